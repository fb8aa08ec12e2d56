// Orthogonalised update (Newton-Schulz products) with momentum and weight step.
//
//   m <- mu m + (1 - dampening) g;  u = nesterov ? (1 - dampening) g + mu m : m
//   X = u / (|u|_F + eps);  steps times: A = X X^T, X <- a X + (b A + c A A) X
//   out = scale X;  w <- decay w - lr scale X
//
// X keeps the matrices' own orientation: with rows > cols the products are
// A = X^T X and X (b A + c A A), the same iteration on the shorter side.
// Operands are fp16, scaled by powers of two so that entries keep their 11 bits
// (X by 2^8, A and B = b A + c A A by 2^10); X is carried as a second fp16
// array of what the first one rounds away, used in the a X term: without it the
// rounding of X costs up to 6e-3 of the result on gradients of low rank, with it
// the result is within 2e-3.
#pragma once

#include "ptx.cuh"
#include "vec.cuh"

namespace wg {

struct MuonParams {
    int batch, rows, cols;
    long long ld, bs;
    const void* grad;
    float* mom;
    void* weight;
    void* out;
    int grad_dtype, out_dtype, weight_dtype;
    int nesterov;
    float mu, gain, eps;  // gain = 1 - dampening
    float scale, keep, lr;  // w <- keep w - lr (scale X)
    // workspace
    int ldx, m, ldm;      // row lengths of X and of A and B; m = min(rows, cols)
    long long xs, ms;     // elements between matrices
    __half *x[2], *xlo, *a, *b;
    float* part;          // [batch][nparts] partial sums of squares
    int nparts;
};

constexpr float kMuonXScale = 256.f;

__device__ __forceinline__ float muon_elem(const MuonParams& p, long long i)
{
    if (p.grad_dtype == 2) return static_cast<const float*>(p.grad)[i];
    if (p.grad_dtype == 0) return to_f32(static_cast<const __nv_bfloat16*>(p.grad)[i]);
    return to_f32(static_cast<const __half*>(p.grad)[i]);
}

// Block sum in a fixed order; every thread gets it.
__device__ __forceinline__ float block_sum_256(float s)
{
    __shared__ float red[8];
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += red[i];
    return s;
}

// The momentum's step and the partial sums of u's squares.
__global__ void __launch_bounds__(256) muon_momentum_kernel(const __grid_constant__ MuonParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    const int n = p.rows * p.cols;
    const long long base = (long long)blockIdx.y * p.bs;
    float s = 0.f;
    for (int i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256) {
        const int r = i / p.cols;
        const long long e = base + r * p.ld + (i - r * p.cols);
        float u = muon_elem(p, e);
        if (p.mom) {
            u *= p.gain;
            const float m = fmaf(p.mu, p.mom[e], u);
            p.mom[e] = m;
            u = p.nesterov ? fmaf(p.mu, m, u) : m;
        }
        s = fmaf(u, u, s);
    }
    s = block_sum_256(s);
    if (threadIdx.x == 0) p.part[blockIdx.y * p.nparts + blockIdx.x] = s;
}

// 1 / (|u|_F + eps) of matrix b: 0 for a zero matrix, NaN when the sum of
// squares is not finite.
__device__ __forceinline__ float muon_inv_norm(const MuonParams& p, int b)
{
    float s = 0.f;
    for (int i = threadIdx.x; i < p.nparts; i += 256) s += p.part[b * p.nparts + i];
    s = block_sum_256(s);
    const float d = sqrtf(s) + p.eps;
    return !(s < INFINITY) ? NAN : d > 0.f ? 1.f / d : 0.f;
}

__device__ __forceinline__ void muon_store(void* out, int dtype, long long e, float v)
{
    if (dtype == 2)
        static_cast<float*>(out)[e] = v;
    else if (dtype == 0)
        static_cast<__nv_bfloat16*>(out)[e] = __float2bfloat16_rn(v);
    else
        static_cast<__half*>(out)[e] = __float2half_rn(v);
}

__device__ __forceinline__ float muon_load(const void* in, int dtype, long long e)
{
    if (dtype == 2) return static_cast<const float*>(in)[e];
    if (dtype == 0) return to_f32(static_cast<const __nv_bfloat16*>(in)[e]);
    return to_f32(static_cast<const __half*>(in)[e]);
}

// The results of an element, o = scale X.
__device__ __forceinline__ void muon_finish(const MuonParams& p, long long e, float o)
{
    if (p.out) muon_store(p.out, p.out_dtype, e, o);
    if (p.weight)
        muon_store(p.weight, p.weight_dtype, e, fmaf(p.keep, muon_load(p.weight, p.weight_dtype, e), -p.lr * o));
}

__device__ __forceinline__ void muon_store8(void* out, int dtype, long long e, const float (&v)[8])
{
    if (dtype == 2)
        store_f32<float, 8>(static_cast<float*>(out) + e, v);
    else if (dtype == 0)
        store_f32<__nv_bfloat16, 8>(static_cast<__nv_bfloat16*>(out) + e, v);
    else
        store_f32<__half, 8>(static_cast<__half*>(out) + e, v);
}
__device__ __forceinline__ void muon_load8(const void* in, int dtype, long long e, float (&v)[8])
{
    if (dtype == 2)
        load_f32<float, 8>(static_cast<const float*>(in) + e, v);
    else if (dtype == 0)
        load_f32<__nv_bfloat16, 8>(static_cast<const __nv_bfloat16*>(in) + e, v);
    else
        load_f32<__half, 8>(static_cast<const __half*>(in) + e, v);
}

// The results of eight elements along a row (every address 16-byte aligned).
__device__ __forceinline__ void muon_finish8(const MuonParams& p, long long e, const float (&o)[8])
{
    if (p.out) muon_store8(p.out, p.out_dtype, e, o);
    if (p.weight) {
        float w[8];
        muon_load8(p.weight, p.weight_dtype, e, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = fmaf(p.keep, w[i], -p.lr * o[i]);
        muon_store8(p.weight, p.weight_dtype, e, w);
    }
}

// x times 2^8 as two fp16 values.
__device__ __forceinline__ void muon_split(float x, __half* hi, __half* lo)
{
    *hi = __float2half_rn(x);
    *lo = __float2half_rn(x - __half2float(*hi));
}

// X = u / (|u|_F + eps) (or the results at once when there are no steps).
__global__ void __launch_bounds__(256) muon_normalize_kernel(const __grid_constant__ MuonParams p, int last)
{
    pdl_launch_dependents();
    pdl_wait();
    const int n = p.rows * p.cols;
    const long long base = (long long)blockIdx.y * p.bs;
    const float inv = muon_inv_norm(p, blockIdx.y);
    for (int i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256) {
        const int r = i / p.cols, c = i - r * p.cols;
        const long long e = base + r * p.ld + c;
        float u;
        if (p.mom) {
            u = p.mom[e];
            if (p.nesterov) u = fmaf(p.mu, u, p.gain * muon_elem(p, e));
        } else {
            u = muon_elem(p, e);
        }
        const float x = u * inv;
        if (last) {
            muon_finish(p, e, p.scale * x);
        } else {
            const long long k = blockIdx.y * p.xs + (long long)r * p.ldx + c;
            muon_split(kMuonXScale * x, &p.x[0][k], &p.xlo[k]);
        }
    }
}

// One product of the iteration: D[i, j] = sum over k of P[i, k] Q[k, j], a 64 x 64
// tile per CTA, with the epilogue of its stage:
//   0: A = D;  1: B = b A + c D;  2: X' = a X + D (the results after the last step).
struct MuonGemm {
    const __half *P, *Q;
    long long pi, pk, qk, qj, pb, qb;  // element strides, and between matrices
    int M, N, K;
    int stage, xin, last;
    float a, b, c;
};

__global__ void __launch_bounds__(256)
    muon_gemm_kernel(const __grid_constant__ MuonParams p, const __grid_constant__ MuonGemm g)
{
    pdl_launch_dependents();
    pdl_wait();
    __shared__ float sp[16][65], sq[16][65];
    const int b = blockIdx.z, i0 = blockIdx.y * 64, j0 = blockIdx.x * 64;
    const __half *P = g.P + b * g.pb, *Q = g.Q + b * g.qb;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < g.K; k0 += 16) {
        for (int e = threadIdx.x; e < 1024; e += 256) {
            int i = e >> 4, k = e & 15;
            if (g.pi == 1) i = e & 63, k = e >> 6;
            sp[k][i] = i0 + i < g.M && k0 + k < g.K ? __half2float(P[(i0 + i) * g.pi + (k0 + k) * g.pk]) : 0.f;
            int j = e >> 4;
            k = e & 15;
            if (g.qj == 1) j = e & 63, k = e >> 6;
            sq[k][j] = j0 + j < g.N && k0 + k < g.K ? __half2float(Q[(k0 + k) * g.qk + (j0 + j) * g.qj]) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            float u[4], v[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) u[r] = sp[k][ty * 4 + r], v[r] = sq[k][tx + 16 * r];
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[r][q] = fmaf(u[r], v[q], acc[r][q]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int i = i0 + ty * 4 + r, j = j0 + tx + 16 * q;
            if (i >= g.M || j >= g.N) continue;
            const float d = acc[r][q];
            if (g.stage == 0) {
                p.a[b * p.ms + (long long)i * p.ldm + j] = __float2half_rn(d * 0x1p-6f);
            } else if (g.stage == 1) {
                const long long e = b * p.ms + (long long)i * p.ldm + j;
                p.b[e] = __float2half_rn(fmaf(g.c * 0x1p-10f, d, g.b * __half2float(p.a[e])));
            } else {
                const long long e = b * p.xs + (long long)i * p.ldx + j;
                const float x = __half2float(p.x[g.xin][e]) + __half2float(p.xlo[e]);
                const float y = fmaf(g.a, x, d * 0x1p-10f);
                if (g.last)
                    muon_finish(p, (long long)b * p.bs + i * p.ld + j, p.scale * (y * (1.f / kMuonXScale)));
                else
                    muon_split(y, &p.x[g.xin ^ 1][e], &p.xlo[e]);
            }
        }
}

}  // namespace wg
