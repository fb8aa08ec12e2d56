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
// the result is within 3e-3 after five default steps.  Where the steps make more of
// A's and B's roundings (see muon_single_error) these have second arrays too, and a
// product is three: two of a first and a second value, one of the first ones.
#pragma once

#include "ptx.cuh"
#include "vec.cuh"

namespace wg {

struct MuonParams {
    int batch, rows, cols;
    long long ld, bs;
    long long gld, gbs;  // the same of grad and mom where the Gram kernel reads them
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
    __half *x[2], *xlo[2], *a, *b;  // (xlo: one array twice where products do not read it)
    __half *alo, *blo;              // second values of A and B, or null
    float* part;          // [batch][nparts] partial sums of squares
    int nparts;
    int nv;  // vectors of a row (the elementwise kernels), and i / nv = i * nv_mul >> nv_shift
    unsigned nv_mul;
    int nv_shift;
    int *arrived, narrived;  // counters of the products' parts, zeroed by the first kernel
};

constexpr float kMuonXScale = 256.f;

__device__ __forceinline__ float muon_elem(const MuonParams& p, long long i)
{
    if (p.grad_dtype == 2) return static_cast<const float*>(p.grad)[i];
    if (p.grad_dtype == 0) return to_f32(static_cast<const __nv_bfloat16*>(p.grad)[i]);
    return to_f32(static_cast<const __half*>(p.grad)[i]);
}

__device__ __forceinline__ uint32_t pack_half2(float a, float b)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_bf162(float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half2(uint32_t x)
{
    return __half22float2(*reinterpret_cast<const __half2*>(&x));
}
__device__ __forceinline__ float2 unpack_bf162(uint32_t x)
{
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x));
}

// Eight values as a pair of 16-bit chunks (BF: bf16, else fp16): hi, and what hi rounds away.
template <bool BF>
__device__ __forceinline__ void split8(const float* v, uint4* hi, uint4* lo)
{
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[i] = BF ? pack_bf162(v[2 * i], v[2 * i + 1]) : pack_half2(v[2 * i], v[2 * i + 1]);
        const float2 f = BF ? unpack_bf162(h[i]) : unpack_half2(h[i]);
        l[i] = BF ? pack_bf162(v[2 * i] - f.x, v[2 * i + 1] - f.y) : pack_half2(v[2 * i] - f.x, v[2 * i + 1] - f.y);
    }
    *hi = make_uint4(h[0], h[1], h[2], h[3]);
    *lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// Eight values as three bf16 chunks, each of what those before it round away: 24 bits, fp32's.
__device__ __forceinline__ void split8_bf16x3(const float* v, uint4* hi, uint4* mid, uint4* lo)
{
    float r[8];
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[i] = pack_bf162(v[2 * i], v[2 * i + 1]);
        const float2 f = unpack_bf162(h[i]);
        r[2 * i] = v[2 * i] - f.x, r[2 * i + 1] = v[2 * i + 1] - f.y;
    }
    *hi = make_uint4(h[0], h[1], h[2], h[3]);
    split8<true>(r, mid, lo);
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

// Eight elements as they come from memory: the conversion waits for them, the load does not.
struct MuonRaw8 {
    uint4 a, b;
};
__device__ __forceinline__ MuonRaw8 muon_raw8(const void* in, int dtype, long long e)
{
    MuonRaw8 r;
    r.b = make_uint4(0u, 0u, 0u, 0u);
    if (dtype == 2) {
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(in) + e);
        r.a = q[0], r.b = q[1];
    } else {
        r.a = *reinterpret_cast<const uint4*>(static_cast<const __half*>(in) + e);
    }
    return r;
}
__device__ __forceinline__ void muon_unraw8(int dtype, const MuonRaw8& r, float (&f)[8])
{
    const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
    if (dtype == 2) {
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(w[k]);
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 x = dtype == 0 ? unpack_bf162(w[k]) : unpack_half2(w[k]);
        f[2 * k] = x.x, f[2 * k + 1] = x.y;
    }
}

// The results of eight elements along a row (every address 16-byte aligned), w the old weights.
__device__ __forceinline__ void muon_finish8(const MuonParams& p, long long e, const float (&o)[8], const MuonRaw8& old)
{
    if (p.out) muon_store8(p.out, p.out_dtype, e, o);
    if (p.weight) {
        float w[8];
        muon_unraw8(p.weight_dtype, old, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = fmaf(p.keep, w[i], -p.lr * o[i]);
        muon_store8(p.weight, p.weight_dtype, e, w);
    }
}
__device__ __forceinline__ void muon_finish8(const MuonParams& p, long long e, const float (&o)[8])
{
    MuonRaw8 old = {};
    if (p.weight) old = muon_raw8(p.weight, p.weight_dtype, e);
    muon_finish8(p, e, o, old);
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

// What u at VEC elements along a row is made of.
template <int VEC>
__device__ __forceinline__ void muon_read(const MuonParams& p, long long e, float (&g)[VEC], float (&m)[VEC])
{
    if constexpr (VEC == 8)
        muon_load8(p.grad, p.grad_dtype, e, g);
    else
        g[0] = muon_elem(p, e);
    if (p.mom) load_f32<float, VEC>(p.mom + e, m);
}
// u.  STEP: the momentum's step is taken (m is then the new momentum); otherwise it has been.
template <int VEC, bool STEP>
__device__ __forceinline__ void muon_make(const MuonParams& p, float (&u)[VEC], float (&m)[VEC])
{
    if (!p.mom) return;
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
        const float y = p.gain * u[k];
        if (STEP) m[k] = fmaf(p.mu, m[k], y);
        u[k] = p.nesterov ? fmaf(p.mu, m[k], y) : m[k];
    }
}
// The row of vector i of a matrix of p.nv vectors a row (i < 2^31).
__device__ __forceinline__ int muon_row(const MuonParams& p, int i)
{
    return (int)(((unsigned long long)(unsigned)i * p.nv_mul) >> p.nv_shift);
}

// Vectors in flight per thread: the kernels below are bound by HBM.
template <int VEC>
constexpr int kMuonAhead = VEC == 8 ? 2 : 8;

// The momentum's step and the partial sums of u's squares.
template <int VEC>
__global__ void __launch_bounds__(256) muon_momentum_kernel(const __grid_constant__ MuonParams p)
{
    constexpr int U = kMuonAhead<VEC>;
    pdl_launch_dependents();
    pdl_wait();
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int i = threadIdx.x; i < p.narrived; i += 256) p.arrived[i] = 0;
    const int n = p.rows * p.nv, step = gridDim.x * 256;
    const long long base = (long long)blockIdx.y * p.bs;
    float s = 0.f;
    for (int i0 = blockIdx.x * 256 + threadIdx.x; i0 < n; i0 += U * step) {
        float g[U][VEC], m[U][VEC];
        long long e[U];
#pragma unroll
        for (int q = 0; q < U; ++q) {
            const int i = min(i0 + q * step, n - 1), r = muon_row(p, i);
            e[q] = base + r * p.ld + (i - r * p.nv) * VEC;
            muon_read<VEC>(p, e[q], g[q], m[q]);
        }
#pragma unroll
        for (int q = 0; q < U; ++q) {
            if (i0 + q * step >= n) break;
            muon_make<VEC, true>(p, g[q], m[q]);
            if (p.mom) store_f32<float, VEC>(p.mom + e[q], m[q]);
#pragma unroll
            for (int k = 0; k < VEC; ++k) s = fmaf(g[q][k], g[q][k], s);
        }
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

// X = u / (|u|_F + eps) (or the results at once when there are no steps).
template <int VEC>
__global__ void __launch_bounds__(256) muon_normalize_kernel(const __grid_constant__ MuonParams p, int last)
{
    constexpr int U = kMuonAhead<VEC>;
    pdl_launch_dependents();
    pdl_wait();
    const int n = p.rows * p.nv, step = gridDim.x * 256;
    const long long base = (long long)blockIdx.y * p.bs;
    const float inv = muon_inv_norm(p, blockIdx.y);
    const float f = last ? inv * p.scale : kMuonXScale * inv;
    for (int i0 = blockIdx.x * 256 + threadIdx.x; i0 < n; i0 += U * step) {
        float u[U][VEC], m[U][VEC];
#pragma unroll
        for (int q = 0; q < U; ++q) {
            const int i = min(i0 + q * step, n - 1), r = muon_row(p, i);
            muon_read<VEC>(p, base + r * p.ld + (i - r * p.nv) * VEC, u[q], m[q]);
        }
#pragma unroll
        for (int q = 0; q < U; ++q) {
            const int i = i0 + q * step;
            if (i >= n) break;
            const int r = muon_row(p, i), c = (i - r * p.nv) * VEC;
            const long long k = blockIdx.y * p.xs + (long long)r * p.ldx + c;
            muon_make<VEC, false>(p, u[q], m[q]);
#pragma unroll
            for (int x = 0; x < VEC; ++x) u[q][x] *= f;
            if constexpr (VEC == 8) {
                if (last) {
                    muon_finish8(p, base + r * p.ld + c, u[q]);
                } else {
                    uint4 h, l;
                    split8<false>(u[q], &h, &l);
                    *reinterpret_cast<uint4*>(p.x[0] + k) = h;
                    *reinterpret_cast<uint4*>(p.xlo[0] + k) = l;
                }
            } else if (last) {
                muon_finish(p, base + r * p.ld + c, u[q][0]);
            } else {
                const __half h = __float2half_rn(u[q][0]);
                p.x[0][k] = h;
                p.xlo[0][k] = __float2half_rn(u[q][0] - __half2float(h));
            }
        }
    }
}

}  // namespace wg
