// Orthogonalised update of matrices whose shorter side is at most 128: the iteration
// runs on the Gram matrix, in one launch as long as errors stay small (five default
// steps do).
//
// With A = X X^T and P = a I + b A + c A A a step is X <- P X, so A <- P A P and
// X_k = Q_k X_0 with Q <- P Q.  All of these are polynomials of one symmetric
// matrix: they commute, and one shared-memory copy of each serves as either
// operand of an MMA.  X itself is read twice (A_0 = U U^T and
// X = Q U) instead of twice a step, and the steps touch m x m matrices only.
//
// Precision: errors of A in directions of small singular values grow by a^2 a
// step, so A, P and Q keep 22 bits: every operand is a pair of fp16 values (what
// the first rounds away is the second), a product three MMAs, sums fp32 in
// tensor memory.  (With single fp16 operands gradients of low rank lose every
// digit.)  U U^T takes u as up to three bf16 values, whose range is fp32's: one for
// bf16 gradients, two for fp16, three for fp32 and with momentum (with two of fp32's
// three, noise beside one strong direction came out up to 2% off for 8 x 72 and 8% for
// 3 x 7; now 1.5e-3 and 2.9e-3).  X = Q U takes it as a pair of fp16 values under its
// matrix's power of two, which the norm gives by then, and so has all of Q's 22 bits
// (64 x 576 of rank one 1.0e-3 off, with Q as a pair of bf16 values 2.8e-3).
//
// A block of P = 64 or 128 rows of the Gram matrix holds as many whole matrices
// as fit (the block-diagonal fold of the convolution kernels): entries of A_0
// between different matrices are set to zero, and products keep them so.  Elements that
// are NaN, infinite or at least 2^64 (whose square is beyond fp32, and which bf16 may
// round to infinity) enter as zeros, and their matrix leaves as NaN, so that they
// cannot reach the others of its block.
//
// Errors of A grow by a^2 a step, so a launch takes no more steps than its bits carry
// (see muon_gram_plan): X is multiplied out then, and the next launch starts from X and
// its own Gram matrix.
//
// A cluster of C CTAs takes a block.  Each adds up U U^T over its 64-column
// chunks of the long side (the momentum's step on the way); each adds a slice of
// the C partial sums through distributed shared memory and gives it to all; all
// run the same steps (one that ran them for the others would have to hand Q out,
// 2 us later); and each multiplies its chunks of U, which it reads again (L2), and
// writes its part of the results.
// Bound by latency: three dependent products a step, each MMA -> tensor memory ->
// registers -> shared memory.  One warp does nothing but issue MMAs, so that A P
// is on its way through the other sixteen while P Q runs.
#pragma once

#include <type_traits>

#include "k_muon.cuh"

namespace wg {

constexpr int kGramThreads = 512;            // the warps that move and convert
constexpr int kGramBlock = kGramThreads + 32;  // and the one that issues MMAs
constexpr int kGramMaxSteps = 16;

struct GramParams {
    MuonParams p;
    int N;           // long side
    int F;           // matrices per block
    int wide;        // rows <= cols
    int chunks;      // 64-column chunks of the long side
    int C;           // CTAs of a cluster
    int parts;       // bf16 values that an element of u takes in U U^T
    int kn;          // 16-wide parts of a block's rows that are used
    int steps;
    int raw;         // what is read is X of the launch before: no norm
    // Per step: P = pa I + pb (TA) + pc (T2); S = rs (T2); Q = rq (TQ); A = ra (TA), the
    // tensor-memory sums holding products of operands scaled by sa, sp, ss and sq (powers of two).
    struct Step {
        float pa, pb, pc, rs, rq, ra, sa, sp, ss, sq;
    } step[kGramMaxSteps];
};

__host__ __device__ constexpr int gram_mat_bytes(int P) { return P * P * 2; }  // one fp16 image
// Three pairs of images, and slack for A operands of 128 rows read from images of 64.
__host__ __device__ constexpr int gram_used_bytes(int P) { return 6 * gram_mat_bytes(P) + 8192 + 1024; }
// What is asked for: so much that no other CTA that takes tensor memory and waits for
// its cluster is on the SM, of this kernel or another.  A CTA takes all of tensor memory
// and then waits for its cluster; two clusters of two streams that share a pair of SMs
// would each hold what the other waits for, and tcgen05.alloc has no limit.  The least
// that such a kernel asks for is 35 KB (eight stages of 4 KB, and 3, of a convolution
// reduced over a cluster), and 1 KB per CTA is the system's.  No more than that for P =
// 64, since the rest is L1, from which rows that start anywhere are read (64 x 577 with
// momentum: 34 us, 40 with 224 KB).
__host__ __device__ constexpr int gram_smem_bytes(int P) { return (P == 64 ? 192 : 224) * 1024; }
static_assert(gram_used_bytes(64) <= gram_smem_bytes(64) && gram_used_bytes(128) <= gram_smem_bytes(128), "shared memory");
static_assert(gram_smem_bytes(64) + 1024 + 35 * 1024 + 1024 > 228 * 1024, "one CTA on an SM");

// Byte offset of the 16-byte chunk that holds elements 8 c8 .. 8 c8 + 7 of row r of a K-major image of P rows:
// 64-element (128-byte) columns of P rows, 128-byte swizzle.
template <int P>
__device__ __forceinline__ uint32_t gram_off(int r, int c8)
{
    return (uint32_t)((c8 >> 3) * (P * 128) + r * 128 + (((c8 & 7) ^ (r & 7)) << 4));
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float* v)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(__float_as_uint(v[0])),
        "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])),
        "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])),
        "r"(__float_as_uint(v[7])), "r"(__float_as_uint(v[8])), "r"(__float_as_uint(v[9])),
        "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])), "r"(__float_as_uint(v[12])),
        "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])), "r"(__float_as_uint(v[15])), "r"(taddr)
        : "memory");
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// NC (a multiple of 16) consecutive tensor-memory columns of this warp's lanes.
template <int NC>
__device__ __forceinline__ void gram_ld(uint32_t taddr, float (&v)[NC])
{
    uint32_t r[NC];
#pragma unroll
    for (int i = 0; i < NC; i += 16) tmem_ld16_issue(taddr + i, r + i);
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < NC; i += 16) reg_fence16(r + i);
#pragma unroll
    for (int i = 0; i < NC; ++i) v[i] = __uint_as_float(r[i]);
}

// NC values of row r, columns c0 .., times s, into the image pair at `img` (shared memory).
template <int P, int NC>
__device__ __forceinline__ void gram_put(uint8_t* img, int r, int c0, const float (&v)[NC], float s)
{
#pragma unroll
    for (int i = 0; i < NC; i += 8) {
        float w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = v[i + k] * s;
        uint4 hi, lo;
        split8<false>(w, &hi, &lo);
        uint8_t* o = img + gram_off<P>(r, (c0 + i) >> 3);
        *reinterpret_cast<uint4*>(o) = hi;
        *reinterpret_cast<uint4*>(o + gram_mat_bytes(P)) = lo;
    }
}

// D[tmem] = X Y for two image pairs: hi hi + hi lo + lo hi.  X is read by rows
// (K-major) and Y by columns (MN-major) of the same layout.  Reading Y by rows too
// (symmetric up to roundings) transposes the roundings of Q between a direction
// the matrix has and one it lacks, which are 482 times larger on one side than on
// the other: gradients of rank one were 10% off.
// The small products come first, or apart: MMAs add with truncation, and so each one
// that adds to the large sums makes them smaller.
// (What is left is put back, see muon_put_back.)
// P = 64: the two images of Y lie one after the other, and one MMA of 128 columns
// multiplies both: hi hi in columns 0 .. 63, hi lo (and lo hi) in columns 64 .. 127 (an
// MMA takes some 66 cycles whatever its columns up to 128: 2 instead of 3).
template <int P>
__device__ __forceinline__ void gram_product(uint32_t d, uint32_t x, uint32_t y, int kn)
{
    const uint32_t idesc = make_idesc_f16(false, false, true, 128, P == 64 ? 64 : 16 * kn);
    const uint32_t idesc2 = make_idesc_f16(false, false, true, 128, 128);
    const uint64_t xd = make_sdesc(x, 16u, 1024u, 2u, 0u), yd = make_sdesc(y, P * 128u, 1024u, 2u, 0u);
    constexpr uint64_t lo = gram_mat_bytes(P) >> 4;
#pragma unroll 1
    for (int ks = 0; ks < kn; ++ks) {
        const uint64_t xo = (uint64_t)((ks >> 2) * (P * 8) + 2 * (ks & 3)), yo = (uint64_t)(128 * ks);
        if (P == 64) {
            umma_f16(d, xd + xo, yd + yo, idesc2, ks ? 1u : 0u);
            umma_f16(d + 64, xd + xo + lo, yd + yo, idesc, 1u);
        } else {
            umma_f16(d, xd + xo, yd + yo + lo, idesc, ks ? 1u : 0u);
            umma_f16(d, xd + xo + lo, yd + yo, idesc, 1u);
        }
    }
    if constexpr (P != 64) {
#pragma unroll 1
        for (int ks = 0; ks < kn; ++ks)
            umma_f16(d, xd + (uint64_t)((ks >> 2) * (P * 8) + 2 * (ks & 3)), yd + (uint64_t)(128 * ks), idesc, 1u);
    }
}

// NC columns of a product, from column c0 (and of its second half).
template <int P, int NC>
__device__ __forceinline__ void gram_sums(uint32_t taddr, float (&v)[NC])
{
    if (P == 64) {
        uint32_t r[2 * NC];
#pragma unroll
        for (int i = 0; i < NC; i += 16) tmem_ld16_issue(taddr + i, r + i), tmem_ld16_issue(taddr + 64 + i, r + NC + i);
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
        for (int i = 0; i < 2 * NC; i += 16) reg_fence16(r + i);
#pragma unroll
        for (int i = 0; i < NC; ++i) v[i] = __uint_as_float(r[i]) + __uint_as_float(r[NC + i]);
    } else {
        gram_ld<NC>(taddr, v);
    }
}

__device__ __forceinline__ float2 ld_dsmem_v2(uint32_t addr)
{
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr));
    return v;
}
__device__ __forceinline__ void st_dsmem_v2(uint32_t addr, float2 v)
{
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(v.x), "f"(v.y) : "memory");
}

// What eight values of u are made of, as it comes from memory: a conversion would wait
// for it.  (Rows that start anywhere: an element in each word.)
struct GramRaw {
    MuonRaw8 g, m;
};

// The eight elements from address e0 (-1: outside) one by one, f(k, address, whether
// it is inside): `pos` is the first one's position along the long side (wide) or its
// row of the block (tall; the rows go on in the next matrix).
template <typename F>
__device__ __forceinline__ void gram_each(const GramParams& g, int blk, long long e0, int pos, F f)
{
    const MuonParams& p = g.p;
    const int nf = min(g.F, p.batch - blk * g.F);
    int at = g.wide ? 0 : pos / p.m, idx = g.wide ? pos : pos - at * p.m;
    long long e = e0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        f(k, e, e0 >= 0 && (g.wide ? idx < g.N : at < nf));
        ++e, ++idx;
        if (!g.wide && idx == p.m) idx = 0, ++at, e += p.gbs - p.m;
    }
}

template <bool VEC>
__device__ __forceinline__ void gram_read(const GramParams& g, int blk, long long e, int pos, GramRaw& r)
{
    const MuonParams& p = g.p;
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
    r.g.a = r.g.b = r.m.a = r.m.b = z;
    if (VEC) {
        if (e < 0) return;
        r.g = muon_raw8(p.grad, p.grad_dtype, e);
        if (p.mom) r.m = muon_raw8(p.mom, 2, e);
        return;
    }
    uint32_t w[8] = {}, m[8] = {};
    gram_each(g, blk, e, pos, [&](int k, long long at, bool in) {
        if (!in) return;
        if (p.grad_dtype == 2)
            w[k] = static_cast<const uint32_t*>(p.grad)[at];
        else
            w[k] = static_cast<const uint16_t*>(p.grad)[at];
        if (p.mom) m[k] = __float_as_uint(p.mom[at]);
    });
    r.g.a = make_uint4(w[0], w[1], w[2], w[3]), r.g.b = make_uint4(w[4], w[5], w[6], w[7]);
    r.m.a = make_uint4(m[0], m[1], m[2], m[3]), r.m.b = make_uint4(m[4], m[5], m[6], m[7]);
}

// STEP: the momentum's step is taken and written; otherwise it has been.
template <bool VEC, bool STEP>
__device__ __forceinline__ void gram_make(const GramParams& g, int blk, long long e, int pos, const GramRaw& r, float (&u)[8])
{
    const MuonParams& p = g.p;
    if (VEC || p.grad_dtype == 2) {
        muon_unraw8(VEC ? p.grad_dtype : 2, r.g, u);
    } else {
        const uint32_t w[8] = {r.g.a.x, r.g.a.y, r.g.a.z, r.g.a.w, r.g.b.x, r.g.b.y, r.g.b.z, r.g.b.w};
#pragma unroll
        for (int k = 0; k < 8; ++k)
            u[k] = p.grad_dtype == 0 ? __uint_as_float(w[k] << 16) : __half2float(__ushort_as_half((unsigned short)w[k]));
    }
    if (!p.mom) return;
    float m[8];
    muon_unraw8(2, r.m, m);
    muon_make<8, STEP>(p, u, m);
    if (!STEP) return;
    if (VEC) {
        if (e >= 0) store_f32<float, 8>(p.mom + e, m);
    } else {
        gram_each(g, blk, e, pos, [&](int k, long long at, bool in) {
            if (in) p.mom[at] = m[k];
        });
    }
}

// x[k] of lane l <-> x[l % 16] of lane k, within each half of the warp.
__device__ __forceinline__ void transpose16(float (&x)[16])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int s = 8; s; s >>= 1)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (!(i & s)) {
                const bool up = lane & s;
                const float y = __shfl_xor_sync(0xffffffffu, up ? x[i] : x[i + s], s);
                x[i] = up ? y : x[i];
                x[i + s] = up ? x[i + s] : y;
            }
}

// Results of 16 rows of the block from row r0 on, one column: o[k] belongs to row
// r0 + k, n is the column.  Weights are all loaded before the first is written.
template <typename F>
__device__ __forceinline__ void gram_rows(const GramParams& g, int blk, int r0, int n, F f)
{
    const MuonParams& p = g.p;
    const int nf = min(g.F, p.batch - blk * g.F);
    int at = r0 / p.m, idx = r0 - at * p.m;
    long long e = (long long)(blk * g.F + at) * p.bs + idx * p.ld + n;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        f(k, e, at < nf && n < g.N);
        e += p.ld;
        if (++idx == p.m) idx = 0, ++at, e += p.bs - p.m * p.ld;
    }
}
template <typename T>
__device__ __forceinline__ void gram_put_rows(const GramParams& g, T* out, int blk, int r0, int n, const float (&o)[16])
{
    gram_rows(g, blk, r0, n, [&](int k, long long e, bool in) {
        if (in) out[e] = from_f32<T>(o[k]);
    });
}
template <typename T>
__device__ __forceinline__ void gram_weight_rows(const GramParams& g, T* w, int blk, int r0, int n, const float (&o)[16])
{
    T x[16];
    gram_rows(g, blk, r0, n, [&](int k, long long e, bool in) { x[k] = in ? w[e] : from_f32<T>(0.f); });
    gram_rows(g, blk, r0, n, [&](int k, long long e, bool in) {
        if (in) w[e] = from_f32<T>(fmaf(g.p.keep, to_f32<T>(x[k]), -g.p.lr * o[k]));
    });
}

// n <= 16 results, `step` elements apart: all loads, then all stores.
template <typename T>
__device__ __forceinline__ void gram_put_each(T* out, long long step, int n, const float (&o)[16])
{
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < n) out[i * step] = from_f32<T>(o[i]);
}
template <typename T>
__device__ __forceinline__ void gram_weight_each(const MuonParams& p, T* w, long long step, int n, const float (&o)[16])
{
    T x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = i < n ? w[i * step] : T();
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < n) w[i * step] = from_f32<T>(fmaf(p.keep, to_f32<T>(x[i]), -p.lr * o[i]));
}

// VEC: every eight elements of a row of grad, momentum, weight and out lie in an
// aligned 16 (or 32) bytes.  Otherwise each is a load of its own, as far ahead as the
// wide ones, and results are turned so that neighbouring lanes write neighbouring
// elements: 64 x 577 28 us and 127 x 4001 71 (one element after another and a row per
// lane: 48 and 177); 64 x 576 and 128 x 4000 take 23 and 54.  A kernel of its own,
// since the code of both, inlined, kept the kernel waiting for instructions.
template <int P, bool VEC>
__global__ void __launch_bounds__(kGramBlock, 1) muon_gram_kernel(const __grid_constant__ GramParams g)
{
    constexpr int NC = P / 4;                     // columns per thread: four warps share a row
    constexpr int MAT = gram_mat_bytes(P), PAIR = 2 * MAT;
    constexpr int IMG = P * 128;                  // one staged image of 64 positions of the long side
    constexpr uint32_t TA = 0, T2 = 128, TQ = 256;  // tensor-memory columns: A, (A A | A P), P Q
    constexpr int TCOLS = 512;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bar[3];
    __shared__ uint32_t tslot;
    __shared__ float diag[128], norm2[64];  // of A_0; |u|_F^2 per matrix
    // Per row: the power of two under which u is staged for Q U, and what is left to multiply its results by.
    __shared__ float up[128], fac[128];
    __shared__ int bad[128];
    uint8_t* smem = align_shared<uint8_t>(smem_raw, 1024);
    uint8_t *ba = smem, *bp = smem + PAIR, *bq = smem + 2 * PAIR;  // A (and A P), P, Q
    const MuonParams& p = g.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool issuer = warp == kGramThreads / 32;  // the warp that issues MMAs
    const int rank = (int)cluster_ctarank(), blk = blockIdx.x / g.C;
    // This thread's part of a Gram-sized matrix: row, first column, and which of
    // its columns are of the row's own matrix.
    const int row = (warp & 3) * 32 + lane, c0 = (warp >> 2) * NC;
    // Rows and columns past the matrices are left as they are: nothing reads their products.
    const bool rows = !issuer && (warp & 3) * 32 < 16 * g.kn, act = rows && c0 < 16 * g.kn;
    const int mine = row / p.m, lo = mine * p.m, hi = mine < g.F ? lo + p.m : lo;
    uint32_t own = 0;
#pragma unroll
    for (int i = 0; i < NC; ++i) own |= (c0 + i >= lo && c0 + i < hi ? 1u : 0u) << i;
    bool ok = true;
    uint32_t ph[3] = {0, 0, 0};
    auto wait = [&](int b) {
        if (ok) ok = mbar_wait(&bar[b], ph[b]);
        ph[b] ^= 1u;
        __syncwarp();
        tc_fence_after();
    };
    // What this thread has written to shared memory and read from tensor memory is done, for the next MMAs.
    auto ready = [&] {
        fence_proxy_async_smem();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    };

    pdl_launch_dependents();
    if (tid == 0) {
        for (int i = 0; i < 3; ++i) mbar_init(&bar[i], 1);
        fence_mbar_init();
    }
    if (tid < 128) bad[tid] = 0, up[tid] = 0.f;
    pdl_wait();
    if (warp == 0) {
        // After the wait: a CTA of the kernel before, which may be on this SM, may have yet
        // to take its own.
        tmem_alloc(&tslot, TCOLS);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = tslot, trow = tb + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)c0;

    // ---------------------------------------------------- A_0 = U U^T over this CTA's chunks
    // Two chunks' images (three each), where A, P and Q will be.  Wide: rows of the block,
    // 64 positions along; tall: 64 positions, the block's rows along, in 64-wide atoms.
    const int line = tid >> 3, seg = (tid & 7) * 8;
    // Where this thread's eight elements of chunk 0 lie (-1: no matrix there), and of chunk ch.
    long long at0[P / 64];
#pragma unroll
    for (int j = 0; j < P / 64; ++j) {
        const int i = (g.wide ? line : seg) + 64 * j, f = i / p.m, b = blk * g.F + f, idx = i - f * p.m;
        at0[j] = f >= g.F || b >= p.batch ? -1 : (long long)b * p.gbs + (g.wide ? idx * p.gld + seg : line * p.gld + idx);
    }
    auto addr = [&](int ch, int j) -> long long {
        if (at0[j] < 0 || ch * 64 + (g.wide ? seg : line) >= g.N) return -1;
        return at0[j] + ch * (g.wide ? 64 : 64 * p.gld);
    };
    auto pos = [&](int ch, int j) { return g.wide ? ch * 64 + seg : seg + 64 * j; };
    auto stage = [&](uint8_t* img, int ch, auto step, const GramRaw (&u)[P / 64]) {
#pragma unroll
        for (int j = 0; j < P / 64; ++j) {
            float v[8];
            gram_make<VEC, decltype(step)::value>(g, blk, addr(ch, j), pos(ch, j), u[j], v);
            float odd = 0.f;  // not finite when one of them is a NaN or of 2^64 or more
#pragma unroll
            for (int k = 0; k < 8; ++k) odd = fmaf(v[k], 0x1p64f, odd);
            if (!(fabsf(odd) < INFINITY))
#pragma unroll 1
                for (int k = 0; k < 8; ++k) {
                    float x = 0.f;
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        if (q == k) x = v[q];
                    if (fabsf(x) < 0x1p64f) continue;
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        if (q == k) v[q] = 0.f;
                    bad[g.wide ? line + 64 * j : seg + 64 * j + k] = 1;
                }
            uint8_t* o = img + j * 8192 + line * 128 + ((((tid & 7) ^ (line & 7))) << 4);
            uint4 h, m, l;
            if constexpr (decltype(step)::value) {
                split8_bf16x3(v, &h, &m, &l);
                if (g.parts > 2) *reinterpret_cast<uint4*>(o + 2 * IMG) = l;
            } else {
                // (|u| is below 2^14 then, and 0 where |u|_F is not finite.)
                if (g.wide) {
                    const float f = up[line + 64 * j];
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] *= f;
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] *= up[seg + 64 * j + k];
                }
                split8<false>(v, &h, &m);
            }
            *reinterpret_cast<uint4*>(o) = h;
            if (g.parts > 1) *reinterpret_cast<uint4*>(o + IMG) = m;
        }
    };
    auto load = [&](int ch, GramRaw (&u)[P / 64]) {
        if (ch >= g.chunks) return;
#pragma unroll
        for (int j = 0; j < P / 64; ++j)
            gram_read<VEC>(g, blk, addr(ch, j), pos(ch, j), u[j]);
    };
    const int nch = (g.chunks - rank + g.C - 1) / g.C;  // this CTA's chunks: rank, rank + C, ...
    if (!issuer) {
        // Chunks on their way ahead of the one that is staged: two, or one where two are too many registers.
        constexpr int AHEAD = P == 64 ? 2 : 1;
        GramRaw u[AHEAD][P / 64];
#pragma unroll 1
        for (int it = -AHEAD; it < nch; ++it) {
            if (it >= 2) wait(it & 1);
            if (it >= 0) stage(ba + (it & 1) * 3 * IMG, rank + it * g.C, std::true_type{}, u[0]);
#pragma unroll
            for (int j = 0; j < P / 64; ++j) u[0][j] = u[AHEAD - 1][j];
            load(rank + (it + AHEAD) * g.C, u[AHEAD - 1]);
            if (it >= 0) ready();
        }
        if (nch >= 2) wait(nch & 1);
        if (nch >= 1) wait((nch - 1) & 1);
    } else {
        const uint32_t mn = g.wide ? 0u : 1u;
        const uint32_t idesc = make_idesc_f16(true, mn, mn, 128, P);
        for (int it = 0; it < nch; ++it) {
            __syncthreads();
            tc_fence_after();
            if (elect_one()) {
                const uint32_t a = smem_u32(ba + (it & 1) * 3 * IMG);
                // Tall blocks of 64 rows: the second 64 rows of the MMA read the first again.
                const uint64_t d = g.wide ? make_sdesc(a, 16u, 1024u, 2u, 0u)
                                          : make_sdesc(a, P == 128 ? 8192u : 0u, 1024u, 2u, 0u);
#pragma unroll 1
                for (int ks = 0; ks < 4; ++ks) {
                    const uint64_t h = d + (uint64_t)(ks * (g.wide ? 2 : 128)), m = h + (IMG >> 4), l = m + (IMG >> 4);
                    // The small products have sums of their own (see gram_product).
                    umma_f16(tb + TA, h, h, idesc, (it | ks) ? 1u : 0u);
                    if (g.parts > 1) {
                        umma_f16(tb + T2, h, m, idesc, (it | ks) ? 1u : 0u);
                        umma_f16(tb + T2, m, h, idesc, 1u);
                        umma_f16(tb + T2, m, m, idesc, 1u);
                    }
                    if (g.parts > 2) {  // (What the others make is below 2^-26 of the first.)
                        umma_f16(tb + T2, h, l, idesc, 1u);
                        umma_f16(tb + T2, l, h, idesc, 1u);
                    }
                }
                umma_commit(&bar[it & 1]);
            }
            __syncwarp();
        }
    }
    // This CTA's partial sum in P's place (fp32 rows, 16-byte chunks swizzled by
    // the row); NaN on the diagonal of a row that held a NaN or an infinity.
    __syncthreads();
    if (act) {
#pragma unroll 1
        for (int h = 0; h < NC; h += 16) {
            float v[16];
            gram_ld<16>(trow + TA + h, v);
            if (g.parts > 1) {
                float x[16];
                gram_ld<16>(trow + T2 + h, x);
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] += x[i];
            }
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<float4*>(bp + row * (P * 4) + (((((c0 + h + i) >> 2)) ^ (row & 7)) << 4)) =
                    nch > 0 ? make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if (row >= c0 && row < c0 + NC && bad[row])
            *reinterpret_cast<float*>(bp + row * (P * 4) + ((((row >> 2) ^ (row & 7)) << 4) | (row & 3) << 2)) = NAN;
    }
    cluster_sync_all();
    if (!issuer) {
        // A slice of the sum over the cluster, into every CTA's Q.
        const int pieces = 16 * g.kn * P / 2 / g.C;  // 8-byte pieces of a slice
        const uint32_t src = smem_u32(bp), dst = smem_u32(bq);
        for (int i = tid; i < pieces; i += kGramThreads) {
            const uint32_t o = (uint32_t)(rank * pieces + i) << 3;
            float2 s = make_float2(0.f, 0.f);
#pragma unroll
            for (int c0 = 0; c0 < 16; c0 += 8) {
                if (c0 >= g.C) break;
                float2 x[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) x[c] = ld_dsmem_v2(mapa_shared(src + o, (uint32_t)min(c0 + c, g.C - 1)));
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    if (c0 + c < g.C) s.x += x[c].x, s.y += x[c].y;
            }
            for (int c = 0; c < g.C; ++c) st_dsmem_v2(mapa_shared(dst + o, (uint32_t)c), s);
        }
    }
    cluster_sync_all();

    // ---------------------------------------------------- the steps
    GramRaw u[P / 64];
    if (issuer) {
        const uint32_t sba = smem_u32(ba), sbp = smem_u32(bp), sbq = smem_u32(bq);
        __syncthreads();  // the diagonal
        __syncthreads();  // and its sums
        for (int k = 0; k < g.steps; ++k) {
            const bool last = k == g.steps - 1;
            __syncthreads();
            tc_fence_after();
            if (elect_one()) {
                gram_product<P>(tb + T2, sba, sba, g.kn);
                umma_commit(&bar[0]);
            }
            __syncwarp();
            if (last && k == 0) break;
            __syncthreads();
            tc_fence_after();
            if (elect_one()) {
                if (!last) {
                    gram_product<P>(tb + T2, sba, sbp, g.kn);
                    umma_commit(&bar[0]);
                }
                if (k > 0) {
                    gram_product<P>(tb + TQ, sbp, sbq, g.kn);
                    umma_commit(&bar[1]);
                }
            }
            __syncwarp();
            if (last) break;
            __syncthreads();
            tc_fence_after();
            if (elect_one()) {
                gram_product<P>(tb + TA, sba, sbp, g.kn);  // A <- S P
                umma_commit(&bar[2]);
            }
            __syncwarp();
        }
    } else {
        if (tid < P)
            diag[tid] = *reinterpret_cast<const float*>(bq + tid * (P * 4) + ((((tid >> 2) ^ (tid & 7)) << 4) | (tid & 3) << 2));
        __syncthreads();
        for (int f = warp; f < g.F; f += kGramThreads / 32) {  // |u|_F^2 is the trace: a warp per matrix
            float s = 0.f;
            for (int i = lane; i < p.m; i += 32) s += diag[f * p.m + i];
#pragma unroll
            for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (lane == 0) norm2[f] = s;
        }
        __syncthreads();
        if (act) {
            // A_0 = U U^T / (|u|_F + eps)^2, zero between matrices.
            const float s = mine < g.F ? norm2[mine] : 0.f;
            const float norm = sqrtf(s), d = norm + p.eps;
            const bool fin = s < INFINITY;
            const float inv = g.raw ? 1.f : fin && d > 0.f ? 1.f / d : 0.f;
            if (c0 == 0) {
                // |u| < 2^(e + 1); below 2^-60 s may have lost squares, and u keeps its bits all the same.
                const int e = max((int)(__float_as_uint(norm) >> 23) - 127, -60);
                up[row] = fin ? __uint_as_float((uint32_t)(127 + 13 - e) << 23) : 0.f;
                const float down = __uint_as_float((uint32_t)(127 - 13 + e) << 23);
                fac[row] = fin ? p.scale * (inv * down) / g.step[g.steps - 1].sq : NAN;
            }
#pragma unroll 1
            for (int h = 0; h < NC; h += 16) {
                float v[16];
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const float4 x = *reinterpret_cast<const float4*>(bq + row * (P * 4) +
                                                                      (((((c0 + h + i) >> 2)) ^ (row & 7)) << 4));
                    v[i] = x.x, v[i + 1] = x.y, v[i + 2] = x.z, v[i + 3] = x.w;
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = fin && (own >> (h + i) & 1u) ? v[i] * inv * inv : 0.f;
                tmem_st16(trow + TA + h, v);
                gram_put<P, 16>(ba, row, c0 + h, v, g.step[0].sa);
            }
            if (P == 64) {
                const float z[16] = {};
                tmem_st16(trow + TA + 64, z);
            }
        }
        // f times the sums at t into the pair at img, sixteen columns at a time (all 32 of a
        // block of 128 at once are more than the registers hold).  What A_0 has zero between
        // matrices stays zero: every product adds zeros there.
        auto convert = [&](uint32_t t, float f, uint8_t* img) {
#pragma unroll 1
            for (int h = 0; h < NC; h += 16) {
                float v[16];
                gram_sums<P, 16>(trow + t + h, v);
                gram_put<P, 16>(img, row, c0 + h, v, f);
            }
        };
        const uint32_t diagonal = row >= c0 && row < c0 + NC ? 1u << (row - c0) : 0u;
        for (int k = 0; k < g.steps; ++k) {
            const bool last = k == g.steps - 1;
            const GramParams::Step w = g.step[k];
            ready();
            wait(0);
            if (act) {
                // P = a I + b A + c A A
#pragma unroll 1
                for (int h = 0; h < NC; h += 16) {
                    float v[16], x[16];
                    gram_sums<P, 16>(trow + T2 + h, v);
                    gram_sums<P, 16>(trow + TA + h, x);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        v[i] = fmaf(w.pc, v[i], w.pb * x[i]);
                        if (diagonal >> (h + i) & 1u) v[i] += w.pa;
                    }
                    if (k > 0 || !last) gram_put<P, 16>(bp, row, c0 + h, v, w.sp);
                    if (k == 0) gram_put<P, 16>(bq, row, c0 + h, v, w.sq);
                }
            }
            if (last && k == 0) break;
            ready();
            if (last) break;
            wait(0);
            if (act) convert(T2, w.rs * w.ss, ba);  // S = A P, in A's place
            ready();
            if (k > 0) {
                wait(1);
                if (act) convert(TQ, w.rq * w.sq, bq);
            }
            wait(2);
            if (act) convert(TA, w.ra * g.step[k + 1].sa, ba);
        }
        load(rank, u);  // the first chunk of U comes back
        if (g.steps > 1) {
            wait(1);
            if (act) convert(TQ, g.step[g.steps - 1].rq * g.step[g.steps - 1].sq, bq);
        }
    }

    // ---------------------------------------------------- results: X = Q U over this CTA's chunks
    if (!issuer) {
        const int q0 = (warp >> 2) * 16;
        // A chunk is staged and its MMAs begin before the results of the one before it are written.
#pragma unroll 1
        for (int it = -1; it < nch; ++it) {
            const int ch = rank + it * g.C;
            const int b0 = blk * g.F + mine;
            const bool mat = rows && mine < g.F && b0 < p.batch;
            MuonRaw8 old[2] = {};
            if (VEC && it >= 0 && g.wide && p.weight && mat) {
                const long long e = (long long)b0 * p.bs + (row - lo) * p.ld + ch * 64 + q0;
                if (ch * 64 + q0 < g.N) old[0] = muon_raw8(p.weight, p.weight_dtype, e);
                if (ch * 64 + q0 + 8 < g.N) old[1] = muon_raw8(p.weight, p.weight_dtype, e + 8);
            }
            if (it + 1 < nch) {
                // (The MMAs that read this image two chunks ago are done: their sums have been read.)
                stage((it & 1 ? ba : bp), ch + g.C, std::false_type{}, u);
                load(ch + 2 * g.C, u);
                ready();
            }
            if (it < 0) continue;
            wait(it & 1);
            float x[16];
            if (rows) gram_ld<16>(tb + ((uint32_t)((warp & 3) * 32) << 16) + (it & 1 ? T2 : TA) + (uint32_t)q0, x);
            if (!VEC && g.wide) {
                // A column per lane (a row per lane touches 32 rows an access).
                if (!rows) continue;
                const float f = fac[row];
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] *= f;
                transpose16(x);
                const int r0 = (warp & 3) * 32 + (lane & 16), n = ch * 64 + q0 + (lane & 15);
                if (p.out) {
                    if (p.out_dtype == 2)
                        gram_put_rows(g, static_cast<float*>(p.out), blk, r0, n, x);
                    else if (p.out_dtype == 0)
                        gram_put_rows(g, static_cast<__nv_bfloat16*>(p.out), blk, r0, n, x);
                    else
                        gram_put_rows(g, static_cast<__half*>(p.out), blk, r0, n, x);
                }
                if (p.weight) {
                    if (p.weight_dtype == 2)
                        gram_weight_rows(g, static_cast<float*>(p.weight), blk, r0, n, x);
                    else if (p.weight_dtype == 0)
                        gram_weight_rows(g, static_cast<__nv_bfloat16*>(p.weight), blk, r0, n, x);
                    else
                        gram_weight_rows(g, static_cast<__half*>(p.weight), blk, r0, n, x);
                }
            } else if (mat) {
                const float f = fac[row];
                const long long base = (long long)b0 * p.bs;
                const int n0 = ch * 64 + q0;
                if (VEC && g.wide) {
#pragma unroll
                    for (int i = 0; i < 16; i += 8) {
                        float o[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) o[k] = f * x[i + k];
                        if (n0 + i < g.N) muon_finish8(p, base + (row - lo) * p.ld + n0 + i, o, old[i / 8]);
                    }
                } else {
                    // (Tall: neighbouring lanes write neighbouring elements.)
                    const long long e0 = base + n0 * p.ld + (row - lo), step = p.ld;
                    const int n = min(16, g.N - n0);
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] *= f;
                    if (p.out) {
                        if (p.out_dtype == 2)
                            gram_put_each(static_cast<float*>(p.out) + e0, step, n, x);
                        else if (p.out_dtype == 0)
                            gram_put_each(static_cast<__nv_bfloat16*>(p.out) + e0, step, n, x);
                        else
                            gram_put_each(static_cast<__half*>(p.out) + e0, step, n, x);
                    }
                    if (p.weight) {
                        if (p.weight_dtype == 2)
                            gram_weight_each(p, static_cast<float*>(p.weight) + e0, step, n, x);
                        else if (p.weight_dtype == 0)
                            gram_weight_each(p, static_cast<__nv_bfloat16*>(p.weight) + e0, step, n, x);
                        else
                            gram_weight_each(p, static_cast<__half*>(p.weight) + e0, step, n, x);
                    }
                }
            }
        }
    } else {
        const uint32_t idesc = make_idesc_f16(false, false, g.wide != 0, 128, 64);
        const uint64_t qd = make_sdesc(smem_u32(bq), 16u, 1024u, 2u, 0u);
        for (int it = 0; it < nch; ++it) {
            __syncthreads();
            tc_fence_after();
            if (elect_one()) {
                const uint32_t img = smem_u32(it & 1 ? bp : ba), d = tb + (it & 1 ? T2 : TA);
                const uint64_t ud = g.wide ? make_sdesc(img, 8192u, 1024u, 2u, 0u) : make_sdesc(img, 16u, 1024u, 2u, 0u);
                const uint64_t ql = MAT >> 4, ul = IMG >> 4;
#pragma unroll 1
                for (int i = 0; i < 2 * g.kn; ++i) {  // the small products first (see gram_product)
                    const bool large = i >= g.kn;
                    const int ks = large ? i - g.kn : i;
                    const uint64_t qo = (uint64_t)((ks >> 2) * (P * 8) + 2 * (ks & 3));
                    const uint64_t uo = g.wide ? (uint64_t)(128 * ks) : (uint64_t)((ks >> 2) * 512 + 2 * (ks & 3));
                    umma_f16(d, qd + qo + (large ? 0 : ql), ud + uo, idesc, i ? 1u : 0u);
                    if (!large && g.parts > 1) umma_f16(d, qd + qo, ud + uo + ul, idesc, 1u);
                }
                umma_commit(&bar[it & 1]);
            }
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tb, TCOLS);
    }
}

}  // namespace wg
