// The products of the orthogonalised update of larger matrices, on CTA pairs
// (tcgen05 .cta_group::2):
//
//   stage 0:  A = X X^T (or X^T X)             symmetric: tiles on and below the diagonal
//   stage 1:  B = b A + c A A                  symmetric
//   stage 2:  X' = a X + B X (or X B); after the last step the results
//
// Tiles of 256 x 256 (or 256 x 128, where there are few), 64 of the sum per stage
// of the ring: each CTA of a pair stages 128 rows of A and half of B's by TMA and
// holds 128 x 256 fp32 sums in tensor memory, twice, so that a tile's epilogue
// runs beside the next tile's MMAs.  Operands are read as they lie: along the sum (K-major) or
// across it (MN-major), so nothing is ever transposed.  Tiles above the diagonal
// of a symmetric product are written by the epilogue of their mirror image.
//
// A tile goes to a pair as a whole; where there are fewer tiles than pairs and the
// sum is long (the Gram matrix of 512 x 32000) a tile is cut along the sum.  Parts
// of a tile leave fp32 sums in the workspace; the part that arrives last adds them
// in the order of the sum, so the result does not depend on who that is.  Nothing
// waits for another CTA except within the pair.
//
// Operands of two values: the sum is three times as long, its blocks those of second
// by first values, first by second, and first by first (the small ones first: MMAs add
// with truncation, see gram_product and muon_put_back).
//
// Main loop: 0.33 us per 64 of a 256 x 256 tile's sum on all pairs, 1.9 PFLOP/s,
// the rate of a large library product.  Around it a launch costs some 7 us: 1 from
// the kernel before (2 with the set-up after the wait for it, some 15 us of 1000 x
// 2731), 1.7 to the first operands, 3 to 6 for the last tile's epilogue; 15 of them bound updates of up to some 1024 rows.  Each of the roles that
// touch global memory waits for the kernel before by itself, after it has found its
// first tile.
#pragma once

#include "k_muon_gram.cuh"

namespace wg {

constexpr int kMgEpiWarps = 16;
constexpr int kMgThreads = 64 + 32 * kMgEpiWarps;  // warp 0 TMA, warp 1 MMA (rank 0), then the epilogue
constexpr int kMgWarpStaging = 4096;  // 32 rows by 32 columns of fp32 per epilogue warp
// Tiles of 256 rows by BN columns, 64 of the sum per stage: a CTA's 128 rows of A and BN / 2 of B.
template <int BN>
struct Mg {
    static constexpr int kStageBytes = 16384 + BN * 64;
    static constexpr int kStages = BN == 256 ? 5 : 6;
    // All the shared memory that a CTA may have: no other kernel's CTA is beside this
    // one, so that tensor memory can be taken before the kernel before this one has ended
    // (a CTA of that one which has yet to take its own cannot be on this SM).
    static constexpr int kSmem = 227 * 1024;
    static_assert(kStages * kStageBytes + kMgEpiWarps * kMgWarpStaging + 1024 + 256 <= kSmem, "shared memory of a CTA");
    static constexpr int kTmem = 2 * BN;  // columns: the sums, twice
};

// What a product's epilogue writes.  A kernel each: in one, the registers of the
// results cost the others spills (8 of 1024 x 1024 321 us against 311, 512 x 8192 207
// against 190; 300 x 1000, whose kernels are short, 118 against 120).
enum MuonKind {
    kMuonA,        // stage 0
    kMuonB,        // stage 1
    kMuonX,        // stage 2
    kMuonLast,     // the results, every eight elements of a row in an aligned 16 (or 32) bytes
    kMuonLastAny,  // the results, rows that start anywhere
};

// The operands' tensor maps: A, B, and with TWO those of their second values.  (Kernels of
// their own: 8192 x 4096 with one value each 1,974 us against 1,944 where the maps are
// chosen as the kernel runs.)
template <bool TWO>
struct MgMaps {
    CUtensorMap m[TWO ? 4 : 2];
};

struct MuonProduct {
    int kind, xin;
    // The last two steps take B + t I and a - t: where B's eigenvalues are near -t, the
    // product is small, and so are its roundings beside a X, which has 22 bits.
    float a, b, c;            // (a: less t)
    float tc;                 // t in units of the sums of A A
    int a_mn, b_mn;           // operand is read across its rows
    float sums;               // A A and B X in units of X (2^-10 and what truncation left out)
    int M, N, kb, kb1;        // extents of D, 64-wide blocks of the sum, and of one of its terms
    int tm, tn, sym;          // tiles along M and N of a matrix
    int per;                  // tiles of a matrix
    int tiles;                // of all matrices
    int whole;                // tiles of whole waves
    int pairs;
    int cut;                  // pairs that share the blocks of sums of the other tiles (at most as many as blocks)
    float* part;              // [pairs][2][2][BN][128] sums of parts of tiles
    int* arrived;             // [pairs][2][16] parts of a tile that are there (zero between launches)
};

__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* tm, uint32_t bar_cluster, int c0, int c1,
                                                 int c2)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(c2), "r"(bar_cluster)
        : "memory");
}

// Arrive once on an mbarrier of the cluster (a shared::cluster address).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// One piece of a pair's work: blocks k0 .. k1 - 1 of the sum of tile t.
struct MgPiece {
    int t, k0, k1;
};

// A pair's pieces, one after another.  The tiles after the whole waves are `units`
// blocks of sums in a row; pair c < cut takes units c * units / cut ..
// (c + 1) * units / cut (with cut = the number of tiles: one each), then its whole
// tiles.
__device__ __forceinline__ long long mg_unit0(const MuonProduct& g, int c)
{
    return (long long)(g.tiles - g.whole) * g.kb * min(c, g.cut) / g.cut;
}
struct MgWalk {
    long long u, end;
    int t;
    __device__ __forceinline__ MgWalk(const MuonProduct& g, int c) : u(mg_unit0(g, c)), end(mg_unit0(g, c + 1)), t(c) {}
    __device__ __forceinline__ bool next(const MuonProduct& g, MgPiece& p)
    {
        if (u < end) {
            const int r = (int)(u / g.kb);
            p.t = g.whole + r;
            p.k0 = (int)(u - (long long)r * g.kb);
            p.k1 = (int)min((long long)g.kb, p.k0 + (end - u));
            u += p.k1 - p.k0;
            return true;
        }
        if (t >= g.whole) return false;
        p.t = t, p.k0 = 0, p.k1 = g.kb;
        t += g.pairs;
        return true;
    }
};

struct MgTile {
    int b, m, n;  // matrix, first row and column
    bool mirror;  // below the diagonal of a symmetric product
};
template <int BN>
__device__ __forceinline__ MgTile mg_tile(const MuonProduct& g, int t)
{
    constexpr int W = 256 / BN;  // tiles that cover a diagonal block
    MgTile r;
    r.b = t / g.per;
    const int i = t - r.b * g.per;
    int m, n;
    if (g.sym) {
        // Rows 0 .. m - 1 of tiles have W m (m + 1) / 2 tiles.
        m = (int)((sqrtf(8.f * i / W + 1.f) - 1.f) * 0.5f);
        while (W * (m * (m + 1) / 2) > i) --m;
        while (W * ((m + 1) * (m + 2) / 2) <= i) ++m;
        n = i - W * (m * (m + 1) / 2);
        r.mirror = n < W * m;
    } else {
        n = i / g.tm, m = i - n * g.tm;
        r.mirror = false;
    }
    r.m = m * 256, r.n = n * BN;
    return r;
}

// What a chunk's epilogue reads: A (stage 1), X and what its first value rounds
// away (stage 2), in rows of 64 bytes (four lanes a row).
struct MgRead {
    uint4 x[4], y[4];
};
template <int KIND, bool TWO>
__device__ __forceinline__ void mg_read(const MuonParams& p, const MuonProduct& g, int b, int i0, int j, MgRead& r)
{
    if constexpr (KIND != kMuonA) {
        const int lane = threadIdx.x & 31, sub = lane >> 2, jc = j + 8 * (lane & 3);
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            const int i = i0 + 8 * it + sub;
            r.x[it] = r.y[it] = make_uint4(0u, 0u, 0u, 0u);
            if (i >= g.M || jc >= g.N) continue;
            if (KIND == kMuonB) {
                const long long e = b * p.ms + (long long)i * p.ldm + jc;
                r.x[it] = *reinterpret_cast<const uint4*>(p.a + e);
                if (TWO) r.y[it] = *reinterpret_cast<const uint4*>(p.alo + e);
            } else {
                const long long e = b * p.xs + (long long)i * p.ldx + jc;
                r.x[it] = *reinterpret_cast<const uint4*>(p.x[g.xin] + e);
                r.y[it] = *reinterpret_cast<const uint4*>(p.xlo[g.xin] + e);
            }
        }
    }
}

// Rows i0 + lane, columns j .. j + 31 of a square matrix of fp16 at `base`, from packed
// pairs h, and their mirror image.  Chunk k of row r of the staging at k ^ (r / 2) % 4.
__device__ __forceinline__ void mg_put_square(const MuonParams& p, const MuonProduct& g, uint8_t* stg, __half* base, int i0,
                                              int j, bool mirror, const uint32_t (&h)[16])
{
    const int lane = threadIdx.x & 31, sub = lane >> 2, c4 = lane & 3, jc = j + 8 * c4;
    uint8_t* own = stg + lane * 64;
    const int osw = (lane >> 1) & 3;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        *reinterpret_cast<uint4*>(own + ((k ^ osw) << 4)) = make_uint4(h[4 * k], h[4 * k + 1], h[4 * k + 2], h[4 * k + 3]);
    __syncwarp();
    // Rows are padded to eight elements; the padding may be written.
#pragma unroll
    for (int it = 0; it < 4; ++it) {
        const int r = 8 * it + sub;
        const uint4 y = *reinterpret_cast<const uint4*>(stg + r * 64 + ((c4 ^ ((r >> 1) & 3)) << 4));
        if (i0 + r < g.M && jc < g.N) *reinterpret_cast<uint4*>(base + (long long)(i0 + r) * p.ldm + jc) = y;
    }
    if (mirror) {
        // Neighbouring lanes exchange so that each has two rows' values of one column.
        const bool odd = lane & 1;
        const int i2 = i0 + (lane & ~1);
        __half* col = base + (long long)(j + (odd ? 1 : 0)) * p.ldm + i2;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const uint32_t other = __shfl_xor_sync(0xffffffffu, h[k], 1);
            const uint32_t w = odd ? __byte_perm(other, h[k], 0x7632) : __byte_perm(h[k], other, 0x5410);
            if (j + 2 * k + (odd ? 1 : 0) < g.N && i2 < g.M) *reinterpret_cast<uint32_t*>(col + 2 * k * p.ldm) = w;
        }
    }
    __syncwarp();
}

// The first n of 32 staged rows, a column per lane.
__device__ __forceinline__ float mg_staged(const uint8_t* stg, int r)
{
    const int lane = threadIdx.x & 31;
    return *reinterpret_cast<const float*>(stg + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
}
template <typename T>
__device__ __forceinline__ void mg_put_rows(T* out, long long ld, int n, const uint8_t* stg)
{
#pragma unroll 8
    for (int r = 0; r < 32; ++r, out += ld)
        if (r < n) *out = from_f32<T>(mg_staged(stg, r));
}
template <typename T>
__device__ __forceinline__ void mg_weight_rows(const MuonParams& p, T* w, int n, const uint8_t* stg)
{
#pragma unroll 1
    for (int r0 = 0; r0 < 32; r0 += 8, w += 8 * p.ld) {
        T x[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) x[q] = r0 + q < n ? w[q * p.ld] : from_f32<T>(0.f);
#pragma unroll
        for (int q = 0; q < 8; ++q)
            if (r0 + q < n) w[q * p.ld] = from_f32<T>(fmaf(p.keep, to_f32<T>(x[q]), -p.lr * mg_staged(stg, r0 + q)));
    }
}

// 32 finished sums of row i0 + lane, columns j .. j + 31 of matrix b, by one warp: of a
// square matrix, A or B.  Global memory is read and written in rows of 64 bytes through the warp's 4 KB of
// shared memory, whose 16-byte chunks are swizzled by the row: row by row from the
// lanes, a request touched 32 lines and the epilogue took longer than the MMAs of a
// 4096-long sum.  `mirror`: the tile's mirror image is written too.
template <int KIND, bool TWO>
__device__ __forceinline__ void mg_square(const MuonParams& p, const MuonProduct& g, uint8_t* stg, int b, int i0, int j,
                                          bool mirror, float (&v)[32], const MgRead& rd)
{
    const int lane = threadIdx.x & 31, sub = lane >> 2, c4 = lane & 3;
    uint32_t h[16];
    if constexpr (KIND == kMuonA) {
        const float f = TWO ? 16.f * g.sums : 0x1p-6f;
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] *= f;
    } else {
        const float c = g.c * (TWO ? g.sums : 0x1p-10f);
        if (i0 == j)  // t I (see MuonProduct)
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] += lane == k ? g.tc : 0.f;
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] *= c;
#pragma unroll
        for (int two = 0; two < (TWO ? 2 : 1); ++two) {
            // A's values come by the row: rows of 64 bytes, chunk k of row r at k ^ (r / 2) % 4.
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const int r = 8 * it + sub;
                *reinterpret_cast<uint4*>(stg + r * 64 + ((c4 ^ ((r >> 1) & 3)) << 4)) = two ? rd.y[it] : rd.x[it];
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint4 y = *reinterpret_cast<const uint4*>(stg + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4));
                const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = unpack_half2(w[e]);
                    v[8 * k + 2 * e] = fmaf(g.b, f.x, v[8 * k + 2 * e]);
                    v[8 * k + 2 * e + 1] = fmaf(g.b, f.y, v[8 * k + 2 * e + 1]);
                }
            }
            __syncwarp();
        }
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) h[k] = pack_half2(v[2 * k], v[2 * k + 1]);
    mg_put_square(p, g, stg, (KIND == kMuonA ? p.a : p.b) + b * p.ms, i0, j, mirror, h);
    if constexpr (TWO) {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const float2 f = unpack_half2(h[k]);
            h[k] = pack_half2(v[2 * k] - f.x, v[2 * k + 1] - f.y);
        }
        mg_put_square(p, g, stg, (KIND == kMuonA ? p.alo : p.blo) + b * p.ms, i0, j, mirror, h);
    }
}

// The same of the next X, or of the results.
template <int KIND, bool TWO>
__device__ __forceinline__ void mg_result(const MuonParams& p, const MuonProduct& g, uint8_t* stg, int b, int i0, int j,
                                          float (&v)[32], const MgRead& rd)
{
    const int lane = threadIdx.x & 31, sub = lane >> 2, c4 = lane & 3;
    const int jc = j + 8 * c4;
    const float sums = TWO ? g.sums : 0x1p-10f;
    // fp32 rows of 128 bytes: chunk k of row r at k ^ r % 8.
#pragma unroll
    for (int k = 0; k < 8; ++k)
        *reinterpret_cast<float4*>(stg + lane * 128 + ((k ^ (lane & 7)) << 4)) =
            make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
    __syncwarp();
#pragma unroll
    for (int it = 0; it < 4; ++it) {
        const int r = 8 * it + sub, i = i0 + r;
        float y[8];
        const float4 d0 = *reinterpret_cast<const float4*>(stg + r * 128 + (((2 * c4) ^ (r & 7)) << 4));
        const float4 d1 = *reinterpret_cast<const float4*>(stg + r * 128 + (((2 * c4 + 1) ^ (r & 7)) << 4));
        const float d[8] = {d0.x, d0.y, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w};
        const uint32_t wh[4] = {rd.x[it].x, rd.x[it].y, rd.x[it].z, rd.x[it].w};
        const uint32_t wl[4] = {rd.y[it].x, rd.y[it].y, rd.y[it].z, rd.y[it].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float2 h = unpack_half2(wh[q]), l = unpack_half2(wl[q]);
            y[2 * q] = fmaf(g.a, h.x + l.x, d[2 * q] * sums);
            y[2 * q + 1] = fmaf(g.a, h.y + l.y, d[2 * q + 1] * sums);
        }
        if (i >= g.M || jc >= g.N) continue;
        if constexpr (KIND == kMuonX) {
            const long long e = b * p.xs + (long long)i * p.ldx + jc;
            uint4 h, l;
            split8<false>(y, &h, &l);
            *reinterpret_cast<uint4*>(p.x[g.xin ^ 1] + e) = h;
            *reinterpret_cast<uint4*>(p.xlo[g.xin ^ 1] + e) = l;
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q) y[q] *= p.scale * (1.f / kMuonXScale);
            if (KIND == kMuonLast) {
                muon_finish8(p, (long long)b * p.bs + i * p.ld + jc, y);
            } else {
                *reinterpret_cast<float4*>(stg + r * 128 + (((2 * c4) ^ (r & 7)) << 4)) = make_float4(y[0], y[1], y[2], y[3]);
                *reinterpret_cast<float4*>(stg + r * 128 + (((2 * c4 + 1) ^ (r & 7)) << 4)) = make_float4(y[4], y[5], y[6], y[7]);
            }
        }
    }
    __syncwarp();
    if (KIND == kMuonLastAny) {
        // Results whose rows start anywhere: a row at a time, a column per lane (eight
        // elements per lane, one by one, took the last product of 1000 x 2731 35 us
        // instead of 20, and with X read by the column that of 8 of 1023 x 1023 51
        // instead of 33).
        const long long e = (long long)b * p.bs + i0 * p.ld + j + lane;
        const int n = j + lane < g.N ? g.M - i0 : 0;
        if (p.out) {
            if (p.out_dtype == 2)
                mg_put_rows(static_cast<float*>(p.out) + e, p.ld, n, stg);
            else if (p.out_dtype == 0)
                mg_put_rows(static_cast<__nv_bfloat16*>(p.out) + e, p.ld, n, stg);
            else
                mg_put_rows(static_cast<__half*>(p.out) + e, p.ld, n, stg);
        }
        if (p.weight) {
            if (p.weight_dtype == 2)
                mg_weight_rows(p, static_cast<float*>(p.weight) + e, n, stg);
            else if (p.weight_dtype == 0)
                mg_weight_rows(p, static_cast<__nv_bfloat16*>(p.weight) + e, n, stg);
            else
                mg_weight_rows(p, static_cast<__half*>(p.weight) + e, n, stg);
        }
        __syncwarp();
    }
}

template <int BN, int KIND, bool TWO>
__global__ void __launch_bounds__(kMgThreads, 1)
    muon_product_kernel(const __grid_constant__ MgMaps<TWO> maps, const __grid_constant__ MuonParams p,
                        const __grid_constant__ MuonProduct g)
{
    constexpr int kMgStages = Mg<BN>::kStages, kMgStageBytes = Mg<BN>::kStageBytes;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align_shared<uint8_t>(smem_raw, 1024);
    uint8_t* staging = smem + kMgStages * kMgStageBytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(staging + kMgEpiWarps * kMgWarpStaging);      // [stages], rank 0's count
    uint64_t* empty = full + kMgStages;                                             // [stages]
    uint64_t* accf = empty + kMgStages;                                             // [2] sums complete
    uint64_t* acce = accf + 2;                                                      // [2] sums read (rank 0's count)
    uint32_t* tslot = reinterpret_cast<uint32_t*>(acce + 2);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank(), pair = blockIdx.x >> 1;

    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        for (int i = 0; i < (TWO ? 4 : 2); ++i) tma_prefetch_desc(&maps.m[i]);
        for (int i = 0; i < kMgStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&accf[i], 1);
            mbar_init(&acce[i], 2 * kMgEpiWarps);
        }
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(tslot, Mg<BN>::kTmem);
        tc_fence_before();
    }
    cluster_sync_all();  // both CTAs' barriers are initialised and both hold tensor memory
    tc_fence_after();
    const uint32_t tbase = *tslot;
    // (All of the above runs beside the end of the kernel before this one, which the
    // loads of this one wait for.)

    if (warp == 0) {
        if (lane == 0) {
            const uint32_t full0 = mapa_shared(smem_u32(&full[0]), 0u);
            int st = 0;
            uint32_t ph = 0;
            bool ok = true;
            MgPiece w;
            MgWalk walk(g, pair);
            bool more = walk.next(g, w);
            pdl_wait();
            for (; ok && more; more = walk.next(g, w)) {
                const MgTile t = mg_tile<BN>(g, w.t);
                const int m0 = t.m + rank * 128, n0 = t.n + rank * (BN / 2);
                for (int k = w.k0; k < w.k1; ++k) {
                    if (!mbar_wait(&empty[st], ph ^ 1u)) {
                        ok = false;
                        break;
                    }
                    const CUtensorMap *ma = &maps.m[0], *mb = &maps.m[1];
                    int kc = 64 * k;
                    if constexpr (TWO) {  // the block's term of the sum
                        const int term = k >= 2 * g.kb1 ? 2 : k >= g.kb1 ? 1 : 0;
                        if (term == 0) ma = &maps.m[2];
                        if (term == 1) mb = &maps.m[3];
                        kc -= 64 * g.kb1 * term;
                    }
                    uint8_t* s = smem + st * kMgStageBytes;
                    const uint32_t bar = full0 + (uint32_t)(st * 8);
                    if (rank == 0) mbar_arrive_expect_tx(&full[st], 2 * kMgStageBytes);
                    if (g.a_mn) {
                        tma_load_3d_pair(s, ma, bar, m0, kc, t.b);
                        tma_load_3d_pair(s + 8192, ma, bar, m0 + 64, kc, t.b);
                    } else {
                        tma_load_3d_pair(s, ma, bar, kc, m0, t.b);
                    }
                    if (g.b_mn) {
                        tma_load_3d_pair(s + 16384, mb, bar, n0, kc, t.b);
                        if (BN == 256) tma_load_3d_pair(s + 16384 + 8192, mb, bar, n0 + 64, kc, t.b);
                    } else {
                        tma_load_3d_pair(s + 16384, mb, bar, kc, n0, t.b);
                    }
                    if (++st == kMgStages) st = 0, ph ^= 1u;
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            const uint32_t idesc = make_idesc_f16(false, g.a_mn, g.b_mn, 256, BN);
            const uint32_t sbase = smem_u32(smem);
            const uint64_t ad = make_sdesc(sbase, g.a_mn ? 8192u : 16u, 1024u, 2u, 0u);
            const uint64_t bd = make_sdesc(sbase + 16384u, g.b_mn ? 8192u : 16u, 1024u, 2u, 0u);
            const uint64_t ak = g.a_mn ? 128 : 2, bk = g.b_mn ? 128 : 2;
            int st = 0;
            uint32_t ph = 0;
            bool ok = true;
            MgPiece w;
            MgWalk walk(g, pair);
            for (int i = 0; ok && walk.next(g, w); ++i) {
                const int buf = i & 1;
                if (!mbar_wait(&acce[buf], ((uint32_t)(i >> 1) & 1u) ^ 1u)) break;
                tc_fence_after();
                const uint32_t d = tbase + (uint32_t)(buf * BN);
                for (int k = w.k0; k < w.k1; ++k) {
                    if (!mbar_wait(&full[st], ph)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t so = (uint64_t)(st * (kMgStageBytes >> 4));
                    if (elect_one()) {
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            umma_f16_pair(d, ad + so + ak * ks, bd + so + bk * ks, idesc, (k > w.k0 || ks) ? 1u : 0u);
                        umma_commit_pair(&empty[st]);
                    }
                    __syncwarp();
                    if (++st == kMgStages) st = 0, ph ^= 1u;
                }
                if (!ok) break;
                if (elect_one()) umma_commit_pair(&accf[buf]);
                __syncwarp();
            }
        }
    } else {
        // Warp e of the epilogue: 32 rows (its tensor-memory quadrant) by a quarter of the columns.
        const int e = warp - 2, q = warp & 3, col = (e >> 2) * (BN / 4);
        const uint32_t acce0 = mapa_shared(smem_u32(&acce[0]), 0u);
        const uint32_t trow = tbase + ((uint32_t)(q * 32) << 16) + (uint32_t)col;
        const int row = q * 32 + lane;
        constexpr size_t slot = (size_t)2 * BN * 128;  // floats of a part: both ranks
        const size_t mine = (size_t)rank * BN * 128 + (size_t)col * 128 + row;
        MgPiece w;
        MgWalk walk(g, pair);
        pdl_wait();
        for (int i = 0; walk.next(g, w); ++i) {
            const int buf = i & 1;
            const MgTile t = mg_tile<BN>(g, w.t);
            const int i0 = t.m + rank * 128 + q * 32, j0 = t.n + col;
            const uint32_t tacc = trow + (uint32_t)(buf * BN);
            const bool whole = w.k0 == 0 && w.k1 == g.kb;
            MgRead rd;
            if (whole) mg_read<KIND, TWO>(p, g, t.b, i0, j0, rd);  // on its way while the sums are made
            if (!mbar_wait_sleep(&accf[buf], (uint32_t)(i >> 1) & 1u)) break;
            __syncwarp();
            tc_fence_after();
            int c0 = pair, c1 = pair;
            bool finish = true;
            if (!whole) {
                // Leave this part's sums (columns of 128 rows: coalesced), and see whether it is the last.
                float* out = g.part + (size_t)(2 * pair + (w.k0 ? 0 : 1)) * slot + mine;
#pragma unroll 1
                for (int ch = 0; ch < BN / 128; ++ch) {
                    float v[32];
                    gram_ld<32>(tacc + (uint32_t)(ch * 32), v);
#pragma unroll
                    for (int k = 0; k < 32; ++k) __stcg(out + (ch * 32 + k) * 128, v[k]);
                }
                const long long units = (long long)(g.tiles - g.whole) * g.kb, u0 = (long long)(w.t - g.whole) * g.kb;
                c0 = (int)(((u0 + 1) * g.cut + units - 1) / units) - 1;
                c1 = (int)(((u0 + g.kb) * g.cut + units - 1) / units) - 1;
                __threadfence();
                __syncwarp();
                int* count = g.arrived + ((w.t - g.whole) * 2 + rank) * kMgEpiWarps + e;
                int n = 0;
                if (lane == 0) n = atomicAdd(count, 1);
                n = __shfl_sync(0xffffffffu, n, 0);
                finish = n == c1 - c0;
                if (finish) {
                    __threadfence();
                    if (lane == 0) *count = 0;
                }
            }
            if (finish) {
#pragma unroll 1
                for (int ch = 0; ch < BN / 128; ++ch) {
                    float v[32];
                    if (whole) {
                        if (ch) mg_read<KIND, TWO>(p, g, t.b, i0, j0 + ch * 32, rd);
                        gram_ld<32>(tacc + (uint32_t)(ch * 32), v);
                    } else {
                        // 32 loads in flight at a time (left to the compiler, one after another).
#pragma unroll
                        for (int k = 0; k < 32; ++k) v[k] = 0.f;
#pragma unroll 1
                        for (int c = c0; c <= c1; ++c) {
                            const float* in = g.part + (size_t)(2 * c + (c == c0 ? 1 : 0)) * slot + mine + ch * 32 * 128;
                            float x[32];
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(x[k]) : "l"(in + k * 128));
#pragma unroll
                            for (int k = 0; k < 32; ++k) v[k] += x[k];
                        }
                        mg_read<KIND, TWO>(p, g, t.b, i0, j0 + ch * 32, rd);
                    }
                    uint8_t* stg = staging + e * kMgWarpStaging;
                    if constexpr (KIND < kMuonX)
                        mg_square<KIND, TWO>(p, g, stg, t.b, i0, j0 + ch * 32, t.mirror, v, rd);
                    else
                        mg_result<KIND, TWO>(p, g, stg, t.b, i0, j0 + ch * 32, v, rd);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(acce0 + (uint32_t)(buf * 8));
        }
    }
    // Neither CTA releases tensor memory or leaves while the other may still use it.
    tc_fence_before();
    cluster_sync_all();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tbase, Mg<BN>::kTmem);
    }
}

}  // namespace wg
