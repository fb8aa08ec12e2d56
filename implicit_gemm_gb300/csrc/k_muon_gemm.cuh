// The products of the orthogonalised update of larger matrices, on CTA pairs
// (tcgen05 .cta_group::2):
//
//   stage 0:  A = X X^T (or X^T X)             symmetric: tiles on and below the diagonal
//   stage 1:  B = b A + c A A                  symmetric
//   stage 2:  X' = a X + B X (or X B); after the last step the results
//
// Tiles of 256 x 256, 64 of the sum per stage of the ring: each CTA of a pair
// stages 128 rows of either operand by TMA (32 KB; 5 stages) and holds 128 x 256
// fp32 sums in tensor memory, twice, so that a tile's epilogue runs beside the
// next tile's MMAs.  Operands are read as they lie: along the sum (K-major) or
// across it (MN-major), so nothing is ever transposed.  Tiles above the diagonal
// of a symmetric product are written by the epilogue of their mirror image.
//
// Whole waves of tiles go one tile to a pair; the tiles that are left are cut
// along the sum so that every pair gets the same share (a matrix of 1024 rows has
// ten tiles below the diagonal for 76 pairs).  Parts of a tile leave fp32 sums in
// the workspace; the part that arrives last adds them in the order of the sum,
// so the result does not depend on who that is.  Nothing waits for another CTA
// except within the pair.
#pragma once

#include "k_muon_gram.cuh"

namespace wg {

constexpr int kMgThreads = 320;  // warp 0 TMA, warp 1 MMA (rank 0), warps 2..9 epilogue
constexpr int kMgStages = 5, kMgStageBytes = 32768;
constexpr int kMgWarpStaging = 8192;  // 32 rows by 64 columns of fp32 per epilogue warp
constexpr int kMgSmem = kMgStages * kMgStageBytes + 8 * kMgWarpStaging + 1024 + 256;
constexpr int kMgTile = 256;

struct MuonProduct {
    int stage, xin, last;
    float a, b, c;
    int a_mn, b_mn;           // operand is read across its rows
    int M, N, kb;             // extents of D, 64-wide blocks of the sum
    int tm, tn, sym;          // tiles along M and N of a matrix
    int tiles;                // of all matrices
    int whole;                // tiles taken whole
    int pairs;
    int cut;                  // pairs that share the blocks of sums of the other tiles (at most as many as blocks)
    int ovec;                 // eight elements along a row of weight and out are aligned
    float* part;              // [pairs][2][2][256][128] sums of parts of tiles
    int* arrived;             // [pairs][2][8] parts of a tile that are there (zero between launches)
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

// Piece i of pair c, or false.  The tiles after the whole ones are `units` blocks
// of sums in a row; pair c < cut takes units c * units / cut .. (c + 1) * units / cut.
__device__ __forceinline__ long long mg_unit0(const MuonProduct& g, int c)
{
    return (long long)(g.tiles - g.whole) * g.kb * min(c, g.cut) / g.cut;
}
__device__ __forceinline__ bool mg_piece(const MuonProduct& g, int c, int i, long long& u, MgPiece& p)
{
    const int own = g.whole / g.pairs;  // whole tiles are whole waves
    if (i < own) {
        p.t = c + i * g.pairs, p.k0 = 0, p.k1 = g.kb;
        return true;
    }
    if (i == own) u = mg_unit0(g, c);
    const long long end = mg_unit0(g, c + 1);
    if (u >= end) return false;
    const int r = (int)(u / g.kb);
    p.t = g.whole + r;
    p.k0 = (int)(u - (long long)r * g.kb);
    p.k1 = (int)min((long long)g.kb, p.k0 + (end - u));
    u += p.k1 - p.k0;
    return true;
}

struct MgTile {
    int b, m, n;  // matrix, tile row and column
};
__device__ __forceinline__ MgTile mg_tile(const MuonProduct& g, int t)
{
    MgTile r;
    const int per = g.sym ? g.tm * (g.tm + 1) / 2 : g.tm * g.tn;
    r.b = t / per;
    const int i = t - r.b * per;
    if (g.sym) {
        int m = (int)((sqrtf(8.f * i + 1.f) - 1.f) * 0.5f);
        while (m * (m + 1) / 2 > i) --m;
        while ((m + 1) * (m + 2) / 2 <= i) ++m;
        r.m = m, r.n = i - m * (m + 1) / 2;
    } else {
        r.n = i / g.tm, r.m = i - r.n * g.tm;
    }
    return r;
}

// 64 finished sums of row i0 + lane, columns j .. j + 63 of matrix b, by one warp.
// Global memory is read and written in rows of 128 bytes (eight lanes a row)
// through the warp's 8 KB of shared memory, whose 16-byte chunks are swizzled by
// the row: row by row from the lanes, a request touched 32 lines and the epilogue
// took longer than the MMAs of a 4096-long sum.  `mirror`: the tile's mirror image
// is written too.
__device__ __forceinline__ void mg_epilogue(const MuonParams& p, const MuonProduct& g, uint8_t* stg, int b, int i0, int j,
                                            bool mirror, float (&v)[64])
{
    const int lane = threadIdx.x & 31, sub = lane >> 3, c8 = lane & 7;
    const int jc = j + 8 * c8;
    if (g.stage < 2) {
        __half* base = (g.stage == 0 ? p.a : p.b) + b * p.ms;
        uint8_t* own = stg + lane * 128;
        uint32_t h[32];
        if (g.stage == 0) {
#pragma unroll
            for (int k = 0; k < 32; ++k) h[k] = pack_half2(v[2 * k] * 0x1p-6f, v[2 * k + 1] * 0x1p-6f);
        } else {
            const __half* src = p.a + b * p.ms + (long long)i0 * p.ldm + jc;
            uint4 x[8];
#pragma unroll
            for (int it = 0; it < 8; ++it) {
                const int r = 4 * it + sub;
                x[it] = make_uint4(0u, 0u, 0u, 0u);
                if (i0 + r < g.M && jc < g.N) x[it] = *reinterpret_cast<const uint4*>(src + (long long)r * p.ldm);
            }
#pragma unroll
            for (int it = 0; it < 8; ++it) {
                const int r = 4 * it + sub;
                *reinterpret_cast<uint4*>(stg + r * 128 + ((c8 ^ (r & 7)) << 4)) = x[it];
            }
            __syncwarp();
            const float c = g.c * 0x1p-10f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint4 y = *reinterpret_cast<const uint4*>(own + ((k ^ c8) << 4));
                const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = unpack_half2(w[e]);
                    h[4 * k + e] = pack_half2(fmaf(g.b, f.x, c * v[8 * k + 2 * e]), fmaf(g.b, f.y, c * v[8 * k + 2 * e + 1]));
                }
            }
            __syncwarp();
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
            *reinterpret_cast<uint4*>(own + ((k ^ c8) << 4)) = make_uint4(h[4 * k], h[4 * k + 1], h[4 * k + 2], h[4 * k + 3]);
        __syncwarp();
        // Rows are padded to eight elements; the padding may be written.
#pragma unroll
        for (int it = 0; it < 8; ++it) {
            const int r = 4 * it + sub;
            const uint4 y = *reinterpret_cast<const uint4*>(stg + r * 128 + ((c8 ^ (r & 7)) << 4));
            if (i0 + r < g.M && jc < g.N) *reinterpret_cast<uint4*>(base + (long long)(i0 + r) * p.ldm + jc) = y;
        }
        if (mirror) {
            // Neighbouring lanes exchange so that each has two rows' values of one column.
            const bool odd = lane & 1;
            const int i2 = i0 + (lane & ~1);
#pragma unroll
            for (int k = 0; k < 32; ++k) {
                const uint32_t other = __shfl_xor_sync(0xffffffffu, h[k], 1);
                const uint32_t w = odd ? __byte_perm(other, h[k], 0x7632) : __byte_perm(h[k], other, 0x5410);
                const int c = j + 2 * k + (odd ? 1 : 0);
                if (c < g.N && i2 < g.M) *reinterpret_cast<uint32_t*>(base + (long long)c * p.ldm + i2) = w;
            }
        }
        __syncwarp();
        return;
    }
#pragma unroll
    for (int k = 0; k < 16; ++k)
        *reinterpret_cast<float4*>(stg + lane * 256 + ((k ^ c8) << 4)) =
            make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
    __syncwarp();
#pragma unroll
    for (int h0 = 0; h0 < 8; h0 += 4) {
        uint4 xh[4], xl[4];
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            const int i = i0 + 4 * (h0 + it) + sub;
            xh[it] = xl[it] = make_uint4(0u, 0u, 0u, 0u);
            if (i < g.M && jc < g.N) {
                const long long e = b * p.xs + (long long)i * p.ldx + jc;
                xh[it] = *reinterpret_cast<const uint4*>(p.x[g.xin] + e);
                xl[it] = *reinterpret_cast<const uint4*>(p.xlo + e);
            }
        }
#pragma unroll
        for (int it = 0; it < 4; ++it) {
            const int r = 4 * (h0 + it) + sub, i = i0 + r;
            float y[8];
            const float4 d0 = *reinterpret_cast<const float4*>(stg + r * 256 + (((2 * c8) ^ (r & 7)) << 4));
            const float4 d1 = *reinterpret_cast<const float4*>(stg + r * 256 + (((2 * c8 + 1) ^ (r & 7)) << 4));
            const float d[8] = {d0.x, d0.y, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w};
            const uint32_t wh[4] = {xh[it].x, xh[it].y, xh[it].z, xh[it].w}, wl[4] = {xl[it].x, xl[it].y, xl[it].z, xl[it].w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float2 h = unpack_half2(wh[q]), l = unpack_half2(wl[q]);
                y[2 * q] = fmaf(g.a, h.x + l.x, d[2 * q] * 0x1p-10f);
                y[2 * q + 1] = fmaf(g.a, h.y + l.y, d[2 * q + 1] * 0x1p-10f);
            }
            if (i >= g.M || jc >= g.N) continue;
            if (!g.last) {
                const long long e = b * p.xs + (long long)i * p.ldx + jc;
                uint4 h, l;
                split8<false>(y, &h, &l);
                *reinterpret_cast<uint4*>(p.x[g.xin ^ 1] + e) = h;
                *reinterpret_cast<uint4*>(p.xlo + e) = l;
                continue;
            }
            const long long o = (long long)b * p.bs + i * p.ld + jc;
#pragma unroll
            for (int q = 0; q < 8; ++q) y[q] *= p.scale * (1.f / kMuonXScale);
            if (g.ovec) {
                muon_finish8(p, o, y);
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (jc + q < g.N) muon_finish(p, o + q, y[q]);
            }
        }
    }
    __syncwarp();
}

__global__ void __launch_bounds__(kMgThreads, 1)
    muon_product_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                        const __grid_constant__ MuonParams p, const __grid_constant__ MuonProduct g)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align_shared<uint8_t>(smem_raw, 1024);
    uint8_t* staging = smem + kMgStages * kMgStageBytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(staging + 8 * kMgWarpStaging);      // [stages], rank 0's count
    uint64_t* empty = full + kMgStages;                                             // [stages]
    uint64_t* accf = empty + kMgStages;                                             // [2] sums complete
    uint64_t* acce = accf + 2;                                                      // [2] sums read (rank 0's count)
    uint32_t* tslot = reinterpret_cast<uint32_t*>(acce + 2);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank(), pair = blockIdx.x >> 1;

    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&ta);
        tma_prefetch_desc(&tb);
        for (int i = 0; i < kMgStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&accf[i], 1);
            mbar_init(&acce[i], 16);
        }
        fence_mbar_init();
    }
    if (warp == 1) {
        pdl_wait();  // tensor memory may still be held by the kernel before this one
        tmem_alloc_pair(tslot, 512);
        tc_fence_before();
    }
    cluster_sync_all();  // both CTAs' barriers are initialised and both hold tensor memory
    tc_fence_after();
    const uint32_t tbase = *tslot;
    pdl_wait();

    if (warp == 0) {
        if (lane == 0) {
            const uint32_t full0 = mapa_shared(smem_u32(&full[0]), 0u);
            int st = 0;
            uint32_t ph = 0;
            bool ok = true;
            long long u = 0;
            MgPiece w;
            for (int i = 0; ok && mg_piece(g, pair, i, u, w); ++i) {
                const MgTile t = mg_tile(g, w.t);
                const int m0 = t.m * kMgTile + rank * 128, n0 = t.n * kMgTile + rank * 128;
                for (int k = w.k0; k < w.k1; ++k) {
                    if (!mbar_wait(&empty[st], ph ^ 1u)) {
                        ok = false;
                        break;
                    }
                    uint8_t* s = smem + st * kMgStageBytes;
                    const uint32_t bar = full0 + (uint32_t)(st * 8);
                    if (rank == 0) mbar_arrive_expect_tx(&full[st], 2 * kMgStageBytes);
                    if (g.a_mn) {
                        tma_load_3d_pair(s, &ta, bar, m0, k * 64, t.b);
                        tma_load_3d_pair(s + 8192, &ta, bar, m0 + 64, k * 64, t.b);
                    } else {
                        tma_load_3d_pair(s, &ta, bar, k * 64, m0, t.b);
                    }
                    if (g.b_mn) {
                        tma_load_3d_pair(s + 16384, &tb, bar, n0, k * 64, t.b);
                        tma_load_3d_pair(s + 16384 + 8192, &tb, bar, n0 + 64, k * 64, t.b);
                    } else {
                        tma_load_3d_pair(s + 16384, &tb, bar, k * 64, n0, t.b);
                    }
                    if (++st == kMgStages) st = 0, ph ^= 1u;
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            const uint32_t idesc = make_idesc_f16(false, g.a_mn, g.b_mn, 256, 256);
            const uint32_t sbase = smem_u32(smem);
            const uint64_t ad = make_sdesc(sbase, g.a_mn ? 8192u : 16u, 1024u, 2u, 0u);
            const uint64_t bd = make_sdesc(sbase + 16384u, g.b_mn ? 8192u : 16u, 1024u, 2u, 0u);
            const uint64_t ak = g.a_mn ? 128 : 2, bk = g.b_mn ? 128 : 2;
            int st = 0;
            uint32_t ph = 0;
            bool ok = true;
            long long u = 0;
            MgPiece w;
            for (int i = 0; ok && mg_piece(g, pair, i, u, w); ++i) {
                const int buf = i & 1;
                if (!mbar_wait(&acce[buf], ((uint32_t)(i >> 1) & 1u) ^ 1u)) break;
                tc_fence_after();
                const uint32_t d = tbase + (uint32_t)(buf * 256);
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
        // Warp e of the epilogue: 32 rows (its tensor-memory quadrant) by half of the columns.
        const int e = warp - 2, q = warp & 3, half = e >> 2;
        const uint32_t acce0 = mapa_shared(smem_u32(&acce[0]), 0u);
        const uint32_t trow = tbase + ((uint32_t)(q * 32) << 16) + (uint32_t)(half * 128);
        const int row = q * 32 + lane;
        long long u = 0;
        MgPiece w;
        for (int i = 0; mg_piece(g, pair, i, u, w); ++i) {
            const int buf = i & 1;
            const MgTile t = mg_tile(g, w.t);
            if (!mbar_wait_sleep(&accf[buf], (uint32_t)(i >> 1) & 1u)) break;
            __syncwarp();
            tc_fence_after();
            const bool whole = w.k0 == 0 && w.k1 == g.kb;
            int c0 = pair, c1 = pair;
            bool finish = true;
            const size_t slot = (size_t)2 * 256 * 128;  // floats of a part: both ranks
            const size_t mine = (size_t)rank * 256 * 128 + (size_t)(half * 128) * 128 + row;
            if (!whole) {
                // Leave this part's sums (columns of 128 rows: coalesced), and see whether it is the last.
                float* out = g.part + (size_t)(2 * pair + (w.k0 ? 0 : 1)) * slot + mine;
#pragma unroll 1
                for (int ch = 0; ch < 4; ++ch) {
                    float v[32];
                    gram_ld<32>(trow + (uint32_t)(buf * 256 + ch * 32), v);
#pragma unroll
                    for (int k = 0; k < 32; ++k) __stcg(out + (ch * 32 + k) * 128, v[k]);
                }
                const long long units = (long long)(g.tiles - g.whole) * g.kb, u0 = (long long)(w.t - g.whole) * g.kb;
                c0 = (int)(((u0 + 1) * g.cut + units - 1) / units) - 1;
                c1 = (int)(((u0 + g.kb) * g.cut + units - 1) / units) - 1;
                __threadfence();
                __syncwarp();
                int* count = g.arrived + ((w.t - g.whole) * 2 + rank) * 8 + e;
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
                for (int ch = 0; ch < 2; ++ch) {
                    float v[64];
                    if (whole) {
                        gram_ld<64>(trow + (uint32_t)(buf * 256 + ch * 64), v);
                    } else {
#pragma unroll
                        for (int k = 0; k < 64; ++k) v[k] = 0.f;
                        for (int c = c0; c <= c1; ++c) {
                            const float* in = g.part + (size_t)(2 * c + (c == c0 ? 1 : 0)) * slot + mine;
#pragma unroll
                            for (int k = 0; k < 64; ++k) v[k] += __ldcg(in + (ch * 64 + k) * 128);
                        }
                    }
                    mg_epilogue(p, g, staging + e * kMgWarpStaging, t.b, t.m * kMgTile + rank * 128 + q * 32,
                                t.n * kMgTile + half * 128 + ch * 64, g.sym && t.m != t.n, v);
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
        tmem_dealloc_pair(tbase, 512);
    }
}

}  // namespace wg
