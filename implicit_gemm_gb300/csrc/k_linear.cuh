// Products of a layer, for one weight or one per expert and its rows:
//
//   kForward:  y[t, n]  = sum over k of x[t, k] w[e, n, k]          rows t of expert e
//   kData:     dx[t, k] = sum over n of dy[t, n] w[e, n, k]
//   kWeight:   dw[e, n, k] = sum over the rows t of e of dy[t, n] x[t, k]
//
// with the bias, activation, dropout and residual of a layer's tail on the finished sums.
//
// On CTA pairs (tcgen05 .cta_group::2).  The MMA's 256 rows are columns of the result
// (features), its columns are rows of the result (tokens; of dw the n): the number of MMA
// columns is free in steps of 32, so an expert with 40 rows pays for 64 and not for 256.
// Operands are read as they lie, along the sum (K-major) or across it (MN-major):
//
//   MMA rows     w (K-major) / w (MN-major) / x (MN-major)
//   MMA columns  x (K-major) / dy (K-major) / dy (MN-major)
//
// 64 of the sum per stage of the ring; each CTA stages 128 MMA rows and half of the MMA
// columns by TMA and holds 128 x 256 fp32 sums in tensor memory, twice, so that a tile's
// epilogue runs beside the next tile's MMAs.
//
// MMAs add to their sums with truncation (a sum of equal signs over 16 n elements comes
// out short by some 1e-7 n of itself), so a sum is taken `chunk` blocks at a time and
// the chunks are added in registers, rounded to nearest.
//
// A sum over an expert's rows ends inside a block: its last block's rows that belong to
// the next expert are zeroed in shared memory, in both operands (0 times an infinity is
// NaN), by a warp of their own in each CTA, which then hands the block to the MMA warp.
//
// What bounds it: of long sums the MMAs, at the rate of a large library product (a block of 64
// of a 256 x 256 tile 0.31 us on 76 pairs; the bare product of 8192 x 4096 to 16384 544 us alone; with
// gelu_tanh and z, on inputs that change from call to call, 680 at the power cap); of few rows the
// weights' bytes (24 rows of 4096 to 16384 25 us, 5.4 TB/s); of sums below some 16 to 60 blocks the
// epilogue's instructions (15 a result, 24 with silu, 30 with dropout, 44 with gelu and dropout), experts'
// weight gradients among them (64 of 4096 x 2048, 16384 rows in all, to bf16 337 us, 353 with dbias, where
// their 1.3 GB are 190); of small problems some 7 us from launch to end.
//
// Where there are fewer tiles than pairs the sum is cut into `split` parts, whose fp32
// sums go through the workspace to linear_join_kernel, in the order of the parts.
// Nothing waits for another CTA except within the pair, and no atomics touch data.
#pragma once

#include "k_layer.cuh"

namespace wg {

// Four warps that direct (TMA, MMA, fixing, and one that makes up the warpgroup), then the
// epilogue: sixteen warps of 96 registers, or, where sums of several chunks are added up
// in 128 registers of each, eight of 224, which the first four give up of their 168:
// 384 x 168 = 128 x 56 + 256 x 224.  (Nothing may spill: no L1 is left beside the ring, and what
// spills comes back from L2.  Eight warps of 168: 8.5 us a tile where 4 is what its stores take.)
constexpr int kLinDirect = 4, kLinDirectRegs = 56, kLinChunkedRegs = 224;
constexpr int lin_epi_warps(bool chunked) { return chunked ? 8 : 16; }
constexpr int lin_threads(bool chunked) { return 32 * (kLinDirect + lin_epi_warps(chunked)); }
static_assert(384 * 168 >= 128 * kLinDirectRegs + 256 * kLinChunkedRegs && 384 * 168 <= 65536, "registers of a CTA");
constexpr int kLinMaxStages = 12;
constexpr int kLinMaxExperts = 1024;
constexpr int kLinABytes = 16384;
// All the shared memory that a CTA may have (see muon_product_kernel: tensor memory is
// taken before the kernel before this one has ended).
constexpr int kLinSmem = 227 * 1024;
constexpr int kLinRing = (kLinSmem - 2 * 4 * (kLinMaxExperts + 4) - 512 - 1024) / 1024 * 1024;

// Division of numbers below 2^31 by a number that the host knows.  (A division as the kernel runs
// is some twenty instructions one after another; five of them were 1 us before the first load.)
struct FastDiv {
    unsigned mul, shift;
};
inline FastDiv fast_div(unsigned d)
{
    FastDiv f;
    unsigned bits = 0;
    while ((1ull << bits) < d) ++bits;
    f.shift = 31 + bits;
    f.mul = (unsigned)(((1ull << f.shift) + d - 1) / d);
    return f;
}
__device__ __forceinline__ int div_by(int n, const FastDiv& f) { return (int)(((uint64_t)(unsigned)n * f.mul) >> f.shift); }

// Sums of dy's columns over few rows, made by the weight gradient's own epilogue warps while the first tile's
// products run: 64 columns of an expert at a time.  (A kernel of its own before the product costs 2 to 7 us more,
// because the product has to wait for it: what the calls before have written is promised to be seen only by a
// kernel that has waited for them itself.)
struct FewSums {
    const void* dy;
    long long ld;
    void* out;              // [experts][N]
    int dtype, out_dtype, accumulate, vec;
    int across, units;      // of 64 columns, and of all experts; units 0: none
};

struct LinParams {
    LayerTail t;
    int experts;            // 0: one weight, every row
    const void* offsets;    // [experts + 1] rows before each expert's
    int offsets64;
    long long tokens;
    int M, N;               // columns of the result (MMA rows), and rows of it (kWeight) or 0
    int kb;                 // 64-wide blocks of the sum (not kWeight)
    int bf16;
    int bt;                 // most MMA columns of a tile
    FastDiv by_bt, by_im, by_8im, by_per;  // im: tiles along the columns; per: tiles of an expert (kWeight)
    int stages, stage_bytes;
    int chunk;              // blocks per sum in tensor memory
    int split, pairs;
    float* part;            // [split][rows][ldp] sums of parts (split > 1)
    long long ldp, part_rows;
    FewSums few;            // kWeight: dbias of few rows, or none
    SumParams sums;         // kWeight: dbias's parts, joined at the end (of linear_join_kernel where there is one), or none
    int join_blocks;        // of linear_join_kernel, that join parts of the product
};

// ---------------------------------------------------------------- experts' rows
// off[0 .. experts]: the offsets brought into order and into [0, tokens] (a status bit
// tells of any that were not).  Whole block; ends with a barrier.
__device__ __forceinline__ void load_offsets(int experts, const void* offsets, int is64, long long tokens, int* off)
{
    if (experts == 0) {
        if (threadIdx.x == 0) off[0] = 0, off[1] = (int)tokens;
    } else {
        bool bad = false;
        for (int i = threadIdx.x; i <= experts; i += blockDim.x) {
            const long long v = is64 ? static_cast<const long long*>(offsets)[i] : static_cast<const int*>(offsets)[i];
            bad |= v < 0 || v > tokens;
            off[i] = (int)max(0LL, min(tokens, v));
        }
        __syncthreads();
        if (threadIdx.x < 32) {
            int run = 0;
            for (int i0 = 0; i0 <= experts; i0 += 32) {
                const int i = i0 + (int)threadIdx.x;
                const int v = i <= experts ? off[i] : 0;
                int m = v;
#pragma unroll
                for (int d = 1; d < 32; d *= 2) {
                    const int o = __shfl_up_sync(0xffffffffu, m, d);
                    if ((int)threadIdx.x >= d) m = max(m, o);
                }
                m = max(m, run);
                if (i <= experts) {
                    bad |= m > v;
                    off[i] = m;
                }
                run = __shfl_sync(0xffffffffu, m, 31);
            }
        }
        if (bad) atomicOr(&g_status, kStatusBadOffset);
    }
    __syncthreads();
}

// used[0 .. count - 1]: the experts that have rows.  The first warp; the block synchronises after it.
__device__ __forceinline__ int list_used(const int* off, int n, short* used)
{
    const int lane = threadIdx.x & 31;
    int c = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int i = i0 + lane;
        const bool has = i < n && off[i + 1] > off[i];
        const uint32_t b = __ballot_sync(0xffffffffu, has);
        if (has) used[c + __popc(b & ((1u << lane) - 1u))] = (short)i;
        c += __popc(b);
    }
    return c;
}

// The passes over experts' rows, `most` rows at a time: expert and first row of each.  The first warp; the block
// synchronises after it.
__device__ __forceinline__ int list_passes(const int* off, int n, int most, short* expert, int* row)
{
    const int lane = threadIdx.x & 31;
    int run = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int i = i0 + lane, c = i < n ? (off[i + 1] - off[i] + most - 1) / most : 0;
        int a = c;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int o = __shfl_up_sync(0xffffffffu, a, d);
            if (lane >= d) a += o;
        }
        for (int k = 0; k < c; ++k) expert[run + a - c + k] = (short)i, row[run + a - c + k] = off[i] + most * k;
        run += __shfl_sync(0xffffffffu, a, 31);
    }
    return run;
}

// The last i with first[i] <= v, i < n (first ascending, first[0] <= v): empty experts have the
// same first as the one after them, and the one that holds v is the last of those.
__device__ __forceinline__ int find_last(const int* first, int n, int v)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= v)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// ---------------------------------------------------------------- tiles
struct LinTile {
    int e;           // expert
    int m;           // first column of the result
    int n, rows;     // first row of the result (of e's matrix for kWeight), rows
    int wide;        // MMA columns
    int k0, k1;      // blocks of the sum
    int row0, valid; // kWeight: first row of the sum, and rows of its last block (64: nothing to zero)
    int part;
};

// n rows in tiles of at most bt: as even as steps of 32 allow.
__device__ __forceinline__ void lin_width(int n, const LinParams& p, int& tiles, int& width)
{
    tiles = div_by(n + p.bt - 1, p.by_bt);
    width = tiles > 1 ? ((n + tiles - 1) / tiles + 31) / 32 * 32 : max(32, (n + 31) / 32 * 32);
}

template <int KIND>
struct LinWalk {
    const LinParams& p;
    const int *off, *first;
    int im, total, item;
    int tiles, width;  // along the rows (of every expert's matrix for kWeight)
    __device__ __forceinline__ LinWalk(const LinParams& p_, const int* off_, const int* first_, int pair)
        : p(p_), off(off_), first(first_), im((p_.M + 255) / 256), item(pair)
    {
        if (KIND == kWeight) {
            lin_width(p.N, p, tiles, width);
            total = max(p.experts, 1) * im * tiles * p.split;
        } else {
            total = first[max(p.experts, 1)] * im * p.split;
        }
    }
    __device__ __forceinline__ bool next(LinTile& t)
    {
        if (item >= total) return false;
        int i = item, n, kb = p.kb;
        t.part = 0;
        if (p.split > 1) i = item / p.split, t.part = item - i * p.split;
        item += p.pairs;
        t.e = 0;
        if (KIND == kWeight) {
            n = p.N;
            if (p.experts > 1) {
                t.e = div_by(i, p.by_per);
                i -= t.e * im * tiles;
            }
            t.row0 = off[t.e];
            const int rows = off[t.e + 1] - t.row0;
            kb = (rows + 63) >> 6;
            t.valid = rows & 63 ? rows & 63 : 64;
        } else {
            if (p.experts > 1) {
                t.e = find_last(first, p.experts, div_by(i, p.by_im));
                i -= first[t.e] * im;
            }
            n = off[t.e + 1] - off[t.e];
            lin_width(n, p, tiles, width);
        }
        // Eight tiles along the rows, then the columns: what the pairs work on at one time
        // is about as many rows' operands as columns'.
        const int g = div_by(i, p.by_8im), gs = min(8, tiles - 8 * g), in = i - 8 * g * im;
        const int c = gs == 8 ? in >> 3 : gs == 1 ? in : in / gs, j = 8 * g + in - c * gs;
        t.m = 256 * c;
        t.n = j * width;
        t.rows = min(width, n - t.n);
        t.wide = (t.rows + 31) / 32 * 32;
        if (KIND != kWeight) t.n += off[t.e];
        t.k0 = 0, t.k1 = kb;
        if (p.split > 1) {  // (parts below 17, blocks below 2^25)
            t.k0 = (int)((unsigned)kb * (unsigned)t.part / (unsigned)p.split);
            t.k1 = (int)((unsigned)kb * (unsigned)(t.part + 1) / (unsigned)p.split);
        }
        return true;
    }
};

// Arrive on an mbarrier of the cluster and add to the bytes that its phase expects.  The thread
// has written nothing that another one reads, so the arrival orders nothing (as a release it
// waited for the thread's own traffic, and a block took 0.9 us instead of 0.33).
__device__ __forceinline__ void mbar_arrive_expect_tx_cluster(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// Arrive on an mbarrier of the cluster.  The thread's own CTA sees what it has written: enough where
// the next owner is told of tensor memory that has been read.  (A release to the cluster waits
// for the thread's stores to memory, 1 us of a tile of few blocks.)
__device__ __forceinline__ void mbar_arrive_read(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The same, for what the cluster sees.
__device__ __forceinline__ void mbar_arrive_at(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tma_load_3d_at(void* dst, const CUtensorMap* tm, uint32_t bar_cluster, int c0, int c1, int c2)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(c2), "r"(bar_cluster)
        : "memory");
}

// Whether every lane's wait has ended as it should: where one has run out of time the warp stops as one
// (lanes that went on alone would be missed at the next barrier).
__device__ __forceinline__ bool all_waited(bool mine) { return __all_sync(0xffffffffu, mine); }

// 16 consecutive 32-bit columns of this warp's 32 tensor-memory lanes.  Whole warp, converged.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&v)[16])
{
    uint32_t r[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i]);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 "
        "[%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// Eight columns a thread, 64 columns by 4 WARPS rows at a time, several rows in flight; lanes of one column are eight
// apart, and the warps' sums meet in s (64 WARPS floats), in their order.  `tid` of 32 WARPS threads, converged.
template <int WARPS, int MODE>
__device__ __forceinline__ void few_sums_of(const FewSums& p, int N, const int* off, float* s, int tid)
{
    constexpr int kAhead = MODE == kActWide ? 8 : 4, kRows = 4 * WARPS;
    const int lane = tid & 31;
    for (int u = blockIdx.x; u < p.units; u += gridDim.x) {
        const int e = u / p.across, c = 64 * (u - e * p.across), col = c + 8 * (tid & 7), m = min(8, N - col);
        const int r0 = off[e], r1 = off[e + 1];
        float sum[8] = {};
        if (m > 0)
            for (int r = r0 + (tid >> 3); r < r1; r += kAhead * kRows) {
                Raw8 x[kAhead];
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
                    if (r + i * kRows < r1) x[i] = act_load<MODE>(p.dy, r + i * kRows, p.ld, col, m, N, p.dtype, false);
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    if (r + i * kRows >= r1) continue;
                    float v[8];
                    act_ready<MODE>(x[i], p.dy, r + i * kRows, p.ld, col);
                    act_unpack<kActWide>(x[i], p.dtype, v);
                    add8(v, sum);
                }
            }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 8);
            sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], 16);
            if (lane < 8) s[64 * (tid >> 5) + 8 * lane + k] = sum[k];
        }
        asm volatile("bar.sync 2, %0;" ::"n"(32 * WARPS) : "memory");
        if (tid < 64 && c + tid < N && !(p.accumulate && r0 == r1)) {
            float a = s[tid];
            for (int w = 1; w < WARPS; ++w) a += s[64 * w + tid];
            put_sum(p.out, (long long)e * N + c + tid, p.out_dtype, p.accumulate, a);
        }
        asm volatile("bar.sync 2, %0;" ::"n"(32 * WARPS) : "memory");
    }
}

template <int KIND, bool CHUNKED>
__global__ void __launch_bounds__(lin_threads(CHUNKED), 1)
    linear_product_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                          const __grid_constant__ LinParams p)
{
    constexpr bool kAmn = KIND != kForward, kBmn = KIND == kWeight;
    constexpr int kEpiWarps = lin_epi_warps(CHUNKED);
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align_shared<uint8_t>(smem_raw, 1024);
    int* off = reinterpret_cast<int*>(smem + kLinRing);                            // [experts + 1]
    int* first = off + kLinMaxExperts + 4;                                         // [experts + 1] tiles along the rows
    uint64_t* full = reinterpret_cast<uint64_t*>(first + kLinMaxExperts + 4);      // [stages], rank 0's count
    uint64_t* empty = full + kLinMaxStages;                                        // [stages]
    uint64_t* tail = empty + kLinMaxStages;                                        // [stages] a block to be fixed is there
    uint64_t* accf = tail + kLinMaxStages;                                         // [2] sums complete
    uint64_t* acce = accf + 2;                                                     // [2] sums read (rank 0's count)
    uint32_t* tslot = reinterpret_cast<uint32_t*>(acce + 2);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank(), pair = blockIdx.x >> 1;

    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&map_a);
        tma_prefetch_desc(&map_b);
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(&full[i], 2);
            mbar_init(&empty[i], 1);
            mbar_init(&tail[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&accf[i], 1);
            mbar_init(&acce[i], 2 * kEpiWarps);
        }
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(tslot, 512);
        tc_fence_before();
    }
    if (p.experts) pdl_wait();  // the offsets may be the result of the kernel before
    load_offsets(p.experts, p.offsets, p.offsets64, p.tokens, off);
    if (KIND != kWeight) {
        if (warp == 0) {
            const int n = max(p.experts, 1);
            int run = 0;
            for (int i0 = 0; i0 < n; i0 += 32) {
                int tiles = 0, width;
                if (i0 + lane < n) lin_width(off[i0 + lane + 1] - off[i0 + lane], p, tiles, width);
                int s = tiles;
#pragma unroll
                for (int d = 1; d < 32; d *= 2) {
                    const int o = __shfl_up_sync(0xffffffffu, s, d);
                    if (lane >= d) s += o;
                }
                if (i0 + lane < n) first[i0 + lane] = run + s - tiles;
                run += __shfl_sync(0xffffffffu, s, 31);
            }
            if (lane == 0) first[n] = run;
        }
    }
    cluster_sync_all();  // both CTAs' barriers, offsets and tensor memory are there
    tc_fence_after();
    const uint32_t tbase = *tslot;
    LinTile t;
    LinWalk<KIND> walk(p, off, first, pair);
    if (warp < kLinDirect) {
        if (CHUNKED) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLinDirectRegs));
        if (warp == 0) {
            if (lane == 0) {
                const uint32_t full0 = mapa_shared(smem_u32(&full[0]), 0u), mine = mapa_shared(smem_u32(&tail[0]), (uint32_t)rank);
                int st = 0;
                uint32_t ph = 0;
                bool ok = true, more = walk.next(t);
                if (!p.experts) pdl_wait();
                for (; ok && more; more = walk.next(t)) {
                    const int m0 = t.m + rank * 128, n0 = t.n + rank * (t.wide >> 1);
                    for (int k = t.k0; k < t.k1; ++k) {
                        if (!mbar_wait(&empty[st], ph ^ 1u)) {
                            ok = false;
                            break;
                        }
                        uint8_t* s = smem + st * p.stage_bytes;
                        uint32_t bar = full0 + (uint32_t)(st * 8);
                        int kc = 64 * k;
                        if (KIND == kWeight) {
                            if (t.valid < 64 && kc + 64 > off[t.e + 1] - t.row0) bar = mine + (uint32_t)(st * 8);
                            kc += t.row0;
                        }
                        mbar_arrive_expect_tx_cluster(bar, (uint32_t)p.stage_bytes);
                        if (KIND == kForward) {
                            tma_load_3d_at(s, &map_a, bar, kc, m0, t.e);
                        } else {
                            const int b = KIND == kData ? t.e : 0;
                            tma_load_3d_at(s, &map_a, bar, m0, kc, b);
                            tma_load_3d_at(s + 8192, &map_a, bar, m0 + 64, kc, b);
                        }
                        if (kBmn) {
                            tma_load_3d_at(s + kLinABytes, &map_b, bar, n0, kc, 0);
                            if (p.bt > 128) tma_load_3d_at(s + kLinABytes + 8192, &map_b, bar, n0 + 64, kc, 0);
                        } else {
                            tma_load_3d_at(s + kLinABytes, &map_b, bar, kc, n0, 0);
                        }
                        if (++st == p.stages) st = 0, ph ^= 1u;
                    }
                }
            }
            __syncwarp();
        } else if (warp == 1) {
            if (!p.experts) pdl_wait();  // (the waits below are bounded, and the kernel before may take longer)
            if (rank == 0) {
                const uint32_t sbase = smem_u32(smem);
                const uint64_t ad = make_sdesc(sbase, kAmn ? 8192u : 16u, 1024u, 2u, 0u);
                const uint64_t bd = make_sdesc(sbase + (uint32_t)kLinABytes, kBmn ? 8192u : 16u, 1024u, 2u, 0u);
                constexpr uint64_t ak = kAmn ? 128 : 2, bk = kBmn ? 128 : 2;
                int st = 0, use = 0;
                uint32_t ph = 0;
                bool ok = true;
                while (ok && walk.next(t)) {
                    const uint32_t idesc = make_idesc_f16(p.bf16, kAmn, kBmn, 256, t.wide);
                    for (int c0 = t.k0; ok && c0 < t.k1; c0 += p.chunk, ++use) {
                        const int buf = use & 1, c1 = min(t.k1, c0 + p.chunk);
                        if (!all_waited(mbar_wait(&acce[buf], ((uint32_t)(use >> 1) & 1u) ^ 1u))) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t d = tbase + (uint32_t)(buf * 256);
                        for (int k = c0; k < c1; ++k) {
                            if (!all_waited(mbar_wait(&full[st], ph))) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                            int ks1 = 4;
                            if (KIND == kWeight && 64 * k + 64 > off[t.e + 1] - t.row0) ks1 = (t.valid + 15) >> 4;
                            const uint64_t so = (uint64_t)(st * (p.stage_bytes >> 4));
                            if (elect_one()) {
#pragma unroll
                                for (int ks = 0; ks < 4; ++ks)
                                    if (ks < ks1) umma_f16_pair(d, ad + so + ak * ks, bd + so + bk * ks, idesc, (k > c0 || ks) ? 1u : 0u);
                                umma_commit_pair(&empty[st]);
                            }
                            __syncwarp();
                            if (++st == p.stages) st = 0, ph ^= 1u;
                        }
                        if (!ok) break;
                        if (elect_one()) umma_commit_pair(&accf[buf]);
                        __syncwarp();
                    }
                }
            }
        } else if (warp == 2) {
            if (KIND == kWeight) {
                if (!p.experts) pdl_wait();
                // Rows of an expert's last block that are the next one's become zeros.  (A row is
                // one line of 128 bytes per 64 columns, whatever the swizzle does within it.)
                const uint32_t full0 = mapa_shared(smem_u32(&full[0]), 0u);
                int st = 0;
                uint32_t seen = 0;
                bool ok = true;
                while (ok && walk.next(t)) {
                    const int rows = off[t.e + 1] - t.row0, n = t.k1 - t.k0;
                    if (n <= 0) continue;
                    const int last = (st + n - 1) % p.stages;
                    st = (st + n) % p.stages;
                    if (t.valid == 64 || 64 * t.k1 <= rows) continue;
                    ok = all_waited(mbar_wait_sleep(&tail[last], (seen >> last) & 1u));
                    seen ^= 1u << last;
                    if (!ok) break;
                    uint8_t* s = smem + last * p.stage_bytes;
                    const int zeros = ((t.valid + 15) >> 4 << 4) - t.valid;  // rows, of 8 chunks of 16 bytes each
                    for (int c = 0; c < p.stage_bytes >> 13; ++c)
                        for (int i = lane; i < 8 * zeros; i += 32)
                            *reinterpret_cast<uint4*>(s + 8192 * c + 128 * t.valid + 16 * i) = make_uint4(0u, 0u, 0u, 0u);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_at(full0 + (uint32_t)(last * 8));
                    __syncwarp();
                }
            }
        }
    } else {
        if (CHUNKED) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kLinChunkedRegs));
        // Warp e of the epilogue: 32 columns of the result (its tensor-memory quadrant), one
        // per lane, by every kStep / 16th 16 of the tile's rows.  Results go to memory as they
        // come from tensor memory, a row of 32 columns per instruction, whatever their
        // alignment: shared memory has no bandwidth to spare beside the operands (staged
        // through it, a tile's epilogue took 15 us).
        constexpr int kStep = 4 * kEpiWarps, kOwn = 256 / kStep;
        const int e = warp - kLinDirect, q = warp & 3, first_row = 16 * (e >> 2);
        const uint32_t acce0 = mapa_shared(smem_u32(&acce[0]), 0u);
        const uint32_t trow = tbase + ((uint32_t)(q * 32) << 16) + (uint32_t)first_row;
        int use = 0;
        bool ok = true, more = walk.next(t);
        if (!p.experts) pdl_wait();
        const unsigned long long offset = layer_offset(p.t);
        if (KIND == kWeight && p.few.units) {
            float* s = reinterpret_cast<float*>(first);  // (of use to the other kinds only)
            static_assert(64 * kEpiWarps <= kLinMaxExperts + 4, "the warps' sums");
            if (p.few.vec)
                few_sums_of<kEpiWarps, kActWide>(p.few, p.N, off, s, threadIdx.x - 32 * kLinDirect);
            else
                few_sums_of<kEpiWarps, kActShifted>(p.few, p.N, off, s, threadIdx.x - 32 * kLinDirect);
        }
        for (; ok && more; more = walk.next(t)) {
            const int j = t.m + rank * 128 + q * 32 + lane;
            const int rows = j < p.M ? t.rows : 0;  // of this column
            if (p.split == 1) tail_prefetch<KIND>(p.t, t.e, t.n + first_row, rows - first_row, kStep, j);
            if (CHUNKED && t.k1 - t.k0 > p.chunk) {
                // Sums of several chunks are added up in registers, and the total goes back to
                // where the last one was: no register of it is held while what follows is computed.
                float acc[kOwn][16];
                for (int k = t.k0;;) {
                    ok = all_waited(mbar_wait_sleep(&accf[use & 1], (uint32_t)(use >> 1) & 1u));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t tacc = trow + (uint32_t)((use & 1) * 256);
                    if (k == t.k0) {
#pragma unroll
                        for (int i = 0; i < kOwn; ++i)
                            if (first_row + kStep * i < t.wide) tmem_ld16_issue(tacc + kStep * i, reinterpret_cast<uint32_t*>(acc[i]));
                        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                        for (int i = 0; i < kOwn; ++i) reg_fence16(reinterpret_cast<uint32_t*>(acc[i]));
                    } else {
#pragma unroll
                        for (int i = 0; i < kOwn; ++i) {
                            if (first_row + kStep * i < t.wide) {
                                uint32_t r[16];
                                tmem_ld16_issue(tacc + kStep * i, r);
                                asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
                                reg_fence16(r);
#pragma unroll
                                for (int n = 0; n < 16; ++n) acc[i][n] += __uint_as_float(r[n]);
                            }
                        }
                    }
                    k += p.chunk;
                    if (k >= t.k1) {
#pragma unroll
                        for (int i = 0; i < kOwn; ++i)
                            if (first_row + kStep * i < t.wide) tmem_st16(tacc + kStep * i, acc[i]);
                        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                        break;
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_read(acce0 + (uint32_t)((use & 1) * 8));
                    ++use;
                }
            } else if (t.k0 < t.k1) {
                ok = all_waited(mbar_wait_sleep(&accf[use & 1], (uint32_t)(use >> 1) & 1u));
                tc_fence_after();
            }
            if (!ok) break;
            uint32_t tacc = trow + (uint32_t)((use & 1) * 256);
            const auto read_all = [&]() {  // this warp has read its share of the buffer
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_read(acce0 + (uint32_t)((use & 1) * 8));
            };
#pragma unroll 1
            for (int r0 = first_row; r0 < t.rows; r0 += kStep, tacc += kStep) {
                uint32_t r[16];
                if (t.k0 < t.k1) {
                    tmem_ld16_issue(tacc, r);
                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
                    reg_fence16(r);
                    if (r0 + kStep >= t.rows) read_all();
                } else {
#pragma unroll
                    for (int k = 0; k < 16; ++k) r[k] = 0u;
                }
                const long long row = t.n + r0;
                if (p.split == 1) {
                    column_tail<KIND>(p.t, offset, t.e, row, rows - r0, j, r);
                } else {
                    float* o = p.part + ((long long)t.part * p.part_rows + (KIND == kWeight ? (long long)t.e * p.N : 0) + row) * p.ldp + j;
#pragma unroll
                    for (int k = 0; k < 16; ++k, o += p.ldp)
                        if (k < rows - r0) *o = __uint_as_float(r[k]);
                }
            }
            if (t.k0 < t.k1) {
                if (first_row >= t.rows) read_all();
                ++use;
            }
        }
        if (KIND == kWeight && p.split == 1 && p.sums.part && e < 8) {
            // dbias, by the first eight of these warps (the others have few registers): 2 us here, 4 in a launch of its own.
            // The pair's MMAs and loads are over, so the ring is free.
            const auto sync = [] { asm volatile("bar.sync 1, 256;" ::: "memory"); };
            float* s = reinterpret_cast<float*>(smem);
            for (int u = blockIdx.x; u < p.sums.units; u += gridDim.x) {
                column_join<256>(p.sums, threadIdx.x - 32 * kLinDirect, u % p.sums.across, u / p.sums.across, s, sync);
                sync();
            }
        }
    }
    __syncwarp();
    // Neither CTA releases tensor memory or leaves while the other may still use it.
    tc_fence_before();
    cluster_sync_all();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tbase, 512);
    }
}

// ---------------------------------------------------------------- parts of sums
// The parts of each result in order, and what follows: eight columns a thread, eight parts in
// flight (355 x 7274 to 64, in 14 parts, with its product 18.7 us; a part after another 25.7).
constexpr int kJoinBlock = 64;  // (few results, so many blocks)
template <int KIND>
__global__ void __launch_bounds__(kJoinBlock) linear_join_kernel(const __grid_constant__ LinParams p)
{
    __shared__ int off[kLinMaxExperts + 1];
    pdl_launch_dependents();
    pdl_wait();
    if (KIND == kWeight && (int)blockIdx.x >= p.join_blocks) {
        const int u = (int)blockIdx.x - p.join_blocks;
        column_join<kJoinBlock>(p.sums, threadIdx.x, u % p.sums.across, u / p.sums.across, reinterpret_cast<float*>(off), [] { __syncthreads(); });
        return;
    }
    if (KIND != kWeight) load_offsets(p.experts, p.offsets, p.offsets64, p.tokens, off);
    const unsigned long long offset = layer_offset(p.t);
    const int groups = (p.M + 7) / 8, experts = max(p.experts, 1);
    const long long total = p.part_rows * groups, step = (long long)p.join_blocks * blockDim.x;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += step) {
        const long long r = i / groups;
        const int j = 8 * (int)(i - r * groups), n = min(8, p.M - j);
        int e;
        long long row = r;
        if (KIND == kWeight) {
            e = (int)(r / p.N);
            row = r - (long long)e * p.N;
        } else {
            if (r < off[0] || r >= off[experts]) continue;
            e = find_last(off, experts, (int)r);
        }
        TailRead<KIND> rd;
        tail_read<KIND>(p.t, e, row, j, n, rd);
        float v[8] = {};
        const float* q = p.part + r * p.ldp + j;
        const long long between = p.part_rows * p.ldp;
        for (int s = 0; s < p.split; s += 8, q += 8 * between) {  // eight parts in flight
            float4 a[8], b[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (s + k < p.split) {
                    a[k] = __ldcg(reinterpret_cast<const float4*>(q + k * between));
                    b[k] = __ldcg(reinterpret_cast<const float4*>(q + k * between) + 1);
                }
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (s + k < p.split) {
                    v[0] += a[k].x, v[1] += a[k].y, v[2] += a[k].z, v[3] += a[k].w;
                    v[4] += b[k].x, v[5] += b[k].y, v[6] += b[k].z, v[7] += b[k].w;
                }
        }
        tail_write<KIND>(p.t, offset, e, row, j, n, rd, v);
    }
}

// ---------------------------------------------------------------- few rows
// The forward product of at most 8 XR rows of an expert per pass: a pass reads every byte of its expert's
// weights once, and that is what bounds it (one row of 8192 to 8192 24 us, 5.6 TB/s; of 4096 to 4096 9 us, of
// which 3 to 4 are the launch, the first loads and the warps' sums).  A CTA has 8 FG columns of the result (rows of w) of one
// expert; its eight warps take 32 of the sum each in turn, so that a row of w is read in 512
// bytes at a time, straight to registers: MMAs of 16 rows of x by 8 of w by 16, of which a
// lane's operands are 16 consecutive bytes (the sum's terms may come in any order, as long as it is
// one for both operands).  One batch of loads is in flight while the one before is multiplied;
// x's come with them (loaded where they were needed, each waited for L2: 4096 x 4096 for one
// row 14 us).  The warps' sums meet in shared memory, in the order of the warps.
// Passes of one expert are different CTAs' (64 rows of one of 8 experts'
// 2047 x 2048 24 us; one after another 82).
constexpr int kRowsThreads = 256;
constexpr int kRowsMost = 64;  // rows in all, and so passes
struct RowsParams {
    LayerTail t;
    int experts, offsets64;
    const void* offsets;
    long long tokens;
    const void *x, *w;
    long long ldx, ldw, wstride;
    int K, M;                // terms of the sum, columns of the result
};

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if (BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Eight elements k .. k + 7 (k a multiple of 8) of a row of `end` elements, in two steps: as they lie in
// memory, to be in flight, and then in their places, zeros behind the row and of a row that is not
// there.  VEC 8 and 2: rows whose starts and lengths are multiples of VEC, in accesses of VEC elements;
// 1: rows that start anywhere, as the two aligned chunks that hold the eight (7168 rows of 8191
// 50 us; in the pairs around them 100.  8192 rows of 8190 33 us in pairs, 44 in chunks).
template <int VEC>
struct RowsRaw {
    uint4 a;
};
template <>
struct RowsRaw<1> {
    uint4 a, b;
};
template <int VEC>
__device__ __forceinline__ RowsRaw<VEC> rows_load(const unsigned short* row, int k, int end, bool stream)
{
    RowsRaw<VEC> r = {};
    if (!row || k >= end) return r;
    if constexpr (VEC == 8) {
        if (stream)
            asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.a.x), "=r"(r.a.y), "=r"(r.a.z), "=r"(r.a.w) : "l"(row + k));
        else
            r.a = __ldg(reinterpret_cast<const uint4*>(row + k));
    } else if constexpr (VEC == 2) {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(row + k);
        r.a.x = __ldg(p);
        if (k + 2 < end) r.a.y = __ldg(p + 1);
        if (k + 4 < end) r.a.z = __ldg(p + 2);
        if (k + 6 < end) r.a.w = __ldg(p + 3);
    } else {
        const uintptr_t at = reinterpret_cast<uintptr_t>(row + k), c = at & ~(uintptr_t)15;
        r.a = __ldg(reinterpret_cast<const uint4*>(c));
        if (c != at && c + 16 < reinterpret_cast<uintptr_t>(row + end)) r.b = __ldg(reinterpret_cast<const uint4*>(c + 16));
    }
    return r;
}
template <int VEC>
__device__ __forceinline__ uint4 rows_take(const RowsRaw<VEC>& r, const unsigned short* row, int k, int end)
{
    if constexpr (VEC > 1) {
        return r.a;
    } else {
        const uint32_t s = (uint32_t)reinterpret_cast<uintptr_t>(row) & 15u;  // (each row its own)
        const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
        uint32_t v[6], u[5], o[4];
#pragma unroll
        for (int i = 0; i < 6; ++i) v[i] = s & 8u ? w[i + 2] : w[i];
#pragma unroll
        for (int i = 0; i < 5; ++i) u[i] = s & 4u ? v[i + 1] : v[i];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = __funnelshift_r(u[i], u[i + 1], (s & 2u) * 8u);
        if (k + 8 > end) {
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = k + 2 * i + 1 < end ? o[i] : k + 2 * i < end ? o[i] & 0xffffu : 0u;
        }
        return make_uint4(o[0], o[1], o[2], o[3]);
    }
}

template <int XR, int FG, bool BF16, int VEC>
__global__ void __launch_bounds__(kRowsThreads, 2) linear_rows_kernel(const __grid_constant__ RowsParams p)
{
    constexpr int kAhead = VEC == 1 ? 1 : VEC == 8 && XR == 1 && FG == 2 ? 3 : 2;  // steps of a batch: two of them fill 128 registers
    struct Batch {
        RowsRaw<VEC> w[kAhead][FG], x[kAhead][XR];
    };
    __shared__ int off[kLinMaxExperts + 1];
    __shared__ short pass_expert[kRowsMost];
    __shared__ int pass_row[kRowsMost], count;
    __shared__ float sums[8][8 * XR][8 * FG + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
    pdl_launch_dependents();
    pdl_wait();
    if (p.experts == 0) {
        const int i = threadIdx.x, c = ((int)p.tokens + 8 * XR - 1) / (8 * XR);
        if (i < c) pass_expert[i] = 0, pass_row[i] = 8 * XR * i;
        if (i == 0) count = c;
    }
    load_offsets(p.experts, p.offsets, p.offsets64, p.tokens, off);
    if (p.experts) {
        if (warp == 0) {
            const int c = list_passes(off, p.experts, 8 * XR, pass_expert, pass_row);
            if (lane == 0) count = c;
        }
        __syncthreads();
    }
    const unsigned long long offset = layer_offset(p.t);
    const int per = (p.M + 8 * FG - 1) / (8 * FG);
    const int total = count * per;
    for (int item = blockIdx.x; item < total; item += gridDim.x) {
        const int pass = item / per, e = pass_expert[pass], r0 = pass_row[pass], j0 = 8 * FG * (item - pass * per);
        const unsigned short* w = static_cast<const unsigned short*>(p.w) + e * p.wstride;
        const unsigned short* wrow[FG];
#pragma unroll
        for (int f = 0; f < FG; ++f) wrow[f] = j0 + 8 * f + g < p.M ? w + (j0 + 8 * f + g) * p.ldw : nullptr;
        const int rows = min(8 * XR, off[e + 1] - r0);
        const unsigned short* xrow[XR];
#pragma unroll
        for (int m = 0; m < XR; ++m)
            xrow[m] = 8 * m + g < rows ? static_cast<const unsigned short*>(p.x) + (r0 + 8 * m + g) * p.ldx : nullptr;
        float d[FG][4] = {};
        const auto load = [&](Batch& c, int k) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
#pragma unroll
                for (int f = 0; f < FG; ++f) c.w[u][f] = rows_load<VEC>(wrow[f], k + 256 * u + 8 * tig, p.K, true);
#pragma unroll
                for (int m = 0; m < XR; ++m) c.x[u][m] = rows_load<VEC>(xrow[m], k + 256 * u + 8 * tig, p.K, false);
            }
        };
        const auto multiply = [&](const Batch& c, int k) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int at = k + 256 * u + 8 * tig;
                const uint4 x0 = rows_take<VEC>(c.x[u][0], xrow[0], at, p.K);
                const uint4 x1 = XR > 1 ? rows_take<VEC>(c.x[u][XR - 1], xrow[XR - 1], at, p.K) : make_uint4(0u, 0u, 0u, 0u);
                const uint32_t lo[4] = {x0.x, x1.x, x0.y, x1.y}, hi[4] = {x0.z, x1.z, x0.w, x1.w};
#pragma unroll
                for (int f = 0; f < FG; ++f) {
                    const uint4 v = rows_take<VEC>(c.w[u][f], wrow[f], at, p.K);
                    mma16816<BF16>(d[f], lo, v.x, v.y);
                    mma16816<BF16>(d[f], hi, v.z, v.w);
                }
            }
        };
        // The warp's sums so far, to its own place in shared memory: every 64 MMAs (they add with
        // truncation, see above).
        bool begun = false;
        const auto put = [&]() {
#pragma unroll
            for (int f = 0; f < FG; ++f)
#pragma unroll
                for (int i = 0; i < 2 * XR; ++i) {
                    float& s = sums[warp][g + 8 * (i >> 1)][8 * f + 2 * tig + (i & 1)];
                    s = begun ? s + d[f][i] : d[f][i];
                    d[f][i] = 0.f;
                }
            begun = true;
        };
        constexpr int kStep = 256 * kAhead, kPut = 64 / (2 * kAhead) / 2 * 2 * kStep;
        Batch b0, b1;
        int k = 32 * warp, next = k + kPut;
        if (k < p.K) load(b0, k);
        while (k < p.K) {
            if (k >= next) put(), next += kPut;
            if (k + kStep < p.K) load(b1, k + kStep);
            multiply(b0, k);
            if ((k += kStep) >= p.K) break;
            if (k + kStep < p.K) load(b0, k + kStep);
            multiply(b1, k);
            k += kStep;
        }
        put();
        __syncthreads();
        for (int i = threadIdx.x; i < rows * FG; i += kRowsThreads) {
            const int r = i / FG, f = i - r * FG, j = j0 + 8 * f, nc = min(8, p.M - j);
            if (nc <= 0) continue;
            TailRead<kForward> rd;
            tail_read<kForward>(p.t, e, r0 + r, j, nc, rd);
            float v[8] = {};
#pragma unroll
            for (int q = 0; q < 8; ++q)
#pragma unroll
                for (int c = 0; c < 8; ++c) v[c] += sums[q][r][8 * f + c];
            tail_write<kForward>(p.t, offset, e, r0 + r, j, nc, rd, v);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- operands that TMA cannot read
// Rows of 16-bit elements that start anywhere, copied to rows of whole 16-byte chunks: a warp
// per row and 256 columns.  Few of them are bound by their launch, many by HBM's reads and writes (1009 and
// 1515 rows of 1001 3 us beside their product).  (What comes after a row's last column may be anything: TMA gives
// zeros there.)
struct PackParams {
    const unsigned short* in;
    unsigned short* out;
    long long rows, ld, bs;
    int batch, cols, ldp;
    int segments;        // rows by 256 columns, of a matrix (fewer than 2^31 fit any memory)
    FastDiv by_per, by_segments;
};
// b has one matrix; of a's, experts' weights, those are copied whose expert has rows.
__global__ void __launch_bounds__(256) linear_pack_kernel(const __grid_constant__ PackParams a, const __grid_constant__ PackParams b,
                                                          const void* offsets, int is64, long long tokens)
{
    __shared__ int off[kLinMaxExperts + 1];
    __shared__ short used[kLinMaxExperts];
    __shared__ int count;
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    long long matrices = a.batch;
    if (a.batch > 1) {
        load_offsets(a.batch, offsets, is64, tokens, off);
        if (threadIdx.x < 32) {
            const int c = list_used(off, a.batch, used);
            if (lane == 0) count = c;
        }
        __syncthreads();
        matrices = count;
    }
    const long long step = (long long)gridDim.x * (blockDim.x / 32), of_a = matrices * a.segments;
    for (long long i = (long long)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32; i < of_a + b.segments; i += step) {
        const bool first = i < of_a;
        const PackParams& p = first ? a : b;
        int n = (int)(first ? i : i - of_a);
        long long m = 0;
        if (first && a.batch > 1) {
            const int k = div_by(n, a.by_segments);
            n -= k * a.segments;
            m = used[k];
        }
        const long long r = div_by(n, p.by_per);
        const int j = 256 * (n - (int)r * ((p.cols + 255) / 256)) + 8 * lane;
        const uintptr_t row = reinterpret_cast<uintptr_t>(p.in + m * p.bs + r * p.ld), from = row + 2 * (uintptr_t)j;
        const uint4 v = join_shifted(fetch_shifted(from, row + 2 * (uintptr_t)p.cols), from);
        if (j < p.cols) *reinterpret_cast<uint4*>(p.out + (m * p.rows + r) * p.ldp + j) = v;
    }
}

// ---------------------------------------------------------------- bias gradients
// Sums of dy's columns over an expert's rows, `chunk` rows at a time, to part[chunk][N], with how many chunks come
// before each expert's (first, written by one block): column_join adds them up at the end.  (Few rows: FewSums.)
// HBM's reads bound it, eight rows a thread in flight (8192 x 16384 46 us, 5.8 TB/s).
struct ColumnParams {
    const void* dy;
    long long tokens, ld;
    int N, dtype;
    int experts, offsets64;
    const void* offsets;
    int cx_log, chunk;
    float* part;
    int* first;
};
template <int MODE>
__global__ void __launch_bounds__(256, 4) column_sum_kernel(const __grid_constant__ ColumnParams p)
{
    __shared__ int off[kLinMaxExperts + 1], first[kLinMaxExperts + 1];
    constexpr int kAhead = MODE == kActWide ? 8 : 4;  // rows in flight per thread
    __shared__ float s[8][256];
    pdl_launch_dependents();
    pdl_wait();
    load_offsets(p.experts, p.offsets, p.offsets64, p.tokens, off);
    const int n = max(p.experts, 1);
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int run = 0;
        for (int i0 = 0; i0 < n; i0 += 32) {
            const int c = i0 + lane < n ? (off[i0 + lane + 1] - off[i0 + lane] + p.chunk - 1) / p.chunk : 0;
            int a = c;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int o = __shfl_up_sync(0xffffffffu, a, d);
                if (lane >= d) a += o;
            }
            if (i0 + lane < n) first[i0 + lane] = run + a - c;
            run += __shfl_sync(0xffffffffu, a, 31);
        }
        if (lane == 0) first[n] = run;
    }
    __syncthreads();
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int i = threadIdx.x; i <= n; i += 256) p.first[i] = first[i];
    const int cx = 1 << p.cx_log, tx = threadIdx.x & (cx - 1), ty = threadIdx.x >> p.cx_log, ny = 256 >> p.cx_log;
    const int col = 8 * (blockIdx.x * cx + tx), m = min(8, p.N - col);
    for (int c = blockIdx.y; c < first[n]; c += gridDim.y) {
        const int e = find_last(first, n, c);
        const int r0 = off[e] + (c - first[e]) * p.chunk, r1 = min(off[e + 1], r0 + p.chunk);
        float sum[8] = {};
        if (m > 0)
            for (int r = r0 + ty; r < r1; r += kAhead * ny) {
                Raw8 x[kAhead];
#pragma unroll
                for (int i = 0; i < kAhead; ++i)
                    if (r + i * ny < r1) x[i] = act_load<MODE>(p.dy, r + i * ny, p.ld, col, m, p.N, p.dtype, false);
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    if (r + i * ny >= r1) continue;
                    float v[8];
                    act_ready<MODE>(x[i], p.dy, r + i * ny, p.ld, col);
                    act_unpack<kActWide>(x[i], p.dtype, v);
                    add8(v, sum);
                }
            }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 8; ++k) s[k][threadIdx.x] = sum[k];
        __syncthreads();
        for (int i = threadIdx.x; i < 8 * cx; i += 256) {
            const int k = i & 7, x = i >> 3, j = 8 * (blockIdx.x * cx + x) + k;
            float a = 0.f;
            for (int y = 0; y < ny; ++y) a += s[k][(y << p.cx_log) + x];
            if (j < p.N) p.part[(long long)c * p.N + j] = a;
        }
    }
}

}  // namespace wg
