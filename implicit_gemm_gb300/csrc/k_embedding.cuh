// Embedding lookup and the gradient of the embedding table.
//
//   lookup:    out[t, :]    = scale * table[token[t], :]
//   gradient:  dtable[v, :] = scale * sum over the t with token[t] = v of dy[t, :]
//
// The gradient runs in two kernels, without atomics on data:
//
//  emb_sort_kernel    a stable counting sort of the positions by token.  Every CTA
//                     owns a range of table rows and reads all tokens (a broadcast
//                     from L2: 256 KB for 65,536 tokens), counts those of its rows
//                     per warp (each warp a contiguous range of positions), and
//                     writes its rows' positions in ascending order; the tokens
//                     below its range are its place in the list, so CTAs need
//                     nothing from each other.  It also writes the zeros of the
//                     rows that no token names.
//  emb_reduce_kernel  a segmented sum over the sorted list: a warp takes W entries
//                     (a window) by 256 columns.  A run of at most 2 W entries is
//                     summed by the warp of the window it starts in, to its end;
//                     a longer one leaves an fp32 partial row per window, and the
//                     partial rows of 16 windows, then of 16 such groups and so on,
//                     are added in order by whichever warp brings the last of them.
//                     So no warp has more than 3 W entries, however often a token
//                     occurs, and the order of every sum is fixed.
#pragma once

#include "ptx.cuh"
#include "vec.cuh"

namespace wg {

struct EmbParams {
    long long T;  // tokens
    int V, D;     // table rows, row length
    long long ld_table, ld_out;
    const void* token;
    int token64;
    int padding;
    float scale;
    const void* in;  // table (lookup) or dy (gradient)
    void* out;       // out (lookup) or dtable (gradient)
    int accumulate;
    int R;          // table rows of a CTA of emb_sort_kernel
    int keep;       // matches that a warp of it keeps from the count
    int W;          // entries of a window: 8, 16 or 32
    int tiles;      // 256-column tiles of a row
    int level[8];   // first partial row of a level: windows, groups of 16 of them, ...
    int narrived;   // counters
    int* meta;      // [0] entries of the list
    int* count;     // [V] occurrences of a row's token
    int* start;     // [V] first entry of its run
    int* list;      // [T] positions, by (row, position)
    int* row;       // [T] their rows
    float* part;    // [level rows][2][D] partial rows: of a run from before the child, of a run that starts in it
    int* arrived;   // [level rows][2][tiles] partial rows of a run that are there, counted at its first child of a group
};

// The token at position t as a table row, or -1 when it is out of range.
__device__ __forceinline__ int emb_token(const EmbParams& p, long long t)
{
    if (p.token64) {
        const long long v = static_cast<const long long*>(p.token)[t];
        return v >= 0 && v < p.V ? (int)v : -1;
    }
    const int v = static_cast<const int*>(p.token)[t];
    return v >= 0 && v < p.V ? v : -1;
}

template <typename TT, typename TO, int VEC>
__global__ void __launch_bounds__(256) emb_lookup_kernel(const __grid_constant__ EmbParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    const long long nv = p.D / VEC, n = p.T * nv;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
        const long long t = i / nv;
        const int c = (int)(i - t * nv) * VEC;
        const int v = emb_token(p, t);
        float f[VEC] = {};
        if (v >= 0)
            load_f32<TT, VEC>(static_cast<const TT*>(p.in) + v * p.ld_table + c, f);
        else if (c == 0)
            atomicOr(&g_status, kStatusBadToken);
#pragma unroll
        for (int k = 0; k < VEC; ++k) f[k] *= p.scale;
        store_f32<TO, VEC>(static_cast<TO*>(p.out) + t * p.ld_out + c, f);
    }
}

constexpr int kEmbSortThreads = 1024, kEmbSortWarps = kEmbSortThreads / 32;
constexpr int kEmbSortMaxRows = 1472;     // 32 counters of 4 bytes a row: 184 KB of shared memory
constexpr int kEmbSortRowBits = 11;       // a row of the range in a kept match
constexpr int kEmbSortMaxSmem = 220 << 10;  // counters and kept matches
constexpr int kEmbTile = 256, kEmbFan = 16;

// n elements of zero from any element-aligned address, by one warp.
template <typename T>
__device__ __forceinline__ void emb_zero_row(T* row, int n, int lane)
{
    const int head = min(n, (int)((16u - ((unsigned)reinterpret_cast<uintptr_t>(row) & 15u)) & 15u) / (int)sizeof(T));
    const int body = (n - head) * (int)sizeof(T) / 16, tail = head + body * (16 / (int)sizeof(T));
    if (lane < head) row[lane] = from_f32<T>(0.f);
    uint4* q = reinterpret_cast<uint4*>(row + head);
    for (int i = lane; i < body; i += 32) q[i] = make_uint4(0u, 0u, 0u, 0u);
    if (tail + lane < n) row[tail + lane] = from_f32<T>(0.f);
}

// Block-wide exclusive sum of one value per thread (1024 threads); *total gets the sum.
__device__ __forceinline__ int block_exclusive_1024(int v, int* total)
{
    __shared__ int wsum[kEmbSortWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    int w = wsum[lane], s = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    *total = __shfl_sync(0xffffffffu, s, 31);
    return x - v + __shfl_sync(0xffffffffu, s - w, warp);
}

template <typename TG>
__global__ void __launch_bounds__(kEmbSortThreads, 1) emb_sort_kernel(const __grid_constant__ EmbParams p)
{
    // [warps][R]: counts, then each warp's next entry of a row; [warps][keep]: matches
    // (position in the warp's range, row of the CTA's range).
    extern __shared__ int hist[];
    __shared__ int first[kEmbSortMaxRows];
    const int R = p.R, lo = blockIdx.x * R, nr = min(R, p.V - lo);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_launch_dependents();
    for (int i = threadIdx.x; i < kEmbSortWarps * R; i += kEmbSortThreads) hist[i] = 0;
    __syncthreads();
    pdl_wait();
    int* mine = hist + warp * R;
    for (int i = blockIdx.x * kEmbSortThreads + threadIdx.x; i < p.narrived; i += gridDim.x * kEmbSortThreads)
        p.arrived[i] = 0;
    // Each warp's positions: a multiple of 32.  Eight loads per lane are in flight at
    // a time (one at a time their latency alone took 30 us for 65,536 tokens).
    constexpr int kAhead = 8;
    const long long per = (p.T + 32 * kEmbSortWarps - 1) / (32 * kEmbSortWarps) * 32;
    const long long t0 = min(p.T, warp * per), t1 = min(p.T, t0 + per);
    unsigned* keep = reinterpret_cast<unsigned*>(hist + kEmbSortWarps * R) + warp * p.keep;
    const int cap = per < (1LL << (32 - kEmbSortRowBits)) ? p.keep : 0;
    int below = 0, kept = 0;
    bool bad = false;
    auto take = [&](int at, unsigned r, bool in) {  // 32 positions from t0 + at
        const unsigned who = __ballot_sync(0xffffffffu, in);
        if (!who) return;
        if (in) {
            const int k = kept + __popc(who & ((1u << lane) - 1u));
            atomicAdd(&mine[r], 1);
            if (k < cap) keep[k] = (unsigned)(at + lane) << kEmbSortRowBits | r;
        }
        kept += __popc(who);
    };
    long long t = t0;
    if (!p.token64 && p.padding < 0) {
        const int* tok = static_cast<const int*>(p.token) + lane;
        for (; t + 32 * kAhead <= t1; t += 32 * kAhead) {
            int v[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) v[k] = tok[t + 32 * k];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                // (A token out of range is a large unsigned number: neither below nor in the range.)
                const unsigned r = (unsigned)v[k] - (unsigned)lo;
                if ((unsigned)v[k] < (unsigned)lo) ++below;
                take((int)(t - t0) + 32 * k, r, r < (unsigned)nr);
            }
            if (blockIdx.x == 0)
#pragma unroll
                for (int k = 0; k < kAhead; ++k) bad |= (unsigned)v[k] >= (unsigned)p.V;
        }
    }
    for (; t < t1; t += 32) {
        const int v = t + lane < t1 ? emb_token(p, t + lane) : -2;
        const unsigned r = (unsigned)v - (unsigned)lo;
        bad |= v == -1;
        if ((unsigned)v < (unsigned)lo && v != p.padding) ++below;
        take((int)(t - t0), r, r < (unsigned)nr && v != p.padding);
    }
    if (blockIdx.x == 0 && bad) atomicOr(&g_status, kStatusBadToken);
    int base, total;
    block_exclusive_1024(below, &base);  // (its barriers also complete the counts)
    // Two rows of the range per thread: their sizes, first entries and each warp's place in them.
    int n[2], own = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int r = threadIdx.x + k * kEmbSortThreads;
        n[k] = 0;
        if (r < nr)
#pragma unroll 8
            for (int w = 0; w < kEmbSortWarps; ++w) n[k] += hist[w * R + r];
    }
    int at[2];
    at[0] = base + block_exclusive_1024(n[0], &own);
    at[1] = base + own + block_exclusive_1024(n[1], &total);
    total += own;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int r = threadIdx.x + k * kEmbSortThreads;
        if (r < nr) {
            p.count[lo + r] = n[k];
            p.start[lo + r] = at[k];
            first[r] = n[k];
            int o = at[k];
            if (n[k])
#pragma unroll 8
                for (int w = 0; w < kEmbSortWarps; ++w) {
                    const int c = hist[w * R + r];
                    hist[w * R + r] = o;
                    o += c;
                }
        }
    }
    if (threadIdx.x == 0 && blockIdx.x == gridDim.x - 1) p.meta[0] = base + total;
    __syncthreads();
    // The matches in order; equal rows of 32 of them take consecutive entries.
    auto place = [&](bool in, long long t, int r) {
        const unsigned who = __ballot_sync(0xffffffffu, in);
        if (in) {
            const unsigned same = __match_any_sync(who, r);
            const int rank = __popc(same & ((1u << lane) - 1u));
            const int e = mine[r] + rank;
            p.list[e] = (int)t;
            p.row[e] = lo + r;
            __syncwarp(who);
            if (rank == 0) mine[r] += __popc(same);
        }
        __syncwarp();
    };
    if (kept <= cap) {
        for (int i = 0; i < kept; i += 32) {
            const bool in = i + lane < kept;
            const unsigned m = in ? keep[i + lane] : 0u;
            place(in, t0 + (m >> kEmbSortRowBits), (int)(m & ((1u << kEmbSortRowBits) - 1u)));
        }
    } else {  // more than were kept (many tokens for a small table): the positions again
        for (long long t = t0; t < t1; t += 128) {
            int v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[k] = t + 32 * k + lane < t1 ? emb_token(p, t + 32 * k + lane) : -1;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const bool in = v[k] >= 0 && v[k] != p.padding && (unsigned)(v[k] - lo) < (unsigned)nr;
                if (__any_sync(0xffffffffu, in)) place(in, t + 32 * k + lane, v[k] - lo);
            }
        }
    }
    // Zeros of the rows without a token: a warp per row.
    if (!p.accumulate)
        for (int r = warp; r < nr; r += kEmbSortWarps)
            if (!first[r]) emb_zero_row(static_cast<TG*>(p.out) + (long long)(lo + r) * p.ld_table, p.D, lane);
}

// A finished row's 256 columns: scaled, added to what is there when accumulating, rounded.
template <typename TG, int VEC>
__device__ __forceinline__ void emb_write(const EmbParams& p, int v, int c0, const float (&s)[8])
{
    TG* out = static_cast<TG*>(p.out) + v * p.ld_table;
#pragma unroll
    for (int j = 0; j < 8 / VEC; ++j) {
        const int c = c0 + j * 32 * VEC;
        if (c >= p.D) continue;
        float f[VEC];
        if (p.accumulate) {
            load_f32<TG, VEC>(out + c, f);
#pragma unroll
            for (int k = 0; k < VEC; ++k) f[k] += p.scale * s[j * VEC + k];
        } else {
#pragma unroll
            for (int k = 0; k < VEC; ++k) f[k] = p.scale * s[j * VEC + k];
        }
        store_f32<TG, VEC>(out + c, f);
    }
}

// The partial row (one tile of it, in s) of a run that begins at entry `start` and
// has n entries, from window w: kept, and added to its neighbours' by the warp that
// finds all of a group there.
template <typename TG, int VEC>
__device__ __forceinline__ void emb_join(const EmbParams& p, int v, int w, int tile, float (&s)[8])
{
    constexpr int NV = 8 / VEC;
    const int lane = threadIdx.x & 31, c0 = tile * kEmbTile + lane * VEC;
    const int start = p.start[v];
    int a = start / p.W, b = (start + p.count[v] - 1) / p.W, child = w;
    for (int l = 0;; ++l) {
        const long long base = p.level[l];
        float* q = p.part + ((base + child) * 2 + (child == a ? 1 : 0)) * p.D;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = c0 + j * 32 * VEC;
            float g[VEC];
#pragma unroll
            for (int x = 0; x < VEC; ++x) g[x] = s[j * VEC + x];
            if (c < p.D) store_f32<float, VEC>(q + c, g);
        }
        __threadfence();
        __syncwarp();
        const int group = child / kEmbFan;
        const int first = max(a, group * kEmbFan), last = min(b, group * kEmbFan + kEmbFan - 1);
        int seen = 0;
        if (lane == 0) seen = atomicAdd(&p.arrived[((base + first) * 2 + (first == a ? 1 : 0)) * p.tiles + tile], 1);
        if (__shfl_sync(0xffffffffu, seen, 0) != last - first) return;
        __threadfence();
#pragma unroll
        for (int x = 0; x < 8; ++x) s[x] = 0.f;
        for (int h = first; h <= last; h += 4) {
            float f[4][8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int c = min(h + k, last);
                const float* in = p.part + ((base + c) * 2 + (c == a ? 1 : 0)) * p.D;
#pragma unroll
                for (int j = 0; j < NV; ++j)
#pragma unroll
                    for (int x = 0; x < VEC; ++x) f[k][j * VEC + x] = __ldcg(in + min(c0 + j * 32 * VEC + x, p.D - 1));
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (h + k <= last)
#pragma unroll
                    for (int x = 0; x < 8; ++x) s[x] += f[k][x];
        }
        if (a / kEmbFan == b / kEmbFan) {
            emb_write<TG, VEC>(p, v, c0, s);
            return;
        }
        a /= kEmbFan, b /= kEmbFan, child = group;
    }
}

// Rows of dy come into a ring of shared memory per warp, two batches of 4 KB, by
// bulk copies: 24 warps on an SM have 192 KB on their way with few registers.
// (Loads into registers, eight rows per warp ahead, left the kernel waiting for
// memory two thirds of the time: 94 us for 65,536 rows of 2,048.)  A row piece that
// does not start or end at 16 bytes is copied with what surrounds it, unless that
// lies outside dy: then the warp loads it itself.
template <typename TY, int VEC>
struct EmbRing {
    static constexpr int kPiece = kEmbTile * (int)sizeof(TY) + (VEC == 1 ? 16 : 0);
    static constexpr int kBatch = 4096 / (kEmbTile * (int)sizeof(TY));
    static constexpr int kBytes = 2 * kBatch * kPiece;
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

template <typename TG, typename TY, int VEC>
__global__ void __launch_bounds__(256, 3) emb_reduce_kernel(const __grid_constant__ EmbParams p)
{
    typedef EmbRing<TY, VEC> Ring;
    constexpr int B = Ring::kBatch, SZ = (int)sizeof(TY);
    extern __shared__ __align__(16) uint8_t rings[];
    __shared__ uint64_t bars[8][2];
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = p.W;
    uint8_t* ring = rings + warp * Ring::kBytes;
    uint64_t* bar = bars[warp];
    if (lane == 0) {
        mbar_init(&bar[0], 1);
        mbar_init(&bar[1], 1);
        fence_mbar_init();
    }
    __syncwarp();
    const long long item = (long long)blockIdx.x * (blockDim.x >> 5) + warp;
    const int w = (int)(item / p.tiles), tile = (int)(item - (long long)w * p.tiles);
    pdl_wait();
    // Three times 32 entries from the window's first on, their rows and positions, asked
    // for before it is known how many of them there are (what lies past the list's end is
    // within its memory, and not used).
    const int e0 = w * W, last_t = (int)p.T - 1;
    int pos[3], row[3];
#pragma unroll
    for (int c = 0; c < 3; ++c) {
        const int i = min(e0 + 32 * c + lane, last_t);
        pos[c] = p.list[i], row[c] = p.row[i];
    }
    const int before = e0 > 0 ? p.row[e0 - 1] : -1;
    const int n = p.meta[0];
    if (e0 >= n) return;
    const int m = min(W, n - e0);
    // The runs that cross the window's borders.
    const int head = __shfl_sync(0xffffffffu, row[0], 0), tail = __shfl_sync(0xffffffffu, row[0], m - 1);
    const int row32 = __shfl_sync(0xffffffffu, row[1], 0);
    const int next = e0 + m < n ? (m < 32 ? __shfl_sync(0xffffffffu, row[0], m & 31) : row32) : -1;
    const int nhead = head == before ? p.count[head] : 0, ntail = tail == next ? p.count[tail] : 0;
    const bool entered = nhead > 2 * W, leaves = ntail > 2 * W;  // long runs that cross
    int b = 0, e = m;  // this warp's entries, from e0 on
    if (nhead && !entered) b = __popc(__ballot_sync(0xffffffffu, lane < m && row[0] == head));  // an earlier window's run
    if (ntail && !leaves && b < e)  // this window's run, to its end
        e = m - __popc(__ballot_sync(0xffffffffu, lane < m && row[0] == tail)) + ntail;
    if (b >= e) return;
    unsigned ends[3];  // where runs end
#pragma unroll
    for (int c = 0; c < 3; ++c) {
        int after = __shfl_down_sync(0xffffffffu, row[c], 1);
        const int over = c < 2 ? __shfl_sync(0xffffffffu, row[c < 2 ? c + 1 : 2], 0) : -1;
        if (lane == 31) after = over;
        ends[c] = __ballot_sync(0xffffffffu, after != row[c] || 32 * c + lane == e - 1);
    }
    const int col0 = tile * kEmbTile, ncol = min(kEmbTile, p.D - col0);
    const TY* dy = static_cast<const TY*>(p.in) + col0;
    const uintptr_t dy0 = reinterpret_cast<uintptr_t>(p.in);
    const uintptr_t dy1 = dy0 + (uintptr_t)((p.T - 1) * p.ld_out + p.D) * SZ;
    // Batches are aligned to the window: the first may begin at b.
    const int q0 = b / B, q1 = (e + B - 1) / B;
    auto pick = [&](const int (&x)[3], int i) {  // entry i's
        const int y = i < 32 ? x[0] : i < 64 ? x[1] : x[2];
        return __shfl_sync(0xffffffffu, y, i & 31);
    };
    auto outside = [&](uintptr_t a) {  // the piece at a cannot be copied
        return VEC == 1 && ((a & ~(uintptr_t)15) < dy0 || ((a + ncol * SZ + 15) & ~(uintptr_t)15) > dy1);
    };
    auto issue = [&](int q) {
        if (q >= q1) return;
        const int i = q * B + lane;
        const int y = q * B < 32 ? pos[0] : q * B < 64 ? pos[1] : pos[2];
        const long long t = __shfl_sync(0xffffffffu, y, i & 31);
        const uintptr_t a = reinterpret_cast<uintptr_t>(dy + t * p.ld_out), lo = a & ~(uintptr_t)15;
        uint32_t bytes = (uint32_t)(((a + ncol * SZ + 15) & ~(uintptr_t)15) - lo);
        if (lane >= B || i < b || i >= e || outside(a)) bytes = 0;
        const uint32_t total = __reduce_add_sync(0xffffffffu, bytes);
        if (lane == 0) mbar_arrive_expect_tx(&bar[q & 1], total);
        __syncwarp();
        if (bytes) bulk_load(ring + ((q & 1) * B + lane) * Ring::kPiece, reinterpret_cast<const void*>(lo), bytes, &bar[q & 1]);
    };
    issue(q0);
    issue(q0 + 1);
    const int c0 = col0 + lane * VEC;
    float s[8] = {}, first[8] = {};
    bool partial = entered;  // the run being summed came from before the window
    for (int q = q0; q < q1; ++q) {
        if (!mbar_wait(&bar[q & 1], (uint32_t)((q - q0) >> 1) & 1u)) {
            if (q + 1 < q1) mbar_wait(&bar[(q + 1) & 1], (uint32_t)((q + 1 - q0) >> 1) & 1u);  // copies in flight
            return;
        }
        __syncwarp();
        const unsigned end = (q * B < 32 ? ends[0] : q * B < 64 ? ends[1] : ends[2]) >> (q * B & 31);
#pragma unroll
        for (int a = 0; a < B; ++a) {
            const int i = q * B + a;
            if (i >= e) break;
            if (i < b) continue;
            const uint8_t* piece = ring + ((q & 1) * B + a) * Ring::kPiece;
            if constexpr (VEC == 8) {
                float f[8];
                load_f32<TY, 8>(reinterpret_cast<const TY*>(piece) + lane * 8, f);
#pragma unroll
                for (int x = 0; x < 8; ++x) s[x] += f[x];
            } else {
                const long long t = pick(pos, i);
                const TY* src = dy + t * p.ld_out;
                const uintptr_t at = reinterpret_cast<uintptr_t>(src);
                if (!outside(at)) src = reinterpret_cast<const TY*>(piece + (at & 15u));
#pragma unroll
                for (int x = 0; x < 8; ++x) s[x] += to_f32<TY>(src[min(lane + 32 * x, ncol - 1)]);
            }
            if (!(end >> a & 1u)) continue;
            if (partial) {  // (joined below)
#pragma unroll
                for (int x = 0; x < 8; ++x) first[x] = s[x];
            } else if (leaves && i == e - 1) {
                break;
            } else {
                emb_write<TG, VEC>(p, pick(row, i), c0, s);
            }
#pragma unroll
            for (int x = 0; x < 8; ++x) s[x] = 0.f;
            partial = false;
        }
        __syncwarp();
        issue(q + 2);
    }
    // The partial rows: of the long run that entered, of the one that leaves (unless it is the same).
    const bool through = entered && leaves && head == tail;
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
        if (i == 0 ? !entered : !leaves || through) continue;
        if (i == 0) {
            float x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = s[k], s[k] = first[k], first[k] = x[k];
        } else if (entered) {
#pragma unroll
            for (int k = 0; k < 8; ++k) s[k] = first[k];
        }
        emb_join<TG, VEC>(p, i == 0 ? head : tail, w, tile, s);
    }
}

}  // namespace wg
