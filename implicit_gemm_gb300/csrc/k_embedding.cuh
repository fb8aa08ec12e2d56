// Embedding lookup and the gradient of the embedding table.
//
//   lookup:    out[t, :]    = scale * table[token[t], :]
//   gradient:  dtable[v, :] = scale * sum over the t with token[t] = v of dy[t, :]
//
// The gradient runs in three kernels, without atomics on data:
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
//                     (a window) by 512 columns.  A run of at most 2 W entries is
//                     summed by the warp of the window it starts in, to its end;
//                     a longer one leaves an fp32 partial row per window.  So no
//                     warp has more than 3 W entries, however often a token occurs.
//  emb_join_kernel    adds the partial rows of the long runs, in the windows' order.
//                     (Joined by whichever warp brought the last partial row instead,
//                     the fences took longer than this kernel does.)
#pragma once

#include <type_traits>

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
    int tiles;      // 512-column tiles of a row
    int* meta;      // [0] entries of the list, [1] long runs that cross windows
    int* count;     // [V] occurrences of a row's token
    int* list;      // [T] positions, by (row, position)
    int* row;       // [T] their rows
    int4* cross;    // (row, first entry, entries, 0) of the long runs that cross windows
    float* part;    // [windows][2][D] partial rows: of a run from before the window, of a run that goes on after it
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

// The same for rows that start anywhere: a warp per row and 256 columns, VEC (1 or 2)
// neighbouring elements per lane and access.  (Element by element over all rows, as
// above, the divisions and one load in flight took 32,768 rows of 2,047 154 us.)
constexpr int kEmbLookCols = 256;
template <typename TT, typename TO, int VEC>
__global__ void __launch_bounds__(256) emb_lookup_any_kernel(const __grid_constant__ EmbParams p)
{
    constexpr int U = kEmbLookCols / (32 * VEC);
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const unsigned tiles = (unsigned)((p.D + kEmbLookCols - 1) / kEmbLookCols);
    const long long n = p.T * tiles;
    for (long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); i < n; i += (long long)gridDim.x * 8) {
        const long long t = n <= 0xffffffffLL ? (unsigned)i / tiles : i / tiles;
        const int tile = (int)(i - t * tiles), c0 = tile * kEmbLookCols + lane * VEC, v = emb_token(p, t);
        if (v < 0 && tile == 0 && lane == 0) atomicOr(&g_status, kStatusBadToken);
        const TT* in = static_cast<const TT*>(p.in) + v * p.ld_table + c0;
        TO* out = static_cast<TO*>(p.out) + t * p.ld_out + c0;
        float f[U][VEC];
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int k = 0; k < VEC; ++k) f[u][k] = 0.f;
            if (v >= 0 && c0 + 32 * VEC * u < p.D) load_f32<TT, VEC>(in + 32 * VEC * u, f[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (c0 + 32 * VEC * u >= p.D) break;
#pragma unroll
            for (int k = 0; k < VEC; ++k) f[u][k] *= p.scale;
            store_f32<TO, VEC>(out + 32 * VEC * u, f[u]);
        }
    }
}

constexpr int kEmbSortThreads = 1024, kEmbSortWarps = kEmbSortThreads / 32;
constexpr int kEmbSortMaxRows = 1472;     // 32 counters of 4 bytes a row: 184 KB of shared memory
constexpr int kEmbSortRowBits = 11;       // a row of the range in a kept match
constexpr int kEmbSortMaxSmem = 220 << 10;  // counters and kept matches
constexpr int kEmbCols = 16, kEmbTile = 32 * kEmbCols;  // columns per lane and per warp

// n elements of zero from any element-aligned address, by one warp.
template <typename T>
__device__ __forceinline__ void emb_zero_row(T* row, int n, int lane)
{
    const int head = min(n, (int)((16u - ((unsigned)reinterpret_cast<uintptr_t>(row) & 15u)) & 15u) / (int)sizeof(T));
    const int body = (n - head) * (int)sizeof(T) / 16, tail = head + body * (16 / (int)sizeof(T));
    if (lane < head) row[lane] = from_f32<T>(0.f);
    uint4* q = reinterpret_cast<uint4*>(row + head);
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    int i = lane;
    for (; i + 96 < body; i += 128) __stcs(q + i, zero), __stcs(q + i + 32, zero), __stcs(q + i + 64, zero), __stcs(q + i + 96, zero);
    for (; i < body; i += 32) __stcs(q + i, zero);
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
    auto scan = [&](auto* token) {
        typedef std::remove_const_t<std::remove_pointer_t<decltype(token)>> I;
        typedef std::make_unsigned_t<I> U;
        token += lane;
        for (; t + 32 * kAhead <= t1; t += 32 * kAhead) {
            I v[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) v[k] = token[t + 32 * k];
            if (blockIdx.x == 0)
#pragma unroll
                for (int k = 0; k < kAhead; ++k) bad |= (U)v[k] >= (U)p.V;
            if (p.padding >= 0)
#pragma unroll
                for (int k = 0; k < kAhead; ++k) v[k] = v[k] == (I)p.padding ? (I)-1 : v[k];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                // (A token out of range is a large unsigned number: neither below nor in the range.)
                const U r = (U)v[k] - (U)lo;
                if ((U)v[k] < (U)lo) ++below;
                take((int)(t - t0) + 32 * k, (unsigned)r, r < (U)nr);
            }
        }
    };
    if (p.token64)
        scan(static_cast<const long long*>(p.token));
    else
        scan(static_cast<const int*>(p.token));
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
    if (threadIdx.x == 0 && blockIdx.x == gridDim.x - 1) p.meta[0] = base + total, p.meta[1] = 0;
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

// A finished row's 512 columns: scaled, added to what is there when accumulating, rounded.
template <typename TG, int VEC>
__device__ __forceinline__ void emb_write(const EmbParams& p, int v, int c0, const float (&s)[kEmbCols])
{
    TG* out = static_cast<TG*>(p.out) + v * p.ld_table;
#pragma unroll
    for (int j = 0; j < kEmbCols / VEC; ++j) {
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

// Rows of dy come into a ring of shared memory per warp, two batches of 4 KB, by
// asynchronous copies: 24 warps on an SM have 192 KB on their way with few
// registers (loads into registers, eight rows per warp ahead, left the kernel
// waiting for memory two thirds of the time: 94 us for 65,536 rows of 2,048), and
// with aligned rows every lane reads back what it copied itself, so nothing waits
// for another lane.  (Bulk copies, one per row and lane, took the kernel three times
// the instructions.)  Rows that start anywhere are copied in the aligned 16-byte
// chunks that hold them (16,001 rows of 999: 19 us, 30 in 4-byte words), unless such a
// chunk lies partly outside dy: then the warp loads the row when it needs it.
template <typename TY, int VEC>
struct EmbRing {
    static constexpr int kPiece = kEmbTile * (int)sizeof(TY) + (VEC == 1 ? 16 : 0);
    static constexpr int kBatch = 4096 / (kEmbTile * (int)sizeof(TY));
    static constexpr int kEntries = 2 * kBatch * kPiece;  // then 96 positions, and 96 rows
    static constexpr int kBytes = kEntries + 96 * 8;
};

__device__ __forceinline__ void async_copy(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the last group of this thread's copies are there.
__device__ __forceinline__ void async_wait_1() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

template <typename TG, typename TY, int VEC>
__global__ void __launch_bounds__(256, 3) emb_reduce_kernel(const __grid_constant__ EmbParams p)
{
    typedef EmbRing<TY, VEC> Ring;
    constexpr int B = Ring::kBatch, SZ = (int)sizeof(TY);
    extern __shared__ __align__(16) uint8_t rings[];
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = p.W;
    uint8_t* ring = rings + warp * Ring::kBytes;
    int* const pos = reinterpret_cast<int*>(ring + Ring::kEntries);
    int* const row = pos + 96;
    const unsigned item = blockIdx.x * (blockDim.x >> 5) + warp;
    const int w = (int)(item / (unsigned)p.tiles), tile = (int)(item - (unsigned)w * p.tiles);
    pdl_wait();
    // Three times 32 entries from the window's first on, their rows and positions, asked
    // for before it is known how many of them there are (what lies past the list's end is
    // within its memory, and not used).
    const int e0 = w * W, last_t = (int)p.T - 1;
    int r[3], head, next;
#pragma unroll
    for (int c = 0; c < 3; ++c) {
        const int i = min(e0 + 32 * c + lane, last_t);
        pos[32 * c + lane] = p.list[i];
        r[c] = p.row[i];
    }
    const int before = e0 > 0 ? p.row[e0 - 1] : -1;
    const int n = p.meta[0];
    if (e0 >= n) return;
#pragma unroll
    for (int c = 0; c < 3; ++c) row[32 * c + lane] = r[c];
    __syncwarp();
    const int m = min(W, n - e0);
    // The runs that cross the window's borders.
    head = row[0], next = e0 + m < n ? row[m] : -1;
    const int tail = row[m - 1];
    const int nhead = head == before ? p.count[head] : 0, ntail = tail == next ? p.count[tail] : 0;
    const bool leaves = ntail > 2 * W;  // a long run that goes on
    bool partial = nhead > 2 * W;       // the run being summed is a long one from before the window
    int b = 0, e = m;                   // this warp's entries, from e0 on
    if (nhead && !partial) b = __popc(__ballot_sync(0xffffffffu, lane < m && r[0] == head));  // an earlier window's run
    if (ntail && !leaves && b < e)  // this window's run, to its end
        e = m - __popc(__ballot_sync(0xffffffffu, lane < m && r[0] == tail)) + ntail;
    if (b >= e) return;
    const int col0 = tile * kEmbTile, ncol = min(kEmbTile, p.D - col0), c0 = col0 + lane * VEC;
    const TY* dy = static_cast<const TY*>(p.in) + col0;
    const uintptr_t dy0 = reinterpret_cast<uintptr_t>(p.in);
    const uintptr_t dy1 = dy0 + (uintptr_t)((p.T - 1) * p.ld_out + p.D) * SZ;
    auto outside = [&](uintptr_t a) {  // the chunks that hold the piece at a are not all in dy
        return VEC == 1 && ((a & ~(uintptr_t)15) < dy0 || ((a + ncol * SZ + 15) & ~(uintptr_t)15) > dy1);
    };
    const uint32_t ring0 = smem_u32(ring);
    // Entries i0 .. i0 + B - 1 (batches are aligned to the window).
    auto issue = [&](int i0) {
        const int lo = max(i0, b), hi = min(i0 + B, e);
#pragma unroll 2
        for (int i = lo; i < hi; ++i) {
            const TY* src = dy + pos[i] * p.ld_out;
            const uint32_t dst = ring0 + (uint32_t)((i & (2 * B - 1)) * Ring::kPiece);
            if constexpr (VEC == 8) {
#pragma unroll
                for (int j = 0; j < kEmbCols / 8; ++j)
                    if (c0 + 256 * j < p.D)
#pragma unroll
                        for (int x = 0; x < SZ / 2; ++x)
                            async_copy(dst + (uint32_t)((256 * j + lane * 8) * SZ + 16 * x),
                                       src + 256 * j + lane * 8 + x * (16 / SZ));
            } else {
                const uintptr_t at = reinterpret_cast<uintptr_t>(src);
                const int chunks = outside(at) ? 0 : (int)((at & 15u) + ncol * SZ + 15) / 16;
                const uint4* chunk = reinterpret_cast<const uint4*>(at & ~(uintptr_t)15);
#pragma unroll
                for (int x = 0; x < Ring::kPiece / 512 + 1; ++x)
                    if (lane + 32 * x < chunks) async_copy(dst + (uint32_t)((lane + 32 * x) * 16), chunk + lane + 32 * x);
            }
        }
        async_commit();  // (an empty group counts too)
    };
    const int q0 = b & ~(B - 1);
    issue(q0);
    issue(q0 + B);
    float s[kEmbCols] = {};
    for (int q = q0; q < e; q += B) {
        async_wait_1();
        if (VEC == 1) __syncwarp();  // other lanes' copies are read
        const int lo = max(q, b), hi = min(q + B, e);
#pragma unroll 1
        for (int i = lo; i < hi; ++i) {
            const uint8_t* piece = ring + (i & (2 * B - 1)) * Ring::kPiece;
            if constexpr (VEC == 8) {
#pragma unroll
                for (int j = 0; j < kEmbCols / 8; ++j) {
                    float f[8];
                    load_f32<TY, 8>(reinterpret_cast<const TY*>(piece) + 256 * j + lane * 8, f);
#pragma unroll
                    for (int x = 0; x < 8; ++x) s[8 * j + x] += f[x];
                }
            } else {
                const TY* src = dy + pos[i] * p.ld_out;
                const uintptr_t at = reinterpret_cast<uintptr_t>(src);
                if (!outside(at)) src = reinterpret_cast<const TY*>(piece + (at & 15u));
#pragma unroll
                for (int x = 0; x < kEmbCols; ++x) s[x] += to_f32<TY>(src[min(lane + 32 * x, ncol - 1)]);
            }
            const int v = row[i];
            if (i + 1 < e && row[i + 1] == v) continue;
            if (partial || (leaves && i == e - 1)) {
                float* q = p.part + ((long long)w * 2 + (partial ? 0 : 1)) * p.D;
#pragma unroll
                for (int j = 0; j < kEmbCols / VEC; ++j) {
                    const int c = c0 + j * 32 * VEC;
                    float g[VEC];
#pragma unroll
                    for (int x = 0; x < VEC; ++x) g[x] = s[j * VEC + x];
                    if (c < p.D) store_f32<float, VEC>(q + c, g);
                }
                // (The run's first entry: those of its row in this window are its first ones.)
                if (!partial && tile == 0 && lane == 0) {
                    int first = i;
                    while (first > 0 && row[first - 1] == v) --first;
                    p.cross[atomicAdd(&p.meta[1], 1)] = make_int4(v, e0 + first, ntail, 0);
                }
            } else {
                emb_write<TG, VEC>(p, v, c0, s);
            }
            partial = false;
#pragma unroll
            for (int x = 0; x < kEmbCols; ++x) s[x] = 0.f;
        }
        if (VEC == 1) __syncwarp();
        issue(q + 2 * B);
    }
}

// The partial rows of a long run, in the windows' order: eight warps a
// contiguous range each, then the eight sums.
constexpr int kEmbJoinWarps = 8, kEmbJoinCols = 128;

template <typename TG>
__global__ void __launch_bounds__(32 * kEmbJoinWarps) emb_join_kernel(const __grid_constant__ EmbParams p)
{
    constexpr int NK = kEmbJoinCols / 32;
    __shared__ float sums[kEmbJoinWarps][kEmbJoinCols];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int runs = p.meta[1], tiles = (p.D + kEmbJoinCols - 1) / kEmbJoinCols;
    for (long long item = blockIdx.x; item < (long long)runs * tiles; item += gridDim.x) {
        const int4 run = p.cross[item / tiles];
        const int tile = (int)(item % tiles), c0 = tile * kEmbJoinCols + lane;
        const int a = run.y / p.W, b = (run.y + run.z - 1) / p.W;
        const int per = (b - a + kEmbJoinWarps) / kEmbJoinWarps;
        const int w0 = a + warp * per, w1 = min(b + 1, w0 + per);
        float s[NK] = {};
#pragma unroll 8
        for (int w = w0; w < w1; ++w) {
            const float* q = p.part + ((long long)w * 2 + (w == a ? 1 : 0)) * p.D;
#pragma unroll
            for (int k = 0; k < NK; ++k) s[k] += q[min(c0 + 32 * k, p.D - 1)];
        }
#pragma unroll
        for (int k = 0; k < NK; ++k) sums[warp][lane + 32 * k] = s[k];
        __syncthreads();
        const int c = tile * kEmbJoinCols + (int)threadIdx.x;
        if (threadIdx.x < kEmbJoinCols && c < p.D) {
            float t = 0.f;
#pragma unroll
            for (int w = 0; w < kEmbJoinWarps; ++w) t += sums[w][threadIdx.x];
            TG* out = static_cast<TG*>(p.out) + run.x * p.ld_table + c;
            t *= p.scale;
            if (p.accumulate) t += to_f32<TG>(*out);
            *out = from_f32<TG>(t);
        }
        __syncthreads();
    }
}

// The whole gradient in one kernel, for few tokens: every CTA finds the positions of
// its table rows (every G-th one: the grid then writes the table from its beginning
// to its end) and sums them itself.  A warp takes a row
// by 256 columns (zeros, or a run of at most 32), a run that is longer all warps of
// the CTA, a contiguous range each.  One launch instead of three that wait for one
// another (512 tokens of an 8192 x 512 table: 14 us before), at the price of one SM
// reading all rows of a frequent token.
constexpr int kEmbSmallThreads = 512, kEmbSmallWarps = kEmbSmallThreads / 32;
constexpr int kEmbSmallMaxRows = 2048, kEmbSmallTokens = 1024;

template <typename TG, typename TY, int VEC>
__global__ void __launch_bounds__(kEmbSmallThreads, 2) emb_small_kernel(const __grid_constant__ EmbParams p)
{
    constexpr int NV = 8 / VEC, AHEAD = 4;
    extern __shared__ int small_smem[];
    __shared__ float part[kEmbSmallWarps][256];
    __shared__ int wsum[kEmbSmallWarps];
    const int T = (int)p.T, R = p.R, G = gridDim.x, nr = (p.V - (int)blockIdx.x + G - 1) / G;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int *count = small_smem, *next = count + R, *match_t = next + R, *match_r = match_t + T, *sorted = match_r + T;
    pdl_launch_dependents();
    for (int i = threadIdx.x; i < R; i += kEmbSmallThreads) count[i] = 0;
    __syncthreads();
    pdl_wait();
    // The positions of this range's tokens, in order: counted per warp, then written.
    const int per = (T + 32 * kEmbSmallWarps - 1) / (32 * kEmbSmallWarps) * 32;
    const int t0 = min(T, warp * per), t1 = min(T, t0 + per);
    int mine = 0;
    for (int t = t0; t < t1; t += 32) {
        const int v = t + lane < t1 ? emb_token(p, t + lane) : -2;
        const bool in = v >= 0 && v != p.padding && v % G == (int)blockIdx.x;
        if (in) atomicAdd(&count[v / G], 1);
        mine += __popc(__ballot_sync(0xffffffffu, in));
        if (blockIdx.x == 0 && v == -1) atomicOr(&g_status, kStatusBadToken);
    }
    if (lane == 0) wsum[warp] = mine;
    __syncthreads();
    int at = 0, total = 0;
    for (int w = 0; w < kEmbSmallWarps; ++w) {
        at += w < warp ? wsum[w] : 0;
        total += wsum[w];
    }
    for (int t = t0; t < t1 && mine; t += 32) {
        const int v = t + lane < t1 ? emb_token(p, t + lane) : -2;
        const bool in = v >= 0 && v != p.padding && v % G == (int)blockIdx.x;
        const unsigned who = __ballot_sync(0xffffffffu, in);
        if (in) {
            const int k = at + __popc(who & ((1u << lane) - 1u));
            match_t[k] = t + lane, match_r[k] = v / G;
        }
        at += __popc(who);
    }
    __syncthreads();
    if (warp == 0 && total > 0) {
        // Where each row's positions begin, then the positions: equal rows of 32 take consecutive places.
        int base = 0;
        for (int r = 0; r < nr; r += 32) {
            const int n = r + lane < nr ? count[r + lane] : 0;
            int x = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (r + lane < nr) next[r + lane] = base + x - n;
            base += __shfl_sync(0xffffffffu, x, 31);
        }
        __syncwarp();
        for (int i = 0; i < total; i += 32) {
            const bool in = i + lane < total;
            const unsigned who = __ballot_sync(0xffffffffu, in);
            if (in) {
                const int r = match_r[i + lane];
                const unsigned same = __match_any_sync(who, r);
                const int rank = __popc(same & ((1u << lane) - 1u));
                sorted[next[r] + rank] = match_t[i + lane];
                __syncwarp(who);
                if (rank == 0) next[r] += __popc(same);
            }
            __syncwarp();
        }
    }
    const int tiles = (p.D + 255) / 256;
    const TY* dy = static_cast<const TY*>(p.in);
    // Entries a .. b - 1 of `sorted`, this lane's columns of a tile.
    auto sum = [&](int a, int b, int c0, float (&s)[8]) {
        int col[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) col[j] = min(c0 + j * 32 * VEC, p.D - VEC);  // columns past the row read its last ones
        for (int i = a; i < b; i += AHEAD) {
            Vec<TY, VEC> f[AHEAD][NV];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                const long long t = sorted[min(i + k, b - 1)];
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    f[k][j] = *reinterpret_cast<const Vec<TY, VEC>*>(dy + t * p.ld_out + col[j]);
            }
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
                if (i + k < b)
#pragma unroll
                    for (int j = 0; j < NV; ++j)
#pragma unroll
                        for (int q = 0; q < VEC; ++q) s[j * VEC + q] += to_f32<TY>(f[k][j].v[q]);
        }
    };
    auto write = [&](int r, int c0, const float (&s)[8]) {
        TG* out = static_cast<TG*>(p.out) + ((long long)r * G + blockIdx.x) * p.ld_table;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = c0 + j * 32 * VEC;
            if (c >= p.D) continue;
            float f[VEC];
            if (p.accumulate) load_f32<TG, VEC>(out + c, f);
#pragma unroll
            for (int k = 0; k < VEC; ++k) f[k] = p.accumulate ? f[k] + p.scale * s[j * VEC + k] : p.scale * s[j * VEC + k];
            store_f32<TG, VEC>(out + c, f);
        }
    };
    __syncthreads();
    // Zeros of the rows without a token: a warp per row.
    if (!p.accumulate)
        for (int r = warp; r < nr; r += kEmbSmallWarps)
            if (!count[r]) emb_zero_row(static_cast<TG*>(p.out) + ((long long)r * G + blockIdx.x) * p.ld_table, p.D, lane);
    if (total == 0) return;
    // (next[r] is now the end of row r's positions.)
    for (int i = warp; i < nr * tiles; i += kEmbSmallWarps) {
        const int r = i / tiles, n = count[r], c0 = i % tiles * 256 + lane * VEC;
        if (n == 0 || n > 32) continue;
        float s[8] = {};
        sum(next[r] - n, next[r], c0, s);
        write(r, c0, s);
    }
    for (int r = 0; r < nr; ++r) {
        const int n = count[r];
        if (n <= 32) continue;
        const int each = (n + kEmbSmallWarps - 1) / kEmbSmallWarps, a = next[r] - n;
        for (int tile = 0; tile < tiles; ++tile) {
            const int c0 = tile * 256 + lane * VEC;
            float s[8] = {};
            sum(a + min(n, warp * each), a + min(n, (warp + 1) * each), c0, s);
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int q = 0; q < VEC; ++q) part[warp][lane * VEC + j * 32 * VEC + q] = s[j * VEC + q];
            __syncthreads();
            if (warp == 0) {
                float u[8] = {};
                for (int w = 0; w < kEmbSmallWarps; ++w)
#pragma unroll
                    for (int j = 0; j < NV; ++j)
#pragma unroll
                        for (int q = 0; q < VEC; ++q) u[j * VEC + q] += part[w][lane * VEC + j * 32 * VEC + q];
                write(r, c0, u);
            }
            __syncthreads();
        }
    }
}

}  // namespace wg
