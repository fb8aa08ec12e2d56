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
//  emb_reduce_kernel  a segmented sum over the sorted list: a warp takes 32 entries
//                     (a window) by 256 columns.  A run of at most 64 entries is
//                     summed by the warp of the window it starts in, to its end;
//                     a longer one leaves an fp32 partial row per window.  So no
//                     warp has more than 95 entries, however often a token occurs.
//  emb_join_kernel    adds the partial rows of the long runs, in the windows' order.
//
// Windows are fixed places of the sorted list, so every sum has one order.
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
    int R;        // table rows of a CTA of emb_sort_kernel
    int* meta;    // [0] entries of the list, [1] long runs that cross windows
    int* count;   // [V] occurrences of a row's token
    int* list;    // [T] positions, by (row, position)
    int* row;     // [T] their rows
    int4* cross;  // (row, first entry, entries, 0) of the long runs that cross windows
    float* part;  // [windows][2][D] partial rows: of a run from before the window, of a run that goes on after it
    int token16;  // token is 16-byte aligned
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
constexpr int kEmbSortKept = 64;       // positions of its rows that a warp keeps from the count
constexpr int kEmbSortMaxRows = 1536;  // 32 counters of 4 bytes a row: 192 KB of shared memory
constexpr int kEmbWindow = 32, kEmbTile = 256, kEmbShort = 64;

// The tokens at positions t .. t + 3 as table rows; -1: out of range, -2: past the last position.
__device__ __forceinline__ void emb_tokens4(const EmbParams& p, long long t, int (&v)[4])
{
    if (!p.token64 && p.token16 && t + 4 <= p.T) {
        const int4 x = *reinterpret_cast<const int4*>(static_cast<const int*>(p.token) + t);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if ((unsigned)v[j] >= (unsigned)p.V) v[j] = -1;
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = t + j < p.T ? emb_token(p, t + j) : -2;
}

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
    extern __shared__ int hist[];  // [warps][R]: counts, then each warp's next entry of a row
    __shared__ int first[kEmbSortMaxRows];
    __shared__ int kept_t[kEmbSortWarps][kEmbSortKept], kept_r[kEmbSortWarps][kEmbSortKept];
    const int R = p.R, lo = blockIdx.x * R, nr = min(R, p.V - lo);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_launch_dependents();
    for (int i = threadIdx.x; i < kEmbSortWarps * R; i += kEmbSortThreads) hist[i] = 0;
    __syncthreads();
    pdl_wait();
    int* mine = hist + warp * R;
    // Each warp's positions: a multiple of 128, four consecutive ones per lane and
    // load.  Sixteen positions per lane are in flight at a time (one at a time the
    // loads' latency alone took 30 us for 65,536 tokens).
    constexpr int kAhead = 4;
    const long long per = ((p.T + kEmbSortThreads * 4 - 1) / (kEmbSortThreads * 4)) * 128;
    const long long t0 = warp * per, t1 = min(p.T, t0 + per);
    int below = 0, kept = 0;
    bool bad = false;
    for (long long t = t0; t < t1; t += 128 * kAhead) {
        int v[kAhead][4];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const long long u = t + 128 * k + 4 * lane;
            if (u < t1)
                emb_tokens4(p, u, v[k]);
            else
                v[k][0] = v[k][1] = v[k][2] = v[k][3] = -2;
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            unsigned in = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                bad |= v[k][j] == -1;
                const bool ok = v[k][j] >= 0 && v[k][j] != p.padding;
                below += ok && v[k][j] < lo;
                if (ok && (unsigned)(v[k][j] - lo) < (unsigned)nr) in |= 1u << j;
            }
            if (!__any_sync(0xffffffffu, in)) continue;
            // Keep the matches in the order of their positions: lane by lane, four in each.
            const int n = __popc(in);
            int at = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, at, o);
                if (lane >= o) at += y;
            }
            const int all = __shfl_sync(0xffffffffu, at, 31);
            at += kept - n;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (in >> j & 1u) {
                    const int r = v[k][j] - lo;
                    atomicAdd(&mine[r], 1);
                    if (at < kEmbSortKept) kept_t[warp][at] = (int)(t + 128 * k + 4 * lane + j), kept_r[warp][at] = r;
                    ++at;
                }
            kept += all;
        }
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
    if (kept <= kEmbSortKept) {
        for (int i = 0; i < kept; i += 32) {
            const bool in = i + lane < kept;
            place(in, in ? kept_t[warp][i + lane] : 0, in ? kept_r[warp][i + lane] : 0);
        }
    } else {  // more than were kept (a frequent token, or a small table): the positions again
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

template <typename TG, typename TY, int VEC>
__global__ void __launch_bounds__(256) emb_reduce_kernel(const __grid_constant__ EmbParams p, int tiles)
{
    constexpr int NV = 8 / VEC, AHEAD = 8;
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long item = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int w = (int)(item / tiles), tile = (int)(item - (long long)w * tiles);
    pdl_wait();
    const int n = p.meta[0], e0 = w * kEmbWindow;
    if (e0 >= n) return;
    const int m = min(kEmbWindow, n - e0);
    // The window's rows, where runs end in it, and the runs that cross its borders.
    const int wrow = p.row[min(e0 + lane, e0 + m - 1)];
    const int prev = e0 > 0 ? p.row[e0 - 1] : -1, next = e0 + m < n ? p.row[e0 + m] : -1;
    const int head = __shfl_sync(0xffffffffu, wrow, 0), tail = __shfl_sync(0xffffffffu, wrow, m - 1);
    const int ncut = head == prev ? p.count[head] : 0, ntail = tail == next ? p.count[tail] : 0;
    const bool entered = ncut > kEmbShort, leaves = ntail > kEmbShort;  // long runs that cross
    int b = e0, e = e0 + m;
    if (ncut && !entered) b += __popc(__ballot_sync(0xffffffffu, lane < m && wrow == head));  // an earlier window's run
    int tail0 = 0;  // first entry in the window of the run that goes on after it
    if (ntail) tail0 = e0 + m - __popc(__ballot_sync(0xffffffffu, lane < m && wrow == tail));
    if (ntail && !leaves && b < e) e = tail0 + ntail;  // this window's run, to its end
    const int c0 = tile * kEmbTile + lane * VEC;
    int col[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) col[j] = min(c0 + j * 32 * VEC, p.D - VEC);  // columns past the row read its last ones
    const TY* dy = static_cast<const TY*>(p.in);
    float s[8] = {};
    bool from_before = entered;
    for (int base = b; base < e; base += 32) {
        const int k = min(32, e - base);
        const int pos = p.list[min(base + lane, e - 1)], row = p.row[min(base + lane, e - 1)];
        const int after = base + lane + 1 < e ? p.row[base + lane + 1] : -1;
        const unsigned ends = __ballot_sync(0xffffffffu, after != row);
        for (int i0 = 0; i0 < k; i0 += AHEAD) {
            // Eight rows in flight; entries past the last read its row again.
            Vec<TY, VEC> f[AHEAD][NV];
#pragma unroll
            for (int a = 0; a < AHEAD; ++a) {
                const long long t = __shfl_sync(0xffffffffu, pos, i0 + a);
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    f[a][j] = *reinterpret_cast<const Vec<TY, VEC>*>(dy + t * p.ld_out + col[j]);
            }
#pragma unroll
            for (int a = 0; a < AHEAD; ++a) {
                const int i = i0 + a;
                if (i >= k) break;
#pragma unroll
                for (int j = 0; j < NV; ++j)
#pragma unroll
                    for (int q = 0; q < VEC; ++q) s[j * VEC + q] += to_f32<TY>(f[a][j].v[q]);
                if (!(ends >> i & 1u)) continue;
                const int v = __shfl_sync(0xffffffffu, row, i);
                const bool on = leaves && base + i == e - 1;
                if (!from_before && !on) {
                    emb_write<TG, VEC>(p, v, c0, s);
                } else {
                    float* q = p.part + ((long long)w * 2 + (from_before ? 0 : 1)) * p.D;
#pragma unroll
                    for (int j = 0; j < NV; ++j) {
                        const int c = c0 + j * 32 * VEC;
                        float g[VEC];
#pragma unroll
                        for (int x = 0; x < VEC; ++x) g[x] = s[j * VEC + x];
                        if (c < p.D) store_f32<float, VEC>(q + c, g);
                    }
                    if (!from_before && tile == 0 && lane == 0)
                        p.cross[atomicAdd(&p.meta[1], 1)] = make_int4(v, tail0, ntail, 0);
                }
#pragma unroll
                for (int x = 0; x < 8; ++x) s[x] = 0.f;
                from_before = false;
            }
        }
    }
}

// The partial rows of a long run, in the windows' order: eight warps a contiguous
// range each, then the eight sums.
template <typename TG, int VEC>
__global__ void __launch_bounds__(256) emb_join_kernel(const __grid_constant__ EmbParams p, int tiles)
{
    __shared__ float sums[8][kEmbTile];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int runs = p.meta[1];
    for (long long item = blockIdx.x; item < (long long)runs * tiles; item += gridDim.x) {
        const int4 run = p.cross[item / tiles];
        const int tile = (int)(item % tiles), c0 = tile * kEmbTile + lane;
        const int a = run.y / kEmbWindow, b = (run.y + run.z - 1) / kEmbWindow;
        const int per = (b - a + 1 + 7) / 8;
        const int w0 = a + warp * per, w1 = min(b + 1, w0 + per);
        float s[8] = {};
#pragma unroll 4
        for (int w = w0; w < w1; ++w) {
            const float* q = p.part + ((long long)w * 2 + (w == a ? 1 : 0)) * p.D;
#pragma unroll
            for (int k = 0; k < 8; ++k) s[k] += q[min(c0 + 32 * k, p.D - 1)];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) sums[warp][lane + 32 * k] = s[k];
        __syncthreads();
        if (warp == 0) {
            const int l = lane * VEC;
            float t[8] = {};
            for (int w = 0; w < 8; ++w)
#pragma unroll
                for (int j = 0; j < 8 / VEC; ++j)
#pragma unroll
                    for (int k = 0; k < VEC; ++k) t[j * VEC + k] += sums[w][l + j * 32 * VEC + k];
            emb_write<TG, VEC>(p, run.x, tile * kEmbTile + l, t);
        }
        __syncthreads();
    }
}

}  // namespace wg
