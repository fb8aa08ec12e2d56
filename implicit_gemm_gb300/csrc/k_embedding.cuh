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
//                     (a window) by 256 columns.  Runs of one token inside the
//                     window are final rows; those that cross its borders leave
//                     fp32 partial rows.  Every warp has the same work, however
//                     often a token occurs.
//  emb_join_kernel    adds the partial rows of the runs that cross windows, in order.
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
    int* meta;    // [0] entries of the list, [1] runs that cross windows
    int* count;   // [V] occurrences of a row's token
    int* list;    // [T] positions, by (row, position)
    int* row;     // [T] their rows
    int4* cross;  // [windows] (row, first entry, entries, 0) of the runs that cross windows
    float* part;  // [windows][2][D] partial rows: of a run from before the window, of a run that goes on after it
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
constexpr int kEmbSortMaxRows = 1600;  // 32 counters of 4 bytes a row: 205 KB of shared memory
constexpr int kEmbWindow = 32, kEmbTile = 256;

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

template <typename TG, int VEC>
__global__ void __launch_bounds__(kEmbSortThreads, 1) emb_sort_kernel(const __grid_constant__ EmbParams p)
{
    extern __shared__ int hist[];  // [warps][R]: counts, then each warp's next entry of a row
    __shared__ int first[kEmbSortMaxRows];
    const int R = p.R, lo = blockIdx.x * R, nr = min(R, p.V - lo);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_launch_dependents();
    for (int i = threadIdx.x; i < kEmbSortWarps * R; i += kEmbSortThreads) hist[i] = 0;
    __syncthreads();
    pdl_wait();
    int* mine = hist + warp * R;
    // Each warp's positions: a multiple of 32 * 4 of them.
    const long long per = ((p.T + kEmbSortThreads * 4 - 1) / (kEmbSortThreads * 4)) * 128;
    const long long t0 = warp * per, t1 = min(p.T, t0 + per);
    int below = 0;
    bool bad = false;
    for (long long t = t0 + lane; t < t1; t += 128) {
        int v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = t + 32 * k < t1 ? emb_token(p, t + 32 * k) : -2;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            bad |= v[k] == -1;
            if (v[k] >= 0 && v[k] != p.padding) {
                below += v[k] < lo;
                if ((unsigned)(v[k] - lo) < (unsigned)nr) atomicAdd(&mine[v[k] - lo], 1);
            }
        }
    }
    if (blockIdx.x == 0 && bad) atomicOr(&g_status, kStatusBadToken);
    int base, total;
    block_exclusive_1024(below, &base);  // (its barriers also complete the counts)
    // Two rows of the range per thread: their sizes, first entries and each warp's place in them.
    int n[2], own = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int r = threadIdx.x * 2 + k;
        n[k] = 0;
        if (r < nr)
            for (int w = 0; w < kEmbSortWarps; ++w) n[k] += hist[w * R + r];
        own += n[k];
    }
    int at = base + block_exclusive_1024(own, &total);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int r = threadIdx.x * 2 + k;
        if (r < nr) {
            p.count[lo + r] = n[k];
            first[r] = n[k];
            int o = at;
            for (int w = 0; w < kEmbSortWarps; ++w) {
                const int c = hist[w * R + r];
                hist[w * R + r] = o;
                o += c;
            }
        }
        at += n[k];
    }
    if (threadIdx.x == 0 && blockIdx.x == gridDim.x - 1) p.meta[0] = base + total, p.meta[1] = 0;
    __syncthreads();
    if (total > 0) {
        // The positions again, each warp's in order; equal rows of 32 positions take consecutive entries.
        for (long long t = t0; t < t1; t += 128) {
            int v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[k] = t + 32 * k + lane < t1 ? emb_token(p, t + 32 * k + lane) : -1;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const bool in = (unsigned)(v[k] - lo) < (unsigned)nr && v[k] >= 0 && v[k] != p.padding;
                const unsigned who = __ballot_sync(0xffffffffu, in);
                if (!who) continue;
                if (in) {
                    const unsigned same = __match_any_sync(who, v[k]);
                    const int rank = __popc(same & ((1u << lane) - 1u));
                    const int e = mine[v[k] - lo] + rank;
                    p.list[e] = (int)(t + 32 * k + lane);
                    p.row[e] = v[k];
                    __syncwarp(who);
                    if (rank == 0) mine[v[k] - lo] += __popc(same);
                }
                __syncwarp();
            }
        }
    }
    // Zeros of the rows without a token: a warp per row.
    if (!p.accumulate) {
        const float zero[VEC] = {};
        for (int r = warp; r < nr; r += kEmbSortWarps) {
            if (first[r]) continue;
            TG* out = static_cast<TG*>(p.out) + (long long)(lo + r) * p.ld_table;
            for (int c = lane * VEC; c < p.D; c += 32 * VEC) store_f32<TG, VEC>(out + c, zero);
        }
    }
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
    int pos = 0, row = -1;
    if (lane < m) pos = p.list[e0 + lane], row = p.row[e0 + lane];
    // The run that enters the window, and the one that leaves it.
    const int prev = e0 > 0 ? p.row[e0 - 1] : -1, next = e0 + m < n ? p.row[e0 + m] : -1;
    const int up = __shfl_down_sync(0xffffffffu, row, 1);
    const unsigned ends = __ballot_sync(0xffffffffu, lane < m && (lane == m - 1 || up != row));
    const int c0 = tile * kEmbTile + lane * VEC;
    const TY* dy = static_cast<const TY*>(p.in);
    float s[8] = {};
    bool entered = __shfl_sync(0xffffffffu, row, 0) == prev;
    int begin = 0;
    for (int i0 = 0; i0 < m; i0 += AHEAD) {
        float f[AHEAD][8];
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            const long long t = __shfl_sync(0xffffffffu, pos, (i0 + a) & 31);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = c0 + j * 32 * VEC;
                float g[VEC] = {};
                if (i0 + a < m && c < p.D) load_f32<TY, VEC>(dy + t * p.ld_out + c, g);
#pragma unroll
                for (int k = 0; k < VEC; ++k) f[a][j * VEC + k] = g[k];
            }
        }
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            const int i = i0 + a;
            if (i >= m) break;
#pragma unroll
            for (int k = 0; k < 8; ++k) s[k] += f[a][k];
            if (!(ends >> i & 1u)) continue;
            const int v = __shfl_sync(0xffffffffu, row, i);
            const bool leaves = i == m - 1 && v == next;
            if (!entered && !leaves) {
                emb_write<TG, VEC>(p, v, c0, s);
            } else {
                float* q = p.part + ((long long)w * 2 + (entered ? 0 : 1)) * p.D;
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const int c = c0 + j * 32 * VEC;
                    float g[VEC];
#pragma unroll
                    for (int k = 0; k < VEC; ++k) g[k] = s[j * VEC + k];
                    if (c < p.D) store_f32<float, VEC>(q + c, g);
                }
                if (!entered && tile == 0 && lane == 0)
                    p.cross[atomicAdd(&p.meta[1], 1)] = make_int4(v, e0 + begin, p.count[v], 0);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) s[k] = 0.f;
            entered = false;
            begin = i + 1;
        }
    }
}

// The partial rows of a run, in the windows' order: eight warps a contiguous range each, then the eight sums.
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
        const int tile = (int)(item % tiles), c0 = tile * kEmbTile;
        const int a = run.y / kEmbWindow, b = (run.y + run.z - 1) / kEmbWindow;
        const int per = (b - a + 1 + 7) / 8;
        const int w0 = a + warp * per, w1 = min(b + 1, w0 + per);
        float s[8] = {};
#pragma unroll 4
        for (int w = w0; w < w1; ++w) {
            const float* q = p.part + ((long long)w * 2 + (w == a ? 1 : 0)) * p.D + c0;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (c0 + lane + 32 * k < p.D) s[k] += q[lane + 32 * k];
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
            emb_write<TG, VEC>(p, run.x, c0 + l, t);
        }
        __syncthreads();
    }
}

}  // namespace wg
