// Embedding lookup and the gradient of the embedding table.
//
//   lookup:    out[t, :]    = scale * table[token[t], :]
//   gradient:  dtable[v, :] = scale * sum over the t with token[t] = v of dy[t, :]
//
// The gradient groups the positions t by token without sorting the tokens
// themselves: a count per table row, a segment per row of a position list, and
// the positions written into the segments.
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
    int* count;   // [V] occurrences of a row's token
    int* offset;  // [V] first entry of its segment
    int* rank;    // [T] an occurrence's index within the segment
    int* list;    // [T] positions
    int* cursor;  // [1] entries handed out
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

__global__ void __launch_bounds__(256) emb_zero_kernel(const __grid_constant__ EmbParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    for (int i = blockIdx.x * 256 + threadIdx.x; i < p.V; i += gridDim.x * 256) p.count[i] = 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.cursor = 0;
}

__global__ void __launch_bounds__(256) emb_count_kernel(const __grid_constant__ EmbParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    for (long long t = (long long)blockIdx.x * 256 + threadIdx.x; t < p.T; t += (long long)gridDim.x * 256) {
        const int v = emb_token(p, t);
        if (v < 0)
            atomicOr(&g_status, kStatusBadToken);
        else if (v != p.padding)
            p.rank[t] = atomicAdd(&p.count[v], 1);
    }
}

__global__ void __launch_bounds__(256) emb_offset_kernel(const __grid_constant__ EmbParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    for (int v = blockIdx.x * 256 + threadIdx.x; v < p.V; v += gridDim.x * 256) {
        const int n = p.count[v];
        p.offset[v] = n ? atomicAdd(p.cursor, n) : 0;
    }
}

__global__ void __launch_bounds__(256) emb_fill_kernel(const __grid_constant__ EmbParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    for (long long t = (long long)blockIdx.x * 256 + threadIdx.x; t < p.T; t += (long long)gridDim.x * 256) {
        const int v = emb_token(p, t);
        if (v >= 0 && v != p.padding) p.list[p.offset[v] + p.rank[t]] = (int)t;
    }
}

// One warp per table row: the row's positions in ascending order, each found as
// the least one above the last.
template <typename TG, typename TY>
__global__ void __launch_bounds__(256) emb_reduce_kernel(const __grid_constant__ EmbParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const TY* dy = static_cast<const TY*>(p.in);
    TG* g = static_cast<TG*>(p.out);
    for (int v = blockIdx.x * 8 + (threadIdx.x >> 5); v < p.V; v += gridDim.x * 8) {
        const int n = p.count[v], o = n ? p.offset[v] : 0;
        if (!n && p.accumulate) continue;
        TG* row = g + v * p.ld_table;
        for (int c0 = 0; c0 < p.D; c0 += 32) {
            const int c = c0 + lane;
            float s = 0.f;
            int last = -1;
            for (int k = 0; k < n; ++k) {
                int t = 0x7fffffff;
                for (int i = lane; i < n; i += 32) {
                    const int e = p.list[o + i];
                    if (e > last && e < t) t = e;
                }
                t = __reduce_min_sync(0xffffffffu, t);
                last = t;
                if (c < p.D) s += to_f32<TY>(dy[t * p.ld_out + c]);
            }
            if (c < p.D) {
                s *= p.scale;
                if (p.accumulate) s += to_f32<TG>(row[c]);
                row[c] = from_f32<TG>(s);
            }
        }
    }
}

}  // namespace wg
