// What follows a product, and the same alone:
//
//   y = residual + D(act(v + bias))          forward (z = v + bias kept on request)
//   y = residual + D(act'(z) v)              input gradient (z: what the layer below was made of)
//
// D(a) = keep ? a / (1 - p) : 0.  Which elements are kept is a function of the seed, the
// offset, the row and the column alone, so a mask is never stored: Philox 4x32 with ten
// rounds (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3",
// 2011), counter (column / 8, row, offset), key = seed; sixteen bits of its 128 an
// element, which is kept where they are at least 65536 p (p rounded to that grid, and
// 1 / (1 - p) with it).  Eight elements a counter: some nine integer instructions each.
//
// All arithmetic is fp32, rounded once when it is stored.
#pragma once

#include "ptx.cuh"
#include "vec.cuh"

namespace wg {

enum LayerAct { kActNone, kActRelu, kActGelu, kActGeluTanh, kActSilu };
enum LayerKind { kForward, kData, kWeight };
// 16-byte accesses of eight columns; 4-byte accesses of two.
enum { kVecBias = 1, kVecRes = 2, kVecY = 4, kVecZ = 8, kPairRes = 16, kPairY = 32, kPairZ = 64 };

struct LayerTail {
    const void* bias;
    const void* res;  // of y's type; may be y itself
    void* y;
    void* z;          // written (forward) or read (data); 16-bit
    long long bias_stride;            // elements between experts' biases
    long long ldr, ldy, ldz;          // elements between rows
    long long y_stride;               // elements between experts' results (and res's), of the weight gradient
    int bias_dtype, y_dtype, z_dtype;
    int act, vec;
    unsigned thr;                     // 0: no dropout
    float gain;
    unsigned long long seed, offset;
    const unsigned long long* counter;  // added to the offset, or null
};

// ---------------------------------------------------------------- dropout
__device__ __forceinline__ uint4 philox(uint4 c, uint2 k)
{
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint32_t h0 = __umulhi(c.x, 0xD2511F53u), l0 = c.x * 0xD2511F53u;
        const uint32_t h1 = __umulhi(c.z, 0xCD9E8D57u), l1 = c.z * 0xCD9E8D57u;
        c = make_uint4(h1 ^ c.y ^ k.x, l1, h0 ^ c.w ^ k.y, l0);
        k.x += 0x9E3779B9u, k.y += 0xBB67AE85u;
    }
    return c;
}

// Elements 8 * group .. + 7 of a row times what dropout makes of them.
__device__ __forceinline__ void drop8(const LayerTail& t, unsigned long long offset, long long row, int group,
                                      float (&v)[8])
{
    const uint4 r = philox(make_uint4((uint32_t)group, (uint32_t)row, (uint32_t)offset, (uint32_t)(offset >> 32)),
                           make_uint2((uint32_t)t.seed, (uint32_t)(t.seed >> 32)));
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = (w[i] & 0xffffu) >= t.thr ? v[2 * i] * t.gain : 0.f;
        v[2 * i + 1] = (w[i] >> 16) >= t.thr ? v[2 * i + 1] * t.gain : 0.f;
    }
}

__device__ __forceinline__ unsigned long long layer_offset(const LayerTail& t)
{
    return t.offset + (t.thr && t.counter ? *t.counter : 0ull);
}

// ---------------------------------------------------------------- activations
__device__ __forceinline__ float sigmoid_f(float a) { return __fdividef(1.f, 1.f + __expf(-a)); }

// gelu's tanh form is v sigmoid(2 u): (1 + tanh u) / 2 is sigmoid(2 u).  (__expf is off by
// some 2^-24 |a| of itself beyond its last places, and 1 + exp(-a) is that near 1 wherever
// the result is not small beside v.  __fdividef gives 0 for divisors above 2^126, where
// the quotient is below 2^-126.)
// Squares are held below 1e10, where every sigmoid has long been 0 or 1, so that no 0 meets
// an infinity.
__device__ __forceinline__ float square_f(float v) { return fminf(v * v, 1e10f); }
__device__ __forceinline__ float gelu_2u(float v) { return v * fmaf(0.0713548162726f, square_f(v), 1.59576912161f); }

template <int ACT>
__device__ __forceinline__ float act_f(float v)
{
    if (ACT == kActRelu) return v < 0.f ? 0.f : v;
    if (ACT == kActGelu) return 0.5f * v * (1.f + erff(v * 0.70710678118654752f));
    if (ACT == kActGeluTanh) return v * sigmoid_f(gelu_2u(v));
    if (ACT == kActSilu) return v * sigmoid_f(v);
    return v;
}

template <int ACT>
__device__ __forceinline__ float slope_f(float v)
{
    if (ACT == kActGelu)
        return fmaf(v * 0.39894228040143268f, __expf(-0.5f * v * v), 0.5f * (1.f + erff(v * 0.70710678118654752f)));
    if (ACT == kActGeluTanh) {
        const float s = sigmoid_f(gelu_2u(v));  // d(2u)/dv = 1.5957... + 3 * 0.0713... v^2
        return fmaf(v * s * (1.f - s), fmaf(0.2140644488178f, square_f(v), 1.59576912161f), s);
    }
    if (ACT == kActSilu) {
        const float s = sigmoid_f(v);
        return s * fmaf(v, 1.f - s, 1.f);
    }
    return 1.f;
}

__device__ __forceinline__ void act8(int act, float (&v)[8])
{
#define WG_EACH(A)                                     \
    _Pragma("unroll") for (int i = 0; i < 8; ++i) v[i] = act_f<A>(v[i]);
    if (act == kActRelu) {
        WG_EACH(kActRelu)
    } else if (act == kActGelu) {
        WG_EACH(kActGelu)
    } else if (act == kActGeluTanh) {
        WG_EACH(kActGeluTanh)
    } else if (act == kActSilu) {
        WG_EACH(kActSilu)
    }
#undef WG_EACH
}
// v times the activation's slope at z.
__device__ __forceinline__ void slope8(int act, const float (&z)[8], float (&v)[8])
{
#define WG_EACH(A)                                     \
    _Pragma("unroll") for (int i = 0; i < 8; ++i) v[i] *= slope_f<A>(z[i]);
    if (act == kActRelu) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = z[i] <= 0.f ? 0.f : v[i];
    } else if (act == kActGelu) {
        WG_EACH(kActGelu)
    } else if (act == kActGeluTanh) {
        WG_EACH(kActGeluTanh)
    } else if (act == kActSilu) {
        WG_EACH(kActSilu)
    }
#undef WG_EACH
}

// ---------------------------------------------------------------- eight elements of a row
// As they lie in memory (dtypes as in the ABI: 0 bf16, 1 fp16, 2 fp32).
struct Raw8 {
    uint4 a, b;
};

__device__ __forceinline__ const char* at(const void* p, long long e, int dtype)
{
    return static_cast<const char*>(p) + (e << (dtype == 2 ? 2 : 1));
}

// n of 8 elements from element e of p; `vec`: all eight are there, 16-byte aligned.
__device__ __forceinline__ Raw8 load_raw8(const void* p, long long e, int dtype, bool vec, int n)
{
    Raw8 r;
    r.a = r.b = make_uint4(0u, 0u, 0u, 0u);
    const char* q = at(p, e, dtype);
    if (vec) {
        r.a = *reinterpret_cast<const uint4*>(q);
        if (dtype == 2) r.b = *reinterpret_cast<const uint4*>(q + 16);
        return r;
    }
    uint32_t w[8] = {};
    if (dtype == 2) {
        const uint32_t* s = reinterpret_cast<const uint32_t*>(q);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) w[i] = s[i];
    } else {
        const unsigned short* s = reinterpret_cast<const unsigned short*>(q);
        uint32_t h[8] = {};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) h[i] = s[i];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = h[2 * i] | h[2 * i + 1] << 16;
    }
    r.a = make_uint4(w[0], w[1], w[2], w[3]);
    r.b = make_uint4(w[4], w[5], w[6], w[7]);
    return r;
}

__device__ __forceinline__ void unpack8(const Raw8& r, int dtype, float (&f)[8])
{
    const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
    if (dtype == 2) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
    } else if (dtype == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(w[i] << 16), f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            f[2 * i] = h.x, f[2 * i + 1] = h.y;
        }
    }
}

__device__ __forceinline__ uint32_t pack2(float a, float b, int dtype)
{
    if (dtype == 0) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void store8(void* p, long long e, int dtype, bool vec, int n, const float (&f)[8])
{
    char* q = const_cast<char*>(at(p, e, dtype));
    if (dtype == 2) {
        if (vec) {
            *reinterpret_cast<float4*>(q) = make_float4(f[0], f[1], f[2], f[3]);
            *reinterpret_cast<float4*>(q + 16) = make_float4(f[4], f[5], f[6], f[7]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) reinterpret_cast<float*>(q)[i] = f[i];
        }
        return;
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack2(f[2 * i], f[2 * i + 1], dtype);
    if (vec) {
        *reinterpret_cast<uint4*>(q) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) reinterpret_cast<unsigned short*>(q)[i] = (unsigned short)(i & 1 ? w[i / 2] >> 16 : w[i / 2]);
    }
}

// What eight results of a row need besides their sums, loaded ahead of them.
template <int KIND>
struct TailRead {
    Raw8 res, z;
};
template <int KIND>
__device__ __forceinline__ void tail_read(const LayerTail& t, int expert, long long row, int col, int n, TailRead<KIND>& r)
{
    if (t.res)
        r.res = load_raw8(t.res, (KIND == kWeight ? expert * t.y_stride : 0) + row * t.ldr + col, t.y_dtype, t.vec & kVecRes, n);
    if (KIND == kData && t.z) r.z = load_raw8(t.z, row * t.ldz + col, t.z_dtype, t.vec & kVecZ, n);
}

// Columns col .. col + n - 1 (col a multiple of 8) of a row from their sums.
template <int KIND>
__device__ __forceinline__ void tail_write(const LayerTail& t, unsigned long long offset, int expert, long long row, int col,
                                           int n, const TailRead<KIND>& r, float (&v)[8])
{
    float x[8];
    if (KIND == kForward) {
        if (t.bias) {
            unpack8(load_raw8(t.bias, expert * t.bias_stride + col, t.bias_dtype, t.vec & kVecBias, n), t.bias_dtype, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += x[i];
        }
        if (t.z) store8(t.z, row * t.ldz + col, t.z_dtype, t.vec & kVecZ, n, v);
        act8(t.act, v);
    }
    if (KIND == kData && t.z) {
        unpack8(r.z, t.z_dtype, x);
        slope8(t.act, x, v);
    }
    if (KIND != kWeight && t.thr) drop8(t, offset, row, col >> 3, v);
    if (t.res) {
        unpack8(r.res, t.y_dtype, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += x[i];
    }
    store8(t.y, (KIND == kWeight ? expert * t.y_stride : 0) + row * t.ldy + col, t.y_dtype, t.vec & kVecY, n, v);
}

// ---------------------------------------------------------------- a column per lane
// What sixteen rows of 32 neighbouring columns, a column per lane, become.
__device__ __forceinline__ float bias_at(const LayerTail& t, int expert, int col)
{
    const char* q = at(t.bias, expert * t.bias_stride + col, t.bias_dtype);
    if (t.bias_dtype == 2) return *reinterpret_cast<const float*>(q);
    if (t.bias_dtype == 0) return __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(q));
    return __half2float(*reinterpret_cast<const __half*>(q));
}

// The first n of sixteen elements, ld apart, as they lie in memory.
template <typename T>
__device__ __forceinline__ void load_each(const void* p, long long e, long long ld, int n, uint32_t (&w)[16])
{
    const T* q = static_cast<const T*>(p) + e;
#pragma unroll
    for (int k = 0; k < 16; ++k, q += ld) w[k] = k < n ? *q : 0;
}
template <typename T>
__device__ __forceinline__ void store_each(void* p, long long e, long long ld, int n, const uint32_t (&v)[16])
{
    T* q = static_cast<T*>(p) + e;
#pragma unroll
    for (int k = 0; k < 16; ++k, q += ld)
        if (k < n) *q = from_f32<T>(__uint_as_float(v[k]));
}
// The same of 16-bit elements whose columns lie on 4 bytes by twos: a lane of a pair has two
// columns of the even rows in memory, the other those of the odd rows.  Half the accesses,
// and half the instructions (the addresses are most of them).
__device__ __forceinline__ void load_pairs(const void* p, long long e, long long ld, int n, uint32_t (&w)[16])
{
    const int odd = threadIdx.x & 1;
    const unsigned short* q = static_cast<const unsigned short*>(p) + e + (odd ? ld - 1 : 0);
    const uint32_t sel = odd ? 0x3276u : 0x5410u;
    uint32_t x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k, q += 2 * ld) x[k] = 2 * k + odd < n ? *reinterpret_cast<const uint32_t*>(q) : 0u;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        // Even lanes: own low half (row 2 k), the other's low half (row 2 k + 1); odd lanes the high ones.
        const uint32_t o = __shfl_xor_sync(0xffffffffu, x[k], 1), b = __byte_perm(x[k], o, sel);
        w[2 * k] = b & 0xffffu, w[2 * k + 1] = b >> 16;
    }
}
template <typename T>
__device__ __forceinline__ void store_pairs(void* p, long long e, long long ld, int n, const uint32_t (&v)[16])
{
    const int odd = threadIdx.x & 1;
    unsigned short* q = static_cast<unsigned short*>(p) + e + (odd ? ld - 1 : 0);
    const uint32_t sel = odd ? 0x3276u : 0x5410u;
#pragma unroll
    for (int k = 0; k < 8; ++k, q += 2 * ld) {
        const uint32_t w = pack2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1]), is_half<T> ? 1 : 0);
        const uint32_t o = __shfl_xor_sync(0xffffffffu, w, 1);
        if (2 * k + odd < n) *reinterpret_cast<uint32_t*>(q) = __byte_perm(w, o, sel);
    }
}
__device__ __forceinline__ void load_rows(const void* p, long long e, long long ld, int dtype, bool pair, int n, uint32_t (&w)[16])
{
    if (dtype == 2)
        load_each<uint32_t>(p, e, ld, n, w);
    else if (pair)
        load_pairs(p, e, ld, n, w);
    else
        load_each<unsigned short>(p, e, ld, n, w);
}
__device__ __forceinline__ void store_rows(void* p, long long e, long long ld, int dtype, bool pair, int n, const uint32_t (&v)[16])
{
    if (dtype == 2)
        store_each<float>(p, e, ld, n, v);
    else if (dtype == 0 && pair)
        store_pairs<__nv_bfloat16>(p, e, ld, n, v);
    else if (dtype == 0)
        store_each<__nv_bfloat16>(p, e, ld, n, v);
    else if (pair)
        store_pairs<__half>(p, e, ld, n, v);
    else
        store_each<__half>(p, e, ld, n, v);
}
__device__ __forceinline__ float as_float(uint32_t w, int dtype)
{
    if (dtype == 0) return __uint_as_float(w << 16);
    if (dtype == 1) return __half2float(__ushort_as_half((unsigned short)w));
    return __uint_as_float(w);
}

// Dropout of rows row .. row + 7 of the warp's 32 columns (the first a multiple of 8): bit k is
// row k's.  Lane l draws for row l % 8 of the columns of lanes l / 8 * 8 .. + 7; its eight
// answers reach the lanes of those columns by a ballot each.
__device__ __forceinline__ uint32_t keep_columns(const LayerTail& t, unsigned long long offset, long long row, int col)
{
    const int lane = threadIdx.x & 31;
    const uint4 r = philox(make_uint4((uint32_t)(col >> 3), (uint32_t)(row + (lane & 7)), (uint32_t)offset, (uint32_t)(offset >> 32)),
                           make_uint2((uint32_t)t.seed, (uint32_t)(t.seed >> 32)));
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    uint32_t mine = 0;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const uint32_t h = c & 1 ? w[c >> 1] >> 16 : w[c >> 1] & 0xffffu;
        const uint32_t b = __ballot_sync(0xffffffffu, h >= t.thr);
        if ((lane & 7) == c) mine = b;
    }
    return mine >> (lane & 24);
}

// What column_tail will read of `rows` rows from `row` on, 16 of every `step`, is brought to L2.
template <int KIND>
__device__ __forceinline__ void tail_prefetch(const LayerTail& t, int expert, long long row, int rows, int step, int col)
{
    const bool z = KIND == kData && t.z;
    if (!t.res && !z) return;
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += step) {
        const int lane = threadIdx.x & 31, r = lane & 15;  // a row per lane; the warp's columns are a line or two
        if (r0 + r >= rows) continue;
        const long long c = col - lane;
        if (t.res && lane < 16)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(at(t.res, (KIND == kWeight ? expert * t.y_stride : 0) + (row + r0 + r) * t.ldr + c, t.y_dtype)));
        if (z && lane >= 16) asm volatile("prefetch.global.L2 [%0];" ::"l"(at(t.z, (row + r0 + r) * t.ldz + c, t.z_dtype)));
    }
}

// The sums v of rows row .. row + 15, of which the first n are there (none: the column is not).
// The whole warp, converged.
template <int KIND>
__device__ __forceinline__ void column_tail(const LayerTail& t, unsigned long long offset, int expert, long long row, int n, int col,
                                            uint32_t (&v)[16])
{
    const long long base = KIND == kWeight ? expert * t.y_stride : 0;
    uint32_t x[16];
    if (KIND == kForward) {
        if (t.bias && n > 0) {
            const float b = bias_at(t, expert, col);
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) + b);
        }
        if (t.z) store_rows(t.z, row * t.ldz + col, t.ldz, t.z_dtype, t.vec & kPairZ, n, v);
        if (t.act != kActNone) {
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {  // one copy of the activations: eight rows, then the other eight
                float f[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(v[k]);
                act8(t.act, f);
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = v[8 + k], v[8 + k] = __float_as_uint(f[k]);
            }
        }
    }
    if (KIND == kData && t.z) {
        load_rows(t.z, row * t.ldz + col, t.ldz, t.z_dtype, t.vec & kPairZ, n, x);
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            float f[8], z[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(v[k]), z[k] = as_float(x[k], t.z_dtype);
            slope8(t.act, z, f);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = v[8 + k], v[8 + k] = __float_as_uint(f[k]), x[k] = x[8 + k];
        }
    }
    if (t.res)  // (on its way while the mask is made)
        load_rows(t.res, base + row * t.ldr + col, t.ldr, t.y_dtype, t.vec & kPairRes, n, x);
    if (KIND != kWeight && t.thr) {
#pragma unroll
        for (int h = 0; h < 16; h += 8) {
            const uint32_t keep = keep_columns(t, offset, row + h, col);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[h + k] = keep >> k & 1 ? __float_as_uint(__uint_as_float(v[h + k]) * t.gain) : 0u;
        }
    }
    if (t.res) {
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) + as_float(x[k], t.y_dtype));
    }
    store_rows(t.y, base + row * t.ldy + col, t.ldy, t.y_dtype, t.vec & kPairY, n, v);
}

// ---------------------------------------------------------------- activation alone
// y = residual + D(act(x + bias)), or dx = D(act'(x + bias) dy) and dbias's partial sums.
// A thread has eight columns and walks down rows, kActRows in flight; 2^cx_log threads side by side.
constexpr int kActThreads = 256, kActRows = 4;

struct ActParams {
    LayerTail t;          // forward: y, res; gradient: y = dx, res = null
    const void* x;        // 16- or 32-bit, may be null in a gradient without an activation
    const void* dy;
    long long rows, ldx, lddy;
    int dim, x_dtype, dy_dtype, vec_x, vec_dy;
    int cx_log, chunk;    // threads side by side; rows of a block
    float* part;          // [chunks][dim] sums of dx, or null
};

template <bool BWD>
__global__ void __launch_bounds__(kActThreads) activation_kernel(const __grid_constant__ ActParams p)
{
    pdl_launch_dependents();
    const int cx = 1 << p.cx_log, tx = threadIdx.x & (cx - 1), ty = threadIdx.x >> p.cx_log, ny = kActThreads >> p.cx_log;
    const int col = 8 * (blockIdx.x * cx + tx), n = min(8, p.dim - col);
    const LayerTail& t = p.t;
    float sum[8] = {}, bias[8] = {};
    pdl_wait();
    const unsigned long long offset = layer_offset(t);
    if (n > 0) {
        if (t.bias) unpack8(load_raw8(t.bias, col, t.bias_dtype, t.vec & kVecBias, n), t.bias_dtype, bias);
        const long long r1 = min(p.rows, (long long)(blockIdx.y + 1) * p.chunk);
        for (long long r0 = (long long)blockIdx.y * p.chunk + ty; r0 < r1; r0 += kActRows * ny) {
            Raw8 x[kActRows], o[kActRows];
#pragma unroll
            for (int i = 0; i < kActRows; ++i) {
                const long long r = r0 + i * ny;
                if (r >= r1) continue;
                if (p.x) x[i] = load_raw8(p.x, r * p.ldx + col, p.x_dtype, p.vec_x, n);
                if (BWD)
                    o[i] = load_raw8(p.dy, r * p.lddy + col, p.dy_dtype, p.vec_dy, n);
                else if (t.res)
                    o[i] = load_raw8(t.res, r * t.ldr + col, t.y_dtype, t.vec & kVecRes, n);
            }
#pragma unroll
            for (int i = 0; i < kActRows; ++i) {
                const long long r = r0 + i * ny;
                if (r >= r1) continue;
                float v[8], z[8];
                if (p.x) {
                    unpack8(x[i], p.x_dtype, z);
#pragma unroll
                    for (int k = 0; k < 8; ++k) z[k] += bias[k];
                }
                if (BWD) {
                    unpack8(o[i], p.dy_dtype, v);
                    slope8(t.act, z, v);
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] = z[k];
                    act8(t.act, v);
                }
                if (t.thr) drop8(t, offset, r, col >> 3, v);
                if (!BWD && t.res) {
                    unpack8(o[i], t.y_dtype, z);
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] += z[k];
                }
                if (t.y) store8(t.y, r * t.ldy + col, t.y_dtype, t.vec & kVecY, n, v);
                if (BWD)
#pragma unroll
                    for (int k = 0; k < 8; ++k) sum[k] += v[k];
            }
        }
    }
    if (BWD && p.part) {
        // Threads of the same columns, in order.
        __shared__ float s[8][kActThreads];
#pragma unroll
        for (int k = 0; k < 8; ++k) s[k][threadIdx.x] = sum[k];
        __syncthreads();
        for (int i = threadIdx.x; i < 8 * cx; i += kActThreads) {
            const int k = i & 7, c = i >> 3, j = 8 * (blockIdx.x * cx + c) + k;
            float a = 0.f;
            for (int y = 0; y < ny; ++y) a += s[k][(y << p.cx_log) + c];
            if (j < p.dim) p.part[(long long)blockIdx.y * p.dim + j] = a;
        }
    }
}

// dbias from its partial sums: those of part[first .. first + count - 1][dim] that are ny apart
// by each of ny threads of a column, then the threads' in order.
constexpr int kJoinThreads = 256;
struct SumParams {
    const float* part;
    void* out;
    int dim, dtype, accumulate;
    int ny_log;
    int chunks;            // of a problem without experts
    const int* first;      // [experts + 1] chunks before each expert's, or null
};
__global__ void __launch_bounds__(kJoinThreads) column_join_kernel(const __grid_constant__ SumParams p)
{
    pdl_launch_dependents();
    __shared__ float s[kJoinThreads];
    const int nx = kJoinThreads >> p.ny_log, ny = 1 << p.ny_log, tx = threadIdx.x & (nx - 1), ty = threadIdx.x / nx;
    const int j = blockIdx.x * nx + tx, e = blockIdx.y;
    pdl_wait();
    const int c0 = p.first ? p.first[e] : 0, c1 = p.first ? p.first[e + 1] : p.chunks;
    float a = 0.f;
    if (j < p.dim)
#pragma unroll 8
        for (int c = c0 + ty; c < c1; c += ny) a += p.part[(long long)c * p.dim + j];
    s[threadIdx.x] = a;
    __syncthreads();
    if (ty || j >= p.dim || (p.accumulate && c0 == c1)) return;
    for (int y = 1; y < ny; ++y) a += s[y * nx + tx];
    const long long i = (long long)e * p.dim + j;
    if (p.dtype == 2) {
        float* o = static_cast<float*>(p.out) + i;
        *o = p.accumulate ? *o + a : a;
    } else if (p.dtype == 0) {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + i;
        *o = __float2bfloat16_rn(p.accumulate ? __bfloat162float(*o) + a : a);
    } else {
        __half* o = static_cast<__half*>(p.out) + i;
        *o = __float2half_rn(p.accumulate ? __half2float(*o) + a : a);
    }
}

}  // namespace wg
