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
    unsigned thr;                     // of an element's 16 bits, times 2^16; 0: no dropout
    float gain;
    uint2 key[10];                    // the generator's keys, a round each
    unsigned long long offset;
    const unsigned long long* counter;  // added to the offset, or null
};

// ---------------------------------------------------------------- dropout
__device__ __forceinline__ uint4 philox(uint4 c, const uint2 (&key)[10])
{
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t a = (uint64_t)c.x * 0xD2511F53u, b = (uint64_t)c.z * 0xCD9E8D57u;
        c = make_uint4((uint32_t)(b >> 32) ^ c.y ^ key[i].x, (uint32_t)b, (uint32_t)(a >> 32) ^ c.w ^ key[i].y, (uint32_t)a);
    }
    return c;
}

// Elements 8 * group .. + 7 of a row, zeros where they are dropped (the gain is still to come).
__device__ __forceinline__ void drop8(const LayerTail& t, unsigned long long offset, long long row, int group,
                                      float (&v)[8])
{
    const uint4 r = philox(make_uint4((uint32_t)group, (uint32_t)row, (uint32_t)offset, (uint32_t)(offset >> 32)), t.key);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = w[i] << 16 >= t.thr ? v[2 * i] : 0.f;
        v[2 * i + 1] = w[i] >= t.thr ? v[2 * i + 1] : 0.f;
    }
}

__device__ __forceinline__ unsigned long long layer_offset(const LayerTail& t)
{
    return t.offset + (t.thr && t.counter ? *t.counter : 0ull);
}

// ---------------------------------------------------------------- activations
// The hardware's reciprocal and power of two, each one instruction (2^-23 or so of the result;
// numbers below 2^-126 count as zeros, an infinity's reciprocal is 0).
__device__ __forceinline__ float rcp_f(float a)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
    return r;
}
__device__ __forceinline__ float exp2_f(float a)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
    return r;
}
// Two values at a time: fp32 operations on pairs issue once.
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b)
{
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void split(F2 x, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x.v)); }
__device__ __forceinline__ F2 mul(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 both(float a) { return f2(a, a); }
__device__ __forceinline__ F2 add(F2 a, F2 b)
{
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

// 1 / (1 + exp(-a)), and e = exp(-a).
__device__ __forceinline__ F2 sigmoid2(F2 a, F2& e)
{
    float x, y;
    split(mul(a, both(-1.4426950408889634f)), x, y);
    e = f2(exp2_f(x), exp2_f(y));
    split(add(e, both(1.f)), x, y);
    return f2(rcp_f(x), rcp_f(y));
}
__device__ __forceinline__ F2 sigmoid2(F2 a)
{
    F2 e;
    return sigmoid2(a, e);
}

// gelu's tanh form is v sigmoid(2 u): (1 + tanh u) / 2 is sigmoid(2 u).  (The exponential is off by
// some 2^-24 |a| of itself beyond its last places, and 1 + exp(-a) is that near 1 wherever
// the result is not small beside v.)  Squares are held below 1e10, where every sigmoid has
// long been 0 or 1, so that no 0 meets an infinity.
__device__ __forceinline__ F2 square2(F2 v)
{
    float x, y;
    split(mul(v, v), x, y);
    return f2(fminf(x, 1e10f), fminf(y, 1e10f));
}

// The normal distribution's tails by Abramowitz and Stegun's 7.1.26 (Hastings, 1955):
// erfc(x) = t (a1 + ... + a5 t^4) exp(-x^2), t = 1 / (1 + p x), off by 1.5e-7 at most, in a third
// of erff's instructions (instructions are what bounds the activation alone).
// q = erfc(|v| / sqrt 2) / 2 and e = exp(-v^2 / 2) of a pair.
__device__ __forceinline__ F2 tails(float a, float b, F2& e)
{
    const F2 v = f2(a, b), x = f2(fabsf(a), fabsf(b));
    const F2 d = fma(x, f2(0.23164190f, 0.23164190f), f2(1.f, 1.f)), g = mul(mul(v, v), f2(-0.72134752f, -0.72134752f));
    float d0, d1, g0, g1;
    split(d, d0, d1), split(g, g0, g1);
    const F2 t = f2(rcp_f(d0), rcp_f(d1));
    e = f2(exp2_f(g0), exp2_f(g1));
    F2 q = fma(t, f2(0.5f * 1.061405429f, 0.5f * 1.061405429f), f2(0.5f * -1.453152027f, 0.5f * -1.453152027f));
    q = fma(t, q, f2(0.5f * 1.421413741f, 0.5f * 1.421413741f));
    q = fma(t, q, f2(0.5f * -0.284496736f, 0.5f * -0.284496736f));
    q = fma(t, q, f2(0.5f * 0.254829592f, 0.5f * 0.254829592f));
    return mul(mul(q, t), e);
}
__device__ __forceinline__ void gelu2(float& a, float& b)
{
    F2 e;
    float q0, q1;
    split(tails(a, b, e), q0, q1);
    // v - v q above 0, v q below: the size of v q taken off what is above 0 (an infinity times
    // a tail of 0 is 0).
    a = fmaxf(a, 0.f) - fminf(fabsf(a), 1e30f) * q0;
    b = fmaxf(b, 0.f) - fminf(fabsf(b), 1e30f) * q1;
}
__device__ __forceinline__ void gelu_slope2(float& a, float& b)
{
    F2 e;
    float q0, q1, p0, p1;
    split(tails(a, b, e), q0, q1);
    split(mul(mul(e, f2(0.39894228f, 0.39894228f)), f2(a, b)), p0, p1);
    a = (a < 0.f ? q0 : 1.f - q0) + p0;
    b = (b < 0.f ? q1 : 1.f - q1) + p1;
}

// The activation of each of a pair.
__device__ __forceinline__ F2 gelu2(F2 v)
{
    float a, b;
    split(v, a, b);
    gelu2(a, b);
    return f2(a, b);
}
__device__ __forceinline__ F2 gelu_tanh2(F2 v) { return mul(v, sigmoid2(mul(v, fma(both(0.0713548162726f), square2(v), both(1.59576912161f))))); }
__device__ __forceinline__ F2 silu2(F2 v) { return mul(v, sigmoid2(v)); }
// Its slope: of v sigmoid(w), s (1 + v w' (1 - s)).  With gelu's w, v w' reaches 35 where s is still below 1: there
// 1 - s is taken as exp(-w) s, whose error is of its own size (subtracted from 1 it left the slope 1.002 times
// 2^-19 off at 4.962).  The power is held below 2^100, where s has long been 0, so that no 0 meets an infinity.
__device__ __forceinline__ F2 gelu_slope2(F2 v)
{
    float a, b;
    split(v, a, b);
    gelu_slope2(a, b);
    return f2(a, b);
}
__device__ __forceinline__ F2 gelu_tanh_slope2(F2 v)
{
    F2 e;
    const F2 q = square2(v), s = sigmoid2(mul(v, fma(both(0.0713548162726f), q, both(1.59576912161f))), e);
    float x, y;
    split(e, x, y);
    const F2 r = mul(mul(v, s), mul(f2(fminf(x, 0x1p100f), fminf(y, 0x1p100f)), s));
    return fma(r, fma(both(0.2140644488178f), q, both(1.59576912161f)), s);
}
__device__ __forceinline__ F2 silu_slope2(F2 v)
{
    const F2 s = sigmoid2(v);
    return mul(s, fma(v, fma(s, both(-1.f), both(1.f)), both(1.f)));
}

__device__ __forceinline__ void act8(int act, float (&v)[8])
{
#define WG_EACH(F)                                  \
    _Pragma("unroll") for (int i = 0; i < 8; i += 2) \
    {                                               \
        split(F(f2(v[i], v[i + 1])), v[i], v[i + 1]); \
    }
    if (act == kActRelu) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] < 0.f ? 0.f : v[i];
    } else if (act == kActGelu) {
        WG_EACH(gelu2)
    } else if (act == kActGeluTanh) {
        WG_EACH(gelu_tanh2)
    } else if (act == kActSilu) {
        WG_EACH(silu2)
    }
#undef WG_EACH
}
// v times the activation's slope at z.
__device__ __forceinline__ void slope8(int act, const float (&z)[8], float (&v)[8])
{
#define WG_EACH(F)                                                                      \
    _Pragma("unroll") for (int i = 0; i < 8; i += 2)                                     \
    {                                                                                   \
        split(mul(f2(v[i], v[i + 1]), F(f2(z[i], z[i + 1]))), v[i], v[i + 1]);            \
    }
    if (act == kActRelu) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = z[i] <= 0.f ? 0.f : v[i];
    } else if (act == kActGelu) {
        WG_EACH(gelu_slope2)
    } else if (act == kActGeluTanh) {
        WG_EACH(gelu_tanh_slope2)
    } else if (act == kActSilu) {
        WG_EACH(silu_slope2)
    }
#undef WG_EACH
}

// v * gain + x of eight.
__device__ __forceinline__ void gain8(float gain, const float (&x)[8], float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 8; i += 2) split(fma(f2(v[i], v[i + 1]), both(gain), f2(x[i], x[i + 1])), v[i], v[i + 1]);
}
__device__ __forceinline__ void gain8(float gain, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 8; i += 2) split(mul(f2(v[i], v[i + 1]), both(gain)), v[i], v[i + 1]);
}
__device__ __forceinline__ void add8(const float (&x)[8], float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 8; i += 2) split(add(f2(v[i], v[i + 1]), f2(x[i], x[i + 1])), v[i], v[i + 1]);
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
        gain8(t.gain, x, v);
    } else {
        gain8(t.gain, v);
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
    const uint4 r = philox(make_uint4((uint32_t)(col >> 3), (uint32_t)(row + (lane & 7)), (uint32_t)offset, (uint32_t)(offset >> 32)), t.key);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    uint32_t mine = 0;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const uint32_t b = __ballot_sync(0xffffffffu, (c & 1 ? w[c >> 1] : w[c >> 1] << 16) >= t.thr);
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
            for (int k = 0; k < 8; ++k) v[h + k] = keep >> k & 1 ? v[h + k] : 0u;
        }
    }
    if (t.res) {
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(fmaf(__uint_as_float(v[k]), t.gain, as_float(x[k], t.y_dtype)));
    } else if (KIND != kWeight && t.thr) {
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * t.gain);
    }
    store_rows(t.y, base + row * t.ldy + col, t.ldy, t.y_dtype, t.vec & kPairY, n, v);
}

// ---------------------------------------------------------------- rows that start anywhere
// Eight 16-bit elements per lane of a row whose lanes' elements follow one another, in aligned
// 16-byte accesses: a lane's elements are parts of two of them, of which the second is the
// next lane's first.  Both are loaded (the second comes from L1; taken from the next lane by
// shuffles, the gradient of 5001 x 2047 in fp16 took 35 us instead of 33; an element at a time, eight
// times the requests, 80).  `a` is the address of the lane's first element, `end` that of the row's
// end; chunks that hold no element of the row are not touched.
// In two steps, so that the loads of several rows are in flight before the first is waited for.
struct Fetched {
    uint4 x, l;  // the lane's aligned chunk, and the one behind it
};
__device__ __forceinline__ Fetched fetch_shifted(uintptr_t a, uintptr_t end)
{
    const uintptr_t c = a & ~(uintptr_t)15;
    Fetched f;
    f.x = f.l = make_uint4(0u, 0u, 0u, 0u);
    if (c < end) f.x = *reinterpret_cast<const uint4*>(c);
    if ((a & 15) && c + 16 < end) f.l = *reinterpret_cast<const uint4*>(c + 16);
    return f;
}
__device__ __forceinline__ uint4 join_shifted(const Fetched& f, uintptr_t a)
{
    const uint4 &x = f.x, &l = f.l;
    const uint32_t s = (uint32_t)(a & 15), h = (s & 2u) * 8u;  // (the same for every lane)
    if (s < 4) return make_uint4(__funnelshift_r(x.x, x.y, h), __funnelshift_r(x.y, x.z, h), __funnelshift_r(x.z, x.w, h), __funnelshift_r(x.w, l.x, h));
    if (s < 8) return make_uint4(__funnelshift_r(x.y, x.z, h), __funnelshift_r(x.z, x.w, h), __funnelshift_r(x.w, l.x, h), __funnelshift_r(l.x, l.y, h));
    if (s < 12) return make_uint4(__funnelshift_r(x.z, x.w, h), __funnelshift_r(x.w, l.x, h), __funnelshift_r(l.x, l.y, h), __funnelshift_r(l.y, l.z, h));
    return make_uint4(__funnelshift_r(x.w, l.x, h), __funnelshift_r(l.x, l.y, h), __funnelshift_r(l.y, l.z, h), __funnelshift_r(l.z, l.w, h));
}

// Those of the eight halves at c that lie in [begin, end).
__device__ __forceinline__ void store_halves(uintptr_t c, const uint4& v, uintptr_t begin, uintptr_t end)
{
    const int lo = c < begin ? (int)(begin - c) : 0, hi = c >= end ? 0 : end - c >= 16 ? 16 : (int)(end - c);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (2 * i >= lo && 2 * i < hi) *reinterpret_cast<unsigned short*>(c + 2 * i) = (unsigned short)(i & 1 ? w[i >> 1] >> 16 : w[i >> 1]);
}
// (Stores take the lane before's last bytes by shuffles: the whole warp, converged.)
__device__ __forceinline__ void store_shifted(uintptr_t a, uintptr_t end, const uint4& x)
{
    const uint32_t s = (uint32_t)(a & 15);
    const int lane = threadIdx.x & 31;
    const uintptr_t begin = a - 16 * lane;
    end = min(end, begin + 512);
    if (s == 0) {
        if (a + 16 <= end)
            *reinterpret_cast<uint4*>(a) = x;
        else
            store_halves(a, x, begin, end);
        return;
    }
    // The aligned chunk at c: the last s bytes of the lane before, then the first of this one;
    // and (of the last lane) the chunk after it, which begins with this lane's last s bytes.
    const uintptr_t c = a - s;
    const uint32_t h = ((16 - s) & 2u) * 8u;
    const auto before = [](uint32_t own) { return __shfl_up_sync(0xffffffffu, own, 1); };
    const uint32_t p3 = before(x.w);
    uint4 v, z;
    if (s <= 4) {
        v = make_uint4(__funnelshift_r(p3, x.x, h), __funnelshift_r(x.x, x.y, h), __funnelshift_r(x.y, x.z, h), __funnelshift_r(x.z, x.w, h));
        z = make_uint4(__funnelshift_r(x.w, 0u, h), 0u, 0u, 0u);
    } else if (s <= 8) {
        const uint32_t p2 = before(x.z);
        v = make_uint4(__funnelshift_r(p2, p3, h), __funnelshift_r(p3, x.x, h), __funnelshift_r(x.x, x.y, h), __funnelshift_r(x.y, x.z, h));
        z = make_uint4(__funnelshift_r(x.z, x.w, h), __funnelshift_r(x.w, 0u, h), 0u, 0u);
    } else if (s <= 12) {
        const uint32_t p2 = before(x.z), p1 = before(x.y);
        v = make_uint4(__funnelshift_r(p1, p2, h), __funnelshift_r(p2, p3, h), __funnelshift_r(p3, x.x, h), __funnelshift_r(x.x, x.y, h));
        z = make_uint4(__funnelshift_r(x.y, x.z, h), __funnelshift_r(x.z, x.w, h), __funnelshift_r(x.w, 0u, h), 0u);
    } else {
        const uint32_t p2 = before(x.z), p1 = before(x.y), p0 = before(x.x);
        v = make_uint4(__funnelshift_r(p0, p1, h), __funnelshift_r(p1, p2, h), __funnelshift_r(p2, p3, h), __funnelshift_r(p3, x.x, h));
        z = make_uint4(__funnelshift_r(x.x, x.y, h), __funnelshift_r(x.y, x.z, h), __funnelshift_r(x.z, x.w, h), __funnelshift_r(x.w, 0u, h));
    }
    if (c >= begin && c + 16 <= end)
        *reinterpret_cast<uint4*>(c) = v;
    else
        store_halves(c, v, begin, end);
    if (lane == 31 && c + 16 < end) store_halves(c + 16, z, begin, end);
}

// ---------------------------------------------------------------- activation alone
// y = residual + D(act(x + bias)), or dx = D(act'(x + bias) dy) and dbias's partial sums.
// A thread has eight columns and walks down rows, several in flight; 2^cx_log threads side by
// side.  HBM bound where arithmetic is cheap (16384 x 4096 in bf16 with a residual: 60 us of
// bytes); gelu and dropout together are as many instructions as that leaves time for.
constexpr int kActThreads = 256;
enum ActMode {
    kActWide,     // 16-bit tensors, every chunk of eight columns on 16 bytes
    kActShifted,  // 16-bit tensors, rows of more than 128 columns (a warp is in one row) that start anywhere
    kActAny,      // any types and alignment
};

struct ActParams {
    LayerTail t;          // forward: y, res; gradient: y = dx, res = null
    const void* x;        // may be null in a gradient without an activation
    const void* dy;
    long long rows, ldx, lddy;
    int dim, x_dtype, dy_dtype, vec_x, vec_dy;
    int cx_log, chunk;    // threads side by side; rows of a block
    float* part;          // [chunks][dim] sums of dx, or null
};

// Eight columns of a row as they come from memory: a Raw8, or what join_shifted takes.
template <int MODE>
__device__ __forceinline__ Raw8 act_load(const void* p, long long row, long long ld, int col, int n, int dim, int dtype, bool vec)
{
    if (MODE == kActShifted) {
        const uintptr_t b = reinterpret_cast<uintptr_t>(p) + 2 * row * ld;
        const Fetched f = fetch_shifted(b + 2 * (uintptr_t)col, b + 2 * (uintptr_t)dim);
        return {f.x, f.l};
    }
    if (MODE == kActWide) {
        Raw8 r;
        r.a = *reinterpret_cast<const uint4*>(at(p, row * ld + col, 0));
        return r;
    }
    return load_raw8(p, row * ld + col, dtype, vec, n);
}
// The eight columns that act_load has loaded.
template <int MODE>
__device__ __forceinline__ void act_ready(Raw8& r, const void* p, long long row, long long ld, int col)
{
    if (MODE == kActShifted) r.a = join_shifted({r.a, r.b}, reinterpret_cast<uintptr_t>(p) + 2 * (uintptr_t)(row * ld + col));
}
template <int MODE>
__device__ __forceinline__ void act_unpack(const Raw8& r, int dtype, float (&f)[8])
{
    if (MODE != kActAny && dtype == 2) __builtin_unreachable();
    unpack8(r, dtype, f);
}

template <bool BWD, int MODE>
__global__ void __launch_bounds__(kActThreads, MODE == kActAny ? 2 : BWD && MODE == kActShifted ? 3 : 4) activation_kernel(const __grid_constant__ ActParams p)
{
    // Rows in flight, as many as leave four blocks of an SM their registers (16384 x 4096: forward 88 us
    // with two, 92 with four and three blocks, 92 with one; gradient 103 with one, 111 with two).
    constexpr int kRows = MODE == kActWide && !BWD ? 2 : MODE == kActAny ? 2 : 1;
    pdl_launch_dependents();
    const int cx = 1 << p.cx_log, tx = threadIdx.x & (cx - 1), ty = threadIdx.x >> p.cx_log, ny = kActThreads >> p.cx_log;
    const int col = 8 * (blockIdx.x * cx + tx), n = min(8, p.dim - col);
    const LayerTail& t = p.t;
    float sum[8] = {}, bias[8] = {};
    pdl_wait();
    const unsigned long long offset = layer_offset(t);
    if (t.bias && n > 0) unpack8(load_raw8(t.bias, col, t.bias_dtype, t.vec & kVecBias, n), t.bias_dtype, bias);
    if (n > 0 || MODE == kActShifted) {  // (there, lanes behind the row's end store what is left of the last ones')
        const long long r1 = min(p.rows, (long long)(blockIdx.y + 1) * p.chunk);
        for (long long r0 = (long long)blockIdx.y * p.chunk + ty; r0 < r1; r0 += kRows * ny) {
            Raw8 x[kRows], o[kRows];
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const long long r = r0 + i * ny;
                if (r >= r1) continue;
                if (p.x) x[i] = act_load<MODE>(p.x, r, p.ldx, col, n, p.dim, p.x_dtype, p.vec_x);
                if (BWD)
                    o[i] = act_load<MODE>(p.dy, r, p.lddy, col, n, p.dim, p.dy_dtype, p.vec_dy);
                else if (t.res)
                    o[i] = act_load<MODE>(t.res, r, t.ldr, col, n, p.dim, t.y_dtype, t.vec & kVecRes);
            }
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const long long r = r0 + i * ny;
                if (r >= r1) continue;
                float v[8], z[8];
                if (p.x) {
                    act_ready<MODE>(x[i], p.x, r, p.ldx, col);
                    act_unpack<MODE>(x[i], p.x_dtype, z);
                    add8(bias, z);
                }
                if (BWD) {
                    act_ready<MODE>(o[i], p.dy, r, p.lddy, col);
                    act_unpack<MODE>(o[i], p.dy_dtype, v);
                    slope8(t.act, z, v);
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] = z[k];
                    act8(t.act, v);
                }
                if (t.thr) drop8(t, offset, r, col >> 3, v);
                if (!BWD && t.res) {
                    act_ready<MODE>(o[i], t.res, r, t.ldr, col);
                    act_unpack<MODE>(o[i], t.y_dtype, z);
                    gain8(t.gain, z, v);
                } else {
                    gain8(t.gain, v);
                }
                if (t.y) {
                    if (MODE == kActAny) {
                        store8(t.y, r * t.ldy + col, t.y_dtype, t.vec & kVecY, n, v);
                    } else {
                        const int d = t.y_dtype == 1;
                        const uint4 w = make_uint4(pack2(v[0], v[1], d), pack2(v[2], v[3], d), pack2(v[4], v[5], d), pack2(v[6], v[7], d));
                        const uintptr_t b = reinterpret_cast<uintptr_t>(t.y) + 2 * r * t.ldy;
                        if (MODE == kActWide)
                            *reinterpret_cast<uint4*>(b + 2 * (uintptr_t)col) = w;
                        else
                            store_shifted(b + 2 * (uintptr_t)col, b + 2 * (uintptr_t)p.dim, w);
                    }
                }
                if (BWD) add8(v, sum);
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
    int across, units;     // blocks of threads along the columns, and of all experts (where another kernel does it)
};
// A finished sum into element i of dbias, or added to it.
__device__ __forceinline__ void put_sum(void* out, long long i, int dtype, bool accumulate, float a)
{
    if (dtype == 2) {
        float* o = static_cast<float*>(out) + i;
        *o = accumulate ? *o + a : a;
    } else if (dtype == 0) {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out) + i;
        *o = __float2bfloat16_rn(accumulate ? __bfloat162float(*o) + a : a);
    } else {
        __half* o = static_cast<__half*>(out) + i;
        *o = __float2half_rn(accumulate ? __half2float(*o) + a : a);
    }
}

// Block bx along the columns of expert e's, by THREADS threads that `sync` brings together; s: a float each.
template <int THREADS, typename Sync>
__device__ __forceinline__ void column_join(const SumParams& p, int tid, int bx, int e, float* s, Sync sync)
{
    const int nx = THREADS >> p.ny_log, ny = 1 << p.ny_log, tx = tid & (nx - 1), ty = tid / nx;
    const int j = bx * nx + tx;
    const int c0 = p.first ? p.first[e] : 0, c1 = p.first ? p.first[e + 1] : p.chunks;
    float a = 0.f;
    if (j < p.dim)
#pragma unroll 8
        for (int c = c0 + ty; c < c1; c += ny) a += p.part[(long long)c * p.dim + j];
    s[tid] = a;
    sync();
    if (ty == 0 && j < p.dim && !(p.accumulate && c0 == c1)) {
        for (int y = 1; y < ny; ++y) a += s[y * nx + tx];
        put_sum(p.out, (long long)e * p.dim + j, p.dtype, p.accumulate, a);
    }
}

__global__ void __launch_bounds__(kJoinThreads) column_join_kernel(const __grid_constant__ SumParams p)
{
    pdl_launch_dependents();
    __shared__ float s[kJoinThreads];
    pdl_wait();
    column_join<kJoinThreads>(p, threadIdx.x, blockIdx.x, blockIdx.y, s, [] { __syncthreads(); });
}

}  // namespace wg
