// gemm_quant.hpp -- rows to 8-bit integers with one scale each, and back (gfx950).
//
//   top = max_k |x[k]|,  scale = top / 127,  q[k] = the integer nearest 127 x[k] / top, ties to even
//   x'[k] = q[k] * scale
//
// The quotient is rounded as if it were exact.  For 16-bit x the product 127 x
// is exact in fp32; one Newton step with its exact remainder gives the quotient
// as fp32 rounds it, and no quotient of such numbers other than an exact half
// comes closer than 2^-19 of itself to one, so rounding that to an integer is
// right.  For fp32 x a quotient within 2^-14 of a half is compared with it by the
// exact products 127 x and half * top, each as two fp32 numbers.
//
// Bound by memory: a row is read once, held in registers by the waves it is
// given, and written once.
#pragma once

#include "gemm_kernel.hpp"

namespace mg {

typedef int i32x2 __attribute__((ext_vector_type(2)));

// Vectors at any element: the hardware takes any alignment, and where rows are
// 16-byte aligned the accesses are.
typedef i32x4 i32x4_any __attribute__((aligned(2)));
typedef i32x2 i32x2_any __attribute__((aligned(1)));
typedef int int_any __attribute__((aligned(1)));

struct Quant {
    const char* x;        // rows of x (quantising) or of q (restoring)
    char* y;              // the other
    float* scales;
    int64_t M, ldx, ldy;  // leading dimensions in elements
    int K;
};

template <In T>
struct QuantType {
    static constexpr int ES = T == In::F32 ? 4 : 2, E = 16 / ES;      // values in 16 bytes
    // The values of a chunk as fp32.
    __device__ static __forceinline__ void unpack(const i32x4& v, float (&f)[E])
    {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if constexpr (T == In::F32) f[e] = __int_as_float(v[e]);
            else if constexpr (T == In::BF16) f[e] = __int_as_float(e & 1 ? v[e / 2] & 0xffff0000 : v[e / 2] << 16);
            else f[e] = (float)__builtin_bit_cast(_Float16, (uint16_t)((uint32_t)v[e / 2] >> (16 * (e & 1))));
        }
    }
    // The largest magnitude's bits: magnitudes compare as unsigned integers,
    // with infinities and NaN above every number.
    __device__ static __forceinline__ uint32_t top(const i32x4& v, uint32_t m)
    {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const uint32_t w = (uint32_t)v[d] & (T == In::F32 ? 0x7fffffffu : 0x7fff7fffu);
            if constexpr (T == In::F32) {
                m = m > w ? m : w;
            } else {
                typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
                m = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, m),
                                                                          __builtin_bit_cast(u16x2, w)));
            }
        }
        return m;
    }
    // ... of a wave's lanes, as the bits of an fp32 number.
    __device__ static __forceinline__ uint32_t wave_top(uint32_t m)
    {
        if constexpr (T != In::F32) {
            const uint32_t hi = m >> 16, lo = m & 0xffffu;
            m = hi > lo ? hi : lo;
        }
#pragma unroll
        for (int d = 32; d >= 1; d /= 2) {
            const uint32_t o = (uint32_t)__shfl_xor((int)m, d);
            m = m > o ? m : o;
        }
        if constexpr (T == In::BF16) m <<= 16;
        else if constexpr (T == In::F16)
            m = m >= 0x7c00u ? 0x7fc00000u : (uint32_t)__float_as_int((float)__builtin_bit_cast(_Float16, (uint16_t)m));
        return m;
    }
};

// What a row's values are divided by.  The numerator 127 x is scaled by a power
// of two (mul holds both) where the largest magnitude is so small that its
// reciprocal, or so large that 127 x, would leave fp32's range.
struct RowScale {
    float mul, top, inv, wide;      // wide: the unscaled largest magnitude
    bool live;                      // false: all zeros, or a NaN or infinity: q is 0
    float scale;

    __device__ __forceinline__ explicit RowScale(uint32_t bits)
    {
        const bool bad = bits >= 0x7f800000u;
        live = bits != 0 && !bad;
        wide = __int_as_float((int)bits);
        scale = bad ? __int_as_float(0x7fc00000) : wide / 127.f;
        const float k = bits < 0x21800000u ? 0x1p80f : bits > 0x71800000u ? 0x1p-20f : 1.f;   // below 2^-60, above 2^100
        mul = 127.f * k;
        top = live ? wide * k : 1.f;
        inv = 1.f / top;
    }
};

// The value as it stands, rounded to fp32: the compiler may otherwise join the
// product that it comes from with what follows, an addition or a conversion to
// 16 bits, and round only there.
__device__ __forceinline__ float settled(float v)
{
    asm("" : "+v"(v));
    return v;
}

// One value's integer, in the low byte (the others hold anything).
template <In T>
__device__ __forceinline__ uint32_t quantize_one(float x, const RowScale& r)
{
    const float a = settled(x * r.mul);
    float t = a * r.inv;
    t = __builtin_fmaf(__builtin_fmaf(-t, r.top, a), r.inv, t);
    // Adding 3 * 2^22 rounds to an integer (to even), whose low bits are the sum's.
    float n = t + 12582912.f;
    if constexpr (T == In::F32) {
        const float i = n - 12582912.f, f = t - i;
        if (__builtin_fabsf(f) > 0.5f - 0x1p-14f) {
            // 127 x against half * top, both as a product and its rounding's error.
            const float s = __builtin_copysignf(1.f, f), half = i + 0.5f * s, p = settled(half * r.top);
            const float d = ((a - p) + (__builtin_fmaf(x, r.mul, -a) - __builtin_fmaf(half, r.top, -p))) * s;
            const bool odd = __float_as_int(n) & 1;
            n = d > 0.f || (d == 0.f && odd) ? n + s : n;
        }
    }
    return (uint32_t)__float_as_int(n);
}

// Four values' low bytes.
__device__ __forceinline__ int pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0c0c0400u), hi = __builtin_amdgcn_perm(d, c, 0x04000c0cu);
    return (int)(lo | hi);
}

template <In T>
__device__ __forceinline__ void quantize_chunk(i32x4 v, const RowScale& r, char* dst)
{
    using Q = QuantType<T>;
    float f[Q::E];
    asm volatile("" : "+v"(v));       // (what follows stays here: every chunk's values at once would fill the registers)
    Q::unpack(v, f);
    uint32_t n[Q::E];
#pragma unroll
    for (int e = 0; e < Q::E; ++e) n[e] = quantize_one<T>(f[e], r);
    int w[Q::E / 4];
#pragma unroll
    for (int d = 0; d < Q::E / 4; ++d) w[d] = r.live ? pack4(n[4 * d], n[4 * d + 1], n[4 * d + 2], n[4 * d + 3]) : 0;
    if constexpr (Q::E == 4) *(int_any*)dst = w[0];
    else *(i32x2_any*)dst = i32x2{w[0], w[1]};
}

// The largest of W waves' maxima.
template <int W>
__device__ __forceinline__ uint32_t join_top(uint32_t m, int wave)
{
    if constexpr (W == 1) {
        return m;
    } else {
        __shared__ uint32_t part[W];
        if ((threadIdx.x & 63) == 0) part[wave] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W; ++w) m = m > part[w] ? m : part[w];
        return m;
    }
}

constexpr int kQuantThreads = 256;
constexpr int kRestoreSteps = 4;

// W waves a row, which hold it in U chunks of 16 bytes a lane.
template <In T, int W, int U>
__global__ void __launch_bounds__(W == 1 ? kQuantThreads : W * 64)
quantize_kernel(Quant p)
{
    using Q = QuantType<T>;
    constexpr int E = Q::E, LANES = W * 64, ROWS = W == 1 ? kQuantThreads / 64 : 1;
    const int tid = threadIdx.x, wave = tid >> 6, lane = W == 1 ? tid & 63 : tid;
    const int64_t row = (int64_t)blockIdx.x * ROWS + (W == 1 ? wave : 0);
    if (row >= p.M) return;
    const char* const x = p.x + row * p.ldx * Q::ES;
    char* const y = p.y + row * p.ldy;
    i32x4 v[U], last = {0, 0, 0, 0};
    uint32_t m = 0;
    if (p.K >= E) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // Past the end: the first chunk again (a branch a chunk would cost 150 registers).
            const int k = (u * LANES + lane) * E, at = k + E <= p.K ? k : 0;
            v[u] = *(const i32x4_any*)(x + (int64_t)at * Q::ES);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) m = Q::top(v[u], m);
    }
    // What is left of a chunk at the row's end, an element a lane.
    const int end = p.K / E * E + lane;
    if (end < p.K) {
        if constexpr (Q::ES == 4) last[0] = ((const int*)x)[end];
        else last[0] = ((const uint16_t*)x)[end];
    }
    m = Q::top(last, m);
    const RowScale r(join_top<W>(Q::wave_top(m), wave));
    if (lane == 0) p.scales[row] = r.scale;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int k = (u * LANES + lane) * E;
        if (k + E <= p.K) quantize_chunk<T>(v[u], r, y + k);
    }
    if (end < p.K) {
        float f[E];
        Q::unpack(last, f);
        y[end] = r.live ? (char)quantize_one<T>(f[0], r) : 0;
    }
}

// Rows longer than registers hold: a workgroup a row, read twice (the second
// time mostly from L2), element by element.
template <In T>
__global__ void __launch_bounds__(kQuantThreads)
quantize_long_kernel(Quant p)
{
    using Q = QuantType<T>;
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x;
    const char* const x = p.x + row * p.ldx * Q::ES;
    char* const y = p.y + row * p.ldy;
    auto value = [&](int k) {
        i32x4 v = {0, 0, 0, 0};
        if constexpr (Q::ES == 4) v[0] = ((const int*)x)[k];
        else v[0] = ((const uint16_t*)x)[k];
        return v;
    };
    uint32_t m = 0;
    for (int k = tid; k < p.K; k += kQuantThreads) m = Q::top(value(k), m);
    const RowScale r(join_top<kQuantThreads / 64>(Q::wave_top(m), tid >> 6));
    if (tid == 0) p.scales[row] = r.scale;
    for (int k = tid; k < p.K; k += kQuantThreads) {
        float f[Q::E];
        Q::unpack(value(k), f);
        y[k] = r.live ? (char)quantize_one<T>(f[0], r) : 0;
    }
}

// The fp32 value of byte e of a word.
__device__ __forceinline__ float byte_value(int w, int e) { return (float)((w << (24 - 8 * e)) >> 24); }

template <In T>
__device__ __forceinline__ uint16_t round16(float v)
{
    if constexpr (T == In::F16) return __builtin_bit_cast(uint16_t, (_Float16)v);
    else return __builtin_bit_cast(uint16_t, (__bf16)v);
}

// A wave takes a span of a row, 16 bytes of restored values a lane and step.
template <In T>
__global__ void __launch_bounds__(kQuantThreads)
dequantize_kernel(Quant p, int spans)
{
    using Q = QuantType<T>;
    constexpr int E = Q::E, LANES = 64, U = kRestoreSteps;
    const int lane = threadIdx.x & 63;
    const int64_t w = (int64_t)blockIdx.x * (kQuantThreads / 64) + (threadIdx.x >> 6);
    const int64_t row = w / spans;
    if (row >= p.M) return;
    const int k0 = (int)(w % spans) * (LANES * E * U) + lane * E;
    const char* const q = p.x + row * p.ldx;
    char* const y = p.y + row * p.ldy * Q::ES;
    const float s = p.scales[row];
    int v[U][E / 4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int k = k0 + u * LANES * E;
        if (k + E > p.K) continue;
        if constexpr (E == 4) {
            v[u][0] = *(const int_any*)(q + k);
        } else {
            const i32x2 t = *(const i32x2_any*)(q + k);
            v[u][0] = t[0];
            v[u][1] = t[1];
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int k = k0 + u * LANES * E;
        if (k + E <= p.K) {
            i32x4 o;
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                if constexpr (E == 4) {
                    o[d] = __float_as_int(byte_value(v[u][0], d) * s);
                } else {
                    const uint32_t lo = round16<T>(settled(byte_value(v[u][d / 2], d % 2 * 2) * s));
                    const uint32_t hi = round16<T>(settled(byte_value(v[u][d / 2], d % 2 * 2 + 1) * s));
                    o[d] = (int)(lo | (hi << 16));
                }
            }
            *(i32x4_any*)(y + (int64_t)k * Q::ES) = o;
        } else {
            for (int e = 0; e < E; ++e)
                if (k + e < p.K) {
                    const float f = settled((float)(signed char)q[k + e] * s);
                    if constexpr (Q::ES == 4) ((float*)y)[k + e] = f;
                    else ((uint16_t*)y)[k + e] = round16<T>(f);
                }
        }
    }
}

}  // namespace mg
