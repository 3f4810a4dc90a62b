// Arithmetic shared by the selective scan's kernels.
#pragma once

#include "common.cuh"
#include "vec.cuh"

namespace xlstm {

// log(1 + e) for e in [0, 1] by the series of the inverse hyperbolic tangent,
// log(1 + e) = 2 atanh(s) with s = e / (2 + e) <= 1/3: the first term left out is
// s^15 / 15 against s, under 2e-8, and a small e keeps its relative accuracy
// (which log(1 + e) through a rounded 1 + e loses).
__device__ __forceinline__ float log1p_unit(float e) {
    const float s = e * reciprocal_fast(2.f + e), q = s * s;
    float p = 1.f / 13.f;
    p = fmaf(p, q, 1.f / 11.f);
    p = fmaf(p, q, 1.f / 9.f);
    p = fmaf(p, q, 1.f / 7.f);
    p = fmaf(p, q, 1.f / 5.f);
    p = fmaf(p, q, 1.f / 3.f);
    return 2.f * fmaf(s * q, p, s);
}
// softplus(v) = max(v, 0) + log(1 + e^-|v|)
__device__ __forceinline__ float softplus(float v) {
    return fmaxf(v, 0.f) + log1p_unit(exp2_fast(-fabsf(v) * kLog2e));
}
// The same for two numbers, on packed operations.
__device__ __forceinline__ float2 softplus2(float2 v) {
    const float2 e = make_float2(exp2_fast(-fabsf(v.x) * kLog2e), exp2_fast(-fabsf(v.y) * kLog2e));
    const float2 den = add2(e, both(2.f));
    const float2 s = mul2(e, make_float2(reciprocal_fast(den.x), reciprocal_fast(den.y))), q = mul2(s, s);
    float2 p = fma2(both(1.f / 13.f), q, both(1.f / 11.f));
    p = fma2(p, q, both(1.f / 9.f));
    p = fma2(p, q, both(1.f / 7.f));
    p = fma2(p, q, both(1.f / 5.f));
    p = fma2(p, q, both(1.f / 3.f));
    return fma2(both(2.f), fma2(mul2(s, q), p, s), make_float2(fmaxf(v.x, 0.f), fmaxf(v.y, 0.f)));
}
__device__ __forceinline__ float step_size(float v, bool soft) { return soft ? softplus(v) : v; }

__device__ __forceinline__ float2 exp2_fast2(float2 v) { return make_float2(exp2_fast(v.x), exp2_fast(v.y)); }

// own + 2^(2 half) h: a state carried over many tokens.  Where it grows, the power alone may
// be past fp32 and the product within it, and a state of zero has to stay one: so by its
// root twice, the root held below infinity (and a NaN kept, which fminf would drop).  The
// exponentials of single tokens stay as they are: one that leaves fp32 is the result's.
__device__ __forceinline__ float root_of(float half) {
    float e;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(e) : "f"(half), "f"(127.f));
    return exp2_fast(e);
}
__device__ __forceinline__ float carried(float half, float h, float own) {
    const float w = root_of(half);
    return fmaf(w, w * h, own);
}
__device__ __forceinline__ float2 carried(float2 half, float2 h, float2 own) {
    const float2 w = make_float2(root_of(half.x), root_of(half.y));
    return fma2(w, mul2(w, h), own);
}

// Adds p[i] of LN / R tokens over the lanes of a group until R partial sums a token
// are left: lane j of the group ends with partial j % R of token j / R.  Each round
// halves the values a lane holds, one shuffle a value (no round where LN == R).
template <int LN, int R> __device__ __forceinline__ float partial_sum(float *p, int sub) {
#pragma unroll
    for (int m = LN / 2; m >= R; m >>= 1) {
        const bool up = sub & m;
#pragma unroll
        for (int i = 0; i < m / R; ++i) {
            const float keep = up ? p[i + m / R] : p[i], give = up ? p[i] : p[i + m / R];
            p[i] = keep + __shfl_xor_sync(0xffffffffu, give, m);
        }
    }
    return p[0];
}

// Four neighbouring channels.
template <typename T> __device__ __forceinline__ void unpack4(const T *p, float *f);
template <> __device__ __forceinline__ void unpack4<float>(const float *p, float *f) {
    const float4 v = *reinterpret_cast<const float4 *>(p);
    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
}
template <> __device__ __forceinline__ void unpack4<__nv_bfloat16>(const __nv_bfloat16 *p, float *f) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    f[0] = __uint_as_float(v.x << 16); f[1] = __uint_as_float(v.x & 0xffff0000u);
    f[2] = __uint_as_float(v.y << 16); f[3] = __uint_as_float(v.y & 0xffff0000u);
}
// Two neighbouring states as they lie in memory, and in fp32.
template <typename T> struct PairOf;
template <> struct PairOf<float> { using type = float2; };
template <> struct PairOf<__nv_bfloat16> { using type = uint32_t; };
template <typename T> using Pair = typename PairOf<T>::type;
__device__ __forceinline__ float2 widen(float2 v) { return v; }
__device__ __forceinline__ float2 widen(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
template <typename T> __device__ __forceinline__ void store4(T *p, const float *f);
template <> __device__ __forceinline__ void store4<float>(float *p, const float *f) {
    __stcs(reinterpret_cast<float4 *>(p), make_float4(f[0], f[1], f[2], f[3]));
}
template <> __device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16 *p, const float *f) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
    __stcs(reinterpret_cast<uint2 *>(p), make_uint2(*reinterpret_cast<const uint32_t *>(&a),
                                                    *reinterpret_cast<const uint32_t *>(&b)));
}

}  // namespace xlstm
