// fp8.cuh -- the 8-bit format shared by the norm, gated-norm and weight
// kernels: e4m3 codes in groups of 128 channels with one fp32 scale each,
// scale = max(max |y|, 1e-12) / 448, code = y / scale rounded to nearest even (of
// activations: y times 1 / scale to 2 ulp, see fp8_codes).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

namespace gdr {

constexpr int kFp8Group = 128;

inline int fp8_groups(int64_t width) { return (int)((width + kFp8Group - 1) / kFp8Group); }

// Eight consecutive values of a row ("octet"): one or two 16-byte accesses.
template <typename T>
struct Octet;

template <>
struct Octet<__nv_bfloat16> {
    uint4 raw;
    __device__ __forceinline__ void zero() { raw = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        raw = __ldcs(reinterpret_cast<const uint4*>(p));
    }
    __device__ __forceinline__ void to_float(float* f) const {
        const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&f)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    }
};

template <>
struct Octet<float> {
    float4 lo, hi;
    __device__ __forceinline__ void zero() { lo = hi = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void load(const float* p) {
        lo = __ldcs(reinterpret_cast<const float4*>(p));
        hi = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void to_float(float* f) const {
        f[0] = lo.x; f[1] = lo.y; f[2] = lo.z; f[3] = lo.w;
        f[4] = hi.x; f[5] = hi.y; f[6] = hi.z; f[7] = hi.w;
    }
    static __device__ __forceinline__ void store(float* p, const float (&f)[8]) {
        reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
};

// max |f| as its bit pattern: ordered like the values, infinity above every
// finite value and NaN above infinity, so a maximum of patterns keeps a NaN
// (fmaxf would drop it).
template <int N>
__device__ __forceinline__ uint32_t abs_bits_max(const float (&f)[N]) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < N; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
    return m;
}

// Maximum over the aligned LANES lanes that hold one group.
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t m) {
#pragma unroll
    for (int s = LANES / 2; s > 0; s >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, s));
    return m;
}

__device__ __forceinline__ float fp8_scale(uint32_t amax_bits) {
    const float a = __uint_as_float(amax_bits);
    return (a < 1e-12f ? 1e-12f : a) / 448.f;      // a NaN stays
}

// 1 / scale to 2 ulp (a scale lies between 2e-15 and 8e35, where the approximate
// division is good; 0 for an infinite one, NaN stays).
__device__ __forceinline__ float fp8_inverse(float scale) { return __fdividef(1.f, scale); }

// Codes of eight values: y * (1 / scale), saturating (the rounding of 1 / scale
// may lift the largest value a few fp32 steps above 448).  Off by up to 2^-21 of the
// quotient (2^-22 the inverse, 2^-24 the product), far below the rounding of the y
// that the norms give; the quotient itself (below) would cost them time: 32768 rows of
// 4096 bf16 without a residual 117 us in a graph instead of 96, 8192 of 896 with one
// 9.5 instead of 9.1.
__device__ __forceinline__ uint2 fp8_codes(const float* y, float inv_scale) {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        h[i] = __nv_cvt_float2_to_fp8x2(make_float2(y[2 * i] * inv_scale, y[2 * i + 1] * inv_scale),
                                        __NV_SATFINITE, __NV_E4M3);
    return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// The same with the quotient y / scale itself: where y is given and not rounded
// before, as a weight is, quotients on the border between two codes are common, and
// they have to come out exact to go to the even code.  The first quotient's remainder
// y - q scale, exact in one fused operation, gives the second (P. Markstein, IBM J.
// Res. Dev. 34, 1990); a quotient that fp32 holds comes out as it is.  16416 x 4096
// bf16 take 33 us in a graph, no more than without the correction; a division per value
// takes twice that.
// An infinite scale's inverse is 0, and 0 times y is left.
__device__ __forceinline__ uint2 fp8_codes_divided(const float* y, float scale, float inv_scale) {
    float q[8];
    const float2 inv = make_float2(inv_scale, inv_scale), neg = make_float2(-scale, -scale);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const float2 v = make_float2(y[i], y[i + 1]);
        float2 t = __fmul2_rn(v, inv);
        if (inv_scale > 0.f) t = __ffma2_rn(__ffma2_rn(t, neg, v), inv, t);
        q[i] = t.x;
        q[i + 1] = t.y;
    }
    return fp8_codes(q, 1.f);
}

}  // namespace gdr
