// What the kernels around the scans share (short convolution, selective scan, norms): 16-byte
// vectors of bf16 or fp32 values as fp32 registers, and the activations.
#pragma once

#include "common.cuh"

namespace drscan {

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t&>(r))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)),
          "l"(reinterpret_cast<uint64_t&>(c)));
    return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(r))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(r))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return r;
}
// The two bf16 of a word, and back.
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack2(float2 x) { return pack_bf16(x.x, x.y); }

// VEC values of a tensor's type in one 16-byte access, unpacked to fp32.
template <typename T>
struct Vec16;

template <>
struct Vec16<float> {
    static constexpr int N = 4;
    __device__ __forceinline__ static void unpack(const uint4& r, float* x) {
        x[0] = __uint_as_float(r.x), x[1] = __uint_as_float(r.y);
        x[2] = __uint_as_float(r.z), x[3] = __uint_as_float(r.w);
    }
    __device__ __forceinline__ static uint4 pack(const float* x) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                          __float_as_uint(x[3]));
    }
};

template <>
struct Vec16<__nv_bfloat16> {
    static constexpr int N = 8;
    // a bf16 value is the upper half of its fp32 value
    __device__ __forceinline__ static void unpack(const uint4& r, float* x) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ static uint4 pack(const float* x) {
        return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                          pack_bf16(x[6], x[7]));
    }
};

// 2^x and 1 / x, approximate (2 ulp, 1 ulp), denormals as zeros.
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 1 / (1 + e^-x), of two values. e^-x overflows to infinity for x < -88, where the quotient is 0. The
// rounding of x log2(e) moves the result by up to 1.3 |x| half steps of fp32 for x < 0, more than the
// approximate functions do. That is far below a step of bf16, and for fp32 a choice: by way of expf
// and a division the gated norm of 8 x 4096 tokens of 16 heads of 128 takes 164 us instead of 123, the
// convolution of 8 x 2048 tokens of 6144 channels 163 instead of 155.
__device__ __forceinline__ float2 sigmoid2(float2 x) {
    const float2 z = mul2(x, make_float2(-1.4426950408889634f, -1.4426950408889634f));
    const float2 d = add2(make_float2(ex2(z.x), ex2(z.y)), make_float2(1.f, 1.f));
    return make_float2(rcp(d.x), rcp(d.y));
}

// log(1 + e^x) without overflow: max(x, 0) + log1p(e^-|x|).
__device__ __forceinline__ float softplus_f32(float x) {
    return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x)));
}

// e^l, the factor a state decays by. Near 1, where a state remembers thousands of steps, by way of
// e^l - 1: the exponential's own error there, up to an ulp and mostly to one side, would add up
// step after step, where the rounded sum's is half an ulp to either.
__device__ __forceinline__ float decay_f32(float l) {
    return l > -0.25f ? 1.f + expm1f(l) : expf(l);
}

}  // namespace drscan
