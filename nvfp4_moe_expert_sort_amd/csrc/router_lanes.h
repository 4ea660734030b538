// router_lanes.h -- a router's row of logits on the lanes of a wavefront: LT
// lanes (16, or 64) share a token, each with runs of four experts; loads,
// reductions over a token's lanes, and the values that unusable logits take.
// Shared by the expert selection and the balance loss.
#pragma once

#include "nvfp4_device.h"

namespace nvfp4 {

namespace {

__device__ __forceinline__ double max64(double a, double b) {
    double r;
    asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
__device__ __forceinline__ float max32(float a, float b) {
    float r;
    asm("v_max_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}

__device__ __forceinline__ float min32(float a, float b) {
    float r;
    asm("v_min_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}

// The value of the lane N places further in the row of 16 lanes (cyclic).
template <int N>
__device__ __forceinline__ uint32_t ror(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N, 0xF, 0xF, true);
}
template <int N>
__device__ __forceinline__ double ror(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, ((uint64_t)ror<N>((uint32_t)(u >> 32)) << 32) | ror<N>((uint32_t)u));
}
template <int N>
__device__ __forceinline__ float ror(float v) {
    return __uint_as_float(ror<N>(__float_as_uint(v)));
}

// Reductions over a token's LT lanes, the result in all of them.  A rotation
// adds the lanes in another order in each lane, so a sum is taken from the
// token's first lane: one fixed order, the same bits in every lane.
template <int LT>
__device__ __forceinline__ double tok_max(double v) {
    v = max64(v, ror<8>(v));
    v = max64(v, ror<4>(v));
    v = max64(v, ror<2>(v));
    v = max64(v, ror<1>(v));
    if (LT == 64) {
        v = max64(v, __shfl_xor(v, 16, kWave));
        v = max64(v, __shfl_xor(v, 32, kWave));
    }
    return v;
}
template <int LT>
__device__ __forceinline__ float tok_max(float v) {
    v = max32(v, ror<8>(v));
    v = max32(v, ror<4>(v));
    v = max32(v, ror<2>(v));
    v = max32(v, ror<1>(v));
    if (LT == 64) {
        v = max32(v, __shfl_xor(v, 16, kWave));
        v = max32(v, __shfl_xor(v, 32, kWave));
    }
    return v;
}
template <int LT, typename F>
__device__ __forceinline__ F tok_sum(F v) {
    v += ror<8>(v);
    v += ror<4>(v);
    v += ror<2>(v);
    v += ror<1>(v);
    if (LT == 64) {
        v += __shfl_xor(v, 16, kWave);
        v += __shfl_xor(v, 32, kWave);
    }
    return __shfl(v, 0, LT);
}

constexpr float kFltMax = 3.402823466e+38f;
// A logit as the definitions take it: -inf where it is unusable, at most the largest finite value.
__device__ __forceinline__ float clean(float l) {
    return l > -__builtin_inff() ? __builtin_amdgcn_fmed3f(l, -kFltMax, kFltMax) : -__builtin_inff();
}

// Element j (of 4) of the chunk that starts at expert e0; -inf past E.
template <typename L>
__device__ __forceinline__ void load4(const L* __restrict__ row, int e0, int E, bool vec, float (&v)[4]);
template <>
__device__ __forceinline__ void load4(const float* __restrict__ row, int e0, int E, bool vec, float (&v)[4]) {
    if (vec && e0 + 4 <= E) {
        const float4 q = *reinterpret_cast<const float4*>(row + e0);
        v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; j++) v[j] = e0 + j < E ? row[e0 + j] : -__builtin_inff();
}
template <>
__device__ __forceinline__ void load4(const uint16_t* __restrict__ row, int e0, int E, bool vec, float (&v)[4]) {
    if (vec && e0 + 4 <= E) {
        const u32x2 q = *reinterpret_cast<const u32x2*>(row + e0);
        v[0] = __uint_as_float(q[0] << 16), v[1] = __uint_as_float(q[0] & 0xFFFF0000u);
        v[2] = __uint_as_float(q[1] << 16), v[3] = __uint_as_float(q[1] & 0xFFFF0000u);
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; j++) v[j] = e0 + j < E ? bf16_to_f32(row[e0 + j]) : -__builtin_inff();
}
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return bf16_to_f32(*p); }

}  // namespace

}  // namespace nvfp4
