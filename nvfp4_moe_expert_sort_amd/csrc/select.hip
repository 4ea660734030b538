// select.hip -- expert selection from router logits (scores, balance bias,
// groups of experts, top-k, weights) and its gradient.
//
// Definitions (include/nvfp4moe.h, nvfp4moe_router_select): with usable
// logits l_e (not NaN, not -inf; +inf as the largest finite value), scores s
// are their softmax or sigmoid; the value that selects is v_e = s_e + b_e, or
// l_e without a bias; groups are ranked by their best v or by the sum of
// their two best s + b, the top groups stay, and the K experts of largest v
// in them are taken, ties to the lower id.
//
// The discrete choice must not depend on FP32 rounding (another side that
// recomputes it from the same logits has to agree), so v is formed in FP64.
// FP64 vector instructions issue at the FP32 rate here, and one v_max_f64
// compares a whole (value, id) key: the id sits in the key's low 10 mantissa
// bits (complemented for v >= 0, so that the lower id is the larger key).
// Without a bias v is an FP32 number whose low 29 bits are zero, and the
// order is exact; with one, values are told apart down to about 2^-41 relative
// (42 bits of key), and where s and b cancel down to the 2^-45 of s that the
// scores are within.
//
// LT lanes (16, or 64 for more than 256 experts or 16 slots) share a token, so
// a wavefront takes 4 tokens or one, each lane NV experts.  The lane sorts its
// keys once with a network; every slot then takes the maximum of the lanes'
// list heads (rotations within a row of 16 lanes) and the owner moves its list
// up.
#include <algorithm>

#include "nvfp4_device.h"
#include "nvfp4_kernels.h"

namespace nvfp4 {

namespace {

constexpr int kSelWaves = 4;         // wavefronts per workgroup
// Keys below every value: an unavailable expert, and one that cannot be taken
// (past E, or in a group that does not stay).  Only the high words differ.
constexpr double kUnavailable = -0x1p+1000, kNotKept = -0x1p+1016;
constexpr uint32_t kUnavailableHi = 0xFE700000u, kNotKeptHi = 0xFF700000u;

__device__ __forceinline__ double max64(double a, double b) {
    double r;
    asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
__device__ __forceinline__ double min64(double a, double b) {
    double r;
    asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
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

// e^x for x in [-746, 746], within 2^-46 relative where FP64 has such a normal
// number (0 at -746, inf from 709.8 on): x = n ln 2 + r with
// |r| <= ln 2 / 2 (n is read from the low bits of t = x log2 e + 1.5 2^52),
// Taylor's series of e^r to r^11 (the next term is below 2^-47), and n added
// to the exponent.  The series is written as one block of instructions that
// take the coefficients from scalar registers: from plain code the compiler
// moves each into vector registers first, two moves a term.
__device__ __forceinline__ double exp64(double x) {
    double p, t, r;
    asm("v_fma_f64 %1, %3, %4, %5\n\t"
        "v_add_f64 %0, %1, -%5\n\t"
        "v_fma_f64 %2, %0, %6, %3\n\t"
        "v_fma_f64 %2, %0, %7, %2\n\t"
        "v_fma_f64 %0, %2, %8, %9\n\t"
        "v_fma_f64 %0, %0, %2, %10\n\t"
        "v_fma_f64 %0, %0, %2, %11\n\t"
        "v_fma_f64 %0, %0, %2, %12\n\t"
        "v_fma_f64 %0, %0, %2, %13\n\t"
        "v_fma_f64 %0, %0, %2, %14\n\t"
        "v_fma_f64 %0, %0, %2, %15\n\t"
        "v_fma_f64 %0, %0, %2, %16\n\t"
        "v_fma_f64 %0, %0, %2, 0.5\n\t"
        "v_fma_f64 %0, %0, %2, 1.0\n\t"
        "v_fma_f64 %0, %0, %2, 1.0"
        : "=&v"(p), "=&v"(t), "=&v"(r)
        : "v"(x), "s"(1.4426950408889634), "v"(0x1.8p+52), "s"(-0x1.62e42fefa39efp-1), "s"(-0x1.abc9e3b39803fp-56),
          "s"(1.0 / 39916800.0), "v"(1.0 / 3628800.0), "s"(1.0 / 362880.0), "s"(1.0 / 40320.0), "s"(1.0 / 5040.0),
          "s"(1.0 / 720.0), "s"(1.0 / 120.0), "s"(1.0 / 24.0), "s"(1.0 / 6.0));
    return __builtin_ldexp(p, (int)(uint32_t)__builtin_bit_cast(uint64_t, t));
}
// 1 / d for normal d > 0, within 2^-45: the hardware estimate (2^-23) and one Newton step.
__device__ __forceinline__ double rcp64(double d) {
    const double r = __builtin_amdgcn_rcp(d);
    return __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
}
// The same within some 2^-52, by a second step: for weights whose distance from 1 counts.
__device__ __forceinline__ double rcp64_full(double d) {
    const double r = rcp64(d);
    return __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
}
// e^x for x <= 0, 0 where FP64 has no number so small: experts masked with the
// type's lowest value have scores of exactly 0 and tie.
__device__ __forceinline__ double exp64_neg(double x) { return exp64(max64(x, -746.0)); }
// 1 / (1 + e^-l), 0 where e^-l exceeds FP64 for the same reason: there the
// Newton step of 1 / inf is a NaN, which the clamp to [0, 1] (a modifier of its
// last instruction) makes 0.
__device__ __forceinline__ double sigmoid64(float l) {
    const double d = 1.0 + exp64((double)__builtin_amdgcn_fmed3f(-l, -746.0f, 746.0f));
    return fmin(fmax(rcp64(d), 0.0), 1.0);
}

constexpr float kFltMax = 3.402823466e+38f;
// A logit as the definitions take it: -inf where it is unusable, at most the largest finite value.
__device__ __forceinline__ float clean(float l) {
    return l > -__builtin_inff() ? __builtin_amdgcn_fmed3f(l, -kFltMax, kFltMax) : -__builtin_inff();
}

// Weight (before the scale) of a chosen expert in lane k < K, in FP64; `live`
// is false in the other lanes and for unavailable experts.  `max_l`, `inv`:
// the softmax's maximum and inverse denominator over all usable logits (only
// read for softmax weights without renormalisation).
template <int LT>
__device__ __forceinline__ double slot_weight(float l, bool live, bool sigmoid, bool renorm, float max_l, double inv) {
    if (!renorm) {
        if (!live) return 0.0;
        return sigmoid ? sigmoid64(l) : exp64_neg((double)l - (double)max_l) * inv;
    }
    // The sum over the selection, shifted by its largest term so that it
    // cannot vanish: sigma(l) e^-m = e^(l - m) / (1 + e^l) with m = min(top, 0).
    const float top = tok_max<LT>(live ? l : -kFltMax);
    double w = 0.0;
    if (live) {
        if (!sigmoid)
            w = exp64_neg((double)l - (double)top);
        else if (l < 0.0f)
            w = exp64_neg((double)l - (double)fminf(top, 0.0f)) * rcp64(1.0 + exp64_neg((double)l));
        else
            w = sigmoid64(l);
    }
    const double sum = tok_sum<LT>(w);
    return live ? w * rcp64_full(sum) : 0.0;
}

// Keeps LDS accesses before it before those after it: a wavefront's LDS
// instructions take effect in order, so its lanes see each other's.
__device__ __forceinline__ void lds_order() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
}

// Batcher's odd-even merge network: a[0..N) descending, N a power of two.
template <int N>
__device__ __forceinline__ void sort_desc(double (&a)[N]) {
#pragma unroll
    for (int p = 1; p < N; p <<= 1)
#pragma unroll
        for (int k = p; k >= 1; k >>= 1)
#pragma unroll
            for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; i++)
                    if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const double x = a[i + j], y = a[i + j + k];
                        a[i + j] = max64(x, y);
                        a[i + j + k] = min64(x, y);
                    }
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

// A lane mask (all ones or zero) that the compiler takes as plain bits: from a
// condition it would turn the choice between two array elements into a choice
// of their index, and that into a search through the whole array.
__device__ __forceinline__ uint32_t lane_mask(bool c) {
    uint32_t m = c ? ~0u : 0u;
    asm("" : "+v"(m));
    return m;
}
__device__ __forceinline__ uint32_t able_mask(uint32_t able, int i) {
    return (uint32_t)__builtin_amdgcn_sbfe((int32_t)able, (uint32_t)i, 1);
}
// v, or the key constant of that high word where the mask is zero.
__device__ __forceinline__ double pick(uint32_t mask, double v, uint32_t other) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t hi = ((uint32_t)(u >> 32) & mask) | (other & ~mask), lo = (uint32_t)u & mask;
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ double blend(uint32_t m, double a, double b) {
    const uint64_t x = __builtin_bit_cast(uint64_t, a), y = __builtin_bit_cast(uint64_t, b);
    const uint32_t lo = ((uint32_t)x & m) | ((uint32_t)y & ~m), hi = ((uint32_t)(x >> 32) & m) | ((uint32_t)(y >> 32) & ~m);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
// v with expert e in its low 10 bits: e, or 1023 - e where v >= 0, so that of
// equal values the lower expert is the larger key.
__device__ __forceinline__ double tag(double v, int e) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t hi = (uint32_t)(u >> 32), id = (uint32_t)e ^ ~(uint32_t)((int32_t)hi >> 31);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | (((uint32_t)u & ~1023u) | (id & 1023u)));
}
__device__ __forceinline__ int key_expert(double key) {
    const uint64_t u = __builtin_bit_cast(uint64_t, key);
    const int low = (int)(u & 1023u);
    return (u >> 63) ? low : 1023 - low;
}

}  // namespace

// LT lanes per token, NV experts per lane (E <= LT * NV) in runs of four,
// lists of LEN keys (the longest that K slots can take from one lane).
//
// Bound by its instructions.  T = 16384, E = 256, K = 8, sigmoid scores with
// bias and 8 groups: 14.6 us, 1420 vector instructions a wavefront (4 tokens),
// four wavefronts a SIMD: about 400 for the FP64 scores, 330 for the network
// and the slots; the 16.8 MB of logits take 3.2 us at the card's copy rate.
// T = 5, E = 128: 3.1 us, a launch.
template <int LT, int NV, int LEN, typename L>
__global__ void __launch_bounds__(kSelWaves * 64, 4) router_select_kernel(SelectParams P) {
    constexpr int kTok = kWave / LT;     // tokens per wavefront
    constexpr int kGroupRounds = kMaxGroups / LT;
    extern __shared__ __attribute__((aligned(16))) double smem[];  // only with groups
    const int lane = threadIdx.x & (LT - 1), slot = threadIdx.x / LT;
    const int64_t t = (int64_t)blockIdx.x * (kSelWaves * kTok) + slot;
    const int64_t tr = min(t, P.T - 1);  // rows past T repeat the last one, not stored
    const L* row = (const L*)P.logits + tr * P.ld;
    const bool sigmoid = P.sigmoid, biased = P.bias != nullptr, grouped = P.n_groups > 1;
    const bool top2 = grouped && P.top2, scores = biased || top2;
    const bool runs = (P.group_size & 3) == 0;  // a run of four experts lies in one group

    float l[NV], bias[NV];
#pragma unroll
    for (int i = 0; i < NV / 4; i++) {
        float v[4];
        load4(row, (i * LT + lane) * 4, P.E, P.vec, v);
#pragma unroll
        for (int j = 0; j < 4; j++) l[4 * i + j] = v[j];
    }
    if (biased) {
#pragma unroll
        for (int i = 0; i < NV / 4; i++) {
            float v[4];
            load4(P.bias, (i * LT + lane) * 4, P.E, P.vec_bias, v);
#pragma unroll
            for (int j = 0; j < 4; j++) bias[4 * i + j] = clean(v[j]);
        }
    }
#pragma unroll
    for (int i = 0; i < NV; i++) l[i] = clean(l[i]);
    float max_l = 0.0f;
    double inv = 1.0;  // 1 / the softmax's denominator
    double key[NV];    // v, or the scores that TOP2 groups add up
    if (sigmoid && scores) {
#pragma unroll
        for (int i = 0; i < NV; i++) key[i] = sigmoid64(l[i]);
    } else if (!sigmoid && (scores || !P.renorm)) {
        float mx = l[0];
#pragma unroll
        for (int i = 1; i < NV; i++) mx = fmaxf(mx, l[i]);
        max_l = fmaxf(tok_max<LT>(mx), -kFltMax);
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < NV; i++) sum += key[i] = exp64_neg((double)l[i] - (double)max_l);
        inv = rcp64(fmax(tok_sum<LT>(sum), 1e-300));  // (no usable expert: 0)
#pragma unroll
        for (int i = 0; i < NV; i++) key[i] *= inv;
    }
    if (!scores) {
#pragma unroll
        for (int i = 0; i < NV; i++) key[i] = (double)(l[i] + 0.0f);  // (-0 as +0)
    } else if (biased) {
#pragma unroll
        for (int i = 0; i < NV; i++) key[i] += (double)bias[i];
    }
    // Unavailable experts: an unusable logit or bias.
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const float worse = biased ? min32(l[i], bias[i]) : l[i];
        key[i] = pick(lane_mask(worse > -__builtin_inff()), key[i], kUnavailableHi);
    }
    uint32_t able = 0;  // bit i: expert i of the lane exists and its group stays
#pragma unroll
    for (int i = 0; i < NV / 4; i++) able |= ((1u << min(max(P.E - (i * LT + lane) * 4, 0), 4)) - 1) << (4 * i);
    if (grouped) {
        double* gv = smem + (size_t)slot * P.lds_token;  // this token's values, and its groups'
        double* gs = gv + P.lds_token - P.n_groups;
        if (runs) {  // the two best of each run: [run in group][best, second][group]
#pragma unroll
            for (int i = 0; i < NV / 4; i++) {
                const int u = i * LT + lane;
                const double a = max64(key[4 * i], key[4 * i + 1]), b = min64(key[4 * i], key[4 * i + 1]);
                const double c = max64(key[4 * i + 2], key[4 * i + 3]), d = min64(key[4 * i + 2], key[4 * i + 3]);
                if (u * 4 < P.E) {
                    const int g = (int)(((uint32_t)(u * 4) * P.group_magic) >> 22);
                    double* at = gv + (u - g * (P.group_size >> 2)) * 2 * P.n_groups + g;
                    at[0] = max64(a, c);
                    at[P.n_groups] = max64(min64(a, c), max64(b, d));
                }
            }
        } else {
#pragma unroll
            for (int n = 0; n < NV; n++) {
                const int e = ((n >> 2) * LT + lane) * 4 + (n & 3);
                if (e < P.E) {
                    const int g = (int)(((uint32_t)e * P.group_magic) >> 22);
                    gv[(e - g * P.group_size) * P.n_groups + g] = key[n];
                }
            }
        }
        __syncthreads();
        // Lane g ranks group g (and g + LT, ...): its value, then the count of
        // groups before it; the kept ones become a bit mask.
#pragma unroll
        for (int r = 0; r < kGroupRounds; r++) {
            const int g = r * LT + lane;
            if (g < P.n_groups) {
                double b1 = kNotKept, b2 = kNotKept;
                if (runs) {
                    for (int w = 0; w < P.group_size / 4; w++) {
                        const double c1 = gv[2 * w * P.n_groups + g], c2 = gv[(2 * w + 1) * P.n_groups + g];
                        b2 = max64(min64(b1, c1), max64(b2, c2));
                        b1 = max64(b1, c1);
                    }
                } else {
                    for (int w = 0; w < P.group_size; w++) {
                        const double v = gv[w * P.n_groups + g];
                        b2 = max64(b2, min64(b1, v));
                        b1 = max64(b1, v);
                    }
                }
                gs[g] = top2 && b2 > kUnavailable ? b1 + b2 : b1;
            }
        }
        __syncthreads();
        uint64_t kept = 0;
#pragma unroll
        for (int r = 0; r < kGroupRounds; r++) {
            const int g = r * LT + lane;
            int before = kMaxGroups;
            if (g < P.n_groups) {
                const double mine = gs[g];
                before = 0;
                for (int h = 0; h < P.n_groups; h++) {
                    const double o = gs[h];
                    before += (o > mine || (o == mine && h < g)) ? 1 : 0;
                }
            }
            const uint64_t all = __ballot(before < P.top_groups);
            kept |= LT == 64 ? all : ((all >> ((threadIdx.x & 63) / LT * LT)) & ((1ull << (LT & 63)) - 1)) << (r * LT);
        }
#pragma unroll
        for (int i = 0; i < NV / 4; i++) {
            const uint32_t e0 = (i * LT + lane) * 4;
            if (runs) {
                able &= ((kept >> (((e0 * P.group_magic) >> 22) & 63)) & 1) ? ~0u : ~(15u << (4 * i));
            } else {
#pragma unroll
                for (int j = 0; j < 4; j++)
                    able &= ((kept >> ((((e0 + j) * P.group_magic) >> 22) & 63)) & 1) ? ~0u : ~(1u << (4 * i + j));
            }
        }
        if (top2 && !biased) {  // groups by their scores, experts by their logits
#pragma unroll
            for (int i = 0; i < NV; i++)
                key[i] = pick(lane_mask(l[i] > -__builtin_inff()), (double)(l[i] + 0.0f), kUnavailableHi);
        }
    }
#pragma unroll
    for (int i = 0; i < NV; i++)
        key[i] = tag(pick(able_mask(able, i), key[i], kNotKeptHi), ((i >> 2) * LT + lane) * 4 + (i & 3));
    sort_desc(key);
    double mine = kNotKept;
    // Slot k takes the best list head; its owner moves its list up (after slot
    // k of at most LEN only LEN - 1 - k more keys of a list can be needed).
#pragma unroll
    for (int k = 0; k < (LEN <= 8 ? LEN : 0); k++)
        if (k < P.K) {
            const double best = tok_max<LT>(key[0]);
            if (lane == k) mine = best;
            const uint32_t pop = lane_mask(key[0] == best);  // keys are unique: one owner
#pragma unroll
            for (int i = 0; i < (LEN < NV ? LEN - 1 - k : LEN); i++)
                key[i] = blend(pop, i + 1 < NV ? key[i + 1] : kNotKept, key[i]);
        }
    if (LEN == NV)
        for (int k = LEN <= 8 ? LEN : 0; k < P.K; k++) {
            const double best = tok_max<LT>(key[0]);
            if (lane == k) mine = best;
            const uint32_t pop = lane_mask(key[0] == best);
#pragma unroll
            for (int i = 0; i < NV; i++) key[i] = blend(pop, i + 1 < NV ? key[i + 1] : kNotKept, key[i]);
        }
    const bool have = lane < P.K;
    const int e = have ? min(key_expert(mine), P.E - 1) : 0;
    const bool taken = have && mine > kUnavailable * 0.5;
    const float lk = taken ? clean(load1(row + e)) : 0.0f;
    const double w = slot_weight<LT>(lk, taken, sigmoid, P.renorm, max_l, inv);
    if (have && t < P.T) {
        P.ids[t * P.K + lane] = e;
        P.probs[t * P.K + lane] = (float)(w * (double)P.scale);
    }
}

// The gradient of the weights with respect to the logits.  With c the scale,
// dp the upstream gradient and w the weights of the chosen experts:
//   renormalised  d_k = c w_k (dp_k - sum_j dp_j w_j), times (1 - sigma_k) for sigmoid scores;
//   sigmoid       d_k = c w_k dp_k (1 - sigma_k);
//   softmax       d_k = c w_k (dp_k - sum_j dp_j w_j) at the chosen experts, and -c s_e sum_j dp_j w_j at the others.
// One pass: lane k forms d_k and puts it into the token's row in LDS, which only
// its own wavefront uses, and the row is written whole.  All of it is FP64, the
// softmax's terms too: dp_k - sum_j dp_j w_j is a small difference where one
// expert has nearly all the weight.  Each value is rounded to FP32 once, and a
// BF16 one from there (half a step of BF16 and 2^-24 more).  T = 4096, E = 256, FP32, renormalised: 4.4 us for 4.3 MB (a launch and
// one chain of loads); T = 32749, E = 128, BF16, softmax over all: 9.0 us for
// 18.9 MB, of which the copy rate allows 3.6 (with FP32 terms 7.2).
template <int LT, int NV, typename L>
__global__ void __launch_bounds__(kSelWaves * 64) router_select_backward_kernel(SelectParams P) {
    constexpr int kTok = kWave / LT;
    __shared__ __attribute__((aligned(16))) float rows[kSelWaves * kTok][LT * NV];
    const int lane = threadIdx.x & (LT - 1), slot = threadIdx.x / LT;
    const int64_t t = (int64_t)blockIdx.x * (kSelWaves * kTok) + slot;
    const int64_t tr = min(t, P.T - 1);
    const L* row = (const L*)P.logits + tr * P.ld;
    const bool sigmoid = P.sigmoid, dense = !sigmoid && !P.renorm;
    int e = -1;
    float dp = 0.0f;
    if (lane < P.K) {
        e = P.ids_in[tr * P.K + lane];
        dp = P.dprobs[tr * P.K + lane];
    }
    float l[NV];
    if (dense) {
#pragma unroll
        for (int i = 0; i < NV / 4; i++) {
            float v[4];
            load4(row, (i * LT + lane) * 4, P.E, P.vec, v);
#pragma unroll
            for (int j = 0; j < 4; j++) l[4 * i + j] = v[j];
        }
    }
    const bool in = e >= 0 && e < P.E;
    const float lk = in ? clean(load1(row + e)) : 0.0f;
    const bool live = in && lk > -__builtin_inff() && !(P.bias && !(P.bias[in ? e : 0] > -__builtin_inff()));
    // An expert listed twice: every lane leaves its number at its expert; a
    // lane that finds another's there has a double.
    uint32_t* tags = reinterpret_cast<uint32_t*>(rows[slot]);
    if (live) tags[e] = lane;
    lds_order();
    const bool twice = __ballot(live && tags[e] != (uint32_t)lane) != 0;
    lds_order();
    float max_l = 0.0f;
    double inv = 1.0;  // 1 / the softmax's denominator
    double s[NV];      // its terms
    if (dense) {
        float mx = -kFltMax;
#pragma unroll
        for (int i = 0; i < NV; i++) mx = max32(mx, l[i] = clean(l[i]));
        max_l = tok_max<LT>(mx);
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < NV; i++) sum += s[i] = exp64_neg((double)l[i] - (double)max_l);
        inv = rcp64_full(fmax(tok_sum<LT>(sum), 1e-300));
    }
    const double w = slot_weight<LT>(lk, live, sigmoid, P.renorm, max_l, inv);
    double mean = 0.0;
    if (P.renorm || dense) mean = tok_sum<LT>(live ? w * (double)dp : 0.0);
    // dp and the slots of the lane's expert: its first slot takes them all
    double up = (double)dp, slots = 1.0;
    bool first = live;
    if (twice) {
        up = slots = 0.0;
        for (int k = 0; k < P.K; k++) {
            const int ek = __shfl(live ? e : -1, k, LT);
            const float dk = __shfl(dp, k, LT);
            if (ek == e) {
                up += (double)dk;
                slots += 1.0;
                first = first && k >= lane;
            }
        }
    }
    double d = 0.0;
    if (first) {
        d = w * (up - (P.renorm ? slots : 1.0) * mean) * (double)P.scale;
        if (sigmoid) d *= sigmoid64(-lk);  // 1 - sigma(l)
    }
    const double all = -mean * (double)P.scale * inv;
#pragma unroll
    for (int i = 0; i < NV / 4; i++) {
        float4 q = {0.0f, 0.0f, 0.0f, 0.0f};
        if (dense) {  // (+0 where the term is 0)
            q.x = (float)__builtin_fma(s[4 * i], all, 0.0), q.y = (float)__builtin_fma(s[4 * i + 1], all, 0.0);
            q.z = (float)__builtin_fma(s[4 * i + 2], all, 0.0), q.w = (float)__builtin_fma(s[4 * i + 3], all, 0.0);
        }
        *reinterpret_cast<float4*>(&rows[slot][(i * LT + lane) * 4]) = q;
    }
    lds_order();
    if (first) rows[slot][e] = (float)d;
    lds_order();
    if (t >= P.T) return;
    L* out = (L*)P.dlogits + t * P.ld_out;
#pragma unroll
    for (int i = 0; i < NV / 4; i++) {
        const int e0 = (i * LT + lane) * 4;
        if (e0 >= P.E) continue;
        const float4 q = *reinterpret_cast<const float4*>(&rows[slot][e0]);
        const float v[4] = {q.x, q.y, q.z, q.w};
        if constexpr (sizeof(L) == 4) {
            if (P.vec_out && e0 + 4 <= P.E)
                *reinterpret_cast<float4*>(out + e0) = float4{v[0], v[1], v[2], v[3]};
            else
                for (int j = 0; j < 4; j++)
                    if (e0 + j < P.E) out[e0 + j] = v[j];
        } else {
            if (P.vec_out && e0 + 4 <= P.E)
                *reinterpret_cast<u32x2*>(out + e0) =
                    u32x2{bf16_hw(v[0]) | (bf16_hw(v[1]) << 16), bf16_hw(v[2]) | (bf16_hw(v[3]) << 16)};
            else
                for (int j = 0; j < 4; j++)
                    if (e0 + j < P.E) out[e0 + j] = (uint16_t)bf16_hw(v[j]);
        }
    }
}

namespace {

// A dispatch holds fewer than 2^32 work-items, so this many tokens at most go
// into one launch; more take several.
template <int LT>
constexpr int64_t kTokensPerLaunch = (((int64_t)1 << 32) / (kSelWaves * 64) - 1) * kSelWaves * (kWave / LT);
// P for its tokens [t0, T), as many as one launch takes.
template <int LT, typename L>
SelectParams launch_share(SelectParams P, int64_t t0) {
    P.logits = (const L*)P.logits + t0 * P.ld;
    P.T = std::min(P.T - t0, kTokensPerLaunch<LT>);
    if (P.ids) {
        P.ids += t0 * P.K;
        P.probs += t0 * P.K;
    } else {
        P.ids_in += t0 * P.K;
        P.dprobs += t0 * P.K;
        P.dlogits = (L*)P.dlogits + t0 * P.ld_out;
    }
    return P;
}

template <int LT, int NV, int LEN, typename L>
hipError_t select_run(const SelectParams& P, hipStream_t s) {
    constexpr int kTok = kSelWaves * (kWave / LT);
    const size_t lds = P.n_groups > 1 ? (size_t)kTok * P.lds_token * sizeof(double) : 0;
    for (int64_t t0 = 0; t0 < P.T; t0 += kTokensPerLaunch<LT>) {
        const SelectParams Q = launch_share<LT, L>(P, t0);
        hipLaunchKernelGGL((router_select_kernel<LT, NV, LEN, L>), dim3((unsigned)((Q.T + kTok - 1) / kTok)),
                           dim3(kSelWaves * 64), lds, s, Q);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}
template <int LT, int NV, typename L>
hipError_t select_len(const SelectParams& P, hipStream_t s) {
    if constexpr (NV > 8)
        return P.K <= 8 ? select_run<LT, NV, 8, L>(P, s) : select_run<LT, NV, NV, L>(P, s);
    else
        return select_run<LT, NV, NV, L>(P, s);
}
// 16 lanes a token hold up to 256 experts (16 a lane) and 16 slots; four times
// as many tokens a wavefront as with 64 lanes (T = 16384, K = 8: E = 256 with
// bias and groups 14.6 against 23.8 us, E = 128 softmax 5.9 against 14.1).
template <typename L>
hipError_t select_type(const SelectParams& P, hipStream_t s) {
    if (P.K <= 16 && P.E <= 64) return select_len<16, 4, L>(P, s);
    if (P.K <= 16 && P.E <= 128) return select_len<16, 8, L>(P, s);
    if (P.K <= 16 && P.E <= 256) return select_len<16, 16, L>(P, s);
    if (P.E <= 256) return select_len<64, 4, L>(P, s);
    if (P.E <= 512) return select_len<64, 8, L>(P, s);
    return select_len<64, 16, L>(P, s);
}
template <int LT, int NV, typename L>
hipError_t backward_run(const SelectParams& P, hipStream_t s) {
    constexpr int kTok = kSelWaves * (kWave / LT);
    for (int64_t t0 = 0; t0 < P.T; t0 += kTokensPerLaunch<LT>) {
        const SelectParams Q = launch_share<LT, L>(P, t0);
        hipLaunchKernelGGL((router_select_backward_kernel<LT, NV, L>), dim3((unsigned)((Q.T + kTok - 1) / kTok)),
                           dim3(kSelWaves * 64), 0, s, Q);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}
template <typename L>
hipError_t backward_type(const SelectParams& P, hipStream_t s) {
    if (P.K <= 16 && P.E <= 64) return backward_run<16, 4, L>(P, s);
    if (P.K <= 16 && P.E <= 128) return backward_run<16, 8, L>(P, s);
    if (P.K <= 16 && P.E <= 256) return backward_run<16, 16, L>(P, s);
    if (P.E <= 256) return backward_run<64, 4, L>(P, s);
    if (P.E <= 512) return backward_run<64, 8, L>(P, s);
    return backward_run<64, 16, L>(P, s);
}

}  // namespace

hipError_t launch_router_select(SelectParams P, bool bf16, hipStream_t stream) {
    // LDS of a token, in doubles: two values a run of four experts where groups
    // are whole runs, else one an expert; the groups' values; odd, so that the
    // tokens of a wavefront start in different banks.
    P.lds_token = ((P.group_size % 4 == 0 ? P.E / 2 : P.E) + P.n_groups) | 1;
    return bf16 ? select_type<uint16_t>(P, stream) : select_type<float>(P, stream);
}
hipError_t launch_router_select_backward(const SelectParams& P, bool bf16, hipStream_t stream) {
    return bf16 ? backward_type<uint16_t>(P, stream) : backward_type<float>(P, stream);
}

}  // namespace nvfp4
