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
// order is exact; with one, values closer than 2^-42 relative count as equal.
//
// LT lanes (16, or 64 for more than 256 experts or 16 slots) share a token, so
// a wavefront takes 4 tokens or one, each lane NV experts.  The lane sorts its
// keys once with a network; every slot then takes the maximum of the lanes'
// list heads (rotations within a row of 16 lanes) and the owner moves its list
// up.
#include "nvfp4_device.h"
#include "nvfp4_kernels.h"

namespace nvfp4 {

namespace {

constexpr int kSelWaves = 4;         // wavefronts per workgroup
constexpr double kUnavailable = -0x1p+1000;  // below every value, above "not kept" (-inf)
constexpr double kNotKept = -__builtin_inf();

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
    v = fmaxf(v, ror<8>(v));
    v = fmaxf(v, ror<4>(v));
    v = fmaxf(v, ror<2>(v));
    v = fmaxf(v, ror<1>(v));
    if (LT == 64) {
        v = fmaxf(v, __shfl_xor(v, 16, kWave));
        v = fmaxf(v, __shfl_xor(v, 32, kWave));
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

// e^x for x in [-708, 709]: x = n ln 2 + r, |r| <= ln 2 / 2, Taylor's series of
// e^r to r^12 (the next term is below 1.7e-16), scaled by 2^n.
__device__ __forceinline__ double exp64(double x) {
    const double n = __builtin_rint(x * 1.4426950408889634);
    double r = __builtin_fma(-n, 0x1.62e42fefa39efp-1, x);
    r = __builtin_fma(-n, 0x1.abc9e3b39803fp-56, r);
    double p = 1.0 / 479001600.0;
    p = __builtin_fma(p, r, 1.0 / 39916800.0);
    p = __builtin_fma(p, r, 1.0 / 3628800.0);
    p = __builtin_fma(p, r, 1.0 / 362880.0);
    p = __builtin_fma(p, r, 1.0 / 40320.0);
    p = __builtin_fma(p, r, 1.0 / 5040.0);
    p = __builtin_fma(p, r, 1.0 / 720.0);
    p = __builtin_fma(p, r, 1.0 / 120.0);
    p = __builtin_fma(p, r, 1.0 / 24.0);
    p = __builtin_fma(p, r, 1.0 / 6.0);
    p = __builtin_fma(p, r, 0.5);
    p = __builtin_fma(p, r, 1.0);
    p = __builtin_fma(p, r, 1.0);
    return __builtin_ldexp(p, (int)n);
}
// 1 / d for normal d > 0: the hardware estimate and two Newton steps.
__device__ __forceinline__ double rcp64(double d) {
    double r = __builtin_amdgcn_rcp(d);
    r = __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
    return __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
}
// e^x for x <= 0; 0 below the range of exp64.
__device__ __forceinline__ double exp64_neg(double x) { return x < -708.0 ? 0.0 : exp64(x); }
__device__ __forceinline__ double sigmoid64(float l) { return rcp64(1.0 + exp64(fmax(fmin(-(double)l, 708.0), -708.0))); }

constexpr float kFltMax = 3.402823466e+38f;
// A logit as the definitions take it: -inf where it is unusable, at most the largest finite value.
__device__ __forceinline__ float clean(float l) { return l > -__builtin_inff() ? fminf(l, kFltMax) : -__builtin_inff(); }

// Weight (before the scale) of a chosen expert in lane k < K, in FP64; `live`
// is false in the other lanes and for unavailable experts.  `max_l`, `den`:
// the softmax's maximum and denominator over all usable logits (only read for
// softmax weights without renormalisation).
template <int LT>
__device__ __forceinline__ double slot_weight(float l, bool live, bool sigmoid, bool renorm, float max_l, double den) {
    if (!renorm) {
        if (!live) return 0.0;
        return sigmoid ? sigmoid64(l) : exp64_neg((double)l - (double)max_l) / den;
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
    return live ? w / sum : 0.0;
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

__device__ __forceinline__ double key_of(double v, int e) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);  // -0 as +0
    return __builtin_bit_cast(double, (u & ~1023ull) | (uint64_t)((u >> 63) ? e : 1023 - e));
}
__device__ __forceinline__ int key_expert(double key) {
    const uint64_t u = __builtin_bit_cast(uint64_t, key);
    const int low = (int)(u & 1023u);
    return (u >> 63) ? low : 1023 - low;
}

}  // namespace

// LT lanes per token, NV experts per lane (E <= LT * NV), lists of LEN keys
// (the longest that K slots can take from one lane).
template <int LT, int NV, int LEN, typename L>
__global__ void __launch_bounds__(kSelWaves * 64) router_select_kernel(SelectParams P) {
    constexpr int kTok = kWave / LT;     // tokens per wavefront
    constexpr int kGroupRounds = kMaxGroups / LT;
    extern __shared__ __attribute__((aligned(16))) double smem[];  // only with groups
    const int lane = threadIdx.x & (LT - 1), slot = threadIdx.x / LT;
    const int64_t t = (int64_t)blockIdx.x * (kSelWaves * kTok) + slot;
    const int64_t tr = min(t, P.T - 1);  // rows past T repeat the last one, not stored
    const L* row = (const L*)P.logits + tr * P.ld;
    const bool sigmoid = P.sigmoid, biased = P.bias != nullptr, grouped = P.n_groups > 1;
    const bool top2 = grouped && P.top2, scores = biased || top2;

    float l[NV];
#pragma unroll
    for (int i = 0; i < NV / 4; i++) {
        float v[4];
        load4(row, (i * LT + lane) * 4, P.E, P.vec, v);
#pragma unroll
        for (int j = 0; j < 4; j++) l[4 * i + j] = clean(v[j]);
    }
    float max_l = 0.0f;
    double den = 1.0;
    const bool softmax_all = !sigmoid && (scores || !P.renorm);
    if (softmax_all) {
        float mx = l[0];
#pragma unroll
        for (int i = 1; i < NV; i++) mx = fmaxf(mx, l[i]);
        max_l = fmaxf(tok_max<LT>(mx), -kFltMax);
    }
    if (softmax_all && !scores) {  // the denominator alone: FP32 terms, no choice depends on it
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; i++) sum += __builtin_amdgcn_exp2f((l[i] - max_l) * 1.4426950408889634f);
        den = (double)tok_sum<LT>(sum);
    }
    double key[NV];
    double* gv = smem + (size_t)slot * (P.E + 8);  // this token's values, [expert in group][group]
    if (scores) {
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            double s;
            if (sigmoid)
                s = sigmoid64(fmaxf(l[i], -kFltMax));
            else
                s = exp64_neg((double)l[i] - (double)max_l);
            if (!(l[i] > -__builtin_inff())) s = 0.0;
            key[i] = s;
            sum += s;
        }
        if (!sigmoid) {
            den = fmax(tok_sum<LT>(sum), 1e-300);  // a row with nothing usable: all scores 0
            const double inv = 1.0 / den;
#pragma unroll
            for (int i = 0; i < NV; i++) key[i] *= inv;
        }
    }
#pragma unroll
    for (int i = 0; i < NV / 4; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const int n = 4 * i + j, e = (i * LT + lane) * 4 + j;
            bool live = l[n] > -__builtin_inff();
            double s = scores ? key[n] : 0.0;
            if (biased && e < P.E) {
                const float b = clean(P.bias[e]);
                live = live && b > -__builtin_inff();
                s += (double)b;
            }
            const double v = biased ? s : (double)l[n];
            if (grouped && e < P.E) {
                const int g = (int)(((uint32_t)e * P.group_magic) >> 22);
                gv[(e - g * P.group_size) * P.n_groups + g] = live ? (top2 ? s : v) : kNotKept;
            }
            key[n] = e < P.E ? key_of(live ? v : kUnavailable, e) : kNotKept;
        }
    if (grouped) {
        // Lane g ranks group g (and g + LT, ...): its value, then the count of
        // groups before it; the kept ones become a bit mask.
        double* gs = smem + (size_t)kSelWaves * kTok * (P.E + 8) + slot * kMaxGroups;
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kGroupRounds; r++) {
            const int g = r * LT + lane;
            if (g < P.n_groups) {
                double b1 = kNotKept, b2 = kNotKept;
                for (int w = 0; w < P.group_size; w++) {
                    const double v = gv[w * P.n_groups + g];
                    b2 = max64(b2, min64(b1, v));
                    b1 = max64(b1, v);
                }
                gs[g] = top2 && b2 > kNotKept ? b1 + b2 : b1;
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
        for (int n = 0; n < NV; n++) {
            const int e = ((n >> 2) * LT + lane) * 4 + (n & 3);
            const int g = (int)(((uint32_t)e * P.group_magic) >> 22);
            if (!((kept >> (g & 63)) & 1)) key[n] = kNotKept;
        }
    }
    sort_desc(key);
    double mine = kNotKept;
    for (int k = 0; k < P.K; k++) {
        const double best = tok_max<LT>(key[0]);
        if (lane == k) mine = best;
        const bool pop = key[0] == best;  // keys are unique: one owner
#pragma unroll
        for (int i = 0; i < LEN; i++) {
            const double next = i + 1 < LEN ? key[i + 1] : kNotKept;
            key[i] = pop ? next : key[i];
        }
    }
    const bool have = lane < P.K;
    const int e = have ? min(key_expert(mine), P.E - 1) : 0;
    const bool live = have && mine > kUnavailable * 0.5;
    const float lk = live ? clean(load1(row + e)) : 0.0f;
    const double w = slot_weight<LT>(lk, live, sigmoid, P.renorm, max_l, den);
    if (have && t < P.T) {
        P.ids[t * P.K + lane] = e;
        P.probs[t * P.K + lane] = (float)(w * (double)P.scale);
    }
}

// The gradient of the weights with respect to the logits.  With c the scale,
// dp the upstream gradient and w the weights of the chosen experts:
//   renormalised  d_k = c w_k (dp_k - sum_j dp_j w_j), times (1 - sigma_k) for sigmoid scores;
//   sigmoid       d_k = c w_k dp_k (1 - sigma_k);
//   softmax       d_k = c w_k dp_k at the chosen experts, and -c s_e sum_j dp_j w_j at every expert.
// One pass: lane k forms d_k in FP64 (K values a token), slots of one expert
// are added in slot order into the token's row in LDS, and the row is written
// whole, so the kernel is bound by writing [T, E].
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
    float max_l = 0.0f;
    double den = 1.0;
    if (dense) {
        float mx = -kFltMax;
#pragma unroll
        for (int i = 0; i < NV / 4; i++) {
            float v[4];
            load4(row, (i * LT + lane) * 4, P.E, P.vec, v);
#pragma unroll
            for (int j = 0; j < 4; j++) mx = fmaxf(mx, l[4 * i + j] = clean(v[j]));
        }
        max_l = tok_max<LT>(mx);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; i++) sum += l[i] = __builtin_amdgcn_exp2f((l[i] - max_l) * 1.4426950408889634f);
        den = fmax((double)tok_sum<LT>(sum), 1e-300);
    }
#pragma unroll
    for (int i = 0; i < NV / 4; i++)
        *reinterpret_cast<float4*>(&rows[slot][(i * LT + lane) * 4]) = float4{0.0f, 0.0f, 0.0f, 0.0f};
    const bool in = e >= 0 && e < P.E;
    const float lk = in ? clean(load1(row + e)) : 0.0f;
    const bool live = in && lk > -__builtin_inff() && !(P.bias && !(P.bias[in ? e : 0] > -__builtin_inff()));
    const double w = slot_weight<LT>(lk, live, sigmoid, P.renorm, max_l, den);
    const double mean = tok_sum<LT>(live ? w * (double)dp : 0.0);
    double d = 0.0;
    if (live) {
        d = w * (P.renorm ? (double)dp - mean : (double)dp) * (double)P.scale;
        if (sigmoid) d *= sigmoid64(-lk);  // 1 - sigma(l)
    }
    // A repeated expert: its first slot takes the sum, in slot order.
    float acc = 0.0f;
    bool first = live;
    for (int k = 0; k < P.K; k++) {
        const int ek = __shfl(live ? e : -1, k, LT);
        const float dk = __shfl((float)d, k, LT);
        if (ek == e) {
            acc += dk;
            first = first && k >= lane;
        }
    }
    __syncthreads();
    if (first) rows[slot][e] = acc;
    __syncthreads();
    if (t >= P.T) return;
    const float all = dense ? (float)(-mean * (double)P.scale / den) : 0.0f;
    L* out = (L*)P.dlogits + t * P.ld_out;
#pragma unroll
    for (int i = 0; i < NV / 4; i++) {
        const int e0 = (i * LT + lane) * 4;
        if (e0 >= P.E) continue;
        const float4 q = *reinterpret_cast<const float4*>(&rows[slot][e0]);
        float v[4] = {q.x, q.y, q.z, q.w};
        if (dense)
#pragma unroll
            for (int j = 0; j < 4; j++) v[j] = __builtin_fmaf(l[4 * i + j], all, v[j]);
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

template <int LT, int NV, int LEN, typename L>
hipError_t select_run(const SelectParams& P, hipStream_t s) {
    constexpr int kTok = kSelWaves * (kWave / LT);
    const size_t lds = P.n_groups > 1 ? (size_t)kTok * (P.E + 8 + kMaxGroups) * 8 : 0;
    hipLaunchKernelGGL((router_select_kernel<LT, NV, LEN, L>), dim3((unsigned)((P.T + kTok - 1) / kTok)),
                       dim3(kSelWaves * 64), lds, s, P);
    return hipGetLastError();
}
template <int LT, int NV, typename L>
hipError_t select_len(const SelectParams& P, hipStream_t s) {
    if constexpr (NV > 8)
        return P.K <= 8 ? select_run<LT, NV, 8, L>(P, s) : select_run<LT, NV, NV, L>(P, s);
    else
        return select_run<LT, NV, NV, L>(P, s);
}
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
    hipLaunchKernelGGL((router_select_backward_kernel<LT, NV, L>), dim3((unsigned)((P.T + kTok - 1) / kTok)),
                       dim3(kSelWaves * 64), 0, s, P);
    return hipGetLastError();
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

hipError_t launch_router_select(const SelectParams& P, bool bf16, hipStream_t stream) {
    return bf16 ? select_type<uint16_t>(P, stream) : select_type<float>(P, stream);
}
hipError_t launch_router_select_backward(const SelectParams& P, bool bf16, hipStream_t stream) {
    return bf16 ? backward_type<uint16_t>(P, stream) : backward_type<float>(P, stream);
}

}  // namespace nvfp4
