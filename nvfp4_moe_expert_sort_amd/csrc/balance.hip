// balance.hip -- the router's balance loss, the experts' token counts, and the
// loss's gradient (include/nvfp4moe.h, nvfp4moe_router_balance_loss).
//
// With n_se the slots of sequence s that name expert e, p_t the token's
// probabilities over all experts and T' the tokens of all sequences:
//   loss = coef E / (K T') sum_s 1 / T_s sum_e n_se sum_{t in s} p_te
//   d/dl_te = coef E / (K T' T_s) p_te (n_se - sum_j n_sj p_tj)  [(1 - sigma_te)]
// The counts are constants of the gradient.
#include <algorithm>

#include "nvfp4_device.h"
#include "nvfp4_kernels.h"
#include "router_lanes.h"

namespace nvfp4 {

namespace {

constexpr int kBalThreads = 256;     // of the gradient
constexpr int kChunkThreads = 1024;  // of the loss: 64 tokens at a time, or 16
constexpr int kJoinThreads = 1024;   // 16 stripes of 64 experts

// e^d for d <= 0 within a few 2^-24 wherever it is a normal number: the part
// of d log2 e that its rounding to FP32 drops is put back to first order.
__device__ __forceinline__ float exp_neg(float d) {
    d = max32(d, -150.0f);
    const float t = d * 1.44269502f;
    float r = __builtin_fmaf(d, 1.44269502f, -t);
    r = __builtin_fmaf(d, 1.92596299e-8f, r);
    const float e = __builtin_amdgcn_exp2f(t);
    return __builtin_fmaf(e, r * 0.693147182f, e);
}

// Sum over a wavefront, in all lanes, in one order.
template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
    return v;
}

// Terms w_e >= 0 of the token's probabilities, p_e = w_e / sum w, from its
// clean logits; for sigmoid scores other = 1 - sigma.  Both are shifted so
// that the sum cannot vanish: by the largest logit, or for sigmoid scores by
// m = min(largest, 0), sigma(l) e^-m = e^(l - m) / (1 + e^l).
template <int LT, int NV>
__device__ __forceinline__ void score_terms(const float (&l)[NV], bool sigmoid, float (&w)[NV], float (&other)[NV]) {
    float mx = l[0];
#pragma unroll
    for (int i = 1; i < NV; i++) mx = max32(mx, l[i]);
    mx = max32(tok_max<LT>(mx), -kFltMax);
    if (sigmoid && __ballot(mx < 0.0f) == 0) {  // (no token of the wavefront has m < 0: e^(l - m) is e^-|l| again)
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const bool neg = l[i] < 0.0f;
            const float t = exp_neg(-fabsf(l[i])), inv = __builtin_amdgcn_rcpf(1.0f + t), ti = t * inv;
            w[i] = neg ? ti : inv;
            w[i] = l[i] > -__builtin_inff() ? w[i] : 0.0f;
            other[i] = neg ? inv : ti;
        }
    } else if (sigmoid) {
        mx = min32(mx, 0.0f);
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const bool neg = l[i] < 0.0f;
            const float t = exp_neg(-fabsf(l[i])), inv = __builtin_amdgcn_rcpf(1.0f + t);
            w[i] = l[i] > -__builtin_inff() ? (neg ? exp_neg(l[i] - mx) * inv : inv) : 0.0f;
            other[i] = neg ? inv : t * inv;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; i++) {
            w[i] = l[i] > -__builtin_inff() ? exp_neg(l[i] - mx) : 0.0f;
            other[i] = 1.0f;
        }
    }
}

// First row of sequence s (of S; s == S: the end of the last), within [0, T].
__device__ __forceinline__ int64_t seq_start(const BalanceParams& P, int32_t s) {
    if (!P.offsets) return s == 0 ? 0 : P.T;
    return min(max((int64_t)P.offsets[s], (int64_t)0), P.T);
}
// The sequence that holds row t, -1 before the first and S behind the last:
// how many of the S + 1 offsets are <= t, less one.  All threads call it.
template <int kThreads>
__device__ __forceinline__ int32_t find_sequence(const BalanceParams& P, int64_t t, int32_t* lds) {
    if (!P.offsets) return 0;
    int32_t n = 0;
    if (P.S < 256) {  // every wavefront by itself
        for (int32_t i = threadIdx.x & 63; i <= P.S; i += 64) n += seq_start(P, i) <= t ? 1 : 0;
        return wave_sum(n) - 1;
    }
    // Of many, first every step-th one.
    auto count = [&](int32_t from, int32_t step, int32_t len) {
        int32_t c = 0;
        for (int32_t i = threadIdx.x; i < len; i += kThreads) c += seq_start(P, from + i * step) <= t ? 1 : 0;
        c = wave_sum(c);
        __syncthreads();
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = c;
        __syncthreads();
        c = 0;
        for (int w = 0; w < kThreads / 64; w++) c += lds[w];
        return c;
    };
    int32_t from = 0, len = P.S + 1;
    if (len > kThreads) {
        const int32_t step = (len + kThreads - 1) / kThreads;
        n = count(0, step, (len + step - 1) / step);
        if (n == 0) return -1;
        from = (n - 1) * step;
        len = min(step, len - from);
    }
    return from + count(from, 1, len) - 1;
}

// The last sequence that starts at row t or before it (S: t lies behind them all),
// of which sequence s is one.  64 offsets a step, by every wavefront for itself.
__device__ __forceinline__ int32_t last_start(const BalanceParams& P, int32_t s, int64_t t) {
    for (int32_t left = P.S - s; left > 0;) {
        const int32_t step = (left + 63) / 64, at = s + ((threadIdx.x & 63) + 1) * step;
        s += __popcll(__ballot(at <= P.S && seq_start(P, min(at, P.S)) <= t)) * step;
        left = min(step - 1, P.S - s);
    }
    return s;
}

// The loss of sum_s 1 / T_s sum_e n_se sum_t p_te.
__device__ __forceinline__ float balance_scaled(const BalanceParams& P, double total) {
    const double tokens = (double)max(seq_start(P, P.S) - seq_start(P, 0), (int64_t)1);
    return (float)(total * (double)P.coef * (double)P.E / ((double)P.K * tokens));
}

template <int LT, int NV, typename L>
__device__ __forceinline__ void load_row(const L* row, const BalanceParams& P, int lane, float (&l)[NV]) {
#pragma unroll
    for (int i = 0; i < NV / 4; i++) {
        float v[4];
        load4(row, (i * LT + lane) * 4, P.E, P.vec, v);
#pragma unroll
        for (int j = 0; j < 4; j++) l[4 * i + j] = clean(v[j]);
    }
}

}  // namespace

// A workgroup takes P.chunk rows, kTok at a time.  Their probabilities are
// formed once, whatever sequences they belong to, and then added up sequence by
// sequence (a lane its own experts over its tokens, then the wavefront's token
// slots by exchanges, then the wavefronts in LDS), like the counts: a workgroup
// whose rows belong to several, which the kernel's end waits for, repeats only
// the sums (16384 rows of 256 experts in 13 sequences 13.5 us; with the whole pass
// repeated 18).
// Chunk b's part of sequence s goes to slot b + s: a walk along the rows raises
// b or s at every step, so no two parts share one.  A call of one chunk has its
// sequences whole here and needs no join.
// 16384 rows of 256 experts: 11 us for 17 MB (3.3 us at the rate of a large
// copy).  3 of it is the launch, 2 the exponentials; the rest is one chain from
// the loads to the sums in LDS, a pass a workgroup.
template <int LT, int NV, typename L>
__global__ void __launch_bounds__(kChunkThreads) balance_chunk_kernel(BalanceParams P) {
    constexpr int kTok = kChunkThreads / LT, kWaves = kChunkThreads / 64;
    constexpr int kIds = (kTok * kMaxTopK + kChunkThreads - 1) / kChunkThreads;
    __shared__ __attribute__((aligned(16))) float part[kWaves][LT * NV];
    __shared__ int32_t hist[LT * NV];
    __shared__ int32_t found[kWaves];
    __shared__ double shares[kWaves];
    const int lane = threadIdx.x & (LT - 1), slot = threadIdx.x / LT, wave = threadIdx.x >> 6;
    const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;  // (past the last chunk, no rows)
    const int64_t first = block * P.chunk, past = min(P.T, first + P.chunk);
    const bool whole = gridDim.x == 1;
    double total = 0.0;  // whole: the thread's part of loss / factor
    int32_t s_next = 0;  // whole: the first sequence whose counts are not written
    if (!whole && block == 0 && threadIdx.x == 0) *P.done = 0;
    float l[NV], acc[NV];
    int32_t id[kIds], id_tok[kIds];  // the thread's ids of a pass, and which token's each is
    auto load = [&](int64_t t0) {
        load_row<LT, NV, L>((const L*)P.logits + min(t0 + slot, past - 1) * P.ld, P, lane, l);
#pragma unroll
        for (int j = 0; j < kIds; j++)
            id[j] = id_tok[j] < min((int64_t)kTok, past - t0) ? P.ids[t0 * P.K + j * kChunkThreads + threadIdx.x] : -1;
    };
#pragma unroll
    for (int j = 0; j < kIds; j++) id_tok[j] = (j * kChunkThreads + (int)threadIdx.x) / P.K;
    if (first < past) load(first);  // (on its way while the sequence is looked up)
#pragma unroll
    for (int i = 0; i < NV; i++) acc[i] = 0.0f;
    for (int e = threadIdx.x; e < P.E; e += kChunkThreads) hist[e] = 0;
    // The sequence that the walk has come to, and its rows.
    int32_t s = max(find_sequence<kChunkThreads>(P, first, found), 0);
    int64_t lo = seq_start(P, min(s, P.S)), hi = seq_start(P, min(s + 1, P.S)), next = seq_start(P, min(s + 2, P.S));
    __syncthreads();
    // Writes the sums and counts of the sequence's rows in this chunk, and clears them.
    auto flush = [&] {
        if constexpr (LT == 16) {
            // Of each two values, the half of the wavefront that adds up the first
            // gives the other half its part of the second; so do the halves' rows of
            // 16 lanes.  Row r is left with the sums of acc[r NV / 4] and on (every lane
            // fetching all of its counterparts' values: 3 us more of 13).
            constexpr int kLeft = NV / 4;
            float sum2[2 * kLeft], sum4[kLeft];
#pragma unroll
            for (int i = 0; i < 2 * kLeft; i++) {
                const auto v = __builtin_amdgcn_permlane32_swap(__float_as_uint(acc[i]), __float_as_uint(acc[i + 2 * kLeft]),
                                                                false, false);
                sum2[i] = __uint_as_float(v[0]) + __uint_as_float(v[1]);
            }
#pragma unroll
            for (int i = 0; i < kLeft; i++) {
                const auto v = __builtin_amdgcn_permlane16_swap(__float_as_uint(sum2[i]), __float_as_uint(sum2[i + kLeft]),
                                                                false, false);
                sum4[i] = __uint_as_float(v[0]) + __uint_as_float(v[1]);
            }
            const int first_acc = (threadIdx.x & 63) / 16 * kLeft;
            float* to = &part[wave][(first_acc / 4 * LT + lane) * 4 + first_acc % 4];
#pragma unroll
            for (int i = 0; i < kLeft; i++) to[i] = sum4[i];
        } else {
#pragma unroll
            for (int i = 0; i < NV / 4; i++)
                *reinterpret_cast<float4*>(&part[wave][(i * LT + lane) * 4]) =
                    float4{acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]};
        }
#pragma unroll
        for (int i = 0; i < NV; i++) acc[i] = 0.0f;
        __syncthreads();
        const int64_t at = (whole ? s : block + s) * P.E;
        static_assert(kMaxExperts <= kChunkThreads, "an expert a thread");
        if (const int e = threadIdx.x; e < P.E) {
            float sum = 0.0f;
#pragma unroll
            for (int k = 0; k < kWaves; k++) sum += part[k][e];
            const int32_t n = hist[e];
            hist[e] = 0;
            if (whole) {
                P.counts[at + e] = n;
                total += (double)sum * (double)n / (double)(hi - lo);
            } else {
                P.psum[at + e] = sum;
                P.csum[at + e] = n;
            }
        }
        if (whole) {
            for (int64_t i = (int64_t)s_next * P.E + threadIdx.x; i < (int64_t)s * P.E; i += kChunkThreads) P.counts[i] = 0;
            s_next = s + 1;
        }
        __syncthreads();
    };
    for (int64_t t0 = first; t0 < past; t0 += kTok) {
        if (t0 > first) load(t0);
        const int64_t end = min(t0 + kTok, past);
        float w[NV], other[NV];
        score_terms<LT, NV>(l, P.sigmoid, w, other);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; i++) sum += w[i];
        sum = tok_sum<LT>(sum);
        const float inv = t0 + slot < end && sum > 0.0f ? 1.0f / sum : 0.0f;
        while (s < P.S && lo < end) {
            if (hi > max(lo, t0)) {
                const int from = (int)max(lo - t0, (int64_t)0), to = (int)min(hi - t0, end - t0);  // of the pass's tokens
                const float in = slot >= from && slot < to ? inv : 0.0f;
#pragma unroll
                for (int i = 0; i < NV; i++) acc[i] = __builtin_fmaf(w[i], in, acc[i]);
#pragma unroll
                for (int j = 0; j < kIds; j++)
                    if (id_tok[j] >= from && id_tok[j] < to && id[j] >= 0 && id[j] < P.E) atomicAdd(&hist[id[j]], 1);
                if (hi <= end || end == past) flush();
            }
            if (hi > end || (hi == end && end == past)) break;
            s++;
            lo = hi;
            hi = next;
            if (hi == lo && s < P.S) {  // without rows: on to the next that has some (40000 such one by one: 15 ms)
                s = last_start(P, s, lo);
                hi = seq_start(P, min(s + 1, P.S));
            }
            next = seq_start(P, min(s + 2, P.S));  // (on its way until the sequence after this one)
        }
    }
    if (whole) {  // (sequences without rows have no counts)
        for (int64_t i = (int64_t)s_next * P.E + threadIdx.x; i < (int64_t)P.S * P.E; i += kChunkThreads) P.counts[i] = 0;
        total = wave_sum(total);
        if ((threadIdx.x & 63) == 0) shares[wave] = total;
        __syncthreads();
        if (threadIdx.x == 0) {
            total = 0.0;
            for (int k = 0; k < kWaves; k++) total += shares[k];
            *P.loss = balance_scaled(P, total);
        }
    }
}

// Adds the slots of one sequence and 64 experts in FP64, in one order: a
// workgroup by 16 stripes of slots or, of so many that a workgroup each would
// queue at the counter below (16384 of one row: 466 us a call, so 94), a wavefront.
// The workgroup that is last to finish adds up the workgroups' shares of the
// loss.  Each share is one value, stored and loaded at the scope of the device,
// which no L2 keeps for itself, and stored for certain before its workgroup is
// counted: with nothing else handed over, no cache has to be written back or
// dropped (two fences: 7.8 us a launch at 13 sequences of 256 experts; so: 5.0).
constexpr int kStripes = kJoinThreads / 64, kJoinItems = 1024;  // items up to which each has a workgroup
__global__ void __launch_bounds__(kJoinThreads) balance_join_kernel(BalanceParams P) {
    constexpr int kAhead = 4;
    __shared__ double sums[kStripes][64];
    __shared__ int32_t cnts[kStripes][64];
    __shared__ bool last;
    const int32_t groups = (P.E + 63) / 64, items = P.S * groups;
    const int col = threadIdx.x & 63, stripe = threadIdx.x >> 6;
    double sum = 0.0, share = 0.0;
    int32_t n = 0;
    // Every `step`-th slot of a sequence's.
    auto add = [&](int64_t lo, int64_t hi, int32_t s, int32_t e, int32_t first, int32_t step) {
        sum = 0.0;
        n = 0;
        if (hi <= lo || e >= P.E) return;
        const int64_t b1 = (hi - 1) / P.chunk;
        for (int64_t b = lo / P.chunk + first; b <= b1; b += step * kAhead) {
            float p[kAhead];
            int32_t c[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; k++) {
                const int64_t at = (min(b + k * step, b1) + s) * P.E + e;
                p[k] = P.psum[at];
                c[k] = P.csum[at];
            }
#pragma unroll
            for (int k = 0; k < kAhead; k++)
                if (b + k * step <= b1) {
                    sum += (double)p[k];
                    n += c[k];
                }
        }
    };
    auto end = [&](int64_t lo, int64_t hi, int32_t s, int32_t e) {
        if (e >= P.E) return;
        P.counts[(int64_t)s * P.E + e] = n;
        if (hi > lo) share += sum * (double)n / (double)(hi - lo);
    };
    if (items > kJoinItems) {
        for (int32_t item = blockIdx.x * kStripes + stripe; item < items; item += gridDim.x * kStripes) {
            const int32_t s = item / groups, e = item % groups * 64 + col;
            const int64_t lo = seq_start(P, s), hi = seq_start(P, s + 1);
            add(lo, hi, s, e, 0, 1);
            end(lo, hi, s, e);
        }
    } else {
        const int32_t s = blockIdx.x / groups, e = blockIdx.x % groups * 64 + col;
        const int64_t lo = seq_start(P, s), hi = seq_start(P, s + 1);
        add(lo, hi, s, e, stripe, kStripes);
        sums[stripe][col] = sum;
        cnts[stripe][col] = n;
        __syncthreads();
        if (stripe == 0) {
            sum = 0.0;
            n = 0;
#pragma unroll
            for (int k = 0; k < kStripes; k++) {
                sum += sums[k][col];
                n += cnts[k][col];
            }
            end(lo, hi, s, e);
        }
        __syncthreads();
    }
    // The workgroup's share, from its wavefronts' (of few items, the first has it).
    share = wave_sum(share);
    if (col == 0) sums[0][stripe] = share;
    __syncthreads();
    if (threadIdx.x == 0) {
        share = 0.0;
        for (int k = 0; k < kStripes; k++) share += sums[0][k];
        __hip_atomic_store(&P.part[blockIdx.x], share, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0);  // the store has reached memory
        asm volatile("" ::: "memory");
        last = __hip_atomic_fetch_add(P.done, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    double total = 0.0;
    for (uint32_t i = threadIdx.x; i < gridDim.x; i += kJoinThreads)
        total += __hip_atomic_load(&P.part[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    total = wave_sum(total);
    if (col == 0) sums[0][stripe] = total;
    __syncthreads();
    if (threadIdx.x == 0) {
        total = 0.0;
        for (int k = 0; k < kStripes; k++) total += sums[0][k];
        *P.loss = balance_scaled(P, total);
    }
}

// One token per LT lanes.  With w the terms of p, D their sum and G = sum w n:
//   d_e = c w_e (n_e D - G) / D^2
// where D, G and the difference are FP64: for a token whose top expert has
// nearly all the probability, n_e - sum n p is small against its terms, and
// here only the relative errors of the w remain (some 2^-23 each).
// 32749 rows of 128 experts in BF16: 12 us for 17 MB, of which 68 vector
// instructions a logit take some 7; then the chain from a sequence's offsets to its
// counts.
template <int LT, int NV, typename L>
__global__ void __launch_bounds__(kBalThreads) balance_backward_kernel(BalanceParams P) {
    constexpr int kTok = kBalThreads / LT;
    __shared__ int32_t found[4];
    const int lane = threadIdx.x & (LT - 1), slot = threadIdx.x / LT;
    const double tokens = (double)max(seq_start(P, P.S) - seq_start(P, 0), (int64_t)1);
    const double factor = (double)(P.dloss ? *P.dloss : 1.0f) * (double)P.coef * (double)P.E;
    for (int64_t tile = blockIdx.x; tile * kTok < P.T; tile += gridDim.x) {
        const int64_t t = tile * kTok + slot, tr = min(t, P.T - 1);
        float l[NV], w[NV], other[NV], add[NV];
        load_row<LT, NV, L>((const L*)P.logits + tr * P.ld, P, lane, l);
#pragma unroll
        for (int i = 0; i < NV / 4; i++) {
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (P.add) load4((const L*)P.add + tr * P.ld_add, (i * LT + lane) * 4, P.E, P.vec_add, v);
#pragma unroll
            for (int j = 0; j < 4; j++) add[4 * i + j] = v[j];
        }
        int32_t s = max(find_sequence<kBalThreads>(P, tile * kTok, found), 0);
        // The token's own, by steps that double and then halve: between the tile's rows
        // there may be thousands of sequences without any (40000 one by one: 8 ms).
        int32_t step = 1;
        for (; s + step <= P.S && seq_start(P, s + step) <= tr; step *= 2) s += step;
        while ((step /= 2) > 0)
            if (s + step <= P.S && seq_start(P, s + step) <= tr) s += step;
        double rows = 0.0;  // of the sequence; rows of none get no gradient
        if (s < P.S) {
            const int64_t lo = seq_start(P, s), hi = seq_start(P, s + 1);
            if (tr >= lo && hi > lo) rows = (double)(hi - lo);
        }
        const int32_t* counts = P.counts_in + (int64_t)min(s, P.S - 1) * P.E;
        float n[NV];
#pragma unroll
        for (int i = 0; i < NV / 4; i++) {
            const int e0 = (i * LT + lane) * 4;
            if (P.vec_counts && e0 + 4 <= P.E) {
                const int4 q = *reinterpret_cast<const int4*>(counts + e0);
                n[4 * i] = __int_as_float(q.x), n[4 * i + 1] = __int_as_float(q.y);
                n[4 * i + 2] = __int_as_float(q.z), n[4 * i + 3] = __int_as_float(q.w);
            } else {
#pragma unroll
                for (int j = 0; j < 4; j++) n[4 * i + j] = __int_as_float(e0 + j < P.E ? counts[e0 + j] : 0);
            }
        }
        score_terms<LT, NV>(l, P.sigmoid, w, other);
        double D = 0.0, G = 0.0;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            D += (double)w[i];
            G = __builtin_fma((double)w[i], (double)__float_as_int(n[i]), G);
        }
        D = tok_sum<LT>(D);
        G = tok_sum<LT>(G);
        // One division for all of c and D^2: an FP64 division is some 35 instructions, of 550 in all.
        const double den = (double)P.K * tokens * rows * (D * D), c = den > 0.0 ? factor / den : 0.0;
        if (t >= P.T) continue;
        L* out = (L*)P.dlogits + t * P.ld_out;
#pragma unroll
        for (int i = 0; i < NV / 4; i++) {
            const int e0 = (i * LT + lane) * 4;
            if (e0 >= P.E) continue;
            float v[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const int k = 4 * i + j;
                const double d = c * (double)(w[k] * other[k]) * __builtin_fma((double)__float_as_int(n[k]), D, -G);
                v[j] = w[k] > 0.0f ? (float)(d + (double)add[k]) : add[k];  // (c may be infinite or NaN, like dloss)
            }
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
}

namespace {

template <int LT, int NV, typename L>
hipError_t loss_run(const BalanceParams& P, hipStream_t s) {
    const int64_t chunks = std::max<int64_t>(1, (P.T + P.chunk - 1) / P.chunk);
    // (a launch has fewer than 2^32 threads along x: 2^22 chunks are too many)
    const int64_t x = std::min<int64_t>(chunks, 1 << 21);
    hipLaunchKernelGGL((balance_chunk_kernel<LT, NV, L>), dim3((unsigned)x, (unsigned)((chunks + x - 1) / x)),
                       dim3(kChunkThreads), 0, s, P);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || chunks == 1) return e;
    const int items = P.S * ((P.E + 63) / 64);
    const int groups = items > kJoinItems ? std::min((items + kStripes - 1) / kStripes, 512) : items;
    hipLaunchKernelGGL(balance_join_kernel, dim3((unsigned)groups), dim3(kJoinThreads), 0, s, P);
    return hipGetLastError();
}
template <int LT, int NV, typename L>
hipError_t balance_backward_run(const BalanceParams& P, hipStream_t s) {
    constexpr int kTok = kBalThreads / LT;
    const int64_t tiles = (P.T + kTok - 1) / kTok;
    hipLaunchKernelGGL((balance_backward_kernel<LT, NV, L>), dim3((unsigned)std::min<int64_t>(tiles, 65536)),
                       dim3(kBalThreads), 0, s, P);
    return hipGetLastError();
}
// 16 lanes a token hold up to 256 experts, 64 lanes up to 1024.
template <typename L>
hipError_t balance_type(const BalanceParams& P, hipStream_t s) {
    const bool back = P.dlogits != nullptr;
    if (P.E <= 64) return back ? balance_backward_run<16, 4, L>(P, s) : loss_run<16, 4, L>(P, s);
    if (P.E <= 128) return back ? balance_backward_run<16, 8, L>(P, s) : loss_run<16, 8, L>(P, s);
    if (P.E <= 256) return back ? balance_backward_run<16, 16, L>(P, s) : loss_run<16, 16, L>(P, s);
    if (P.E <= 512) return back ? balance_backward_run<64, 8, L>(P, s) : loss_run<64, 8, L>(P, s);
    return back ? balance_backward_run<64, 16, L>(P, s) : loss_run<64, 16, L>(P, s);
}

}  // namespace

// Rows of a workgroup of the loss.  All of a few rows, whose single launch takes
// less than a second one would (256 rows of 128 experts: 10.5 against 14.3 us, in 4
// sequences 12.6 against 14.1, in 8 16.1 against 14.2; of 256 experts 14.2 against
// 14.9).  Else one pass of its token slots and, so that there are at most 512
// workgroups (of more than 256 experts 256, one a CU: 16384 rows of 1024 experts 24
// against 31 us), up to 256 (a lane then adds 4 tokens, or 16 in rows of more than 256
// experts, in FP32 before FP64 takes over); but fewer where the sequences are so
// short that a workgroup would add up more than some 4 of them, 0.9 us each (256
// rows in 64 sequences: 23 us by 64 rows, 14.4 by 16).
int32_t balance_chunk(int64_t T, int64_t E, int64_t S) {
    if (T <= kBalanceOneLaunch && T * E <= kBalanceOneLogits && S <= kBalanceOneSequences) return kBalanceOneLaunch;
    int32_t chunk = E <= 256 ? 64 : 16;
    while (chunk < 256 && (T + chunk - 1) / chunk > (E <= 256 ? 512 : 256)) chunk *= 2;
    while (chunk > 16 && S * chunk > 4 * T) chunk /= 2;
    return chunk;
}

hipError_t launch_balance(const BalanceParams& P, bool bf16, hipStream_t stream) {
    return bf16 ? balance_type<uint16_t>(P, stream) : balance_type<float>(P, stream);
}

}  // namespace nvfp4
