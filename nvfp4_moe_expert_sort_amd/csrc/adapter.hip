// adapter.hip -- low-rank adapters of many requests beside a shared projection,
// and their gradients (include/nvfp4moe.h, nvfp4moe_adapter_linear).
//
// Row r with adapter a: v = A_a x_r, out_r = base_r + scale_a B_a v.  For dy:
// w = B_a^T dy_r, dx_r = base_r + A_a^T scale_a w, dA_a = scale_a sum w x_r^T,
// dB_a = scale_a sum dy_r v^T.  The gradient with respect to x is the forward
// operation with B^T and A^T in the places of A and B, so one kernel serves
// both, on transposed copies of the adapters.
#include <algorithm>

#include "nvfp4_device.h"
#include "nvfp4_kernels.h"

namespace nvfp4 {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kAdWaves = 8;          // wavefronts that share the first product's K
constexpr int kPlanThreads = 1024;
constexpr int kBins = kMaxExperts + 1;  // adapters, and the rows without one

__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ u32x4 load16(const uint16_t* p) { return *reinterpret_cast<const u32x4*>(p); }

// v as the sum of BF16 values of falling size, each the rounding of what the
// ones before it leave; an infinite or NaN v is the first of them alone.
__device__ __forceinline__ uint32_t bf16_piece(float& rest) {
    const uint32_t b = bf16_hw(rest);
    const float r = rest - bf16_to_f32(b);
    rest = fabsf(r) < __builtin_inff() ? r : 0.0f;
    return b;
}

// Sum over the workgroup's earlier entries of a[0..n), in place; every thread calls it.
__device__ __forceinline__ void block_scan(int32_t* a, int n, int32_t* lds) {
    const int per = (n + kPlanThreads - 1) / kPlanThreads, lo = min((int)threadIdx.x * per, n), hi = min(lo + per, n);
    int32_t sum = 0;
    for (int i = lo; i < hi; i++) sum += a[i];
    int32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int32_t v = __shfl_up(incl, o, kWave);
        if ((threadIdx.x & 63) >= o) incl += v;
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 63) lds[threadIdx.x >> 6] = incl;
    __syncthreads();
    int32_t run = incl - sum;
    for (int w = 0; w < (int)(threadIdx.x >> 6); w++) run += lds[w];
    for (int i = lo; i < hi; i++) {
        const int32_t v = a[i];
        a[i] = run;
        run += v;
    }
    __syncthreads();
}

// The bin whose range of a table holds entry i: start[0..n) does not decrease.
__device__ __forceinline__ int find_bin(const int32_t* start, int n, int32_t i) {
    int lo = 0, hi = n;  // start[lo] <= i < start[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        (start[mid] <= i ? lo : hi) = mid;
    }
    return lo;
}

__device__ __forceinline__ int bin_of(const AdapterPlan& P, int32_t id) { return id >= 0 && id < P.n ? id : P.n; }

// Counts the bins of the lanes' four consecutive rows in LDS, of which the
// first `live` exist.  Neighbouring rows mostly share an adapter: one lane then
// adds for all.
__device__ __forceinline__ void count4(int32_t* hist, const AdapterPlan& P, int4 id, int64_t live) {
    if (live <= 0) return;
    const int b0 = bin_of(P, id.x), b1 = bin_of(P, id.y), b2 = bin_of(P, id.z), b3 = bin_of(P, id.w);
    const bool same = live >= 4 && b0 == b1 && b0 == b2 && b0 == b3;
    if (__ballot(same && b0 == __builtin_amdgcn_readfirstlane(b0)) == ~0ull) {
        if ((threadIdx.x & 63) == 0) atomicAdd(&hist[b0], 256);
    } else if (same) {
        atomicAdd(&hist[b0], 4);
    } else {
        atomicAdd(&hist[b0], 1);
        if (live > 1) atomicAdd(&hist[b1], 1);
        if (live > 2) atomicAdd(&hist[b2], 1);
        if (live > 3) atomicAdd(&hist[b3], 1);
    }
}

}  // namespace

// Rows grouped by adapter, each adapter's in their order, rows without one
// behind them; the row tiles and, for the gradients, the row chunks, which the
// last workgroup writes.  Every workgroup counts all rows for itself (16 K rows
// of ids in flight at once), which saves a launch that only counts.
__global__ void __launch_bounds__(kPlanThreads) adapter_plan_kernel(AdapterPlan P) {
    constexpr int kWaves = kPlanThreads / 64, kAhead = 4;
    __shared__ int32_t total[kBins + 1], start[kBins + 1], before[kBins], scan[kWaves];
    __shared__ uint16_t counts[kWaves][kBins];
    __shared__ int32_t tile0[kBins], chunk0[kBins], slot0[kBins];
    const int bins = P.n + 1, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const bool tables = blockIdx.x == gridDim.x - 1;
    const int64_t first = tables ? 0 : (int64_t)blockIdx.x * P.rows;  // a multiple of 256: a wavefront's rows lie on one side
    for (int i = threadIdx.x; i <= bins; i += kPlanThreads) total[i] = 0;
    for (int i = threadIdx.x; i < bins; i += kPlanThreads) before[i] = 0;
    __syncthreads();
    for (int64_t r0 = 0; r0 < P.M; r0 += 4 * kPlanThreads * kAhead) {
        int4 id[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; k++) {
            const int64_t r = r0 + 4 * ((int64_t)k * kPlanThreads + threadIdx.x);
            id[k] = make_int4(-1, -1, -1, -1);
            if (P.vec && r + 4 <= P.M) {
                id[k] = *reinterpret_cast<const int4*>(P.ids + r);
            } else {
                if (r < P.M) id[k].x = P.ids[r];
                if (r + 1 < P.M) id[k].y = P.ids[r + 1];
                if (r + 2 < P.M) id[k].z = P.ids[r + 2];
                if (r + 3 < P.M) id[k].w = P.ids[r + 3];
            }
        }
#pragma unroll
        for (int k = 0; k < kAhead; k++) {
            const int64_t r = r0 + 4 * ((int64_t)k * kPlanThreads + threadIdx.x);
            count4(r < first ? before : total, P, id[k], P.M - r);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i <= bins; i += kPlanThreads) {
        if (i < bins) total[i] += before[i];
        start[i] = total[i];
    }
    __syncthreads();
    block_scan(start, bins + 1, scan);
    if (!tables) {
        // 1024 rows at a time, one a thread.  Lanes of one bin find each other
        // by a ballot for each bit of it; a row's place is the bin's next one,
        // plus the bin's rows in earlier wavefronts and earlier lanes.
        for (int i = threadIdx.x; i < bins; i += kPlanThreads) start[i] += before[i];
        for (int64_t k = 0; k < P.rows && first + k < P.M; k += kPlanThreads) {
            const int64_t r = first + k + threadIdx.x;
            const bool live = r < P.M;
            const int b = live ? bin_of(P, P.ids[r]) : 0;
            uint64_t same = __ballot(live);
            for (int bit = 0; (P.n >> bit) != 0; bit++) {
                const bool on = (b >> bit) & 1;
                const uint64_t m = __ballot(on);
                same &= on ? m : ~m;
            }
            uint16_t* mine = counts[wave];
            for (int i = lane; i < bins; i += 64) mine[i] = 0;
            asm volatile("" ::: "memory");  // (a wavefront's LDS stores take effect in order)
            const int rank = __popcll(same & ((1ull << lane) - 1));
            if (live && rank == 0) mine[b] = (uint16_t)__popcll(same);
            __syncthreads();
            for (int i = threadIdx.x; i < bins; i += kPlanThreads) {
                uint32_t run = 0;
                for (int w = 0; w < kWaves; w++) {
                    const uint32_t n = counts[w][i];
                    counts[w][i] = (uint16_t)run;
                    run += n;
                }
                before[i] = run;
            }
            __syncthreads();
            if (live) P.order[start[b] + mine[b] + rank] = (int32_t)r;
            __syncthreads();
            for (int i = threadIdx.x; i < bins; i += kPlanThreads) start[i] += before[i];
        }
        return;
    }
    for (int i = threadIdx.x; i < bins; i += kPlanThreads) {
        const int32_t chunks = i < P.n && P.chunk ? (total[i] + P.chunk - 1) / P.chunk : 0;
        tile0[i] = i < P.n || P.rest ? (total[i] + P.tile - 1) / P.tile : 0;
        chunk0[i] = chunks;
        slot0[i] = chunks > 1 ? chunks : 0;
    }
    __syncthreads();
    const int32_t last_tiles = tile0[bins - 1];  // (the rows without an adapter have no chunks)
    __syncthreads();
    block_scan(tile0, bins, scan);
    const int32_t n_tiles = tile0[bins - 1] + last_tiles;
    int32_t n_chunks = 0;
    if (P.chunk) {
        block_scan(chunk0, bins, scan);
        block_scan(slot0, bins, scan);
        n_chunks = chunk0[bins - 1];
    }
    if (threadIdx.x == 0) {
        P.n_tables[0] = n_tiles;
        P.n_tables[1] = n_chunks;
    }
    for (int32_t i = threadIdx.x; i < n_tiles; i += kPlanThreads) {
        const int b = find_bin(tile0, bins, i);
        const int32_t at = (i - tile0[b]) * P.tile;
        P.tiles[i] = make_int4(b < P.n ? b : -1, start[b] + at, min(total[b] - at, P.tile), 0);
    }
    if (!P.chunk) return;
    for (int32_t i = threadIdx.x; i < n_chunks; i += kPlanThreads) {
        const int b = find_bin(chunk0, bins, i);
        const int32_t k = i - chunk0[b], at = k * P.chunk;
        P.chunks[i] = make_int4(b, start[b] + at, min(total[b] - at, P.chunk), total[b] > P.chunk ? slot0[b] + k : -1);
    }
    for (int i = threadIdx.x; i < P.n; i += kPlanThreads)
        P.info[i] = make_int2((total[i] + P.chunk - 1) / P.chunk, slot0[i]);
}

// One workgroup: up to 16 MB rows of one adapter, and a share of the columns.
// The first product V = A x^T over K is split over the wavefronts (chunks of
// 64 columns in turn) and joined in LDS in one fixed order, whatever the tile:
// a row's bits do not depend on the rows beside it.  V, an FP32 sum, is passed
// on as two BF16 values (2^-16 of it may be lost, against the 2^-8 of the output's
// one rounding): 32 of the second product's inputs are then 16 ranks twice,
// which costs no instruction at rank 16.
// RB: ranks in blocks of 16; MB: rows in blocks of 16.
template <int RB, int MB>
__global__ void __launch_bounds__(kAdWaves * 64) adapter_kernel(AdapterParams P) {
    constexpr int kR = 16 * RB, kPitch = 2 * kR + 8;
    __shared__ __attribute__((aligned(16))) f32x4 red[kAdWaves][RB * MB][64];
    __shared__ __attribute__((aligned(16))) uint16_t vs[16 * MB][kPitch];
    __shared__ int32_t rows[16 * MB];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, q = lane >> 4;
    const int32_t tile = blockIdx.x / P.slabs, slab = blockIdx.x % P.slabs;
    if (tile >= *P.n_tiles) return;
    const int4 t = P.tiles[tile];
    const int a = t.x, count = t.z;
    if (threadIdx.x < 16 * MB) rows[threadIdx.x] = P.order[t.y + min((int)threadIdx.x, count - 1)];
    __syncthreads();
    if (a < 0) {  // rows without an adapter
        const int pieces = P.N / 8;
        for (int64_t k = slab * (kAdWaves * 64) + threadIdx.x; k < (int64_t)count * pieces; k += P.slabs * (kAdWaves * 64)) {
            const int64_t r = rows[k / pieces], c = k % pieces * 8;
            const u32x4 z = {0, 0, 0, 0};
            *reinterpret_cast<u32x4*>(P.out + r * P.ld_out + c) = P.base ? load16(P.base + r * P.ld_base + c) : z;
        }
        if (P.v && slab == 0)
            for (int k = threadIdx.x; k < count * P.R; k += kAdWaves * 64) P.v[(int64_t)rows[k / P.R] * P.R + k % P.R] = 0.0f;
        return;
    }
    int64_t row[MB];
#pragma unroll
    for (int m = 0; m < MB; m++) row[m] = rows[16 * m + i];

    f32x4 acc[RB][MB];
#pragma unroll
    for (int r = 0; r < RB; r++)
#pragma unroll
        for (int m = 0; m < MB; m++) acc[r][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const uint16_t* A = P.A + (int64_t)a * P.R * P.K;
    for (int k0 = wave * 64; k0 < P.K; k0 += kAdWaves * 64) {
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const int k = k0 + 32 * h + 8 * q;
            u32x4 af[RB], xf[MB];
#pragma unroll
            for (int m = 0; m < MB; m++) xf[m] = u32x4{0, 0, 0, 0};
#pragma unroll
            for (int r = 0; r < RB; r++) af[r] = u32x4{0, 0, 0, 0};
            if (k < P.K) {
#pragma unroll
                for (int m = 0; m < MB; m++) xf[m] = load16(P.x + row[m] * P.ldx + k);
#pragma unroll
                for (int r = 0; r < RB; r++)
                    if (16 * r + i < P.R) af[r] = load16(A + (int64_t)(16 * r + i) * P.K + k);
            }
#pragma unroll
            for (int r = 0; r < RB; r++)
#pragma unroll
                for (int m = 0; m < MB; m++) acc[r][m] = mfma16(af[r], xf[m], acc[r][m]);
        }
    }
#pragma unroll
    for (int r = 0; r < RB; r++)
#pragma unroll
        for (int m = 0; m < MB; m++) red[wave][r * MB + m][lane] = acc[r][m];
    __syncthreads();
    for (int j = wave; j < RB * MB; j += kAdWaves) {
        const int m = j % MB, r = j / MB * 16 + 4 * q;  // the lane's ranks r .. r + 3 of row i
        f32x4 s = red[0][j][lane];
#pragma unroll
        for (int w = 1; w < kAdWaves; w++) s += red[w][j][lane];
        if (r >= P.R) s = f32x4{0.0f, 0.0f, 0.0f, 0.0f};  // (0 times an infinite x)
        if (P.v && slab == 0 && r < P.R && 16 * m + i < count)
            *reinterpret_cast<f32x4*>(P.v + (int64_t)rows[16 * m + i] * P.R + r) = s;
        const float scale = P.scale ? P.scale[a] : 1.0f;
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; e++) {
            float v = s[e] * scale;
            hi[e] = bf16_piece(v);
            lo[e] = bf16_hw(v);
        }
        *reinterpret_cast<u32x2*>(&vs[16 * m + i][r]) = u32x2{hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16)};
        *reinterpret_cast<u32x2*>(&vs[16 * m + i][kR + r]) = u32x2{lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16)};
    }
    __syncthreads();

    // The second product: 64 columns a step.  Row n of its first operand is
    // column c0 + 16 (n / 4) + 4 b + n % 4, so that the four products b leave
    // the lane 16 consecutive columns of its row.
    u32x4 vf[MB][RB];
#pragma unroll
    for (int m = 0; m < MB; m++)
#pragma unroll
        for (int j = 0; j < RB; j++) vf[m][j] = *reinterpret_cast<const u32x4*>(&vs[16 * m + i][32 * j + 8 * q]);
    const uint16_t* B = P.B + (int64_t)a * P.N * P.R;
    for (int c0 = (slab * kAdWaves + wave) * 64; c0 < P.N; c0 += P.slabs * kAdWaves * 64) {
        const int n0 = c0 + 16 * q;
        u32x4 old[MB][2];
#pragma unroll
        for (int m = 0; m < MB; m++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
                old[m][h] = u32x4{0, 0, 0, 0};
                if (P.base && n0 + 8 * h < P.N && 16 * m + i < count) old[m][h] = load16(P.base + row[m] * P.ld_base + n0 + 8 * h);
            }
        f32x4 y[MB][4];
#pragma unroll
        for (int b = 0; b < 4; b++) {
            const int n = min(c0 + 16 * (i >> 2) + 4 * b + (i & 3), P.N - 1);
            u32x4 bf[(RB + 1) / 2];
#pragma unroll
            for (int j = 0; j < (RB + 1) / 2; j++) {
                const int r = RB == 1 ? 8 * (q & 1) : 32 * j + 8 * q;
                bf[j] = u32x4{0, 0, 0, 0};
                if (r < P.R) bf[j] = load16(B + (int64_t)n * P.R + r);
            }
#pragma unroll
            for (int m = 0; m < MB; m++) {
                y[m][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int j = RB - 1; j >= 0; j--) y[m][b] = mfma16(bf[RB == 1 ? 0 : j % (RB / 2 > 0 ? RB / 2 : 1)], vf[m][j], y[m][b]);
            }
        }
#pragma unroll
        for (int m = 0; m < MB; m++) {
            if (16 * m + i >= count) continue;
#pragma unroll
            for (int h = 0; h < 2; h++) {
                if (n0 + 8 * h >= P.N) continue;
                u32x4 o;
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const f32x4 d = y[m][2 * h + e / 2];
                    const float lo = d[2 * (e & 1)] + __uint_as_float(old[m][h][e] << 16);
                    const float hi = d[2 * (e & 1) + 1] + __uint_as_float(old[m][h][e] & 0xFFFF0000u);
                    o[e] = bf16_hw(lo) | (bf16_hw(hi) << 16);
                }
                *reinterpret_cast<u32x4*>(P.out + row[m] * P.ld_out + n0 + 8 * h) = o;
            }
        }
    }
}

// The adapters that have rows, transposed: At [n][K][R] and Bt [n][R][N].
__global__ void __launch_bounds__(256) adapter_transpose_kernel(AdapterGrad P) {
    __shared__ uint16_t tile[64][66];
    const int a = blockIdx.y, k_tiles = (P.K + 63) / 64;
    if (P.info[a].x == 0) return;
    const bool is_a = (int)blockIdx.x < k_tiles;
    const int c0 = ((int)blockIdx.x - (is_a ? 0 : k_tiles)) * 64;
    // in [rows_in][cols_in] -> out [cols_in][rows_in]
    const int64_t rows_in = is_a ? P.R : P.N, cols_in = is_a ? P.K : P.R;
    const uint16_t* in = (is_a ? P.A : P.B) + (int64_t)a * rows_in * cols_in;
    uint16_t* out = (is_a ? P.At : P.Bt) + (int64_t)a * rows_in * cols_in;
    for (int r0 = 0; r0 < P.R; r0 += 64) {
        const int64_t row0 = is_a ? r0 : c0, col0 = is_a ? c0 : r0;
        for (int k = threadIdx.x; k < 64 * 64; k += 256) {
            const int64_t r = row0 + k / 64, c = col0 + k % 64;
            if (r < rows_in && c < cols_in) tile[k / 64][k % 64] = in[r * cols_in + c];
        }
        __syncthreads();
        for (int k = threadIdx.x; k < 64 * 64; k += 256) {
            const int64_t c = col0 + k / 64, r = row0 + k % 64;
            if (r < rows_in && c < cols_in) out[c * rows_in + r] = tile[k % 64][k / 64];
        }
        __syncthreads();
    }
}

// dA and dB of one row chunk and 128 columns: the sum over rows is the matrix
// instruction's inner dimension, 32 rows a step, the wavefronts taking steps in
// turn.  A lane loads 8 columns of 8 rows; one byte permutation a register
// turns them into operands with 8 rows of one column each, for eight products
// whose columns lie 8 apart.  w and v are FP32 sums and go in as three BF16
// values, which is all of their 24 bits.
// RB: ranks in blocks of 16 (blockIdx.z takes further ones).
template <int RB>
__global__ void __launch_bounds__(256) adapter_wgrad_kernel(AdapterGrad P) {
    __shared__ __attribute__((aligned(16))) float red[4][16][132];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, q = lane >> 4;
    if ((int)blockIdx.y >= P.n_tables[1]) return;
    const int4 t = P.chunks[blockIdx.y];
    const int a = t.x, count = t.z, k_slabs = (P.K + 127) / 128;
    const bool is_a = (int)blockIdx.x < k_slabs;
    const int C = is_a ? P.K : P.N, c0 = ((int)blockIdx.x - (is_a ? 0 : k_slabs)) * 128, rank0 = blockIdx.z * 16 * RB;
    const uint16_t* Z = is_a ? P.x : P.dy;
    const int64_t ldz = is_a ? P.ldx : P.ld_dy;
    const float* W = is_a ? P.w : P.v;
    f32x4 acc[8][RB];
#pragma unroll
    for (int c = 0; c < 8; c++)
#pragma unroll
        for (int r = 0; r < RB; r++) acc[c][r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int col = c0 + 8 * i;
    for (int s = wave * 32; s < count; s += 128) {
        u32x4 z[8];
        float w[RB][8];
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int at = s + 8 * q + j;
            const bool live = at < count;
            const int64_t r = P.order[t.y + min(at, count - 1)];
            z[j] = u32x4{0, 0, 0, 0};
            if (live && col < C) z[j] = load16(Z + r * ldz + col);
#pragma unroll
            for (int b = 0; b < RB; b++) {
                const int rank = rank0 + 16 * b + i;
                w[b][j] = 0.0f;
                if (live && rank < P.R) w[b][j] = W[r * P.R + rank];
            }
        }
        u32x4 wf[RB][3];
#pragma unroll
        for (int b = 0; b < RB; b++)
#pragma unroll
            for (int p = 0; p < 3; p++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const uint32_t lo = bf16_piece(w[b][2 * e]);
                    wf[b][p][e] = lo | (bf16_piece(w[b][2 * e + 1]) << 16);
                }
#pragma unroll
        for (int c = 0; c < 8; c++) {
            u32x4 zf;
#pragma unroll
            for (int e = 0; e < 4; e++)
                zf[e] = __builtin_amdgcn_perm(z[2 * e + 1][c / 2], z[2 * e][c / 2], (c & 1) ? 0x07060302u : 0x05040100u);
#pragma unroll
            for (int b = 0; b < RB; b++)
#pragma unroll
                for (int p = 2; p >= 0; p--) acc[c][b] = mfma16(wf[b][p], zf, acc[c][b]);
        }
    }
    // The wavefronts' sums, added in one order.
    const float scale = P.scale ? P.scale[a] : 1.0f;
    const int64_t each = (int64_t)P.R * (P.K + P.N);
    float* dA = t.w < 0 ? P.dA + (int64_t)a * P.R * P.K : P.slots + t.w * each;
    float* dB = t.w < 0 ? P.dB + (int64_t)a * P.R * P.N : P.slots + t.w * each + (int64_t)P.R * P.K;
#pragma unroll
    for (int b = 0; b < RB; b++) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 4; e++) {
            *reinterpret_cast<f32x4*>(&red[wave][4 * q + e][8 * i]) = f32x4{acc[0][b][e], acc[1][b][e], acc[2][b][e], acc[3][b][e]};
            *reinterpret_cast<f32x4*>(&red[wave][4 * q + e][8 * i + 4]) = f32x4{acc[4][b][e], acc[5][b][e], acc[6][b][e], acc[7][b][e]};
        }
        __syncthreads();
        const int rank = rank0 + 16 * b;
        if (is_a) {
            const int r = threadIdx.x / 16, c = threadIdx.x % 16 * 8;
            if (rank + r < P.R && c0 + c < C)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    f32x4 s[4];
#pragma unroll
                    for (int k = 0; k < 4; k++) s[k] = *reinterpret_cast<const f32x4*>(&red[k][r][c + 4 * h]);
                    *reinterpret_cast<f32x4*>(dA + (int64_t)(rank + r) * P.K + c0 + c + 4 * h) = ((s[0] + s[1]) + (s[2] + s[3])) * scale;
                }
        } else {
            const int c = threadIdx.x / 2, r = threadIdx.x % 2 * 8;
            if (rank + r < P.R && c0 + c < C)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    f32x4 o;
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const int k = r + 4 * h + e;
                        o[e] = ((red[0][k][c] + red[1][k][c]) + (red[2][k][c] + red[3][k][c])) * scale;
                    }
                    *reinterpret_cast<f32x4*>(dB + (int64_t)(c0 + c) * P.R + rank + r + 4 * h) = o;
                }
        }
    }
}

// Adapters whose rows filled several chunks: the chunks' sums, in order.
// Adapters without rows: zeros.
__global__ void __launch_bounds__(256) adapter_join_kernel(AdapterGrad P) {
    const int a = blockIdx.y;
    const int2 info = P.info[a];
    if (info.x == 1) return;
    const int64_t of_a = (int64_t)P.R * P.K, each = of_a + (int64_t)P.R * P.N;
    const int64_t k = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (k >= each) return;
    f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int c = 0; c < info.x; c++) s += *reinterpret_cast<const f32x4*>(P.slots + (info.y + c) * each + k);
    float* out = k < of_a ? P.dA + a * of_a + k : P.dB + a * (each - of_a) + (k - of_a);
    *reinterpret_cast<f32x4*>(out) = s;
}

// The row tile for a rank: RB * MB * 8 KiB of LDS join the wavefronts' sums.
int adapter_tile(int32_t R) { return R <= 64 ? 32 : 16; }

// A workgroup of the plan places 1024 rows, or as many as keep their number to
// 256: each of them counts all rows.
hipError_t launch_adapter_plan(AdapterPlan P, hipStream_t stream) {
    P.rows = std::max<int64_t>(1, (P.M + 256 * kPlanThreads - 1) / (256 * kPlanThreads)) * kPlanThreads;
    P.vec = (uintptr_t)P.ids % 16 == 0;
    const int64_t blocks = (P.M + P.rows - 1) / P.rows + 1;
    hipLaunchKernelGGL(adapter_plan_kernel, dim3((unsigned)blocks), dim3(kPlanThreads), 0, stream, P);
    return hipGetLastError();
}

namespace {

template <int RB, int MB>
hipError_t adapter_run(const AdapterParams& P, int64_t tiles, hipStream_t s) {
    hipLaunchKernelGGL((adapter_kernel<RB, MB>), dim3((unsigned)(tiles * P.slabs)), dim3(kAdWaves * 64), 0, s, P);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_adapter(AdapterParams P, int64_t tiles, hipStream_t stream) {
    // Few tiles: their columns are shared out, and each share repeats the first product.
    P.slabs = (int32_t)std::max<int64_t>(1, std::min<int64_t>((P.N + kAdWaves * 64 - 1) / (kAdWaves * 64), 512 / tiles));
    if (P.R <= 16) return adapter_run<1, 2>(P, tiles, stream);
    if (P.R <= 32) return adapter_run<2, 2>(P, tiles, stream);
    if (P.R <= 64) return adapter_run<4, 2>(P, tiles, stream);
    return adapter_run<8, 1>(P, tiles, stream);
}

// Rows of a chunk of the gradients: the columns' slabs times the chunks are
// about 1024 workgroups.
int32_t adapter_chunk(int64_t M, int64_t K, int64_t N) {
    const int64_t slabs = (K + 127) / 128 + (N + 127) / 128, chunks = std::max<int64_t>(1, 1024 / slabs);
    return (int32_t)std::min<int64_t>((std::max<int64_t>(M, 1) + 128 * chunks - 1) / (128 * chunks) * 128, (int64_t)1 << 30);
}

hipError_t launch_adapter_transpose(const AdapterGrad& P, hipStream_t stream) {
    hipLaunchKernelGGL(adapter_transpose_kernel, dim3((P.K + 63) / 64 + (P.N + 63) / 64, P.n), dim3(256), 0, stream, P);
    return hipGetLastError();
}

hipError_t launch_adapter_wgrad(const AdapterGrad& P, int64_t chunks, hipStream_t stream) {
    const unsigned slabs = (P.K + 127) / 128 + (P.N + 127) / 128;
    if (chunks > 0) {
        const dim3 grid(slabs, (unsigned)chunks, P.R > 64 ? 2 : 1);
        if (P.R <= 16)
            hipLaunchKernelGGL(adapter_wgrad_kernel<1>, grid, dim3(256), 0, stream, P);
        else if (P.R <= 32)
            hipLaunchKernelGGL(adapter_wgrad_kernel<2>, grid, dim3(256), 0, stream, P);
        else
            hipLaunchKernelGGL(adapter_wgrad_kernel<4>, grid, dim3(256), 0, stream, P);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const int64_t each = (int64_t)P.R * (P.K + P.N);
    hipLaunchKernelGGL(adapter_join_kernel, dim3((unsigned)((each / 4 + 255) / 256), P.n), dim3(256), 0, stream, P);
    return hipGetLastError();
}

}  // namespace nvfp4
