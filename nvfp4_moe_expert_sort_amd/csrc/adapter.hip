// adapter.hip -- low-rank adapters of many requests beside a shared projection,
// and their gradients (include/nvfp4moe.h, nvfp4moe_adapter_linear).
//
// Row r with adapter a: v = A_a x_r, out_r = base_r + scale_a B_a v.  For dy:
// w = B_a^T dy_r, dx_r = base_r + A_a^T scale_a w, dA_a = scale_a sum w x_r^T,
// dB_a = scale_a sum dy_r v^T.  The gradient with respect to x is the forward
// operation with B^T and A^T in the places of A and B, so one kernel serves
// both, on transposed copies of the adapters.
#include <algorithm>
#include <type_traits>

#include "nvfp4_device.h"
#include "nvfp4_kernels.h"

namespace nvfp4 {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kAdWaves = 8;          // wavefronts that share the first product's K
constexpr uint32_t kCus = 256;
constexpr int kPlanThreads = 1024;
constexpr int kBins = kMaxExperts + 1;  // adapters, and the rows without one

__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
// Keeps the loads before it ahead of what follows (the scheduler would move
// them down to where their values are needed, to save registers).
__device__ __forceinline__ void issue() { __builtin_amdgcn_sched_barrier(0); }
__device__ __forceinline__ u32x4 load16(const uint16_t* p) { return *reinterpret_cast<const u32x4*>(p); }

// v as the sum of BF16 values of falling size, each the rounding of what the
// ones before it leave (of a finite value to a finite one: above 2^128 - 2^119
// the nearest would be infinity); an infinite or NaN v is the first of them alone.
__device__ __forceinline__ uint32_t bf16_piece(float& rest) {
    uint32_t b = bf16_hw(rest);
    if ((b & 0x7FFF) == 0x7F80 && fabsf(rest) < __builtin_inff()) b--;
    const float r = rest - bf16_to_f32(b);
    rest = fabsf(r) < __builtin_inff() ? r : 0.0f;
    return b;
}

// Element c (of 8) of each of 8 rows.
__device__ __forceinline__ u32x4 column8(const u32x4 (&z)[8], int c) {
    u32x4 f;
#pragma unroll
    for (int e = 0; e < 4; e++)
        f[e] = __builtin_amdgcn_perm(z[2 * e + 1][c / 2], z[2 * e][c / 2], (c & 1) ? 0x07060302u : 0x05040100u);
    return f;
}

// Sums over the earlier entries of an array [n], in place, by one wavefront.
// (All 16 of the workgroup would take a share of the SIMDs each to do as little:
// 1.0 us a scan of 9 entries, and so 0.6.)
__device__ __forceinline__ void wave_scan(int32_t* of, int n) {
    const int lane = threadIdx.x & 63, per = (n + 63) / 64, lo = min(lane * per, n), hi = min(lo + per, n);
    int32_t sum = 0;
    for (int i = lo; i < hi; i++) sum += of[i];
    int32_t run = sum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int32_t v = __shfl_up(run, o, kWave);
        if (lane >= o) run += v;
    }
    run -= sum;
    for (int i = lo; i < hi; i++) {
        const int32_t v = of[i];
        of[i] = run;
        run += v;
    }
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

// Counts of the bins, in copies of which a lane uses one: neighbouring rows
// mostly share an adapter, and additions of many lanes to one address take one
// turn each.  (One copy, and lanes that find the others of their adapter by
// ballots: 32768 rows sorted by adapter counted after 6.0 us, and so after 3.5.)
constexpr int kCopies = 8, kCopyPitch = kBins + 8;
// The lane's four consecutive rows, of which the first `live` exist.
__device__ __forceinline__ void count4(int32_t* hist, const AdapterPlan& P, int4 id, int64_t live) {
    if (live <= 0) return;
    hist += (threadIdx.x & (kCopies - 1)) * kCopyPitch;
    if (live >= 4 && id.x == id.y && id.x == id.z && id.x == id.w) {
        atomicAdd(&hist[bin_of(P, id.x)], 4);
        return;
    }
    atomicAdd(&hist[bin_of(P, id.x)], 1);
    if (live > 1) atomicAdd(&hist[bin_of(P, id.y)], 1);
    if (live > 2) atomicAdd(&hist[bin_of(P, id.z)], 1);
    if (live > 3) atomicAdd(&hist[bin_of(P, id.w)], 1);
}

// B^T and A^T, which take the places of A and B in the gradient's products, of
// the adapters that have rows.  Up to rank 32 (RB 0) as matrices [R][N] and
// [K][R]; from there as operands, ranks padded with zeros to 16 RB, N and K to
// multiples of 64, in units of 16 bytes (8 elements):
//   first product:  rank r, inputs 8 k .. + 7: ((k / 4) RB + r / 16) 64 + k % 4 * 16 + r % 16
//   second product: column c, ranks 8 r .. + 7: ((c / 64 * 4 + c % 4) RB / 2 + r / 4) 64 + r % 4 * 16 + c % 64 / 4
// A thread turns 8 x 8 elements over with one byte permutation each two.
template <int RB>
__device__ __forceinline__ void pack_adapters(const AdapterPack& P, int64_t item) {
    const uint32_t r8 = RB ? 2 * RB : P.R / 8, k8 = RB ? (P.K + 63) / 64 * 8 : P.K / 8, n8 = RB ? (P.N + 63) / 64 * 8 : P.N / 8;
    const uint32_t each = r8 * (k8 + n8);
    const int a = (int)(item / each);
    if (a >= P.n || (P.info && P.info[a].x == 0)) return;
    uint32_t k = (uint32_t)(item % each);
    const bool is_a = k < r8 * k8;
    if (!is_a) k -= r8 * k8;
    // 8 ranks from 8 r on, and 8 columns of A or rows of B from 8 c on
    const uint32_t r = is_a ? k / k8 : k % r8, c = is_a ? k % k8 : k / r8;
    const bool in = RB == 0 || (8 * (int)r < P.R && 8 * (int)c < (is_a ? P.K : P.N));
    const uint16_t* at = in ? is_a ? P.A + ((int64_t)a * P.R + 8 * r) * P.K + 8 * c : P.B + ((int64_t)a * P.N + 8 * c) * P.R + 8 * r : P.A;
    const int64_t ld = in ? is_a ? P.K : P.R : 0;
    u32x4 z[8];
#pragma unroll
    for (int j = 0; j < 8; j++) z[j] = load16(at + j * ld);
    if (!in)
#pragma unroll
        for (int j = 0; j < 8; j++) z[j] = u32x4{0, 0, 0, 0};
    u32x4* out = is_a ? P.second + a * P.units_second : P.first + a * P.units_first;
#pragma unroll
    for (int j = 0; j < 8; j++) {
        // of A: column 8 c + j, ranks 8 r ..; of B: rank 8 r + j, rows 8 c ..
        uint32_t to;
        if (RB == 0)
            to = is_a ? (8 * c + j) * r8 + r : (8 * r + j) * n8 + c;
        else if (is_a)
            to = ((((8 * c + j) >> 6) * 4 + (j & 3)) * (RB / 2) + (r >> 2)) * 64 + (r & 3) * 16 + (((8 * c + j) & 63) >> 2);
        else
            to = ((c >> 2) * RB + ((8 * r + j) >> 4)) * 64 + (c & 3) * 16 + ((8 * r + j) & 15);
        out[to] = column8(z, j);
    }
}
__device__ __forceinline__ void pack_adapters(const AdapterPack& P, int64_t item) {
    if (P.R <= 32)
        pack_adapters<0>(P, item);
    else if (P.R <= 64)
        pack_adapters<4>(P, item);
    else
        pack_adapters<8>(P, item);
}

}  // namespace

// Rows grouped by adapter, each adapter's in their order, rows without one
// behind them; the row tiles and, for the gradients, the row chunks, which the
// last workgroup writes.  Every workgroup counts all rows for itself (16 K rows
// of ids in flight at once), which saves a launch that only counts.
// Workgroups behind those transpose the adapters, if that need not wait for the
// plan to say which of them have rows.
// 5.6 us for 8192 rows, 9.1 for 32768 of 128 adapters: the launch, the chain from
// the ids to the last table, and what 16 wavefronts a CU take to issue it.
__global__ void __launch_bounds__(kPlanThreads) adapter_plan_kernel(AdapterPlan P, AdapterPack pack) {
    constexpr int kWaves = kPlanThreads / 64, kAhead = 8;
    __shared__ int32_t total[kBins], start[kBins], before[kBins];
    __shared__ int32_t hist[2][kCopies * kCopyPitch];  // of the rows ahead of this workgroup's, and of the others
    __shared__ uint16_t counts[kWaves][kBins];
    __shared__ int32_t tile0[kBins], chunk0[kBins], slot0[kBins];  // (a tile is a step of the gradients)
    const int bins = P.n + 1, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    if ((int)blockIdx.x >= P.blocks) {
        pack_adapters(pack, ((int64_t)blockIdx.x - P.blocks) * kPlanThreads + threadIdx.x);
        return;
    }
    const bool tables = (int)blockIdx.x == P.blocks - 1;
    const int64_t first = tables ? 0 : (int64_t)blockIdx.x * P.rows;  // a multiple of 256: a wavefront's rows lie on one side
    for (int i = threadIdx.x; i < bins; i += kPlanThreads)
#pragma unroll
        for (int c = 0; c < 2 * kCopies; c++) hist[c / kCopies][c % kCopies * kCopyPitch + i] = 0;
    __syncthreads();
    // Four rows a thread.  kAhead such pieces of 4096 rows are loaded before any
    // is counted, and the last piece (which may be a part) before all.
    const int64_t last = P.M > 0 ? (P.M - 1) / (4 * kPlanThreads) : 0, r_last = 4 * (last * kPlanThreads + threadIdx.x);
    int4 id_last = make_int4(-1, -1, -1, -1);
    if (r_last < P.M) id_last.x = P.ids[r_last];
    if (r_last + 1 < P.M) id_last.y = P.ids[r_last + 1];
    if (r_last + 2 < P.M) id_last.z = P.ids[r_last + 2];
    if (r_last + 3 < P.M) id_last.w = P.ids[r_last + 3];
    for (int64_t p0 = 0; p0 < last; p0 += kAhead) {
        int4 id[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; k++) {
            const int32_t* at = P.ids + 4 * (min(p0 + k, last - 1) * kPlanThreads + threadIdx.x);
            if (P.vec)
                id[k] = *reinterpret_cast<const int4*>(at);
            else
                id[k] = make_int4(at[0], at[1], at[2], at[3]);
        }
        issue();
#pragma unroll
        for (int k = 0; k < kAhead; k++)
            if (p0 + k < last) count4(hist[4 * ((p0 + k) * kPlanThreads + threadIdx.x) >= first], P, id[k], 4);
    }
    count4(hist[r_last >= first], P, id_last, P.M - r_last);
    __syncthreads();
    for (int i = threadIdx.x; i < bins; i += kPlanThreads) {
        int32_t n[2] = {0, 0};
#pragma unroll
        for (int c = 0; c < 2 * kCopies; c++) n[c / kCopies] += hist[c / kCopies][c % kCopies * kCopyPitch + i];
        before[i] = n[0];
        total[i] = start[i] = n[0] + n[1];
    }
    __syncthreads();
    if (wave == 0) wave_scan(start, bins);
    __syncthreads();
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
                uint32_t run = 0, n[kWaves];
#pragma unroll
                for (int w = 0; w < kWaves; w++) n[w] = counts[w][i];
#pragma unroll
                for (int w = 0; w < kWaves; w++) {
                    counts[w][i] = (uint16_t)run;
                    run += n[w];
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
        // (an adapter without rows has an empty chunk, whose sums are zeros)
        const int32_t chunks = i < P.n && P.chunk ? max(1, (total[i] + P.chunk - 1) / P.chunk) : 0;
        tile0[i] = i < P.n || P.rest ? (total[i] + P.tile - 1) / P.tile : 0;
        chunk0[i] = chunks;
        slot0[i] = chunks > 1 ? chunks : 0;
    }
    __syncthreads();
    const int32_t last_tiles = tile0[bins - 1];  // (the rows without an adapter have no chunks)
    __syncthreads();
    if (wave == 0)
        wave_scan(tile0, bins);
    else if (P.chunk && wave < 3)
        wave_scan(wave == 1 ? chunk0 : slot0, bins);
    __syncthreads();
    const int32_t n_tiles = tile0[bins - 1] + last_tiles, n_chunks = P.chunk ? chunk0[bins - 1] : 0;
    if (threadIdx.x == 0) {
        P.n_tables[0] = n_tiles;
        P.n_tables[1] = n_chunks;
    }
    for (int32_t i = threadIdx.x; i < n_tiles; i += kPlanThreads) {
        const int b = find_bin(tile0, bins, i);
        const int32_t at = (i - tile0[b]) * P.tile;
        P.tiles[i] = make_int4(b < P.n ? b : -1, start[b] + at, min(total[b] - at, P.tile), i);
    }
    if (!P.chunk) return;
    for (int32_t i = threadIdx.x; i < n_chunks; i += kPlanThreads) {
        const int b = find_bin(chunk0, bins, i);
        const int32_t k = i - chunk0[b], at = k * P.chunk;
        P.chunks[i] = make_int4(b, start[b] + at, min(total[b] - at, P.chunk), total[b] > P.chunk ? slot0[b] + k : -1);
        P.chunk_step[i] = tile0[b] + at / P.tile;
    }
    for (int i = threadIdx.x; i < P.n; i += kPlanThreads)
        P.info[i] = make_int2((total[i] + P.chunk - 1) / P.chunk, slot0[i]);
}

// One workgroup: up to 16 MB rows of one adapter, and a share of the columns.
//
// The first product V = A x^T over K is split over the wavefronts and joined in
// LDS in one fixed order, whatever the tile: a row's bits do not depend on the
// rows beside it.  V, an FP32 sum, is passed on as three BF16 values, which is all
// of its 24 bits.  (With two, of the 20480 outputs of 5 rows some 20 lay one BF16
// step off, and 2 at most so.  The third costs nothing measurable up to rank 32; 8192
// rows of 4096 columns: rank 64 42.0 -> 43.2 us a call, rank 128 52 -> 58.)  At rank
// 16 the second product has 32 inputs of 16 ranks of the first two pieces, and 32
// of the third and zeros.
//
// A matrix operand has its rows on neighbouring lanes; read like that, memory
// gives 16 bytes of 16 lines at a time.  So each wavefront reads its operands
// in whole lines and turns them over in a piece of LDS of its own (16-byte
// units, exclusive-ored with the row so that operand reads meet no bank twice),
// the loads a step or two ahead in registers; base and out are accessed in runs of
// 16 lanes a row, with the second product's columns dealt out so that a lane
// holds neighbouring ones.
//
// RB: ranks in blocks of 16; MB: rows in blocks of 16.
// kGrad: V and the forward's v also go, as such values, to the operands of the
// weights' gradients.
// kSmall: at most 512 rows, without a plan: every workgroup groups them itself.
// The gradient's A and B, which are copies anyway, come from rank 33 on as the
// products' operands (pack_adapters) and need not be turned over: 69
// against 92 us at 8192 rows, rank 64 and 4096 columns; at rank 16, where the
// second product's would be twice as long, 88 against 79 us for 128 experts (both
// before the last tiles were shared out).  (A forward pass that packs first gains
// less than the packing takes.)
//
// Bound by memory: 8192 rows, rank 16, 4096 columns, 201 MB 34 us where a part is
// in the last-level cache, 48 from memory (4.2 TB/s); 128 experts' 335 MB 59 us
// (5.5 TB/s); rank 64 gradients, 201 MB and 6 of operands, 46 us in 256 tiles.
// At high ranks by the adapters too, which every tile reads through L2 (rank 128:
// 2 MB for 0.8 of rows).  Few tiles are a chain: two products of 8 steps a
// wavefront, 1 to 1.5 us each (rank 64, 130 tiles: 27 us).
template <int RB, int MB, bool kGrad, bool kBase, bool kSmall>
__global__ void __launch_bounds__(kAdWaves * 64, RB < 4 || (RB == 4 && kGrad) ? 4 : 2) adapter_kernel(AdapterParams P) {
    constexpr bool kPacked = kGrad && RB >= 4;
    constexpr int kR = 16 * RB, kPieces = 3, kPitch = (RB == 1 ? 4 : kPieces) * kR + 8;
    constexpr int kMost = kPacked ? 4 : 8, kRound = RB * MB < kMost ? RB * MB : kMost;  // blocks of V joined at a time
    constexpr int kA = RB < 2 ? RB : 2;                // rank blocks turned over at a time
    // Steps of the first product whose loads are in registers.
    constexpr int kAhead = RB < 2 || (RB < 4 && MB < 2) || (RB == 4 && !kPacked) ? 2 : 1;
    constexpr int NB = 4, kCols = 16 * NB;  // neighbouring columns of a lane; columns of a step
    constexpr int kB = (RB + 1) / 2, kBLoads = NB * RB / 2;  // operands a column; 16-byte loads of B a lane and step
    constexpr int kUnits1 = (MB + (kPacked ? 0 : kA)) * 128, kUnits2 = kPacked ? 0 : kBLoads * 64, kUnits = kUnits1 > kUnits2 ? kUnits1 : kUnits2;
    constexpr int kRed = kRound * kAdWaves * 64;
    // Units of 16 bytes: the wavefronts' pieces, and in between their sums.
    __shared__ __attribute__((aligned(16))) u32x4 lds[kAdWaves * kUnits > kRed ? kAdWaves * kUnits : kRed];
    __shared__ __attribute__((aligned(16))) uint16_t vs[16 * MB][kPitch];
    __shared__ int64_t base_at[16 * MB], out_at[16 * MB];  // where the rows start, in bytes
    const int lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    u32x4* own = lds + wave * kUnits;
    // Whole tiles in multiples of the CUs; the rest are shared out by columns
    // between all CUs (each share repeats the first product).  One tile too many
    // would otherwise be worked on by one CU, at less than half of its speed beside
    // another, long after the others are done: the gradients' 257 tiles of rank 64
    // and 4096 columns 65 us, shared out 50, and 256 tiles 45.  Consecutive tiles,
    // which mostly share an adapter, on one XCD.
    const uint32_t n_all = kSmall ? P.tile_bound : *P.n_tiles, n_whole = kSmall ? 0 : n_all / kCus * kCus;
    const bool is_whole = blockIdx.x < n_whole;
    const uint32_t first = is_whole ? 0 : n_whole, tiles = is_whole ? n_whole : n_all - n_whole;
    uint32_t slabs = is_whole ? 1 : P.slabs;
    if (!kSmall && !is_whole) slabs = max(1u, min(slabs, kCus / max(tiles, 1u)));
    const uint32_t items = tiles * slabs;
    const uint32_t per = (items + 7) / 8, block = blockIdx.x - first, item = (block & 7) * per + (block >> 3);
    if ((block >> 3) >= per || item >= items) return;
    const int32_t tile = first + item / slabs, slab = item % slabs;
    int4 t;
    __shared__ int32_t rows[16];
    if constexpr (kSmall) {
        // Thread r has row r.  Its rank among the rows of its adapter: equal
        // lanes find each other by a ballot for each bit of the adapter; counts
        // of the earlier wavefronts' in LDS.  Every 16th row of an adapter leads
        // a tile; tiles are numbered by their leaders.
        uint16_t* counts = reinterpret_cast<uint16_t*>(lds);  // [kAdWaves][bins]
        const int bins = P.n + 1, r = threadIdx.x;
        const bool live = r < P.M;
        int bin = P.n;
        if (live) bin = P.ids[r];
        if (bin < 0 || bin > P.n) bin = P.n;
        for (int k = threadIdx.x; k < kAdWaves * bins; k += kAdWaves * 64) counts[k] = 0;
        uint64_t same = __ballot(live);
        for (int bit = 0; (P.n >> bit) != 0; bit++) {
            const bool on = (bin >> bit) & 1;
            const uint64_t m = __ballot(on);
            same &= on ? m : ~m;
        }
        int rank = __popcll(same & ((1ull << lane) - 1));
        __syncthreads();
        if (live && rank == 0) counts[wave * bins + bin] = (uint16_t)__popcll(same);
        __syncthreads();
        int total = 0;
#pragma unroll
        for (int w = 0; w < kAdWaves; w++) {
            const int n = counts[w * bins + bin];
            total += n;
            rank += w < wave ? n : 0;
        }
        __shared__ uint64_t leaders[kAdWaves];
        __shared__ int4 lead;  // adapter, its rank, rows of the adapter
        const bool leads = live && rank % 16 == 0 && (bin < P.n || P.rest);
        const uint64_t mine = __ballot(leads);
        if (lane == 0) leaders[wave] = mine;
        __syncthreads();
        int number = __popcll(mine & ((1ull << lane) - 1)), n_tiles = 0;
#pragma unroll
        for (int w = 0; w < kAdWaves; w++) {
            n_tiles += __popcll(leaders[w]);
            number += w < wave ? __popcll(leaders[w]) : 0;
        }
        if (tile >= n_tiles) return;
        if (leads && number == tile) lead = make_int4(bin, rank, total, 0);
        __syncthreads();
        const int rank0 = lead.y;
        t.x = lead.x < P.n ? lead.x : -1;
        t.z = min(lead.z - rank0, 16);
        if (live && bin == lead.x && rank >= rank0 && rank < rank0 + 16) rows[rank - rank0] = r;
        __syncthreads();
    } else {
        t = P.tiles[tile];
    }
    const int a = t.x, count = t.z;
    // Rows past `count` repeat the last one: its values, stored again.
    auto row_of = [&](int m) {
        if constexpr (kSmall) return (int64_t)rows[min(m, count - 1)];
        return (int64_t)P.order[t.y + min(m, count - 1)];
    };
    if (a < 0) {
        // Rows without an adapter, one a wavefront, eight loads in flight (one: 32
        // rows of 4096 columns take 19 us, as long as a tile with an adapter).
        constexpr int kLoads = 8;
        const int pieces = P.N / 8, c0 = (int)((int64_t)pieces * slab / slabs), c1 = (int)((int64_t)pieces * (slab + 1) / slabs);
        for (int m = wave; m < count; m += kAdWaves) {
            const int64_t r = row_of(m);
            uint16_t* to = P.out + r * P.ld_out;
            for (int c = c0 + lane; c < c1; c += 64 * kLoads) {
                u32x4 z[kLoads];
#pragma unroll
                for (int j = 0; j < kLoads; j++) {
                    z[j] = u32x4{0, 0, 0, 0};
                    if (kBase) z[j] = load16(P.base + r * P.ld_base + 8 * min(c + 64 * j, c1 - 1));
                }
                issue();
#pragma unroll
                for (int j = 0; j < kLoads; j++)
                    if (c + 64 * j < c1) *reinterpret_cast<u32x4*>(to + 8 * (c + 64 * j)) = z[j];
            }
        }
        if (!kGrad && P.v && slab == 0)
            for (int k = threadIdx.x; k < count * P.R; k += kAdWaves * 64) P.v[row_of(k / P.R) * P.R + k % P.R] = 0.0f;
        return;
    }

    // The first product: 64 columns a step, of 8 rows a load.  (Ranks past R
    // take other ones' values, which the join makes zeros.)
    const int sub = lane >> 3, piece = lane & 7;  // row in a load, unit in a row
    const uint16_t* xr[2 * MB];
#pragma unroll
    for (int k = 0; k < 2 * MB; k++) xr[k] = P.x + row_of(8 * k + sub) * P.ldx + 8 * piece;
    const uint16_t* ar = P.A + ((int64_t)a * P.R + sub) * P.K + 8 * piece;
    const u32x4* a_pack = reinterpret_cast<const u32x4*>(P.A) + a * P.units_a + lane;
    u32x4 xf[kAhead][2 * MB], af[kAhead][2 * RB];
    f32x4 acc[RB][MB];
#pragma unroll
    for (int r = 0; r < RB; r++)
#pragma unroll
        for (int m = 0; m < MB; m++) acc[r][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto load1 = [&](int s, int c) {
#pragma unroll
        for (int k = 0; k < 2 * MB; k++) xf[s][k] = load16(xr[k] + c * 64);
#pragma unroll
        for (int k = 0; k < 2 * RB; k++)
            if constexpr (kPacked)
                af[s][k] = a_pack[((int64_t)c * (2 * RB) + k) * 64];
            else
                af[s][k] = load16(ar + (int64_t)min(8 * k, P.R - 8) * P.K + c * 64);
        issue();
    };
    auto mul1 = [&](int s, auto next) {
        u32x4* put = own + sub * 8 + (piece ^ sub);
#pragma unroll
        for (int k = 0; k < 2 * MB; k++) put[64 * k] = xf[s][k];
        if constexpr (kPacked) {
            issue();
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const u32x4* at = own + i * 8 + ((4 * h + q) ^ (i & 7));
                u32x4 x[MB];
#pragma unroll
                for (int m = 0; m < MB; m++) x[m] = at[128 * m];
#pragma unroll
                for (int r = 0; r < RB; r++)
#pragma unroll
                    for (int m = 0; m < MB; m++) acc[r][m] = mfma16(af[s][h * RB + r], x[m], acc[r][m]);
            }
            issue();
            next();
            return;
        }
#pragma unroll
        for (int r0 = 0; r0 < RB; r0 += kA) {
#pragma unroll
            for (int k = 0; k < 2 * kA; k++) put[64 * (2 * MB + k)] = af[s][2 * r0 + k];
            if (r0 + kA == RB) {
                issue();
                next();
            }
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const u32x4* at = own + i * 8 + ((4 * h + q) ^ (i & 7));
                u32x4 x[MB];
#pragma unroll
                for (int m = 0; m < MB; m++) x[m] = at[128 * m];
#pragma unroll
                for (int r = 0; r < kA; r++) {
                    const u32x4 w = at[128 * (MB + r)];
#pragma unroll
                    for (int m = 0; m < MB; m++) acc[r0 + r][m] = mfma16(w, x[m], acc[r0 + r][m]);
                }
            }
        }
    };
    auto nothing = [] {};
    {
        // The wavefront's steps: consecutive ones, so that the wavefronts read
        // far apart and rows of a power of two bytes do not all meet in a few
        // channels of L2.  The last one may be a part.
        const int steps = (P.K + 63) / 64, whole = min(steps * (wave + 1) / kAdWaves, P.K / 64);
        int c = steps * wave / kAdWaves;
        const bool rest = wave == kAdWaves - 1 && P.K % 64 != 0;
        auto at = [&](int k) { return c + k; };
#pragma unroll
        for (int s = 0; s < kAhead; s++)
            if (at(s) < whole) load1(s, at(s));
        for (; at(2 * kAhead - 1) < whole; c = at(kAhead))
#pragma unroll
            for (int s = 0; s < kAhead; s++) mul1(s, [&] { load1(s, at(kAhead + s)); });
#pragma unroll
        for (int s = 0; s < kAhead; s++)
            if (at(kAhead + s) < whole)
                mul1(s, [&] { load1(s, at(kAhead + s)); });
            else if (at(s) < whole)
                mul1(s, nothing);
#pragma unroll
        for (int s = 0; s < kAhead - 1; s++)
            if (at(kAhead + s) < whole) mul1(s, nothing);
        if (rest) {
            c = P.K / 64;
            const bool in = c * 64 + 8 * piece < P.K;
            const int k0 = in ? c * 64 : -8 * piece;  // (the row's start)
            const u32x4 z = {0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < 2 * MB; k++) {
                xf[0][k] = load16(xr[k] + k0);
                if (!in) xf[0][k] = z;
            }
#pragma unroll
            for (int k = 0; k < 2 * RB; k++) {
                if constexpr (kPacked) {
                    af[0][k] = a_pack[((int64_t)c * (2 * RB) + k) * 64];
                } else {
                    af[0][k] = load16(ar + (int64_t)min(8 * k, P.R - 8) * P.K + k0);
                    if (!in) af[0][k] = z;
                }
            }
            mul1(0, nothing);
        }
    }

    // The second product, kCols columns a step: lane i has columns NB i .. + NB - 1
    // of rows 4 q .. + 3 of each block; product b takes columns NB n + b.
    typedef uint32_t vec __attribute__((ext_vector_type(NB / 2)));
    if (threadIdx.x < 16 * MB) {
        const int64_t r = row_of(threadIdx.x);
        base_at[threadIdx.x] = 2 * r * P.ld_base;
        out_at[threadIdx.x] = 2 * r * P.ld_out;
    }
    const uint16_t* B = P.B + (int64_t)a * P.N * P.R;
    const int units_b = kCols * P.R / 8;  // of B in a step: consecutive
    u32x4 bf[kPacked ? NB * kB : kBLoads];
    const u32x4* b_pack = reinterpret_cast<const u32x4*>(P.B) + a * P.units_b + lane;
    auto load_b = [&](int n0) {  // (past the last column, its last unit)
        if constexpr (kPacked) {
#pragma unroll
            for (int k = 0; k < NB * kB; k++) bf[k] = b_pack[((int64_t)(n0 / kCols) * (NB * kB) + k) * 64];
            issue();
            return;
        }
        const int units = min(units_b, (P.N - n0) * (P.R / 8));
#pragma unroll
        for (int k = 0; k < kBLoads; k++) bf[k] = load16(B + (int64_t)n0 * P.R + min(64 * k + lane, units - 1) * 8);
        issue();
    };
    const int steps2 = (P.N + kCols - 1) / kCols, share = slab * kAdWaves + wave, shares = slabs * kAdWaves;
    int n0 = (int)((int64_t)steps2 * share / shares) * kCols;
    const int n_end = min((int)((int64_t)steps2 * (share + 1) / shares) * kCols, P.N);

    const float scale = P.scale ? P.scale[a] : 1.0f;
    f32x4* red = reinterpret_cast<f32x4*>(lds);
#pragma unroll
    for (int j0 = 0; j0 < RB * MB; j0 += kRound) {
        __syncthreads();
#pragma unroll
        for (int r = 0; r < RB; r++)
#pragma unroll
            for (int m = 0; m < MB; m++)
                if (r * MB + m >= j0 && r * MB + m < j0 + kRound) red[(wave * kRound + r * MB + m - j0) * 64 + lane] = acc[r][m];
        if (j0 + kRound == RB * MB && n0 < n_end) load_b(n0);
        __syncthreads();
        if (wave < kRound) {
            const int j = j0 + wave, m = j % MB, r = j / MB * 16 + 4 * q;  // the lane's ranks r .. r + 3 of row i
            f32x4 s = red[wave * 64 + lane];
#pragma unroll
            for (int w = 1; w < kAdWaves; w++) s += red[(w * kRound + wave) * 64 + lane];
            if (r >= P.R) s = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            if (!kGrad && P.v && slab == 0 && r < P.R && 16 * m + i < count)
                *reinterpret_cast<f32x4*>(P.v + row_of(16 * m + i) * P.R + r) = s;
            uint32_t part[kPieces][4];
#pragma unroll
            for (int e = 0; e < 4; e++) {
                float v = s[e] * scale;
#pragma unroll
                for (int p = 0; p < kPieces; p++) part[p][e] = bf16_piece(v);
            }
#pragma unroll
            for (int p = 0; p < kPieces; p++)
                *reinterpret_cast<u32x2*>(&vs[16 * m + i][p * kR + r]) =
                    u32x2{part[p][0] | (part[p][1] << 16), part[p][2] | (part[p][3] << 16)};
            // (the third piece's inputs of the second product are 16 ranks and 16 zeros)
            if constexpr (RB == 1) *reinterpret_cast<u32x2*>(&vs[16 * m + i][kPieces * kR + r]) = u32x2{0, 0};
        }
    }
    __syncthreads();
    if constexpr (kGrad) {
        // Operands of the weights' gradients (adapter_wgrad_kernel): lane l of
        // block (rank block, piece) holds rank l % 16 of rows 8 (l / 16) .. + 7.
        if (slab == 0) {
            const int64_t at = (int64_t)t.w * (RB * 3 * 64);
            for (int k = threadIdx.x; k < RB * 64; k += kAdWaves * 64) {
                const int rb = k / 64, l = k % 64, rank = rb * 16 + (l & 15), m0 = (l >> 4) * 8;
                u32x4 w[3], v[3];
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    float f[2];
                    uint32_t keep = 0;  // (rows past `count` count nothing)
#pragma unroll
                    for (int o = 0; o < 2; o++) {
                        const int m = m0 + 2 * e + o;
                        f[o] = 0.0f;
                        if (m < count && rank < P.R) f[o] = P.v_in[row_of(m) * P.R + rank];
                        if (m < count) keep |= 0xFFFFu << (16 * o);
                    }
#pragma unroll
                    for (int p = 0; p < 3; p++) {
                        w[p][e] = (vs[m0 + 2 * e][p * kR + rank] | ((uint32_t)vs[m0 + 2 * e + 1][p * kR + rank] << 16)) & keep;
                        const uint32_t lo = bf16_piece(f[0]);
                        v[p][e] = lo | (bf16_piece(f[1]) << 16);
                    }
                }
#pragma unroll
                for (int p = 0; p < 3; p++) {
                    P.w_pack[at + (rb * 3 + p) * 64 + l] = w[p];
                    P.v_pack[at + (rb * 3 + p) * 64 + l] = v[p];
                }
            }
        }
    }

    // Unit p of B's piece lies at p ^ ((p / 16) ^ (p / 64)) % 16: reads of one
    // product are 16 NB rows apart, and these differ in that term.
    const int r8 = P.R / 8;
    auto step2 = [&](int n0, auto whole) {
        vec old[MB][4];
        const int n = n0 + NB * i;
        if (kBase) {
            const uint8_t* at = reinterpret_cast<const uint8_t*>(P.base + (whole.value ? n : min(n, P.N - NB)));
            if (P.stream) {  // (the fences: or the compiler makes one load of the two kinds)
                asm volatile("" ::: "memory");
#pragma unroll
                for (int m = 0; m < MB; m++)
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        old[m][e] = __builtin_nontemporal_load(reinterpret_cast<const vec*>(at + base_at[16 * m + 4 * q + e]));
                asm volatile("" ::: "memory");
            } else {
#pragma unroll
                for (int m = 0; m < MB; m++)
#pragma unroll
                    for (int e = 0; e < 4; e++) old[m][e] = *reinterpret_cast<const vec*>(at + base_at[16 * m + 4 * q + e]);
            }
        }
        issue();
        if constexpr (!kPacked) {
#pragma unroll
            for (int k = 0; k < kBLoads; k++) own[64 * k + (lane ^ (lane >> 4) ^ ((4 * k ^ k) & 15))] = bf[k];
            issue();
            if (n0 + kCols < n_end) load_b(n0 + kCols);
        }
        f32x4 y[MB][NB];
#pragma unroll
        for (int b = 0; b < NB; b++)
#pragma unroll
            for (int m = 0; m < MB; m++) y[m][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < kB; j++) {
            u32x4 w[NB];
#pragma unroll
            for (int b = 0; b < NB; b++) {
                const int p = (NB * i + b) * r8 + min(RB == 1 ? q & 1 : 4 * j + q, r8 - 1);
                w[b] = kPacked ? bf[kPacked ? b * kB + j : 0] : own[p ^ (((p >> 4) ^ (p >> 6)) & 15)];
            }
#pragma unroll
            for (int h = RB > 1 ? kPieces - 1 : 1; h >= 0; h--) {  // the small parts of V first
                u32x4 v[MB];
#pragma unroll
                for (int m = 0; m < MB; m++) v[m] = *reinterpret_cast<const u32x4*>(&vs[16 * m + i][32 * (j + h * kB) + 8 * q]);
#pragma unroll
                for (int b = 0; b < NB; b++)
#pragma unroll
                    for (int m = 0; m < MB; m++) y[m][b] = mfma16(v[m], w[b], y[m][b]);
            }
        }
        if constexpr (kPacked) {
            issue();
            if (n0 + kCols < n_end) load_b(n0 + kCols);
        }
        if (!whole.value && n >= P.N) return;
#pragma unroll
        for (int m = 0; m < MB; m++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                vec o;
#pragma unroll
                for (int k = 0; k < NB / 2; k++) {
                    float lo = y[m][2 * k][e], hi = y[m][2 * k + 1][e];
                    if (kBase) {
                        lo += __uint_as_float(old[m][e][k] << 16);
                        hi += __uint_as_float(old[m][e][k] & 0xFFFF0000u);
                    }
                    o[k] = bf16_hw(lo) | (bf16_hw(hi) << 16);
                }
                *reinterpret_cast<vec*>(reinterpret_cast<uint8_t*>(P.out + n) + out_at[16 * m + 4 * q + e]) = o;
            }
    };
    for (; n0 + kCols <= n_end; n0 += kCols) step2(n0, std::true_type{});
    if (n0 < n_end) step2(n0, std::false_type{});
}

__global__ void __launch_bounds__(256) adapter_pack_kernel(AdapterPack P) {
    pack_adapters(P, (int64_t)blockIdx.x * 256 + threadIdx.x);
}

// dA and dB of one row chunk and 128 columns: the sum over rows is the matrix
// instruction's inner dimension, 32 rows a step.  A lane loads 8 columns of 8
// rows; one byte permutation a register turns them into operands with 8 rows of
// one column each, for eight products whose columns lie 8 apart.  w and v are
// FP32 sums and go in as three BF16 values, which is all of their 24 bits, laid
// out as operands by adapter_kernel (zeros behind the chunk's last row, where x
// and dy repeat it).
// RB: ranks in blocks of 16 (blockIdx.z takes further ones).  The NW wavefronts
// take steps in turn and join their sums in LDS.  (Wavefronts that take 128
// columns each and all steps have nothing to join, but uneven experts then leave
// CUs idle: 8 us more of 63 for 128 of them.)
// 8192 rows, rank 64, 4096 columns: 47 us for 128 MB of rows and 26 GFLOP in
// pieces, the matrix pipe busy for a quarter; 128 experts, 235 MB, 55 us (4.3
// TB/s).  Bound by the latency of the rows' loads, which the registers of the
// sums leave few of in flight, and uneven chunks.
template <int RB, int NW>
__global__ void __launch_bounds__(NW * 64, RB < 2 ? 4 : 2) adapter_wgrad_kernel(AdapterGrad P) {
    constexpr int kAhead = RB < 2 ? RB : 2;  // rank blocks whose w is in registers
    __shared__ __attribute__((aligned(16))) f32x4 red[NW * 8 * 64];
    const int lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // The last rows first, and of them dy: what adapter_kernel read last is still
    // in the last-level cache.
    const int chunk = P.n_tables[1] - 1 - (int)blockIdx.y;
    if (chunk < 0) return;
    const int4 t = P.chunks[chunk];
    const int a = t.x, count = t.z, n_slabs = (P.N + 127) / 128, slab = blockIdx.x;
    const bool is_a = slab >= n_slabs;
    const int C = is_a ? P.K : P.N, c0 = (is_a ? slab - n_slabs : slab) * 128, block0 = blockIdx.z * RB;
    const int64_t ldz = is_a ? P.ldx : P.ld_dy;
    const uint16_t* Z = (is_a ? P.x : P.dy) + min(c0 + 8 * i, C - 8);
    const u32x4* W = (is_a ? P.w_pack : P.v_pack) + ((int64_t)P.chunk_step[chunk] * P.rank_blocks + block0) * 192 + lane;
    const int32_t* order = P.order + t.y;
    f32x4 acc[8][RB];
#pragma unroll
    for (int c = 0; c < 8; c++)
#pragma unroll
        for (int r = 0; r < RB; r++) acc[c][r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    u32x4 z[8], w[kAhead][3];
    auto load_rows = [&](int s) { return order[min(s + (lane & 31), count - 1)]; };
    auto load_z = [&](int32_t rows) {
#pragma unroll
        for (int j = 0; j < 8; j++) z[j] = load16(Z + (int64_t)__shfl(rows, 8 * q + j, kWave) * ldz);
    };
    auto load_w = [&](int b, int s) {
        const u32x4* at = W + ((int64_t)(s / 32) * P.rank_blocks + b) * 192;
#pragma unroll
        for (int p = 0; p < 3; p++) w[b % kAhead][p] = at[64 * p];
    };
    // One step; `more`: the wavefront's next step is loaded meanwhile.
    constexpr int kStep = 32 * NW;
    int32_t rows = 0;
    auto step = [&](int s, auto more) {
        u32x4 zf[8];
#pragma unroll
        for (int c = 0; c < 8; c++) zf[c] = column8(z, c);
        if constexpr (more.value) {
            load_z(rows);
            rows = load_rows(s + 2 * kStep);
            issue();
        }
#pragma unroll
        for (int b = 0; b < RB; b++) {
#pragma unroll
            for (int c = 0; c < 8; c++)
#pragma unroll
                for (int p = 2; p >= 0; p--) acc[c][b] = mfma16(w[b % kAhead][p], zf[c], acc[c][b]);
            if (b + kAhead < RB)
                load_w(b + kAhead, s);
            else if constexpr (more.value)
                load_w(b + kAhead - RB, s + kStep);
        }
    };
    int s = wave * 32;
    if (s < count) {
        load_z(load_rows(s));
#pragma unroll
        for (int b = 0; b < kAhead; b++) load_w(b, s);
        rows = load_rows(s + kStep);
        for (; s + kStep < count; s += kStep) step(s, std::true_type{});
        step(s, std::false_type{});
    }
    const float scale = P.scale && !is_a ? P.scale[a] : 1.0f;  // (w holds it already)
    const int64_t each = (int64_t)P.R * (P.K + P.N);
    float* dA = t.w < 0 ? P.dA + (int64_t)a * P.R * P.K : P.slots + t.w * each;
    float* dB = t.w < 0 ? P.dB + (int64_t)a * P.R * P.N : P.slots + t.w * each + (int64_t)P.R * P.K;
#pragma unroll
    for (int b = 0; b < RB; b++) {
        const int rank = (block0 + b) * 16 + 4 * q;
        // Piece k of the block: of dA rank 4 q + k / 2 and columns 8 i + 4 (k % 2) .. + 3,
        // of dB column 8 i + k and ranks 4 q .. + 3.
        auto piece = [&](int k) {
            const int e = k >> 1, h = 4 * (k & 1);
            return is_a ? f32x4{acc[h][b][e], acc[h + 1][b][e], acc[h + 2][b][e], acc[h + 3][b][e]} : acc[k][b];
        };
        auto put = [&](int k, f32x4 v) {
            if (is_a) {
                const int c = c0 + 8 * i + 4 * (k & 1);
                if (rank + (k >> 1) < P.R && c < C) *reinterpret_cast<f32x4*>(dA + (int64_t)(rank + (k >> 1)) * P.K + c) = v;
            } else {
                const int c = c0 + 8 * i + k;
                if (rank < P.R && c < C) *reinterpret_cast<f32x4*>(dB + (int64_t)c * P.R + rank) = v * scale;
            }
        };
        if (b) __syncthreads();
#pragma unroll
        for (int k = 0; k < 8; k++) red[(wave * 8 + k) * 64 + lane] = piece(k);
        __syncthreads();
        for (int k = wave; k < 8; k += NW) {  // the wavefronts' sums, in one order
            f32x4 v = red[k * 64 + lane];
#pragma unroll
            for (int j = 1; j < NW; j++) v += red[(j * 8 + k) * 64 + lane];
            put(k, v);
        }
    }
}

// Adapters whose rows filled several chunks: the chunks' sums, in order.
__global__ void __launch_bounds__(256) adapter_join_kernel(AdapterGrad P) {
    const int a = blockIdx.y;
    const int2 info = P.info[a];
    if (info.x <= 1) return;
    const int64_t of_a = (int64_t)P.R * P.K, each = of_a + (int64_t)P.R * P.N;
    const int64_t k = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (k >= each) return;
    f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int c = 0; c < info.x; c++) s += *reinterpret_cast<const f32x4*>(P.slots + (info.y + c) * each + k);
    float* out = k < of_a ? P.dA + a * of_a + k : P.dB + a * (each - of_a) + (k - of_a);
    *reinterpret_cast<f32x4*>(out) = s;
}

int adapter_rank_blocks(int32_t R) { return R <= 16 ? 1 : R <= 32 ? 2 : R <= 64 ? 4 : 8; }
int64_t adapter_units(int64_t cols, int32_t R) {
    return R <= 32 ? cols * R / 8 : (cols + 63) / 64 * 128 * adapter_rank_blocks(R);
}

// A workgroup of the plan places 1024 rows, or as many as keep their number to
// 256: each of them counts all rows.
hipError_t launch_adapter_plan(AdapterPlan P, const AdapterPack* pack, hipStream_t stream) {
    P.rows = std::max<int64_t>(1, (P.M + 256 * kPlanThreads - 1) / (256 * kPlanThreads)) * kPlanThreads;
    P.vec = (uintptr_t)P.ids % 16 == 0;
    P.blocks = (int32_t)((P.M + P.rows - 1) / P.rows + 1);
    AdapterPack k{};
    int64_t more = 0;
    // All adapters, where their bytes are a small part of the rows'; else those with rows, afterwards.
    if (pack && (int64_t)pack->n * pack->R <= P.M / 4) {
        k = *pack;
        k.info = nullptr;
        more = (k.n * (adapter_units(k.K, k.R) + adapter_units(k.N, k.R)) / 8 + kPlanThreads - 1) / kPlanThreads;
    }
    hipLaunchKernelGGL(adapter_plan_kernel, dim3((unsigned)(P.blocks + more)), dim3(kPlanThreads), 0, stream, P, k);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !pack || more) return e;
    const int64_t items = pack->n * (adapter_units(pack->K, pack->R) + adapter_units(pack->N, pack->R)) / 8;
    hipLaunchKernelGGL(adapter_pack_kernel, dim3((unsigned)((items + 255) / 256)), dim3(256), 0, stream, *pack);
    return hipGetLastError();
}

// Rows of a forward tile.  Up to rank 16 always 16 rows, of which a CU holds two
// tiles.  Above, 16 rows are ahead by some where each CU has one tile at most
// (600 rows of 4096 columns: rank 32 14.5 against 15.6 us, rank 64 18.4 against 20.4,
// rank 128 24.8 against 27.9; near the border, 4000 rows, 25.0 against 24.1, 30.3
// against 30.7 and 41.4 against 42.0), and 32 read the adapters half as often (16384
// rows: rank 32 88 against 74 us, rank 64 128 against 97, rank 128 185 against 130).
int adapter_tile(int32_t R, int64_t M, int64_t n) { return R <= 16 || M / 16 + n + 1 <= 256 ? 16 : 32; }

namespace {

template <int RB, bool kBase>
hipError_t adapter_start(const AdapterParams& P, int64_t tiles, hipStream_t s) {
    const dim3 grid((unsigned)((tiles + 7) / 8 * 8)), block(kAdWaves * 64);
    if (P.w_pack)
        hipLaunchKernelGGL((adapter_kernel<RB, kAdTile / 16, true, kBase, false>), grid, block, 0, s, P);
    else if (P.ids)
        hipLaunchKernelGGL((adapter_kernel<RB, 1, false, kBase, true>), grid, block, 0, s, P);
    else if (adapter_tile(P.R, P.M, P.n) == 16)
        hipLaunchKernelGGL((adapter_kernel<RB, 1, false, kBase, false>), grid, block, 0, s, P);
    else if constexpr (RB > 1)
        hipLaunchKernelGGL((adapter_kernel<RB, 2, false, kBase, false>), grid, block, 0, s, P);
    return hipGetLastError();
}
template <int RB>
hipError_t adapter_run(const AdapterParams& P, int64_t tiles, hipStream_t s) {
    return P.base ? adapter_start<RB, true>(P, tiles, s) : adapter_start<RB, false>(P, tiles, s);
}

}  // namespace

// Up to 512 rows, one a thread, take one launch, which groups them itself.
bool adapter_small(int64_t M) { return M <= kAdWaves * 64; }

hipError_t launch_adapter(AdapterParams P, int64_t tiles, hipStream_t stream) {
    const int cols = 64 * kAdWaves;  // of a step
    const int64_t most = (P.N + cols - 1) / cols;  // shares of a tile's columns
    if (P.ids) {
        P.tile_bound = (int32_t)std::min<int64_t>(P.M, P.n + 1 + P.M / 16);
        P.slabs = (int32_t)std::max<int64_t>(1, std::min<int64_t>(most, kCus / P.tile_bound));
        tiles = (int64_t)P.tile_bound * P.slabs;
    } else {  // what the tiles, at most `tiles`, and the shares of the rest of them come to
        P.slabs = (int32_t)most;
        tiles = std::min<int64_t>(tiles * most, tiles + kCus);
    }
    // Where the rows' tensors (of the gradient x too) fill the 256 MB of the
    // last-level cache, base, which is read once, stays out of it: 128 experts'
    // 335 MB forward 73 -> 58 us, their gradient 73 + 63 -> 69 + 55.  Below, it may be
    // there already: 201 MB 33 us, and 40 past the cache.
    P.stream = 2 * P.M * ((P.w_pack ? 2 : 1) * (int64_t)P.K + 2 * P.N) >= ((int64_t)1 << 28);
    switch (adapter_rank_blocks(P.R)) {
        case 1: return adapter_run<1>(P, tiles, stream);
        case 2: return adapter_run<2>(P, tiles, stream);
        case 4: return adapter_run<4>(P, tiles, stream);
        default: return adapter_run<8>(P, tiles, stream);
    }
}

// Rows of a chunk of the weights' gradients, how a workgroup takes them
// (adapter_wgrad_kernel), and whether an adapter may have several.
AdapterSplit adapter_split(int64_t M, int32_t R, int64_t K, int64_t N, int64_t n) {
    const int64_t slabs = (K + 127) / 128 + (N + 127) / 128;
    AdapterSplit s{};
    s.waves = 4;
    if (R <= 16 && M <= 1024) {
        // One chunk an adapter, without sums to join.  By 16 wavefronts, a step or two
        // each, while every CU has a workgroup at most: 1021 rows of one adapter, 2048 x
        // 4096, 7.1 us a launch and by 4 wavefronts 9.2; of 8 adapters 7.1 and 4.7, of 64
        // 32 and 12.
        // All three launches with one chunk an adapter and with several, 2048 x 4096:
        // 1000 rows of one adapter 25.6 against 29.3 us, of 8 24.1 and 25.8, of 64 38.3
        // and 41.2.  (2000 rows in one chunk of 2048 would still gain: 33.4 against 36.2,
        // 29.1 and 33.0, 40.4 and 43.0.)  From rank 24 on the steps of one chunk are
        // longer, and 1000 rows of one adapter lose: rank 64 48.5 against 42.4 us (rank 32
        // 32.3 and 34.5; of 8 adapters 31.0 and 32.3, rank 64 40.4 and 42.0).
        if (n * slabs <= (int64_t)kCus) s.waves = 16;
        s.chunk = 1024;
        s.most = (int32_t)(M / 1024);
    } else {  // the columns' slabs times the chunks are the workgroups that the CUs hold at a time
        const int64_t chunks = std::max<int64_t>(1, (R <= 16 ? 1024 : 512) / slabs);
        s.chunk = (int32_t)std::min<int64_t>((std::max<int64_t>(M, 1) + 128 * chunks - 1) / (128 * chunks) * 128, (int64_t)1 << 30);
        s.most = (int32_t)std::min<int64_t>(chunks, M / 128);
    }
    s.join = M > s.chunk;
    return s;
}

hipError_t launch_adapter_wgrad(const AdapterGrad& P, const AdapterSplit& split, int64_t chunks, hipStream_t stream) {
    const dim3 grid((P.K + 127) / 128 + (P.N + 127) / 128, (unsigned)chunks, P.R > 64 ? 2 : 1);
    if (split.waves == 16)
        hipLaunchKernelGGL((adapter_wgrad_kernel<1, 16>), grid, dim3(1024), 0, stream, P);
    else if (P.R <= 16)
        hipLaunchKernelGGL((adapter_wgrad_kernel<1, 4>), grid, dim3(256), 0, stream, P);
    else if (P.R <= 32)
        hipLaunchKernelGGL((adapter_wgrad_kernel<2, 4>), grid, dim3(256), 0, stream, P);
    else
        hipLaunchKernelGGL((adapter_wgrad_kernel<4, 4>), grid, dim3(256), 0, stream, P);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !split.join) return e;
    const int64_t each = (int64_t)P.R * (P.K + P.N);
    hipLaunchKernelGGL(adapter_join_kernel, dim3((unsigned)((each / 4 + 255) / 256), P.n), dim3(256), 0, stream, P);
    return hipGetLastError();
}

}  // namespace nvfp4
