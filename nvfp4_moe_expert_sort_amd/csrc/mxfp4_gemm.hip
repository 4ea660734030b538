// mxfp4_gemm.hip -- MXFP4 products on gfx950: out[m][n] = bf16(sum_k a[m][k] w[n][k]).
//
// Both operands go into v_mfma_scale_f32_16x16x128_f8f6f4 as they are stored
// (mxfp4.h), so the loop has no decoding.  Every output element is accumulated
// in FP32 over increasing 128-column chunks by that one instruction, whatever
// the kernel, the tile and the number of rows: a row's result has the same
// bits in every batch.
//
//   mx_gemm_wide_kernel    tiles of up to 128 rows x 256 or 64 columns:
//                          activations shared through LDS by direct loads, each
//                          wave's weights straight from memory into registers
//   mx_gemm_small_kernel   few rows a matrix on average (8, or 16 of one matrix):
//                          16 columns per wave, up to 32 rows quantized into
//                          LDS by the workgroup
#include <type_traits>

#include "mxfp4.h"
#include "nvfp4_kernels.h"

namespace nvfp4 {

namespace {

struct MxTile {
    int32_t mat, row0, rows, n0;  // weight matrix, rows of the operand, first output column
    bool live;
};

// The tile of this workgroup.  The XCDs take contiguous ranges of the tile
// list (workgroups are dealt to them round-robin), in which eight row tiles
// walk through the column tiles together, so that they share an L2.
__device__ __forceinline__ MxTile mx_tile(const MxGemmParams& P, int bm, int bn) {
    // (tiles x column tiles < 2^24, checked on the host)
    const uint32_t nm = P.tiles ? (uint32_t)*P.n_tiles : (uint32_t)((P.M + bm - 1) / bm);
    const uint32_t total = nm * (uint32_t)P.col_tiles, per = (total + 7) / 8;
    const uint32_t at = blockIdx.x >> 3, idx = (blockIdx.x & 7) * per + at;
    MxTile t{0, 0, 0, 0, at < per && idx < total};
    if (!t.live) return t;
    const uint32_t band = idx / (8 * (uint32_t)P.col_tiles), in = idx - band * 8 * (uint32_t)P.col_tiles;
    const uint32_t high = min(8u, nm - band * 8);
    const int32_t nt = (int32_t)(in / high), mt = (int32_t)(band * 8 + in - (uint32_t)nt * high);
    t.n0 = nt * bn;
    if (P.tiles) {
        const int4 e = P.tiles[mt];
        t.mat = e.x;
        t.row0 = e.y;
        t.rows = e.z;
    } else {
        t.row0 = mt * bm;
        t.rows = (int32_t)min((int64_t)bm, P.M - t.row0);
    }
    return t;
}

// Four consecutive columns n.. of one output row.
__device__ __forceinline__ void mx_store4(const MxGemmParams& P, int64_t row, int32_t n, f32x4 v) {
    uint16_t* o = P.out + row * P.ld_out + n;
    if (P.vec_out && n + 4 <= P.N) {
        *reinterpret_cast<u32x2*>(o) = u32x2{bf16_hw(v[0]) | (bf16_hw(v[1]) << 16), bf16_hw(v[2]) | (bf16_hw(v[3]) << 16)};
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; j++)
        if (n + j < P.N) o[j] = (uint16_t)bf16_hw(v[j]);
}

// Eight consecutive columns n.. of one output row, as BF16 pairs.
__device__ __forceinline__ void mx_store8(const MxGemmParams& P, int64_t row, int32_t n, u32x4 v) {
    uint16_t* o = P.out + row * P.ld_out + n;
    if (P.vec_out8 && n + 8 <= P.N) {
        *reinterpret_cast<u32x4*>(o) = v;
        return;
    }
    for (int j = 0; j < 8 && n + j < P.N; j++) {
        const uint32_t pair = j < 2 ? v[0] : j < 4 ? v[1] : j < 6 ? v[2] : v[3];
        o[j] = (uint16_t)(pair >> (16 * (j & 1)));
    }
}

__device__ __forceinline__ f32x4 mx_mfma_sel(int sel, u32x4 w, u32x4 a, f32x4 acc, uint32_t ws, uint32_t as) {
    switch (sel) {
        case 0: return mx_mfma<0>(w, a, acc, ws, as);
        case 1: return mx_mfma<1>(w, a, acc, ws, as);
        case 2: return mx_mfma<2>(w, a, acc, ws, as);
        default: return mx_mfma<3>(w, a, acc, ws, as);
    }
}

}  // namespace

constexpr int kWideBM = 128;
constexpr int kWideStages = 3;  // 256-column steps of activations in LDS

struct WideLds {
    uint8_t a[kWideStages][kWideBM * 128];
    uint8_t s[2][kWideBM * 16];  // scale words of a 512-column quad: [row][block]
};

namespace {

// 16 bytes per lane from base + off to LDS at `lds` + 16 lane (one vmcnt event).
// The builtin would make the compiler wait for every load in flight before
// each LDS read, since it cannot tell the buffers apart; here the waits are
// written out (`arrive`).  The load has no output register, and its address
// register is read when it issues.  The LDS address is an operand in m0, so the
// compiler knows what m0 holds; the load must not follow that move directly.
__device__ __forceinline__ void dma16(const uint8_t* base, uint32_t off, uint32_t lds) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

// 8192 x 4096 x 4096: 66-81 us, 3.4-4.2 PFLOP/s.  The matrix pipe is busy in
// 59 % of the cycles, and the card holds 1.4-1.7 GHz there: with zeros for
// operands the same cycles take 50 us, so power is what bounds it.  32768 rows
// over 128 experts of 1536 x 2048: 91 us; 303 MB read and 101 written by the
// counters (weights, quantized rows and outputs once are 350), 4.4 TB/s of the
// 5.2 that a copy moves.
//
// The product of a tile of up to MT 16-row subtiles, NT 16-column tiles per
// wave.  Loop over 128-column chunks, four of them (a quad, one scale word)
// unrolled:
//   - activations come as 256-column steps, three LDS buffers deep: step s + 2
//     is requested when all waves have read step s - 1;
//   - a wave's weights are loaded kAhead chunks ahead, each register group as
//     soon as its last product has been issued;
//   - the next chunk's activation fragments are read under the last column
//     tile's products.
template <int MT, int NT>
__device__ __forceinline__ void wide_tile(const MxGemmParams& P, const MxTile& T, WideLds& S) {
    constexpr int kDma = MT / 2;  // loads per wave and step
    constexpr int kAhead = NT == 1 ? 4 : 2;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), q = lane >> 4, r = lane & 15;
    const int32_t chunks = P.chunks, quads = P.quads, steps = (chunks + 1) / 2;

    // A step is 128 bytes of each row; the 16-byte pieces of row `row` are
    // stored at piece ^ (row / 2) % 8, so that the 16 rows of a fragment read
    // hit different banks.
    // (Addresses are a uniform base and a 32-bit offset per lane: K < 2^24 keeps
    // a tile's rows within it.)
    const uint8_t* a_base = P.a_codes + (int64_t)T.row0 * P.ld_a;
    const uint8_t* s_base = P.a_scales + (int64_t)T.row0 * P.ld_as;
    uint32_t src[kDma];
#pragma unroll
    for (int j = 0; j < kDma; j++) {
        const int row = (wave * kDma + j) * 8 + (lane >> 3), piece = (lane & 7) ^ ((row >> 1) & 7);
        src[j] = (uint32_t)min(row, T.rows - 1) * (uint32_t)P.ld_a + piece * 16;
    }
    const uint32_t lds_a = lds_addr(&S.a[0][wave * kDma * 1024]), lds_s = lds_addr(&S.s[0][wave * MT * 64]);
    auto stage = [&](int s) {  // a step past the end repeats the last one into a buffer that is not read again
        const int at = min(s, steps - 1);
#pragma unroll
        for (int j = 0; j < kDma; j++)
            dma16(a_base + (int64_t)at * 128, src[j], lds_a + (uint32_t)(s % kWideStages) * (kWideBM * 128) + j * 1024);
    };
    // scale words: wave w brings rows [w MT 4, (w + 1) MT 4), 16 bytes each
    const uint32_t ssrc = (uint32_t)min(wave * MT * 4 + min(lane, MT * 4 - 1), T.rows - 1) * (uint32_t)P.ld_as;
    auto stage_scales = [&](int g) {
        if (lane < MT * 4) dma16(s_base + (int64_t)min(g, quads - 1) * 16, ssrc, lds_s + (uint32_t)(g & 1) * (kWideBM * 16));
    };
    const uint8_t* wc[NT];
    const uint8_t* wsp[NT];
#pragma unroll
    for (int t = 0; t < NT; t++) {  // column tiles past the matrix repeat its last one
        const int64_t tile = (int64_t)T.mat * P.row_tiles + min(T.n0 / 16 + wave * NT + t, P.row_tiles - 1);
        wc[t] = P.w_codes + tile * chunks * 1024;
        wsp[t] = P.w_scales + tile * quads * 256;
    }
    const uint32_t lane16 = lane * 16, lane4 = lane * 4;
    f32x4 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; i++)
#pragma unroll
        for (int t = 0; t < NT; t++) acc[i][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    u32x4 w[kAhead][NT], a[MT];
    uint32_t ws[NT], wsn[NT], as[MT];
    const int a_off[2] = {r * 128 + ((q ^ ((r >> 1) & 7)) << 4), r * 128 + (((4 + q) ^ ((r >> 1) & 7)) << 4)};
    auto load_w = [&](int c, int t) {
        return *reinterpret_cast<const u32x4*>(wc[t] + (int64_t)min(c, chunks - 1) * 1024 + lane16);
    };
    auto load_ws = [&](int g, int t) {
        return *reinterpret_cast<const uint32_t*>(wsp[t] + (int64_t)min(g, quads - 1) * 256 + lane4);
    };
    auto read_a = [&](int c, int i) {
        return *reinterpret_cast<const u32x4*>(&S.a[(c >> 1) % kWideStages][a_off[c & 1] + i * 2048]);
    };
    auto read_s = [&](int g, int i) { return *reinterpret_cast<const uint32_t*>(&S.s[g & 1][(i * 16 + r) * 16 + q * 4]); };
    // Waits until a step has landed for every wave; every wave has then also
    // read the step before, whose buffer the next request takes.  Loads return
    // in order and the kDma loads of the next step were issued after it.  (A
    // longer count that leaves the weights in flight too measured the same.)
    auto arrive = [&]() {
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kDma) : "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    stage_scales(0);
    stage(0);
    stage(1);
#pragma unroll
    for (int t = 0; t < NT; t++) ws[t] = load_ws(0, t);
#pragma unroll
    for (int b = 0; b < kAhead; b++)
#pragma unroll
        for (int t = 0; t < NT; t++) w[b][t] = load_w(b, t);
    arrive();
    stage_scales(1);
    stage(2);
#pragma unroll
    for (int i = 0; i < MT; i++) {
        a[i] = read_a(0, i);
        as[i] = read_s(0, i);
    }
    // Holds a column tile's products at their place: they have no side effect,
    // and instruction selection would otherwise sink them all to the end of
    // the loop body and spill their operands.
    auto pin = [&](int t) {
#pragma unroll
        for (int i = 0; i < MT; i += 2) asm volatile("" : "+v"(acc[i][t]), "+v"(acc[i + 1][t]));
    };
    // Chunks 4 g + HALF and the next one: one step.
    auto step = [&](int g, auto half) {
        constexpr int H = decltype(half)::value;
#pragma unroll
        for (int b = 0; b < 2; b++) {
            constexpr int kLast = NT - 1;
            const int c = g * 4 + H + b, k = (H + b) % kAhead;
#pragma unroll
            for (int t = 0; t < kLast; t++) {
#pragma unroll
                for (int i = 0; i < MT; i++) acc[i][t] = mx_mfma_sel(H + b, w[k][t], a[i], acc[i][t], ws[t], as[i]);
                w[k][t] = load_w(c + kAhead, t);
                pin(t);
            }
            if (b == 1) {
                arrive();  // step (c + 1) / 2
                if (H == 2) stage_scales(g + 2);
                stage((c + 1) / 2 + 2);
            }
#pragma unroll
            for (int i = 0; i < MT; i++) {
                acc[i][kLast] = mx_mfma_sel(H + b, w[k][kLast], a[i], acc[i][kLast], ws[kLast], as[i]);
                a[i] = read_a(c + 1, i);
                if (H + b == 3) as[i] = read_s(g + 1, i);
            }
            w[k][kLast] = load_w(c + kAhead, kLast);
            pin(kLast);
        }
    };
    int g = 0;
    for (; (g + 1) * 4 <= chunks; g++) {
#pragma unroll
        for (int t = 0; t < NT; t++) wsn[t] = load_ws(g + 1, t);
        step(g, std::integral_constant<int, 0>{});
        step(g, std::integral_constant<int, 2>{});
#pragma unroll
        for (int t = 0; t < NT; t++) ws[t] = wsn[t];
    }
    // The last, partial quad: activations are padded with zeros to whole
    // steps, so an odd last chunk's partner adds nothing.
    if (g < quads) {
        step(g, std::integral_constant<int, 0>{});
        if (g * 4 + 2 < chunks) step(g, std::integral_constant<int, 2>{});
    }
    // Epilogue: the outputs go through LDS, up to 64 rows at a time, so that
    // eight lanes store 128 bytes of a row: a wave's own 64 columns, or with
    // NT = 1 the workgroup's.  The 16-byte pieces of a row are stored at
    // piece ^ row % 8.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load into LDS is in flight
    __syncthreads();
    constexpr bool kOwn = NT == 4;
    constexpr int kRows = MT < 4 ? MT * 16 : 64;
    uint8_t* out = reinterpret_cast<uint8_t*>(&S) + (kOwn ? wave * (64 * 128) : 0);
    const int piece0 = kOwn ? 0 : wave * 2, reader = kOwn ? lane : threadIdx.x;
    const int32_t n = T.n0 + (kOwn ? wave * 64 : 0) + (reader & 7) * 8;
#pragma unroll
    for (int i0 = 0; i0 < MT; i0 += 4) {
#pragma unroll
        for (int i = i0; i < MT && i < i0 + 4; i++)
#pragma unroll
            for (int t = 0; t < NT; t++) {
                const f32x4 v = acc[i][t];
                const int row = (i - i0) * 16 + r;
                *reinterpret_cast<u32x2*>(out + row * 128 + (((piece0 + t * 2 + (q >> 1)) ^ (row & 7)) << 4) + (q & 1) * 8) =
                    u32x2{bf16_hw(v[0]) | (bf16_hw(v[1]) << 16), bf16_hw(v[2]) | (bf16_hw(v[3]) << 16)};
            }
        const int rows = min(T.rows - i0 * 16, min((MT - i0) * 16, kRows));
        if (kOwn)
            __builtin_amdgcn_wave_barrier();
        else
            __syncthreads();
        for (int row = reader >> 3; row < rows; row += kOwn ? 8 : 32) {
            const u32x4 v = *reinterpret_cast<const u32x4*>(out + row * 128 + (((reader & 7) ^ (row & 7)) << 4));
            mx_store8(P, (int64_t)T.row0 + i0 * 16 + row, n, v);
        }
        if (kOwn)
            __builtin_amdgcn_wave_barrier();
        else
            __syncthreads();
    }
}

}  // namespace

template <int NT>
__global__ void __launch_bounds__(256, 2) mx_gemm_wide_kernel(MxGemmParams P) {
    __shared__ __attribute__((aligned(1024))) WideLds S;
    const MxTile T = mx_tile(P, kWideBM, NT * 64);
    if (!T.live) return;
    if (T.rows > 96)
        wide_tile<8, NT>(P, T, S);
    else if (T.rows > 64)
        wide_tile<6, NT>(P, T, S);
    else if (T.rows > 32)
        wide_tile<4, NT>(P, T, S);
    else
        wide_tile<2, NT>(P, T, S);
}

// Few rows: workgroup (x, y) takes every gridDim.x-th group of 64 columns, 16 per
// wave, for pass y of the product: up to kSmallBM rows of one matrix, so that an
// expert with many rows keeps as many workgroups busy.  It quantizes the rows
// itself, into LDS, while its first weights (12 KiB a wave) are on their way:
// no launch, table or round trip through memory comes before them.  Bound by
// reading the weights: 512 rows over 128 experts of 1536 x 2048 take 36 us for
// 214 MB (6 TB/s, part of it from the last-level cache; 43 us and 5.0 TB/s from
// memory), 19 us if one expert has them all; 7 x 4096 x 2048 takes 6.1 us, a
// launch and one chain of loads.  After the first it streams: each wave keeps a
// ring of kSmallRing quads of weights in flight across its column groups.
constexpr int kSmallRing = 3, kSmallMT = 2, kSmallBM = 16 * kSmallMT;

namespace {

struct MxPass {
    int32_t mat;
    int64_t row0;
    int32_t rows;  // up to kSmallBM
};

// Pass blockIdx.y of a grouped product, of all experts' passes of kSmallBM rows
// in expert order; false past the last.  Offsets count as in build_tiles:
// clamped to [0, M], and the largest up to an expert is where it ends.  Every
// wavefront finds it for itself, each lane with E / 64 consecutive experts.
__device__ __forceinline__ bool mx_pass(const MxGemmParams& P, MxPass& T) {
    constexpr int kPer = kMaxExperts / 64;
    const int lane = threadIdx.x & 63, per = (P.E + 63) / 64, e0 = lane * per;
    const int32_t M = (int32_t)P.M, pass = (int32_t)blockIdx.y;
    int32_t end[kPer], top = 0;
    if (lane == 0) top = max(0, min(P.offsets[0], M));
#pragma unroll
    for (int i = 0; i < kPer; i++) {
        if (i >= per) break;
        end[i] = top = max(top, e0 + i < P.E ? min(P.offsets[e0 + i + 1], M) : 0);
    }
    int32_t before = lane == 0 ? max(0, min(P.offsets[0], M)) : 0;  // where the lane's first expert begins
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int32_t u = __shfl_up(top, o, kWave);
        if (lane >= o) top = max(top, u);
    }
    const int32_t left = __shfl_up(top, 1, kWave);
    if (lane > 0) before = left;
    int32_t sum = 0;  // passes of the lane's experts, then of all up to them
    int32_t begin = before;
#pragma unroll
    for (int i = 0; i < kPer; i++) {
        if (i >= per) break;
        end[i] = max(end[i], begin);
        sum += (end[i] - begin + kSmallBM - 1) / kSmallBM;
        begin = end[i];
    }
    const int32_t own = sum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int32_t u = __shfl_up(sum, o, kWave);
        if (lane >= o) sum += u;
    }
    int32_t at = pass - (sum - own);  // among the lane's passes, if it is one
    const uint64_t owner = __ballot(at >= 0 && at < own);
    if (owner == 0) return false;
    int32_t mat = 0, row0 = 0, rows = 0;
    begin = before;
#pragma unroll
    for (int i = 0; i < kPer; i++) {
        if (i >= per) break;
        const int32_t n = (end[i] - begin + kSmallBM - 1) / kSmallBM;
        if (at >= 0 && at < n) {
            mat = e0 + i;
            row0 = begin + at * kSmallBM;
            rows = min(end[i] - row0, kSmallBM);
        }
        at -= n;
        begin = end[i];
    }
    const int src = __builtin_ctzll(owner);
    T.mat = __builtin_amdgcn_readlane(mat, src);
    T.row0 = __builtin_amdgcn_readlane(row0, src);
    T.rows = __builtin_amdgcn_readlane(rows, src);
    return true;
}

}  // namespace

__global__ void __launch_bounds__(256, 4) mx_gemm_small_kernel(MxGemmParams P) {
    // codes [kSmallBM][lds_codes], then scale words [kSmallBM][lds_scales]
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), q = lane >> 4, r = lane & 15;
    MxPass T{0, 0, (int32_t)P.M};
    if (P.offsets && !mx_pass(P, T)) return;
    const uint32_t rows = (uint32_t)T.rows;
    const int32_t chunks = P.chunks, quads = P.quads;
    const int32_t col_groups = (P.N + 63) / 64;
    const int32_t mine = (col_groups - blockIdx.x + gridDim.x - 1) / gridDim.x;  // this workgroup's
    const int64_t mat_tile = (int64_t)T.mat * P.row_tiles;
    const uint32_t lane16 = lane * 16, lane4 = lane * 4;
    const uint32_t groups = (uint32_t)chunks * 16;  // 8-column groups of a row, padded to whole chunks
    uint8_t* sc = smem + kSmallBM * P.lds_codes;
    u32x4 w[kSmallRing][4];
    uint32_t ws[kSmallRing];
    // The load cursor: quad lg of column group lj (past the last it repeats the last quad).
    int32_t lg, lj;
    const uint8_t *lc, *ls;
    auto column_group = [&](int j) {  // columns past the matrix repeat its last 16, and are not stored
        const int64_t tile = mat_tile + min(((int32_t)blockIdx.x + j * (int32_t)gridDim.x) * 4 + wave, P.row_tiles - 1);
        lc = P.w_codes + tile * chunks * 1024;
        ls = P.w_scales + tile * quads * 256;
    };
    auto load = [&](int slot) {
#pragma unroll
        for (int cc = 0; cc < 4; cc++)
            w[slot][cc] = *reinterpret_cast<const u32x4*>(lc + (int64_t)min(lg * 4 + cc, chunks - 1) * 1024 + lane16);
        ws[slot] = *reinterpret_cast<const uint32_t*>(ls + (int64_t)lg * 256 + lane4);
        if (++lg == quads) {
            if (lj + 1 < mine) {
                lg = 0;
                column_group(++lj);
            } else {
                lg = quads - 1;
            }
        }
    };
    lg = lj = 0;
    column_group(0);
#pragma unroll
    for (int s = 0; s < kSmallRing; s++) load(s);
    for (uint32_t i0 = threadIdx.x; i0 < rows * groups; i0 += 4 * 256) {
        u32x4 v[4];
        uint32_t row[4], col[4];
#pragma unroll
        for (int u = 0; u < 4; u++) {
            const uint32_t i = i0 + u * 256;
            row[u] = __umulhi(i, P.groups_magic);
            col[u] = (i - row[u] * groups) * 8;
            v[u] = u32x4{0u, 0u, 0u, 0u};
            if (i < rows * groups && col[u] < P.cols)
                v[u] = *reinterpret_cast<const u32x4*>(P.x + (T.row0 + row[u]) * P.ldx + col[u]);
        }
#pragma unroll
        for (int u = 0; u < 4; u++) {
            const uint32_t byte = mx_scale_byte(mx_block_max(v[u]), P.up);
            if (i0 + u * 256 >= rows * groups) continue;
            *reinterpret_cast<uint32_t*>(smem + row[u] * P.lds_codes + col[u] / 2) = mx_encode8(v[u], byte);
            const uint32_t b = col[u] / 32, c = b >> 2;
            if ((threadIdx.x & 3) == 0) sc[row[u] * P.lds_scales + (c >> 2) * 16 + (b & 3) * 4 + (c & 3)] = (uint8_t)byte;
        }
    }
    __syncthreads();
    const bool two = rows > 16;
    f32x4 acc[kSmallMT] = {};
    int32_t g = 0, j = 0;  // the product cursor
    while (j < mine) {
#pragma unroll
        for (int s = 0; s < kSmallRing; s++) {
            if (j >= mine) break;
#pragma unroll
            for (int i = 0; i < kSmallMT; i++) {
                if (i > 0 && !two) break;
                const uint32_t as = *reinterpret_cast<const uint32_t*>(sc + (i * 16 + r) * P.lds_scales + g * 16 + q * 4);
#pragma unroll
                for (int cc = 0; cc < 4; cc++)
                    if (g * 4 + cc < chunks) {
                        const u32x4 a = *reinterpret_cast<const u32x4*>(smem + (i * 16 + r) * P.lds_codes +
                                                                        (g * 4 + cc) * 64 + q * 16);
                        acc[i] = mx_mfma_sel(cc, w[s][cc], a, acc[i], ws[s], as);
                    }
            }
            load(s);
            if (++g == quads) {
                const int32_t n = ((int32_t)blockIdx.x + j * (int32_t)gridDim.x) * 64 + wave * 16 + q * 4;
                for (int i = 0; i < kSmallMT; i++) {
                    if (i * 16 + r < (int)rows) mx_store4(P, T.row0 + i * 16 + r, n, acc[i]);
                    acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                }
                g = 0;
                j++;
            }
        }
    }
}

// The small kernel is for few rows a matrix on average (a rule on what the host
// knows), of up to kSmallElements elements together, which each of its
// workgroups quantizes, in rows that fit LDS.  Against the tile kernel, quantizer
// included: one matrix, 8 rows of 4096 to 4096 columns 8.8 against 11.0 us.
// Grouped, rows spread evenly and (in brackets) by a popularity of e^(N(0, 1/4)):
//   128 x 1536 x 2048,  4 rows  36.7 (35.9) against 38.9 (37.9)
//                       8 rows  39.4 (41.1) against 40.1 (39.7)
//                      12 rows  42.2 (47.1) against 40.4 (40.9)
//   128 x 2048 x 768,   8 rows  22.0 (22.8) against 25.3 (24.8)
//                      14 rows  23.6 (28.6) against 25.6 (26.5)
//   60 x 1536 x 2048,   6 rows  20.0 (21.5) against 22.4 (22.4)
//                      12 rows  21.6 (27.1) against 22.5 (23.1)
// Routing is uneven, so grouped products take it up to 8 rows.
constexpr int64_t kSmallRows = 16, kSmallGroupedRows = 8, kSmallElements = 32768;
constexpr int32_t kSmallCols = 4096;
constexpr int64_t kSmallBlocks = 1024;  // workgroups of the small kernel
constexpr int64_t kWideBlocks = 144;    // tiles that make 256 columns worth it
bool mx_small(int64_t rows, int64_t E, int64_t K) {
    return rows <= (E > 1 ? kSmallGroupedRows : kSmallRows) * E && rows * K <= kSmallElements * E && K <= kSmallCols;
}

hipError_t launch_mx_gemm_small(MxGemmParams P, int64_t E, hipStream_t stream) {
    // Rows start 16 bytes further in the banks than the row before.
    P.lds_codes = (P.chunks * 64 + 255) / 256 * 256 + 16;
    P.lds_scales = (P.quads * 16 + 255) / 256 * 256 + 16;
    P.groups_magic = (uint32_t)((((uint64_t)1 << 32) + P.chunks * 16 - 1) / (P.chunks * 16));
    // About four workgroups for each of 256 CUs, as far as the columns give them.
    const int64_t col_groups = (P.N + 63) / 64, used = E < P.M ? E : P.M;
    int64_t share = (kSmallBlocks + used - 1) / used;
    if (share > col_groups) share = col_groups;
    const int64_t each = (col_groups + share - 1) / share;  // evenly
    share = (col_groups + each - 1) / each;
    // A pass of kSmallBM rows is a workgroup row: at most one an expert that is not full.
    const int64_t passes = P.offsets ? P.M / kSmallBM + used : 1;
    P.E = (int32_t)E;
    hipLaunchKernelGGL(mx_gemm_small_kernel, dim3((unsigned)share, (unsigned)passes), dim3(256),
                       kSmallBM * (P.lds_codes + P.lds_scales), stream, P);
    return hipGetLastError();
}

// The column width of a tile: 256, or 64 where 256 would leave CUs without a
// workgroup (512 x 4096 x 4096, 64 tiles of 256: 21.3 against 16.9 us; 1024
// rows, 128 tiles: 24.7 against 23.7; 4096 x 1536 x 2048, 192 tiles: 20.4
// against 22.3).
//
// Measured and not taken: tiles of 256 rows by 8 waves (8192 x 4096 x 4096 with
// its quantizer 84.6 against 83.4 us), 96-row tiles for grouped products (132
// against 125 us), weights four chunks ahead in tiles of up to 96 rows (no
// change), non-temporal output stores (the grouped product 119 against 125 us,
// but with a kernel that reads the output 153 against 151).
int mx_tile_rows() { return kWideBM; }
hipError_t launch_mx_gemm(MxGemmParams P, int64_t tiles_bound, hipStream_t stream) {
    const bool wide = tiles_bound * ((P.N + 255) / 256) >= kWideBlocks;
    P.col_tiles = wide ? (P.N + 255) / 256 : (P.N + 63) / 64;
    const dim3 grid((unsigned)((tiles_bound * P.col_tiles + 7) / 8 * 8)), wg(256);
    if (wide)
        hipLaunchKernelGGL(mx_gemm_wide_kernel<4>, grid, wg, 0, stream, P);
    else
        hipLaunchKernelGGL(mx_gemm_wide_kernel<1>, grid, wg, 0, stream, P);
    return hipGetLastError();
}

}  // namespace nvfp4
