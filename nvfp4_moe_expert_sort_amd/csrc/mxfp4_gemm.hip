// mxfp4_gemm.hip -- MXFP4 products on gfx950: out[m][n] = bf16(sum_k a[m][k] w[n][k]).
//
// Both operands go into v_mfma_scale_f32_16x16x128_f8f6f4 as they are stored
// (mxfp4.h), so the loop has no decoding.  Every output element is accumulated
// in FP32 over increasing 128-column chunks by that one instruction, whatever
// the kernel, the tile and the number of rows: a row's result has the same
// bits in every batch.
//
//   mx_gemm_wide_kernel    128 rows x 256 columns per workgroup: 8 x 4 tiles of
//                          16 x 16 per wave; activations shared through LDS
//                          (direct loads, two 256-column buffers), each wave's
//                          weights straight from memory into registers
//   mx_gemm_direct_kernel  16 MT rows x 16 columns per wave, both operands
//                          straight from memory: few rows, bound by reading
//                          the weights
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
    const int32_t nm = P.tiles ? *P.n_tiles : (int32_t)((P.M + bm - 1) / bm);
    const int64_t total = (int64_t)nm * P.col_tiles, per = (total + 7) / 8;
    const int64_t at = (int64_t)(blockIdx.x >> 3);
    const int64_t idx = (int64_t)(blockIdx.x & 7) * per + at;
    MxTile t{0, 0, 0, 0, at < per && idx < total};
    if (!t.live) return t;
    const int32_t band = (int32_t)(idx / (8 * (int64_t)P.col_tiles));
    const int32_t in = (int32_t)(idx - (int64_t)band * 8 * P.col_tiles);
    const int32_t high = min(8, nm - band * 8);
    const int32_t nt = in / high, mt = band * 8 + in - nt * high;
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

constexpr int kWideMT = 8, kWideNT = 4;
constexpr int kWideBM = kWideMT * 16, kWideBN = kWideNT * 16 * 4;
constexpr int kWideStages = 3;  // 256-column steps of activations in LDS

struct WideLds {
    uint8_t a[kWideStages][kWideBM * 128];
    uint8_t s[2][kWideBM * 16];  // scale words of a 512-column quad: [row][block]
};

namespace {

// 16 bytes per lane from base + off to LDS at `lds` + 16 lane (one vmcnt event).
// The builtin would make the compiler wait for every load in flight before
// each LDS read, since it cannot tell the buffers apart; here the waits are
// written out (`arrive`).  m0, which the compiler does not list as clobbered,
// has no other user in these kernels.
__device__ __forceinline__ void dma16(const uint8_t* base, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(lds) : "memory");
}
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

// The product of a tile of up to MT 16-row subtiles.  Loop over 128-column
// chunks, four of them (a quad, one scale word) unrolled:
//   - activations come as 256-column steps, three LDS buffers deep: step s + 2
//     is requested when all waves have read step s - 1;
//   - a wave's weights are loaded two chunks ahead, each register group as
//     soon as its last product has been issued;
//   - the next chunk's activation fragments are read under the last column
//     tile's products.
template <int MT>
__device__ __forceinline__ void wide_tile(const MxGemmParams& P, const MxTile& T, WideLds& S) {
    constexpr int kDma = MT / 2;  // loads per wave and step
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
    const uint8_t* wc[kWideNT];
    const uint8_t* wsp[kWideNT];
#pragma unroll
    for (int t = 0; t < kWideNT; t++) {  // column tiles past the matrix repeat its last one
        const int64_t tile = (int64_t)T.mat * P.row_tiles + min(T.n0 / 16 + wave * kWideNT + t, P.row_tiles - 1);
        wc[t] = P.w_codes + tile * chunks * 1024;
        wsp[t] = P.w_scales + tile * quads * 256;
    }
    const uint32_t lane16 = lane * 16, lane4 = lane * 4;
    f32x4 acc[MT][kWideNT];
#pragma unroll
    for (int i = 0; i < MT; i++)
#pragma unroll
        for (int t = 0; t < kWideNT; t++) acc[i][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    u32x4 w[2][kWideNT], a[MT];
    uint32_t ws[kWideNT], wsn[kWideNT], as[MT];
    const int a_off[2] = {r * 128 + ((q ^ ((r >> 1) & 7)) << 4), r * 128 + (((4 + q) ^ ((r >> 1) & 7)) << 4)};
    auto load_w = [&](int c, int t) { return *reinterpret_cast<const u32x4*>(wc[t] + (int64_t)min(c, chunks - 1) * 1024 + lane16); };
    auto load_ws = [&](int g, int t) { return *reinterpret_cast<const uint32_t*>(wsp[t] + (int64_t)min(g, quads - 1) * 256 + lane4); };
    auto read_a = [&](int c, int i) { return *reinterpret_cast<const u32x4*>(&S.a[(c >> 1) % kWideStages][a_off[c & 1] + i * 2048]); };
    auto read_s = [&](int g, int i) { return *reinterpret_cast<const uint32_t*>(&S.s[g & 1][(i * 16 + r) * 16 + q * 4]); };
    // Step s (and the scales requested with it) has landed for every wave:
    // at least kDma loads, step s + 1's, were issued after it.  Every wave has
    // read step s - 1, whose buffer step s + 2 takes.
    auto arrive = [&]() {
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kDma) : "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    stage_scales(0);
    stage(0);
    stage(1);
#pragma unroll
    for (int t = 0; t < kWideNT; t++) ws[t] = load_ws(0, t);
#pragma unroll
    for (int t = 0; t < kWideNT; t++) w[0][t] = load_w(0, t);
#pragma unroll
    for (int t = 0; t < kWideNT; t++) w[1][t] = load_w(1, t);
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
            constexpr int kLast = kWideNT - 1;
            const int c = g * 4 + H + b;
#pragma unroll
            for (int t = 0; t < kLast; t++) {
#pragma unroll
                for (int i = 0; i < MT; i++) acc[i][t] = mx_mfma_sel(H + b, w[b][t], a[i], acc[i][t], ws[t], as[i]);
                w[b][t] = load_w(c + 2, t);
                pin(t);
            }
            if (b == 1) {
                arrive();  // step (c + 1) / 2
                if (H == 2) stage_scales(g + 2);
                stage((c + 1) / 2 + 2);
            }
#pragma unroll
            for (int i = 0; i < MT; i++) {
                acc[i][kLast] = mx_mfma_sel(H + b, w[b][kLast], a[i], acc[i][kLast], ws[kLast], as[i]);
                a[i] = read_a(c + 1, i);
                if (H + b == 3) as[i] = read_s(g + 1, i);
            }
            w[b][kLast] = load_w(c + 2, kLast);
            pin(kLast);
        }
    };
    int g = 0;
    for (; (g + 1) * 4 <= chunks; g++) {
#pragma unroll
        for (int t = 0; t < kWideNT; t++) wsn[t] = load_ws(g + 1, t);
        step(g, std::integral_constant<int, 0>{});
        step(g, std::integral_constant<int, 2>{});
#pragma unroll
        for (int t = 0; t < kWideNT; t++) ws[t] = wsn[t];
    }
    // The last, partial quad: activations are padded with zeros to whole
    // steps, so an odd last chunk's partner adds nothing.
    if (g < quads) {
        step(g, std::integral_constant<int, 0>{});
        if (g * 4 + 2 < chunks) step(g, std::integral_constant<int, 2>{});
    }
    // Epilogue: the wave's outputs go through LDS, up to 64 rows at a time, so
    // that eight lanes store a row's whole 128 bytes.  The 16-byte pieces of a
    // row are stored at piece ^ row % 8.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load into LDS is in flight
    __syncthreads();
    uint8_t* mine = reinterpret_cast<uint8_t*>(&S) + wave * (64 * 128);
    const int32_t n0 = T.n0 + wave * (kWideNT * 16);
#pragma unroll
    for (int i0 = 0; i0 < MT; i0 += 4) {
#pragma unroll
        for (int i = i0; i < MT && i < i0 + 4; i++)
#pragma unroll
            for (int t = 0; t < kWideNT; t++) {
                const f32x4 v = acc[i][t];
                const int row = (i - i0) * 16 + r;
                *reinterpret_cast<u32x2*>(mine + row * 128 + (((t * 2 + (q >> 1)) ^ (row & 7)) << 4) + (q & 1) * 8) =
                    u32x2{bf16_hw(v[0]) | (bf16_hw(v[1]) << 16), bf16_hw(v[2]) | (bf16_hw(v[3]) << 16)};
            }
        constexpr int kRows = MT < 4 ? MT * 16 : 64;
        const int rows = min(T.rows - i0 * 16, min((MT - i0) * 16, kRows)), n = n0 + (lane & 7) * 8;
        __builtin_amdgcn_wave_barrier();
        for (int row = lane >> 3; row < rows; row += 8) {
            const u32x4 v = *reinterpret_cast<const u32x4*>(mine + row * 128 + (((lane & 7) ^ (row & 7)) << 4));
            mx_store8(P, (int64_t)T.row0 + i0 * 16 + row, n, v);
        }
        __builtin_amdgcn_wave_barrier();
    }
}

}  // namespace

__global__ void __launch_bounds__(256, 2) mx_gemm_wide_kernel(MxGemmParams P) {
    __shared__ __attribute__((aligned(1024))) WideLds S;
    const MxTile T = mx_tile(P, kWideBM, kWideBN);
    if (!T.live) return;
    if (T.rows > 96)
        wide_tile<8>(P, T, S);
    else if (T.rows > 64)
        wide_tile<6>(P, T, S);
    else if (T.rows > 32)
        wide_tile<4>(P, T, S);
    else
        wide_tile<2>(P, T, S);
}

template <int MT>
__global__ void __launch_bounds__(256) mx_gemm_direct_kernel(MxGemmParams P) {
    const MxTile T = mx_tile(P, 16 * MT, 64);
    if (!T.live) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane >> 4, r = lane & 15;
    const int32_t chunks = P.chunks, nt = T.n0 / 16 + wave;
    if (nt >= P.row_tiles) return;
    const int64_t tile = (int64_t)T.mat * P.row_tiles + nt;
    const uint8_t* wc = P.w_codes + tile * chunks * 1024 + lane * 16;
    const uint8_t* wsp = P.w_scales + tile * P.quads * 256 + lane * 4;
    const uint8_t *ac[MT], *asp[MT];
#pragma unroll
    for (int i = 0; i < MT; i++) {
        const int64_t row = T.row0 + min(i * 16 + r, T.rows - 1);
        ac[i] = P.a_codes + row * P.ld_a + q * 16;
        asp[i] = P.a_scales + row * P.ld_as + q * 4;
    }
    f32x4 acc[MT];
#pragma unroll
    for (int i = 0; i < MT; i++) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    struct Quad {
        u32x4 w[4], a[MT][4];
        uint32_t ws, as[MT];
    };
    auto load = [&](Quad& b, int g) {
        g = min(g, P.quads - 1);
#pragma unroll
        for (int cc = 0; cc < 4; cc++) {
            const int64_t c = min(g * 4 + cc, chunks - 1);
            b.w[cc] = *reinterpret_cast<const u32x4*>(wc + c * 1024);
#pragma unroll
            for (int i = 0; i < MT; i++) b.a[i][cc] = *reinterpret_cast<const u32x4*>(ac[i] + c * 64);
        }
        b.ws = *reinterpret_cast<const uint32_t*>(wsp + (int64_t)g * 256);
#pragma unroll
        for (int i = 0; i < MT; i++) b.as[i] = *reinterpret_cast<const uint32_t*>(asp[i] + (int64_t)g * 16);
    };
    auto mul = [&](const Quad& b, int g) {
#pragma unroll
        for (int cc = 0; cc < 4; cc++)
            if (g * 4 + cc < chunks) {
#pragma unroll
                for (int i = 0; i < MT; i++) acc[i] = mx_mfma_sel(cc, b.w[cc], b.a[i][cc], acc[i], b.ws, b.as[i]);
            }
    };
    Quad b0, b1;
    load(b0, 0);
    for (int g = 0; g < P.quads; g += 2) {
        load(b1, g + 1);
        mul(b0, g);
        load(b0, g + 2);
        mul(b1, g + 1);
    }
#pragma unroll
    for (int i = 0; i < MT; i++)
        if (i * 16 + r < T.rows) mx_store4(P, (int64_t)T.row0 + i * 16 + r, nt * 16 + q * 4, acc[i]);
}

// Rows per tile of the kernel that mx_gemm launches for `rows` rows over E
// matrices.
int mx_tile_rows(int64_t rows, int64_t E) {
    const int64_t per = (rows + E - 1) / E;
    return per <= 16 ? 16 : per <= 32 ? 32 : per <= 64 ? 64 : kWideBM;
}

hipError_t launch_mx_gemm(MxGemmParams P, int64_t tiles_bound, int bm, hipStream_t stream) {
    P.col_tiles = bm == kWideBM ? (P.N + kWideBN - 1) / kWideBN : (P.N + 63) / 64;
    const int64_t blocks = (tiles_bound * P.col_tiles + 7) / 8 * 8;
    const dim3 grid((unsigned)blocks), wg(256);
    switch (bm) {
        case 16: hipLaunchKernelGGL(mx_gemm_direct_kernel<1>, grid, wg, 0, stream, P); break;
        case 32: hipLaunchKernelGGL(mx_gemm_direct_kernel<2>, grid, wg, 0, stream, P); break;
        case 64: hipLaunchKernelGGL(mx_gemm_direct_kernel<4>, grid, wg, 0, stream, P); break;
        default: hipLaunchKernelGGL(mx_gemm_wide_kernel, grid, wg, 0, stream, P); break;
    }
    return hipGetLastError();
}

}  // namespace nvfp4
