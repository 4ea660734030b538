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

__global__ void __launch_bounds__(256, 2) mx_gemm_wide_kernel(MxGemmParams P) {
    __shared__ __attribute__((aligned(1024))) uint8_t sa[2][kWideBM * 128];
    const MxTile T = mx_tile(P, kWideBM, kWideBN);
    if (!T.live) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane >> 4, r = lane & 15;
    const int32_t chunks = P.chunks, steps = (chunks + 1) / 2;

    // Activations: a 256-column step is 128 bytes of each row; the 16-byte
    // pieces of row `row` are stored rotated by its number (xor (row / 2) % 8)
    // so that the 16 rows of a fragment read hit different banks.
    const uint8_t* src[kWideBM / 32];
#pragma unroll
    for (int j = 0; j < kWideBM / 32; j++) {
        const int row = (wave * (kWideBM / 32) + j) * 8 + (lane >> 3), piece = (lane & 7) ^ ((row >> 1) & 7);
        src[j] = P.a_codes + (int64_t)(T.row0 + min(row, T.rows - 1)) * P.ld_a + piece * 16;
    }
    auto stage = [&](int s) {
#pragma unroll
        for (int j = 0; j < kWideBM / 32; j++)
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(src[j] + (int64_t)s * 128),
                                             (__attribute__((address_space(3))) void*)&sa[s & 1][(wave * (kWideBM / 32) + j) * 1024],
                                             16, 0, 0);
    };
    // Weights: whole 1 KiB tiles; columns past the matrix repeat its last tile.
    const uint8_t* wc[kWideNT];
    const uint8_t* wsp[kWideNT];
#pragma unroll
    for (int t = 0; t < kWideNT; t++) {
        const int64_t tile = (int64_t)T.mat * P.row_tiles + min(T.n0 / 16 + wave * kWideNT + t, P.row_tiles - 1);
        wc[t] = P.w_codes + tile * chunks * 1024 + lane * 16;
        wsp[t] = P.w_scales + tile * P.quads * 256 + lane * 4;
    }
    const uint8_t* asp[kWideMT];
#pragma unroll
    for (int i = 0; i < kWideMT; i++)
        asp[i] = P.a_scales + (int64_t)(T.row0 + min(i * 16 + r, T.rows - 1)) * P.ld_as + q * 4;

    f32x4 acc[kWideMT][kWideNT];
#pragma unroll
    for (int i = 0; i < kWideMT; i++)
#pragma unroll
        for (int t = 0; t < kWideNT; t++) acc[i][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    u32x4 wn[kWideNT];
    uint32_t was[kWideNT], aas[kWideMT];
    stage(0);
#pragma unroll
    for (int t = 0; t < kWideNT; t++) wn[t] = *reinterpret_cast<const u32x4*>(wc[t]);
    const int a_off[2] = {r * 128 + ((q ^ ((r >> 1) & 7)) << 4), r * 128 + (((4 + q) ^ ((r >> 1) & 7)) << 4)};
    for (int g = 0; g < P.quads; g++) {
#pragma unroll
        for (int t = 0; t < kWideNT; t++) was[t] = *reinterpret_cast<const uint32_t*>(wsp[t] + (int64_t)g * 256);
#pragma unroll
        for (int i = 0; i < kWideMT; i++) aas[i] = *reinterpret_cast<const uint32_t*>(asp[i] + (int64_t)g * 16);
#pragma unroll
        for (int cc = 0; cc < 4; cc++) {
            const int c = g * 4 + cc;
            if (c >= chunks) break;
            if ((cc & 1) == 0) {
                __syncthreads();  // step c / 2 has landed and the other buffer is no longer read
                if (c / 2 + 1 < steps) stage(c / 2 + 1);
            }
            u32x4 w[kWideNT];
#pragma unroll
            for (int t = 0; t < kWideNT; t++) {
                w[t] = wn[t];
                wn[t] = *reinterpret_cast<const u32x4*>(wc[t] + (int64_t)min(c + 1, chunks - 1) * 1024);
            }
            const uint8_t* buf = &sa[(c >> 1) & 1][a_off[cc & 1]];
#pragma unroll
            for (int i = 0; i < kWideMT; i++) {
                const u32x4 a = *reinterpret_cast<const u32x4*>(buf + i * 2048);
#pragma unroll
                for (int t = 0; t < kWideNT; t++) acc[i][t] = mx_mfma_sel(cc, w[t], a, acc[i][t], was[t], aas[i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kWideMT; i++)
        if (i * 16 + r < T.rows) {
#pragma unroll
            for (int t = 0; t < kWideNT; t++)
                mx_store4(P, (int64_t)T.row0 + i * 16 + r, T.n0 + (wave * kWideNT + t) * 16 + q * 4, acc[i][t]);
        }
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
