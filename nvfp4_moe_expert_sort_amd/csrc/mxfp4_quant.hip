// mxfp4_quant.hip -- MXFP4 quantizers and the dequantizer on gfx950.
//
// Per block of 32 columns: amax, a power-of-two scale from its BF16 exponent
// (integer arithmetic, one answer), E2M1 codes by the hardware conversion.
// All are streaming kernels (2 bytes read and 17/32 written per element, or
// the reverse), bound by HBM: 8192 x 4096 rows to operands 13.7 us (6.2 TB/s),
// 49152 x 2048 to codes and back 56 + 38 us (5.4 TB/s together), weight tiles of
// 196608 x 2048 200 us (5.1 TB/s); a plain copy on this card moves 5.2-5.5.
//   mx_quant_rows_kernel   row-major codes: four lanes share a block (16 bytes
//                          each, so a wave's load is 1 KiB of one row); writes
//                          the public logical layout, or the operand rows of
//                          the products with the row-tile table beside them
//   mx_quant_tiles_kernel  the weights' tile layout: a wave takes 16 rows x 512
//                          columns and stores whole 1 KiB tiles
//   mx_dequant_kernel      either layout back to BF16 (exact below 2^128)
#include "mxfp4.h"
#include "nvfp4_kernels.h"

namespace nvfp4 {

namespace {

// g / n for g < 2^32, n >= 1, with inv = 1.0 / n: the FP64 quotient is off by
// less than one, and the remainder corrects it.
__device__ __forceinline__ uint32_t divide(uint32_t g, uint32_t n, double inv) {
    uint32_t q = (uint32_t)((double)g * inv);
    const int32_t r = (int32_t)(g - q * n);
    if (r < 0) q--;
    if (r >= (int32_t)n) q++;
    return q;
}

// The row tiles of a grouped product, in expert order: {expert, first row,
// rows, 0} for tiles of `bm` rows.  Offsets are clamped to [0, R] and made
// monotone by a running maximum, so no value in them reaches past the rows.
__device__ void build_tiles(const MxRowsParams& P) {
    __shared__ int32_t off[kMaxExperts + 1];
    __shared__ int32_t wsum[4], wmax[4];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    constexpr int kPer = kMaxExperts / 256;
    int32_t hi[kPer];  // end of expert tid * kPer + i
    int32_t m = 0;
#pragma unroll
    for (int i = 0; i < kPer; i++) {
        const int e = tid * kPer + i;
        int32_t v = 0;
        if (e < P.E) v = max(0, min(P.offsets[e + 1], (int32_t)P.rows));
        if (e == 0) v = max(v, max(0, min(P.offsets[0], (int32_t)P.rows)));
        hi[i] = m = max(m, v);
    }
    int32_t s = m;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int32_t u = __shfl_up(s, o, kWave);
        if (lane >= o) s = max(s, u);
    }
    if (lane == 63) wmax[wave] = s;
    __syncthreads();
    int32_t before = __shfl_up(s, 1, kWave);
    if (lane == 0) before = 0;
    for (int w = 0; w < wave; w++) before = max(before, wmax[w]);
#pragma unroll
    for (int i = 0; i < kPer; i++) off[tid * kPer + i + 1] = max(hi[i], before);
    if (tid == 0) off[0] = max(0, min(P.offsets[0], (int32_t)P.rows));
    __syncthreads();
    int32_t n = 0;
#pragma unroll
    for (int i = 0; i < kPer; i++) {
        const int e = tid * kPer + i;
        if (e < P.E) n += (off[e + 1] - off[e] + P.bm - 1) / P.bm;
    }
    int32_t t = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int32_t u = __shfl_up(t, o, kWave);
        if (lane >= o) t += u;
    }
    if (lane == 63) wsum[wave] = t;
    __syncthreads();
    int32_t at = t - n;
    for (int w = 0; w < wave; w++) at += wsum[w];
#pragma unroll
    for (int i = 0; i < kPer; i++) {
        const int e = tid * kPer + i;
        if (e >= P.E) break;
        const int32_t rows = off[e + 1] - off[e], tiles = (rows + P.bm - 1) / P.bm;
        const int32_t high = tiles ? ((rows + tiles - 1) / tiles + 15) / 16 * 16 : 0;  // even shares of whole 16 rows, <= bm
        for (int32_t i = 0; i < tiles; i++, at++)
            P.tiles[at] = int4{e, off[e] + i * high, max(min(high, rows - i * high), 0), 0};
    }
    if (tid == 255) *P.n_tiles = at;  // every expert lies at or before this thread's
}

}  // namespace

// Operand rows (P.operand): the codes of a row padded with zeros to 256
// columns; the scale of chunk c's block q at byte (c / 4) * 16 + q * 4 + c % 4.
__global__ void __launch_bounds__(256) mx_quant_rows_kernel(MxRowsParams P) {
    uint32_t block = blockIdx.x;
    if (P.tiles) {
        if (block == 0) {
            build_tiles(P);
            return;
        }
        block--;
    }
    const uint32_t total = P.groups * (uint32_t)P.rows;  // 8-element groups
    // A wave takes kMxUnroll KiB of consecutive groups (where rows follow each other).
    const uint32_t g0 = (block * 4 + (threadIdx.x >> 6)) * (kMxUnroll * 64) + (threadIdx.x & 63);
    u32x4 v[kMxUnroll];
    if (P.flat) {
        // Rows without gaps, in and out: element 8 g of the input is group g's,
        // bytes 4 g of the codes and scale g / 4 (its bytes within the 16 of a
        // 512-column quad transposed for an operand).
#pragma unroll
        for (int u = 0; u < kMxUnroll; u++) {
            const uint32_t g = g0 + u * 64;
            v[u] = u32x4{0u, 0u, 0u, 0u};
            if (g < total) v[u] = *reinterpret_cast<const u32x4*>(P.x + (int64_t)g * 8);
        }
#pragma unroll
        for (int u = 0; u < kMxUnroll; u++) {
            const uint32_t g = g0 + u * 64, b = g >> 2;
            const uint32_t byte = mx_scale_byte(mx_block_max(v[u]), P.up);
            const uint32_t code = mx_encode8(v[u], byte);
            if (g >= total) continue;
            *reinterpret_cast<uint32_t*>(P.codes + (int64_t)g * 4) = code;
            if ((g & 3) == 0) P.scales[P.operand ? (b & ~15u) | ((b & 3) << 2) | ((b >> 2) & 3) : b] = (uint8_t)byte;
        }
        return;
    }
    uint32_t row[kMxUnroll], col[kMxUnroll];
#pragma unroll
    for (int u = 0; u < kMxUnroll; u++) {
        const uint32_t g = g0 + u * 64;
        v[u] = u32x4{0u, 0u, 0u, 0u};
        row[u] = 0xFFFFFFFFu;
        col[u] = 0;
        if (g < total) {
            row[u] = divide(g, P.groups, P.inv_groups);
            col[u] = (g - row[u] * P.groups) * 8;
            if (col[u] < P.cols) v[u] = *reinterpret_cast<const u32x4*>(P.x + (int64_t)row[u] * P.ld + col[u]);
        }
    }
#pragma unroll
    for (int u = 0; u < kMxUnroll; u++) {
        const uint32_t byte = mx_scale_byte(mx_block_max(v[u]), P.up);
        const uint32_t code = mx_encode8(v[u], byte);
        if (row[u] == 0xFFFFFFFFu) continue;
        *reinterpret_cast<uint32_t*>(P.codes + (int64_t)row[u] * P.ld_codes + col[u] / 2) = code;
        if ((threadIdx.x & 3) == 0) {
            const uint32_t b = col[u] / 32, c = b >> 2, q = b & 3;
            const uint32_t at = P.operand ? (c >> 2) * 16 + q * 4 + (c & 3) : b;
            P.scales[(int64_t)row[u] * P.ld_scales + at] = (uint8_t)byte;
        }
    }
}

// Wave: 16 rows x 512 columns of one matrix; rows and columns past the matrix
// are zeros.
__global__ void __launch_bounds__(256) mx_quant_tiles_kernel(const uint16_t* __restrict__ x, int64_t n_units, int32_t rows,
                                                             int32_t cols, int64_t ld, int32_t row_tiles, int32_t chunks,
                                                             int32_t quads, uint8_t* __restrict__ codes,
                                                             uint8_t* __restrict__ scales, int up) {
    const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (unit >= n_units) return;
    const int lane = threadIdx.x & 63, q = lane >> 4, r = lane & 15;
    const int64_t tile = unit / quads;  // matrix * row_tiles + row tile
    const int32_t g = (int32_t)(unit % quads);
    const int64_t mat = tile / row_tiles;
    const int32_t rl = (int32_t)(tile % row_tiles) * 16 + r;
    const uint16_t* src = x + (mat * rows + rl) * ld;
    u32x4 v[4][4];
#pragma unroll
    for (int c = 0; c < 4; c++) {
        const int32_t col = (g * 4 + c) * 128 + q * 32;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[c][i] = u32x4{0u, 0u, 0u, 0u};
            if (rl < rows && col < cols) v[c][i] = *reinterpret_cast<const u32x4*>(src + col + 8 * i);
        }
    }
    uint32_t word = 0;
#pragma unroll
    for (int c = 0; c < 4; c++) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) m = mx_max2(m, mx_abs(v[c][i][j]));
        const uint32_t byte = mx_scale_byte(max(m & 0xFFFFu, m >> 16), up != 0);
        u32x4 code;
#pragma unroll
        for (int i = 0; i < 4; i++) code[i] = mx_encode8(v[c][i], byte);
        word |= byte << (8 * c);
        if (g * 4 + c < chunks) *reinterpret_cast<u32x4*>(codes + (tile * chunks + g * 4 + c) * 1024 + lane * 16) = code;
    }
    *reinterpret_cast<uint32_t*>(scales + (tile * quads + g) * 256 + lane * 4) = word;
}

// Thread: 8 elements of one row.
__global__ void __launch_bounds__(256) mx_dequant_kernel(MxDequantParams P) {
    const uint32_t total = P.groups * (uint32_t)P.rows;
#pragma unroll
    for (int u = 0; u < kMxUnroll; u++) {
        const uint32_t g = (blockIdx.x * kMxUnroll + u) * 256u + threadIdx.x;
        if (g >= total) return;
        const uint32_t row = divide(g, P.groups, P.inv_groups), col = (g - row * P.groups) * 8;
        int64_t code_at, scale_at;
        if (P.tiled) {
            const uint32_t mat = row / P.mat_rows, rl = row - mat * P.mat_rows;
            const int64_t tile = (int64_t)mat * P.row_tiles + (rl >> 4);
            const uint32_t c = col >> 7, q = (col >> 5) & 3, lane = q * 16 + (rl & 15);
            code_at = (tile * P.chunks + c) * 1024 + lane * 16 + (col & 31) / 2;
            scale_at = (tile * P.quads + (c >> 2)) * 256 + lane * 4 + (c & 3);
        } else {
            code_at = (int64_t)row * (P.cols / 2) + col / 2;
            scale_at = (int64_t)row * (P.cols / 32) + col / 32;
        }
        const uint32_t code = *reinterpret_cast<const uint32_t*>(P.codes + code_at);
        *reinterpret_cast<u32x4*>(P.out + (int64_t)row * P.ld + col) = mx_decode8(code, P.scales[scale_at]);
    }
}

hipError_t launch_mx_quant_rows(MxRowsParams P, hipStream_t stream) {
    P.groups = (uint32_t)((P.operand ? (P.cols + 255) / 256 * 256 : P.cols) / 8);
    P.inv_groups = 1.0 / P.groups;
    P.flat = P.ld == P.cols && (!P.operand || P.cols % 512 == 0);
    const uint64_t per = 256 * kMxUnroll, total = (uint64_t)P.groups * P.rows;
    hipLaunchKernelGGL(mx_quant_rows_kernel, dim3((unsigned)((total + per - 1) / per) + (P.tiles ? 1u : 0u)), dim3(256), 0,
                       stream, P);
    return hipGetLastError();
}

hipError_t launch_mx_quant_tiles(const uint16_t* x, int64_t n_mats, int32_t rows, int32_t cols, int64_t ld, uint8_t* codes,
                                 uint8_t* scales, bool up, hipStream_t stream) {
    const int32_t row_tiles = (rows + 15) / 16, chunks = (cols + 127) / 128, quads = (chunks + 3) / 4;
    const int64_t units = n_mats * row_tiles * quads;
    hipLaunchKernelGGL(mx_quant_tiles_kernel, dim3((unsigned)((units + 3) / 4)), dim3(256), 0, stream, x, units, rows, cols,
                       ld, row_tiles, chunks, quads, codes, scales, up ? 1 : 0);
    return hipGetLastError();
}

hipError_t launch_mx_dequant(MxDequantParams P, hipStream_t stream) {
    P.groups = P.cols / 8;
    P.inv_groups = 1.0 / P.groups;
    P.chunks = (P.cols + 127) / 128;
    P.quads = (P.chunks + 3) / 4;
    P.row_tiles = (P.mat_rows + 15) / 16;
    const uint64_t per = 256 * kMxUnroll, total = (uint64_t)P.groups * P.rows;
    hipLaunchKernelGGL(mx_dequant_kernel, dim3((unsigned)((total + per - 1) / per)), dim3(256), 0, stream, P);
    return hipGetLastError();
}

}  // namespace nvfp4
