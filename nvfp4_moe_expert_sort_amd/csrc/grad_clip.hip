// grad_clip.hip -- the global norm of a list of gradient tensors, and their
// clipping by it.
//
//   norm = sqrt(sum over all elements g^2);  out = g * (norm > max ? max / norm : 1)
//
// Two launches over a plan of chunks (nvfp4moe_grad_plan), both bound by HBM:
// every element is read twice (once for the norm, once to scale it) and
// written once.  Squares are formed and summed in FP64: vector FP64 runs at
// the FP32 rate here, two instructions an element hide under the reads, and no
// FP32 value overflows or loses its square.  A workgroup's partial sum and
// their total are taken in one fixed order, so the norm has the same bits in
// every run.  The second pass walks the plan backwards: what the first read
// last is still in the 256 MB last-level cache.
//
// 604 M FP32 gradients (2.4 GB): 422 us for the norm (5.7 TB/s), 919 us to scale
// them into other buffers (5.25 TB/s); a plain copy moves 5.2-5.5.  61 tensors
// of up to 65537 elements: 3.2 + 4.0 us.
#include "nvfp4_device.h"
#include "nvfp4_kernels.h"

namespace nvfp4 {

namespace {

typedef double f64x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ double block_sum(double v) {
    __shared__ double part[4];
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    return (part[0] + part[1]) + (part[2] + part[3]);
}

__device__ __forceinline__ float grad_at(const GradChunk& c, uint32_t i) {
    return c.bf16 ? bf16_to_f32(((const uint16_t*)c.in)[i]) : ((const float*)c.in)[i];
}

// Sum of the squares of 16 bytes.
__device__ __forceinline__ void add_squares(u32x4 v, bool bf16, double (&s)[4]) {
#pragma unroll
    for (int j = 0; j < 4; j++) {
        if (bf16) {
            const double a = (double)__uint_as_float(v[j] << 16), b = (double)__uint_as_float(v[j] & 0xFFFF0000u);
            s[j] = __builtin_fma(a, a, s[j]);
            s[j] = __builtin_fma(b, b, s[j]);
        } else {
            const double a = (double)__uint_as_float(v[j]);
            s[j] = __builtin_fma(a, a, s[j]);
        }
    }
}

}  // namespace

__global__ void __launch_bounds__(256) grad_norm_kernel(const GradChunk* __restrict__ plan, int64_t n_chunks,
                                                        double* __restrict__ partial) {
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    for (int64_t k = blockIdx.x; k < n_chunks; k += gridDim.x) {
        const GradChunk c = plan[k];
        const uint32_t per = c.bf16 ? 8 : 4, body = (c.n - c.head) / per, tail = c.head + body * per;
        if (threadIdx.x < c.head) {
            const double a = (double)grad_at(c, threadIdx.x);
            s[0] = __builtin_fma(a, a, s[0]);
        }
        const u32x4* v = reinterpret_cast<const u32x4*>((const uint8_t*)c.in + (size_t)c.head * (c.bf16 ? 2 : 4));
        uint32_t i = threadIdx.x;
        for (; i + 3 * 256 < body; i += 4 * 256) {
            u32x4 q[4];
#pragma unroll
            for (int j = 0; j < 4; j++) q[j] = v[i + j * 256];
#pragma unroll
            for (int j = 0; j < 4; j++) add_squares(q[j], c.bf16, s);
        }
        for (; i < body; i += 256) add_squares(v[i], c.bf16, s);
        if (tail + threadIdx.x < c.n) {
            const double a = (double)grad_at(c, tail + threadIdx.x);
            s[1] = __builtin_fma(a, a, s[1]);
        }
    }
    const double total = block_sum((s[0] + s[1]) + (s[2] + s[3]));
    if (threadIdx.x == 0) partial[blockIdx.x] = total;
}

__global__ void __launch_bounds__(256) grad_scale_kernel(const GradChunk* __restrict__ plan, int64_t n_chunks,
                                                         const double* __restrict__ partial, int n_partial,
                                                         double max_norm, double* __restrict__ norm_out) {
    double s = 0.0;
    for (int i = threadIdx.x; i < n_partial; i += 256) s += partial[i];
    const double norm = __builtin_sqrt(block_sum(s));
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm;
    // An Inf or NaN among the gradients leaves them as they are, to the bit: a
    // conversion would make signaling NaNs quiet.
    const double coef = norm > max_norm && norm < __builtin_inf() ? max_norm / norm : 1.0;
    const bool same = coef == 1.0;
    for (int64_t k0 = blockIdx.x; k0 < n_chunks; k0 += gridDim.x) {
        const GradChunk c = plan[n_chunks - 1 - k0];
        if (same && c.in == c.out) continue;
        const uint32_t per = c.bf16 ? 8 : 4, body = (c.n - c.head) / per, tail = c.head + body * per;
        auto one = [&](uint32_t i) {
            const float g = (float)((double)grad_at(c, i) * coef);
            if (c.bf16)
                ((uint16_t*)c.out)[i] = same ? ((const uint16_t*)c.in)[i] : (uint16_t)bf16_hw(g);
            else
                ((uint32_t*)c.out)[i] = same ? ((const uint32_t*)c.in)[i] : __float_as_uint(g);
        };
        if (threadIdx.x < c.head) one(threadIdx.x);
        if (c.out_vec) {
            const size_t skip = (size_t)c.head * (c.bf16 ? 2 : 4);
            const u32x4* v = reinterpret_cast<const u32x4*>((const uint8_t*)c.in + skip);
            u32x4* o = reinterpret_cast<u32x4*>((uint8_t*)c.out + skip);
            auto scale = [&](u32x4 q) {
                if (same) return q;
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    if (c.bf16) {
                        const float a = (float)((double)__uint_as_float(q[j] << 16) * coef);
                        const float b = (float)((double)__uint_as_float(q[j] & 0xFFFF0000u) * coef);
                        q[j] = bf16_hw(a) | (bf16_hw(b) << 16);
                    } else {
                        q[j] = __float_as_uint((float)((double)__uint_as_float(q[j]) * coef));
                    }
                }
                return q;
            };
            uint32_t i = threadIdx.x;
            for (; i + 3 * 256 < body; i += 4 * 256) {
                u32x4 q[4];
#pragma unroll
                for (int j = 0; j < 4; j++) q[j] = v[i + j * 256];
#pragma unroll
                for (int j = 0; j < 4; j++) o[i + j * 256] = scale(q[j]);
            }
            for (; i < body; i += 256) o[i] = scale(v[i]);
        } else {
            for (uint32_t i = c.head + threadIdx.x; i < tail; i += 256) one(i);
        }
        if (tail + threadIdx.x < c.n) one(tail + threadIdx.x);
    }
}

hipError_t launch_clip_grad_norm(const GradChunk* plan, int64_t n_chunks, double max_norm, double* partial, double* norm_out,
                                 hipStream_t stream) {
    const unsigned blocks = (unsigned)(n_chunks < kGradBlocks ? (n_chunks > 0 ? n_chunks : 1) : kGradBlocks);
    hipLaunchKernelGGL(grad_norm_kernel, dim3(blocks), dim3(256), 0, stream, plan, n_chunks, partial);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(grad_scale_kernel, dim3(blocks), dim3(256), 0, stream, plan, n_chunks, partial, (int)blocks, max_norm,
                       norm_out);
    return hipGetLastError();
}

}  // namespace nvfp4
