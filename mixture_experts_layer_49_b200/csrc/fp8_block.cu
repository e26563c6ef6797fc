// fp8_block.cu -- the data movement around the block-scaled e4m3 experts
// (fp8_block_sm100.cu): 1 x 128 quantization of bf16 rows and the gather of
// the packed rows' scales.
//
// For each run of 128 values of a row (the last may be shorter):
//   a = max(max |v|, 2^-100), scale = a / 448, code = e4m3(v * (448 / a))
// with correctly rounded fp32 quotient and product and nearest-even
// conversion; the floor keeps 448 / a finite for blocks of zeros.  Bound by
// memory: 2 bytes in, 1 + 1/32 bytes out per value; 16 threads hold a block
// (eight values each), so a warp reads 512 contiguous bytes.
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads) quant_block_kernel(QuantBlockArgs a) {
    pdl_wait_then_release();
    const int nb = (a.cols + 127) >> 7;
    const int64_t total = a.rows * nb * 16;                   // a multiple of 16: half warps stay whole
    const int64_t step = (int64_t)gridDim.x * kThreads;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; (i & ~31ll) < total; i += step) {
        const int64_t blk = i >> 4;
        const int64_t row = blk / nb;
        const int b = (int)(blk - row * nb);
        const int c = b * 128 + (int)(i & 15) * 8;
        const bool in = i < total && c < a.cols;
        float f[8], amax = 0.f;
        if (in) {
            const uint4 u = *reinterpret_cast<const uint4 *>(a.in + row * a.ld_in + c);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f[2 * j] = __uint_as_float(w[j] << 16);
                f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(f[j]));
        }
#pragma unroll
        for (int s = 8; s > 0; s >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, s));
        amax = fmaxf(amax, 0x1p-100f);
        if (!in) continue;
        const float inv = __fdiv_rn(448.f, amax);
        uint32_t o[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(
                make_float2(__fmul_rn(f[4 * h], inv), __fmul_rn(f[4 * h + 1], inv)), __NV_SATFINITE, __NV_E4M3);
            const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(
                make_float2(__fmul_rn(f[4 * h + 2], inv), __fmul_rn(f[4 * h + 3], inv)), __NV_SATFINITE, __NV_E4M3);
            o[h] = (uint32_t)lo | ((uint32_t)hi << 16);
        }
        *reinterpret_cast<uint2 *>(a.out + row * a.ld_out + c) = make_uint2(o[0], o[1]);
        if ((i & 15) == 0)
            *reinterpret_cast<float *>(reinterpret_cast<char *>(a.scale) + row * a.ld_scale + 4 * b) =
                __fdiv_rn(amax, 448.f);
    }
}

// dst[r][0 .. nb) = src[row_token[r]][0 .. nb) for r < *count; one half warp
// per row.
__global__ void __launch_bounds__(kThreads) gather_scales_kernel(const float *src, int64_t ld_src, float *dst,
                                                                 int64_t ld_dst, int nb, const int32_t *row_token,
                                                                 const int32_t *count, int64_t max_rows) {
    pdl_wait_then_release();
    int64_t n = *count;
    n = n < 0 ? 0 : (n < max_rows ? n : max_rows);
    const int lane = threadIdx.x & 15;
    const int64_t step = (int64_t)gridDim.x * (kThreads / 16);
    for (int64_t r = (int64_t)blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4); r < n; r += step) {
        const float *s = reinterpret_cast<const float *>(reinterpret_cast<const char *>(src) + row_token[r] * ld_src);
        float *d = reinterpret_cast<float *>(reinterpret_cast<char *>(dst) + r * ld_dst);
        for (int b = lane; b < nb; b += 16) d[b] = s[b];
    }
}

}  // namespace

cudaError_t launch_quant_block(const QuantBlockArgs &a, cudaStream_t st) {
    if (a.rows <= 0 || a.cols <= 0) return cudaSuccess;
    const int64_t total = a.rows * ((a.cols + 127) / 128) * 16;
    const int64_t want = (total + kThreads - 1) / kThreads, cap = (int64_t)a.num_sms * 32;
    return launch_kernel(quant_block_kernel, dim3((unsigned)(want < cap ? want : cap)), dim3(kThreads), 0, st, a.pdl, a);
}

cudaError_t launch_gather_scales(const float *src, int64_t ld_src, float *dst, int64_t ld_dst, int nb,
                                 const int32_t *row_token, const int32_t *count, int64_t max_rows, int num_sms,
                                 cudaStream_t st) {
    if (max_rows <= 0) return cudaSuccess;
    const int64_t want = (max_rows + kThreads / 16 - 1) / (kThreads / 16), cap = (int64_t)num_sms * 8;
    return launch_kernel(gather_scales_kernel, dim3((unsigned)(want < cap ? want : cap)), dim3(kThreads), 0, st, true,
                         src, ld_src, dst, ld_dst, nb, row_token, count, max_rows);
}

}  // namespace moe
