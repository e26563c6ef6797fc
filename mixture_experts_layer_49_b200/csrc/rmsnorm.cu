// rmsnorm.cu -- RMS norm of the layer's input with the residual's addition
// and an 8-bit output, forward and backward.
//
// A block adds its attention output x to the residual stream r and hands the
// normalised sum to the MoE layer:
//   z = x + r                           (fp32, not rounded before the norm)
//   v = z * rsqrt(mean(z^2) + eps) * w  (fp32)
//   h = T(z), y = T(v)                  (one rounding each; T bf16 or fp32)
//   per 128 values of a row: a = max(max |v|, 2^-100),
//   scale = a / 448, code = e4m3(v * (448 / a)), nearest even
// The codes come from the fp32 v, not from the rounded y, so an 8-bit value
// is rounded once; the floor 2^-100 keeps 448 / a finite for a block of zeros
// or subnormal values (codes 0, a normal scale).
//
// Backward, for h as stored, dy and the gradient dres that reaches h from the
// residual stream (both x and r get the returned dh):
//   n = h * rstd, u = w * dy
//   dh = dres + rstd * (u - n * mean(u * n)),   dw = sum_t dy * n
//
// Bound by memory: forward 2 reads and 2 writes of T plus a byte and 1/32 for
// the codes and scales per element, backward 3 reads and 1 write.  A row lives
// in the registers of one thread group (8 elements per 16-byte load and
// thread), so every element is read once; a block of 128 is 16 neighbouring
// threads.  Measured, forward with the codes, on the device in a graph and as one
// Python call among others: 8192 x 7168 bf16 82 and 87 us (floor 81), 3001 x 1160
// fp32 11.3 and 12.9 (8.5), 4 x 2048 2.2 and 10.7.
#include <cuda_fp8.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.cuh"

namespace moe {

namespace {

constexpr int kPartRows = 1184;                // rows of partial dw sums at d >= 512: 8 per SM

template <typename T>
struct Vec8;                                   // eight elements of a row as loaded

template <>
struct Vec8<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { u = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void clear() { u = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(float *f) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float *f) {
        uint4 o;
        __nv_bfloat162 *b = reinterpret_cast<__nv_bfloat162 *>(&o);
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        *reinterpret_cast<uint4 *>(p) = o;
    }
};

template <>
struct Vec8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = *reinterpret_cast<const float4 *>(p);
        b = *reinterpret_cast<const float4 *>(p + 4);
    }
    __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float *f) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    static __device__ __forceinline__ void store(float *p, const float *f) {
        *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4 *>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
    }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over the blockDim.x threads of this row (blockDim.x a multiple of 32);
// the warps' partials are added in warp order.  Every thread of the block
// calls it when a row has more than one warp.
__device__ __forceinline__ float row_sum(float v, float (*part)[32]) {
    v = warp_sum(v);
    const int nw = blockDim.x >> 5;
    if (nw == 1) return v;
    if ((threadIdx.x & 31) == 0) part[threadIdx.y][threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < nw; ++i) s += part[threadIdx.y][i];
    __syncthreads();
    return s;
}

// Eight codes of v * inv in two words.
__device__ __forceinline__ uint2 codes8(const float *v, float inv) {
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(
            make_float2(__fmul_rn(v[4 * h], inv), __fmul_rn(v[4 * h + 1], inv)), __NV_SATFINITE, __NV_E4M3);
        const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(
            make_float2(__fmul_rn(v[4 * h + 2], inv), __fmul_rn(v[4 * h + 3], inv)), __NV_SATFINITE, __NV_E4M3);
        w[h] = (uint32_t)lo | ((uint32_t)hi << 16);
    }
    return make_uint2(w[0], w[1]);
}

// blockDim = (threads per row, rows per block); thread x holds vectors
// x, x + blockDim.x, ... of its row.
template <typename T, int VPT, int MAXT>
__global__ void __launch_bounds__(MAXT) rmsnorm_kernel(RmsNormArgs a) {
    pdl_wait_then_release();
    __shared__ float part[8][32];
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = row < a.rows;
    const int nvec = a.d >> 3;
    const T *x = static_cast<const T *>(a.x) + row * a.d;
    const T *r = a.residual ? static_cast<const T *>(a.residual) + row * a.d : nullptr;

    Vec8<T> xv[VPT], rv[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (live && v < nvec) xv[i].load(x + v * 8); else xv[i].clear();
        if (live && r && v < nvec) rv[i].load(r + v * 8); else rv[i].clear();
    }
    float z[VPT][8], ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        float rf[8];
        xv[i].get(z[i]);
        rv[i].get(rf);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (r) z[i][j] += rf[j];              // without a residual -0 stays -0
            ss = fmaf(z[i][j], z[i][j], ss);
        }
    }
    ss = row_sum(ss, part);
    const float rstd = __frsqrt_rn(__fadd_rn(__fdiv_rn(ss, (float)a.d), a.eps));
    if (a.codes == nullptr && !live) return;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        const bool in = live && v < nvec;
        if (in && a.h) Vec8<T>::store(static_cast<T *>(a.h) + row * a.d + v * 8, z[i]);
        float o[8], amax = 0.f;
        if (in) {
            const float4 w0 = __ldg(reinterpret_cast<const float4 *>(a.weight) + 2 * v);
            const float4 w1 = __ldg(reinterpret_cast<const float4 *>(a.weight) + 2 * v + 1);
            const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                o[j] = z[i][j] * rstd * w[j];
                amax = fmaxf(amax, fabsf(o[j]));
            }
            if (a.y) Vec8<T>::store(static_cast<T *>(a.y) + row * a.d + v * 8, o);
        }
        if (a.codes) {                            // uniform: every lane of the warp takes part
#pragma unroll
            for (int s = 8; s > 0; s >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, s));
            amax = fmaxf(amax, 0x1p-100f);
            if (in) {
                *reinterpret_cast<uint2 *>(a.codes + row * a.d + v * 8) = codes8(o, __fdiv_rn(448.f, amax));
                if ((v & 15) == 0)
                    *reinterpret_cast<float *>(reinterpret_cast<char *>(a.scale) + row * a.ld_scale + (v >> 4) * 4) =
                        __fdiv_rn(amax, 448.f);
            }
        }
    }
}

// blockDim = (threads per row, rows at a time), rows of more than one warp one at a
// time; part p of gridDim.x * blockDim.y takes rows p, p + parts, ...; its share of
// dw stays in registers and ends in part[p].  The rows' h, dy and dres come through
// shared memory by cp.async, STAGES - 1 rows ahead: each thread copies and reads
// its own vectors, so nothing but its own wait orders them.  16384 x 2048 bf16: 51
// us against a floor of 41 (rows loaded as needed 76, one row ahead in registers
// 61); 8192 x 7168 bf16 85 of 72, 8192 x 4096 fp32 85 of 82.  STAGES 0: rows too
// wide for 200 KB of stages, loaded as they are needed.  Rows above 8192 have up to
// 1024 threads, whose registers spill: 4096 x 16384 bf16 261 of 82.
template <typename T, int VPT, int MAXT, int STAGES>
__global__ void __launch_bounds__(MAXT) rmsnorm_bwd_kernel(RmsNormBwdArgs a) {
    pdl_wait_then_release();
    extern __shared__ __align__(16) uint8_t stage_mem[];       // [STAGES][h, dy, dres][VPT * blockDim.x] vectors
    __shared__ float2 red[2][32];
    constexpr int VB = 8 * sizeof(T);             // bytes of a vector
    const int nvec = a.d >> 3, nw = blockDim.x >> 5;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t part = (int64_t)blockIdx.x * blockDim.y + threadIdx.y, parts = (int64_t)gridDim.x * blockDim.y;
    const float inv_d = __fdiv_rn(1.f, (float)a.d);
    float dw[VPT][8], w[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = min((int)(threadIdx.x + i * blockDim.x), nvec - 1);        // past the row: unused
        Vec8<float> wv;
        wv.load(a.weight + v * 8);
        wv.get(w[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
    }
    auto src = [&](int which, int64_t row, int i) {
        const void *base = which == 0 ? a.h : which == 1 ? a.dy : a.dres;
        return static_cast<const T *>(base) + row * a.d + (threadIdx.x + i * blockDim.x) * 8;
    };
    auto slot = [&](int stage, int which, int i) {
        return stage_mem + (size_t)((((stage * 3 + which) * VPT + i) * blockDim.y + threadIdx.y) * blockDim.x + threadIdx.x) * VB;
    };
    auto fetch = [&](int stage, int64_t row) {    // this thread's vectors of a row, one group
        if (row < a.rows)
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if ((int)(threadIdx.x + i * blockDim.x) < nvec)
#pragma unroll
                    for (int q = 0; q < 3; ++q)
                        if (q < 2 || a.dres)
#pragma unroll
                            for (int c = 0; c < VB; c += 16)
                                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(slot(stage, q, i)) + c),
                                             "l"(reinterpret_cast<const char *>(src(q, row, i)) + c) : "memory");
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto vec = [&](int stage, int which, int64_t row, int i) {
        Vec8<T> v;
        v.load(STAGES ? reinterpret_cast<const T *>(slot(stage, which, i)) : src(which, row, i));
        return v;
    };
    if (STAGES)
        for (int s = 0; s < STAGES - 1; ++s) fetch(s, part + s * parts);
    int flip = 0, stage = 0;
    for (int64_t row = part; row < a.rows; row += parts, flip ^= 1) {
        if (STAGES) {
            // the slot read last round takes the row STAGES - 1 ahead (dh may be dy
            // or dres: other rows of them)
            fetch(stage == 0 ? STAGES - 1 : stage - 1, row + (STAGES - 1) * parts);
            asm volatile("cp.async.wait_group %0;" ::"n"(STAGES ? STAGES - 1 : 0) : "memory");
        }
        float ss = 0.f, uh = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if ((int)(threadIdx.x + i * blockDim.x) >= nvec) continue;
            float hf[8], gf[8];
            vec(stage, 0, row, i).get(hf);
            vec(stage, 1, row, i).get(gf);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                ss = fmaf(hf[j], hf[j], ss);
                uh = fmaf(gf[j] * w[i][j], hf[j], uh);
            }
        }
        ss = warp_sum(ss);
        uh = warp_sum(uh);
        if (nw > 1) {                             // two buffers: one barrier per row
            if (lane == 0) red[flip][warp] = make_float2(ss, uh);
            __syncthreads();
            ss = 0.f;
            uh = 0.f;
            for (int i = 0; i < nw; ++i) { ss += red[flip][i].x; uh += red[flip][i].y; }
        }
        const float rstd = __frsqrt_rn(__fadd_rn(__fdiv_rn(ss, (float)a.d), a.eps));
        const float m = uh * rstd * inv_d;        // mean(u * n)
        T *dh = static_cast<T *>(a.dh) + row * a.d;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = threadIdx.x + i * blockDim.x;
            if (v >= nvec) continue;
            float hf[8], gf[8], o[8];
            vec(stage, 0, row, i).get(hf);
            vec(stage, 1, row, i).get(gf);
            if (a.dres) {
                vec(stage, 2, row, i).get(o);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float n = hf[j] * rstd;
                dw[i][j] = fmaf(gf[j], n, dw[i][j]);
                o[j] += rstd * (gf[j] * w[i][j] - n * m);
            }
            Vec8<T>::store(dh + v * 8, o);
        }
        if (STAGES) stage = stage + 1 == STAGES ? 0 : stage + 1;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v < nvec) Vec8<float>::store(a.part + part * a.d + v * 8, dw[i]);
    }
}

// dw[c] = the sum of part[.][c]: 32 columns per block, 32 row groups of the parts
// in order, the groups then in order.
__global__ void __launch_bounds__(1024) rmsnorm_dw_kernel(const float *part, int nparts, int d, float *dw) {
    pdl_wait_then_release();
    __shared__ float red[32][33];
    const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < d) {
        const int lo = g * nparts / 32, hi = (g + 1) * nparts / 32;
#pragma unroll 8
        for (int p = lo; p < hi; ++p) s += part[(int64_t)p * d + c];
    }
    red[g][lane] = s;
    __syncthreads();
    if (g == 0 && c < d) {
        float t = red[0][lane];
#pragma unroll
        for (int i = 1; i < 32; ++i) t += red[i][lane];
        dw[c] = t;
    }
}

// Vectors per thread and threads per row.
void row_shape(int d, int *vpt, int *threads) {
    const int nvec = d / 8;
    *vpt = nvec <= 256 ? 1 : (nvec <= 512 ? 2 : 4);
    *threads = (((nvec + *vpt - 1) / *vpt) + 31) / 32 * 32;
}

template <typename T>
cudaError_t launch_fwd(const RmsNormArgs &a, cudaStream_t st) {
    int vpt, tx;
    row_shape(a.d, &vpt, &tx);
    const int ty = tx >= 128 ? 1 : 128 / tx;      // narrow rows share a block (tx 32, 64, 96: 4, 2, 1 rows)
    const dim3 grid((unsigned)((a.rows + ty - 1) / ty)), block(tx, ty);
    if (vpt == 1) return launch_kernel(rmsnorm_kernel<T, 1, 256>, grid, block, 0, st, a.pdl, a);
    if (vpt == 2) return launch_kernel(rmsnorm_kernel<T, 2, 256>, grid, block, 0, st, a.pdl, a);
    if (tx <= 256) return launch_kernel(rmsnorm_kernel<T, 4, 256>, grid, block, 0, st, a.pdl, a);
    return launch_kernel(rmsnorm_kernel<T, 4, 1024>, grid, block, 0, st, a.pdl, a);
}

template <typename T, int VPT, int MAXT, int STAGES>
cudaError_t launch_bwd_stages(const RmsNormBwdArgs &a, int tx, int *nparts, cudaStream_t st) {
    const int ty = tx == 32 ? 4 : 1;
    const size_t smem = (size_t)STAGES * 3 * VPT * tx * ty * 8 * sizeof(T);
    // as many blocks as are resident: 1024 threads and 200 KB of stages per SM
    int per_sm = std::max(1024 / (tx * ty), 1);
    if (STAGES) per_sm = (int)std::min<size_t>(per_sm, 200 * 1024 / smem);
    const int blocks = std::max(1, std::min(*nparts / ty, per_sm * a.num_sms));
    if (smem > 40 * 1024) {                       // with the static part above the default of 48 KB
        cudaError_t e = cudaFuncSetAttribute(rmsnorm_bwd_kernel<T, VPT, MAXT, STAGES>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    *nparts = blocks * ty;
    return launch_kernel(rmsnorm_bwd_kernel<T, VPT, MAXT, STAGES>, dim3(blocks), dim3(tx, ty), smem, st, a.pdl, a);
}

// Three stages where two blocks of them fit an SM, else two, else none.
template <typename T, int VPT, int MAXT>
cudaError_t launch_bwd_rows(const RmsNormBwdArgs &a, int tx, int *nparts, cudaStream_t st) {
    const size_t stage = (size_t)3 * VPT * tx * 8 * sizeof(T);
    if constexpr (MAXT <= 256)
        if (6 * stage <= 200 * 1024) return launch_bwd_stages<T, VPT, MAXT, 3>(a, tx, nparts, st);
    if (2 * stage <= 200 * 1024) return launch_bwd_stages<T, VPT, MAXT, 2>(a, tx, nparts, st);
    return launch_bwd_stages<T, VPT, MAXT, 0>(a, tx, nparts, st);
}

template <typename T>
cudaError_t launch_bwd(const RmsNormBwdArgs &a, int *nparts, cudaStream_t st) {
    const int nvec = a.d / 8;
    const int vpt = nvec <= 64 ? 1 : (nvec <= 512 ? 2 : 4);
    const int tx = ((nvec + vpt - 1) / vpt + 31) / 32 * 32;
    if (vpt == 1) return launch_bwd_rows<T, 1, 128>(a, tx, nparts, st);
    if (tx <= 128) return launch_bwd_rows<T, 2, 128>(a, tx, nparts, st);
    if (vpt == 2) return launch_bwd_rows<T, 2, 256>(a, tx, nparts, st);
    if (tx <= 256) return launch_bwd_rows<T, 4, 256>(a, tx, nparts, st);
    return launch_bwd_rows<T, 4, 1024>(a, tx, nparts, st);
}

}  // namespace

int64_t rmsnorm_bwd_parts(int64_t rows, int d) {
    const int64_t most = d >= 512 ? kPartRows : kPartRows * 512 / (d > 64 ? d : 64);
    const int64_t n = rows < most ? rows : most;
    return n == 0 ? 0 : (n + 3) / 4 * 4;          // narrow rows: four at a time, the last maybe beyond
}

cudaError_t launch_rmsnorm(const RmsNormArgs &a, bool bf16, cudaStream_t st) {
    if (a.rows == 0) return cudaSuccess;
    return bf16 ? launch_fwd<__nv_bfloat16>(a, st) : launch_fwd<float>(a, st);
}

cudaError_t launch_rmsnorm_bwd(const RmsNormBwdArgs &a, bool bf16, cudaStream_t st) {
    int nparts = (int)rmsnorm_bwd_parts(a.rows, a.d);
    cudaError_t e = cudaSuccess;
    if (nparts > 0) e = bf16 ? launch_bwd<__nv_bfloat16>(a, &nparts, st) : launch_bwd<float>(a, &nparts, st);
    if (e != cudaSuccess) return e;
    return launch_kernel(rmsnorm_dw_kernel, dim3((unsigned)((a.d + 31) / 32)), dim3(1024), 0, st, nparts > 0 || a.pdl,
                         static_cast<const float *>(a.part), nparts, a.d, a.dweight);
}

}  // namespace moe
