// fp8_block_decode.cu -- the block-scaled e4m3 experts for one or two tokens.
//
// With at most a handful of rows per expert the products only stream the weights
// of the hit experts once (37.7 MB for one token of the Qwen3 shape: 5.8 us of
// HBM), and the tile kernel of fp8_block_sm100.cu has too few 256-column tiles to
// keep the memory busy (48 and 64 tiles for that token).  Here a block of eight
// warps takes 16, 32, 64 or 128 output columns of one expert and
// splits K over its warps, so the same token has 192 and 256 blocks.
//
// Each warp runs mma.sync.m16n8k32 on e4m3: 16 weight rows as A, up to eight
// activation rows as B, fp32 sums -- the rate does not matter here, and operands
// come straight from global memory in fragment order (tcgen05 wants them in
// shared memory).  Within a block of 128 the order of K is free: lane q of a row's
// four takes the 16-byte pieces q and q + 4, so every load is 16 bytes wide and
// the fragments of A and B agree.  The scaled sums of a warp's K blocks and then
// of the warps are added in a fixed order.
//
// The first product leaves the hidden rows in fp32, because a block of 128 hidden
// values spans several blocks here; the second quantizes them as it loads them
// (the same rule: a = max(max |h|, 2^-100), code = e4m3(h * (448 / a))).
//
// Measured for the whole FFN with other experts in every call: one token of the
// Qwen3 shape 15.1 us (26.9 with the tile kernel), of the Mixtral shape 81 us (110).
#include <cuda_fp8.h>

#include "common.cuh"
#include "fp8_block.cuh"
#include "kernels.cuh"

namespace moe {

namespace {

enum { FB_SWIGLU = 0, FB_GELU = 1, FB_DOWN = 2 };
constexpr int kThreads = 256;
constexpr int kWarps = 8;
constexpr int kRows = 8;                       // activation rows of one pass over the weights

struct Params {
    const int32_t *offsets;
    int32_t *status;
    int E, T, tiles_r, tiles_s, active_max;    // tiles per expert / of the shared expert; hit experts at most
    int64_t routed_rows;
    int K_routed, K_shared, N_routed, N_shared;
    const uint8_t *x, *x_s;                    // codes of A's rows, K bytes apart (first product)
    const float *sa, *sa_s;
    int64_t ld_sa, ld_sa_s;                    // bytes
    const float *h;                            // fp32 hidden rows, ldh apart (second product)
    int64_t ldh;
    int64_t shared_row;                        // first shared row of h and of the output
    const uint8_t *w, *w2, *w_s, *w2_s;
    const float *sw, *sw2, *sw_s, *sw2_s;
    int64_t ld_sw;                             // bytes
    const float *bias, *row_gate;
    float *out_h;                              // fp32 hidden rows (first product)
    __nv_bfloat16 *out;                        // y rows (second product)
    int64_t ldo;
};

__device__ __forceinline__ void mma_e4m3_16x8x32(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                 uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 load16(const uint8_t *p, bool in) {
    return in ? __ldg(reinterpret_cast<const uint4 *>(p)) : make_uint4(0u, 0u, 0u, 0u);
}

// c = the products of one block of 128: lo / hi the pieces of rows g and g + 8.
__device__ __forceinline__ void block_product(float (&c)[4], const uint4 (&lo)[2], const uint4 (&hi)[2], const uint4 (&b)[2]) {
    c[0] = c[1] = c[2] = c[3] = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        mma_e4m3_16x8x32(c, lo[i].x, hi[i].x, lo[i].y, hi[i].y, b[i].x, b[i].y);
        mma_e4m3_16x8x32(c, lo[i].z, hi[i].z, lo[i].w, hi[i].w, b[i].z, b[i].w);
    }
}

__device__ __forceinline__ uint32_t codes4(const float *v, float inv) {
    const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(v[0], inv), __fmul_rn(v[1], inv)),
                                                             __NV_SATFINITE, __NV_E4M3);
    const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(v[2], inv), __fmul_rn(v[3], inv)),
                                                             __NV_SATFINITE, __NV_E4M3);
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

// WN: 16-column tiles of a block; its warps split K over kWarps / WN of them.
template <int MODE, int WN>
__global__ void __launch_bounds__(kThreads, 2) fp8_block_decode(const __grid_constant__ Params p) {
    // The second product reads its weights, which no kernel writes, and offsets,
    // complete before the first product began, ahead of its wait for the hidden rows.
    if (MODE != FB_DOWN) pdl_wait_then_release();
    else asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int WK = kWarps / WN, NM = MODE == FB_SWIGLU ? 2 : 1;
    __shared__ int found[3];
    __shared__ float red[NM][WK][WN * 16][kRows + 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, q = lane & 3;
    const bool sh = (int)blockIdx.x >= p.active_max * p.tiles_r;
    const int tile = sh ? blockIdx.x - p.active_max * p.tiles_r : blockIdx.x % p.tiles_r;
    int e = 0, row0 = 0, n = p.T;
    if (!sh) {                                 // the a-th expert that has rows
        const int a = blockIdx.x / p.tiles_r;
        if (warp == 0) {
            int seen = 0, fe = -1, fr = 0, fn = 0;
            for (int e0 = 0; e0 < p.E && fe < 0; e0 += 32) {
                int64_t r0 = 0, rows = 0;
                if (e0 + lane < p.E) {
                    r0 = p.offsets[e0 + lane];
                    rows = (int64_t)p.offsets[e0 + lane + 1] - r0;
                    if (r0 < 0 || rows < 0 || r0 + rows > p.routed_rows) rows = 0;      // recorded below
                }
                const uint32_t hit = __ballot_sync(0xffffffffu, rows > 0);
                const bool mine = rows > 0 && seen + __popc(hit & ((1u << lane) - 1u)) == a;
                const uint32_t who = __ballot_sync(0xffffffffu, mine);
                if (who) {
                    const int l = __ffs(who) - 1;
                    fe = e0 + l;
                    fr = __shfl_sync(0xffffffffu, (int)r0, l);
                    fn = __shfl_sync(0xffffffffu, (int)rows, l);
                }
                seen += __popc(hit);
            }
            if (lane == 0) { found[0] = fe; found[1] = fr; found[2] = fn; }
        } else if (MODE == FB_DOWN && blockIdx.x == 0 && warp == 1) {
            // the search ends at its expert: one warp looks at all groups, while the second
            // product waits for the first (0.3 us of one token; in the first product 0.5)
            int wrong = -1;
            for (int i = lane; i < p.E; i += 32) {
                const int64_t r0 = p.offsets[i], r1 = p.offsets[i + 1];
                if (r0 < 0 || r1 < r0 || r1 > p.routed_rows) wrong = i;
            }
            if (wrong >= 0) record_error(p.status, MOE_ERR_DEVICE_BOUNDS, wrong);
        }
        __syncthreads();
        e = found[0];
        row0 = found[1];
        n = found[2];
        if (e < 0) {
            if (MODE == FB_DOWN) asm volatile("griddepcontrol.wait;" ::: "memory");    // its end tells of both products'
            return;
        }
    }
    const int K = sh ? p.K_shared : p.K_routed, N = sh ? p.N_shared : p.N_routed;
    const int nk = (K + 127) / 128;
    const int wn = warp % WN, wk = warp / WN;
    const int col0 = tile * WN * 16, wcol = col0 + wn * 16;
    const int64_t nb = (N + 127) / 128;
    const uint8_t *w[NM];
    const float *sw[NM];
#pragma unroll
    for (int m = 0; m < NM; ++m) {
        const uint8_t *base = m ? (sh ? p.w2_s : p.w2) : (sh ? p.w_s : p.w);
        const float *sbase = m ? (sh ? p.sw2_s : p.sw2) : (sh ? p.sw_s : p.sw);
        w[m] = base + ((int64_t)e * N + wcol + g) * K + q * 16;
        sw[m] = reinterpret_cast<const float *>(reinterpret_cast<const char *>(sbase) + (e * nb + (wcol >> 7)) * p.ld_sw);
    }
    const bool wlive = wcol < N;               // N is a multiple of 16: whole tiles of 16
    for (int r0 = 0; r0 < n; r0 += kRows) {
        const int rows = min(kRows, n - r0);
        const bool live = g < rows;
        float acc[NM][4];
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][i] = 0.f;
        const int64_t arow = (int64_t)row0 + r0 + g;
        // two K blocks at a time: all of their weights are asked for before the
        // first product waits
        for (int kb0 = wk; wlive && kb0 < nk; kb0 += 2 * WK) {       // uniform over the warp
            uint4 lo[2][NM][2], hi[2][NM][2];
            float s[2][NM];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int m = 0; m < NM; ++m) {
                    const int kb = kb0 + u * WK;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int k = kb * 128 + i * 64;
                        const bool in = k + q * 16 < K;
                        lo[u][m][i] = load16(w[m] + k, in);
                        hi[u][m][i] = load16(w[m] + (int64_t)8 * K + k, in);
                    }
                    s[u][m] = kb < nk ? __ldg(sw[m] + kb) : 0.f;
                }
            if (MODE == FB_DOWN) asm volatile("griddepcontrol.wait;" ::: "memory");
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int kb = kb0 + u * WK;
                if (kb >= nk) break;
                uint4 b[2];
                float sa0, sa1;
                if (MODE == FB_DOWN) {
                    const float *hr = p.h + ((sh ? p.shared_row : 0) + arow) * p.ldh;
                    float v[32], amax = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int k = kb * 128 + (i >> 2) * 64 + q * 16 + (i & 3) * 4;
                        const float4 f = live && k < K ? *reinterpret_cast<const float4 *>(hr + k) : make_float4(0.f, 0.f, 0.f, 0.f);
                        v[4 * i] = f.x; v[4 * i + 1] = f.y; v[4 * i + 2] = f.z; v[4 * i + 3] = f.w;
                        amax = fmaxf(fmaxf(fmaxf(amax, fabsf(f.x)), fmaxf(fabsf(f.y), fabsf(f.z))), fabsf(f.w));
                    }
                    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                    amax = fmaxf(amax, 0x1p-100f);
                    const float inv = __fdiv_rn(448.f, amax);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        b[i] = make_uint4(codes4(v + 16 * i, inv), codes4(v + 16 * i + 4, inv), codes4(v + 16 * i + 8, inv),
                                          codes4(v + 16 * i + 12, inv));
                    const float sc = __fdiv_rn(amax, 448.f);       // of row g; this lane's sums belong to rows 2 q, 2 q + 1
                    sa0 = __shfl_sync(0xffffffffu, sc, q * 8);
                    sa1 = __shfl_sync(0xffffffffu, sc, q * 8 + 4);
                } else {
                    const uint8_t *xr = (sh ? p.x_s : p.x) + arow * K + q * 16;
                    const char *sr = reinterpret_cast<const char *>(sh ? p.sa_s : p.sa);
                    const int64_t ld = sh ? p.ld_sa_s : p.ld_sa;
#pragma unroll
                    for (int i = 0; i < 2; ++i) b[i] = load16(xr + kb * 128 + i * 64, live && kb * 128 + i * 64 + q * 16 < K);
                    const int64_t t = (int64_t)row0 + r0 + 2 * q;
                    sa0 = 2 * q < rows ? __ldg(reinterpret_cast<const float *>(sr + t * ld) + kb) : 0.f;
                    sa1 = 2 * q + 1 < rows ? __ldg(reinterpret_cast<const float *>(sr + (t + 1) * ld) + kb) : 0.f;
                }
#pragma unroll
                for (int m = 0; m < NM; ++m) {
                    float c[4];
                    block_product(c, lo[u][m], hi[u][m], b);
                    const float s0 = sa0 * s[u][m], s1 = sa1 * s[u][m];
                    acc[m][0] = fmaf(c[0], s0, acc[m][0]);
                    acc[m][1] = fmaf(c[1], s1, acc[m][1]);
                    acc[m][2] = fmaf(c[2], s0, acc[m][2]);
                    acc[m][3] = fmaf(c[3], s1, acc[m][3]);
                }
            }
        }
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            red[m][wk][wn * 16 + g][2 * q] = acc[m][0];
            red[m][wk][wn * 16 + g][2 * q + 1] = acc[m][1];
            red[m][wk][wn * 16 + g + 8][2 * q] = acc[m][2];
            red[m][wk][wn * 16 + g + 8][2 * q + 1] = acc[m][3];
        }
        __syncthreads();
        for (int i = tid; i < WN * 16 * kRows; i += kThreads) {
            const int c = i % (WN * 16), r = i / (WN * 16), col = col0 + c;
            if (r >= rows || col >= N) continue;
            float v[NM];
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                v[m] = red[m][0][c][r];
#pragma unroll
                for (int k = 1; k < WK; ++k) v[m] += red[m][k][c][r];
            }
            const float bias = (!sh && p.bias) ? __ldg(p.bias + (int64_t)e * N + col) : 0.f;
            const int64_t row = (int64_t)row0 + r0 + r, orow = (sh ? p.shared_row : 0) + row;
            if (MODE == FB_DOWN) {
                const float gate = sh ? 1.f : __ldg(p.row_gate + row);
                p.out[orow * p.ldo + col] = __float2bfloat16_rn((v[0] + bias) * gate);
            } else {
                p.out_h[orow * p.ldh + col] = MODE == FB_SWIGLU ? fb_silu(v[0]) * v[NM - 1] : fb_gelu(v[0] + bias);
            }
        }
        __syncthreads();
    }
}

template <int MODE, int WN>
cudaError_t launch_wn(Params p, bool has_sh, cudaStream_t st, bool pdl) {
    p.tiles_r = (p.N_routed + WN * 16 - 1) / (WN * 16);
    p.tiles_s = has_sh ? (p.N_shared + WN * 16 - 1) / (WN * 16) : 0;
    const int64_t grid = (int64_t)p.active_max * p.tiles_r + p.tiles_s;
    return launch_kernel(fp8_block_decode<MODE, WN>, dim3((unsigned)grid), dim3(kThreads), 0, st, pdl, p);
}

// The widest column split that still gives every SM its two blocks: a block has
// about 4 us of latencies (offsets, first weights, the sum over warps) whatever
// its width.
template <int MODE>
cudaError_t launch_product(const Params &p, bool has_sh, int num_sms, cudaStream_t st, bool pdl) {
    const int64_t tiles = (int64_t)p.active_max * ((p.N_routed + 15) / 16) + (has_sh ? (p.N_shared + 15) / 16 : 0);
    const int64_t fit = 2 * (int64_t)num_sms;
    if (tiles <= fit) return launch_wn<MODE, 1>(p, has_sh, st, pdl);
    if (tiles <= 2 * fit) return launch_wn<MODE, 2>(p, has_sh, st, pdl);
    if (tiles <= 4 * fit) return launch_wn<MODE, 4>(p, has_sh, st, pdl);
    return launch_wn<MODE, 8>(p, has_sh, st, pdl);
}

}  // namespace

cudaError_t launch_ffn_fp8_block_decode(const FfnFp8BlockArgs &a, cudaStream_t st) {
    const bool swiglu = a.act == MOE_ACT_SWIGLU;
    const bool has_sh = a.S > 0 && a.T > 0;
    if (a.routed_rows == 0 && !has_sh) return cudaSuccess;
    Params p{};
    p.offsets = a.offsets; p.status = a.status;
    p.E = a.E; p.T = a.T; p.routed_rows = a.routed_rows;
    p.active_max = (int)(a.routed_rows < a.E ? a.routed_rows : a.E);
    p.K_routed = p.K_shared = a.d; p.N_routed = a.F; p.N_shared = a.S;
    p.x = a.x_perm; p.x_s = a.x; p.sa = a.xs_perm; p.sa_s = a.xs; p.ld_sa = a.ld_xs; p.ld_sa_s = a.ld_xs_shared;
    p.ldh = a.hF; p.shared_row = a.shared_base;
    p.w = a.W1; p.w2 = a.Wu; p.w_s = a.Wsg; p.w2_s = a.Wsu;
    p.sw = a.W1s; p.sw2 = a.Wus; p.sw_s = a.Wsgs; p.sw2_s = a.Wsus; p.ld_sw = a.sld;
    p.bias = swiglu ? nullptr : a.b1;
    p.out_h = a.h32;
    cudaError_t e = swiglu ? launch_product<FB_SWIGLU>(p, has_sh, a.num_sms, st, a.pdl)
                           : launch_product<FB_GELU>(p, has_sh, a.num_sms, st, a.pdl);
    if (e != cudaSuccess) return e;
    p.K_routed = a.F; p.K_shared = a.S; p.N_routed = p.N_shared = a.d;
    p.h = a.h32;
    p.w = a.W2; p.w_s = a.Wsd; p.sw = a.W2s; p.sw_s = a.Wsds;
    p.bias = swiglu ? nullptr : a.b2;
    p.row_gate = a.row_gate;
    p.out = a.y_perm; p.ldo = a.d;
    return launch_product<FB_DOWN>(p, has_sh, a.num_sms, st, true);
}

}  // namespace moe
