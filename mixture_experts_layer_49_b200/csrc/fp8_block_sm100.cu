// fp8_block_sm100.cu -- grouped expert FFN with block-scaled e4m3 operands:
// activations with one fp32 scale per row and 128 values of K, weights with
// one fp32 scale per 128 x 128 block.
//
//   C[r][n] = sum_b sa[r][b] * sw[n / 128][b] * sum_{k in block b} a[r][k] w[n][k]
//
// The scales change along K, so they cannot wait for the epilogue: each block
// of 128 of K is one chain of four tcgen05.mma (kind::f8f6f4, K = 32) into a
// fresh TMEM accumulator, and the epilogue warps add it, scaled, to sums in
// their registers while the tensor core fills the other accumulator.  The
// sums never leave fp32 and the partial products of 128 terms are the longest
// chain that the tensor core rounds.
//
// One persistent CTA per SM, tile 128 rows x 256 accumulator columns (SwiGLU:
// 128 gate and 128 up columns), 320 threads:
//   warp 0      TMA producer, 4 stages of A 128 x 128 and B 256 x 128 bytes
//   warp 1      TMEM allocator and tcgen05.mma issuer
//   warps 2..9  the scaled sums (two warps per TMEM lane quadrant, 128 columns
//               each: 128 fp32 registers a thread) and the epilogue
// Epilogues: SwiGLU and GELU quantize the hidden row's block of 128 straight
// from the fp32 sums (one rounding), so the second product reads codes and
// scales and no pass over H runs in between; the down projection adds the bias,
// applies the gate and rounds once to bf16.
//
// Per K block the tensor core needs 512 cycles (128 x 256 x 128 products at
// 8192 per cycle); the sums need 32768 TMEM words (512 bytes a cycle: 256
// cycles) and as many fused multiply-adds (two per lane and cycle: 128 cycles).
//
// Every mbarrier wait is bounded as in the other tensor-core kernels; a wait
// that runs out records MOE_ERR_TIMEOUT, and the CTA lets its copies and
// products in flight finish before it frees its TMEM.
#include <cudaTypedefs.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.cuh"
#include "sm100.cuh"

namespace moe {

namespace {

constexpr int BM = 128, BN = 256, BK = 128;
constexpr int STAGES = 4;
constexpr int kThreads = 320;
constexpr uint32_t A_BYTES = BM * BK;
constexpr uint32_t B_BYTES = BN * BK;
constexpr uint32_t STAGE_BYTES = A_BYTES + B_BYTES;
constexpr uint32_t TMEM_COLS = 512;
constexpr int kMaxGroups = 257;
constexpr uint32_t kIdesc = make_idesc_e4m3(BM, BN);

enum { FB_SWIGLU = 0, FB_GELU = 1, FB_DOWN = 2 };

struct Params {
    const int32_t *offsets;      // [E+1]
    int32_t *status;
    int E, T, has_shared;
    int64_t routed_rows;         // rows of the packed arrays
    int K_routed, K_shared, N_routed, N_shared;
    // scales: rows of A (routed, shared; bytes between rows), then weights:
    // expert stride and bytes between rows of blocks
    const float *sa, *sa_s;
    int64_t ld_sa, ld_sa_s;
    const float *sw, *sw2;       // routed (SwiGLU: gate, up)
    const float *sws, *sws2;     // shared expert
    int64_t ld_sw;
    int64_t shared_a_row;        // first A row of the shared group
    int64_t shared_out_row;      // first output row of the shared group
    const float *bias;           // [E, N_routed] or null
    const float *row_gate;       // FB_DOWN
    void *out;                   // codes (FB_SWIGLU, FB_GELU) or bf16, row stride ldo elements
    int64_t ldo;
    float *out_scale;            // scale rows of the codes, ld_out_scale floats apart
    int64_t ld_out_scale;
    uint64_t timeout_ns;
};

struct Tail {
    uint64_t full[STAGES];
    uint64_t empty[STAGES];
    uint64_t accf[2];
    uint64_t acce[2];
    uint64_t drain;
    uint64_t xch[4];             // SwiGLU: both halves of a quadrant's rows left their maxima
    uint32_t tmem_base;
    int abort_flag;
    int tile_start[kMaxGroups + 1];
    int mtiles[kMaxGroups];
    int rows[kMaxGroups];
    int row0[kMaxGroups];
    float amax[2][2][BM];        // SwiGLU: the two halves' row maxima, two tiles deep
};
constexpr size_t kSmemBytes = 1024 + STAGES * STAGE_BYTES + sizeof(Tail);
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

__device__ __forceinline__ float gelu_erf(float v) { return 0.5f * v * (1.f + erff(v * 0.70710678118654752f)); }
__device__ __forceinline__ float silu(float v) { return __fdividef(v, 1.f + __expf(-v)); }

__device__ __forceinline__ bool aborted(const Tail &s) {
    return *reinterpret_cast<const volatile int *>(&s.abort_flag) != 0;
}
__device__ __forceinline__ void fail(Tail &s, const Params &p, int where) {
    record_error(p.status, MOE_ERR_TIMEOUT, where);
    *reinterpret_cast<volatile int *>(&s.abort_flag) = 1;
}

__device__ __forceinline__ void decode(const Tail &s, int G, int tile, int &g, int &mt, int &nt) {
    int lo = 0, hi = G - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s.tile_start[mid] <= tile) lo = mid; else hi = mid - 1;
    }
    g = lo;
    const int local = tile - s.tile_start[g];
    mt = local % s.mtiles[g];
    nt = local / s.mtiles[g];
}

// Two fp32 fused multiply-adds in one instruction: (a0, a1) += (v0, v1) * s.
__device__ __forceinline__ void fma2(float &a0, float &a1, float v0, float v1, uint64_t s) {
    uint64_t a, v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(a0), "f"(a1));
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(v0), "f"(v1));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(a) : "l"(v), "l"(s));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a0), "=f"(a1) : "l"(a));
}
__device__ __forceinline__ uint64_t both(float s) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %1};" : "=l"(d) : "f"(s));
    return d;
}

// Codes of 16 values v * inv as one 16-byte vector.
__device__ __forceinline__ uint4 codes16(const float *v, float inv) {
    uint32_t w[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(
            make_float2(__fmul_rn(v[4 * h], inv), __fmul_rn(v[4 * h + 1], inv)), __NV_SATFINITE, __NV_E4M3);
        const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(
            make_float2(__fmul_rn(v[4 * h + 2], inv), __fmul_rn(v[4 * h + 3], inv)), __NV_SATFINITE, __NV_E4M3);
        w[h] = (uint32_t)lo | ((uint32_t)hi << 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// What one sums thread knows of its tile: its output row and scale sources.
struct RowCtx {
    bool valid;
    int64_t orow;                // output row
    const float *sa;             // scale row of its A row
    const float *sw0, *sw1;      // weight scale rows of its first and second 64 columns
    int N, half, nt;
    float gate;
    const float *bias;
};

template <int MODE>
__device__ __forceinline__ RowCtx row_ctx(const Params &p, bool sh, int e, int nt, int half, int64_t a_row,
                                          int64_t a_row_first, int64_t orow, bool valid) {
    RowCtx c;
    c.valid = valid;
    c.orow = orow;
    c.half = half;
    c.nt = nt;
    c.N = sh ? p.N_shared : p.N_routed;
    // a row past the group's end reads the group's first scale row (its sums are never stored)
    c.sa = reinterpret_cast<const float *>(reinterpret_cast<const char *>(sh ? p.sa_s : p.sa) +
                                           (valid ? a_row : a_row_first) * (sh ? p.ld_sa_s : p.ld_sa));
    const int64_t nb = (c.N + 127) >> 7;
    const int64_t blk = MODE == FB_SWIGLU ? nt : nt * 2 + half;
    // columns past N belong to no block: their products are zero, any scale row will do
    const int64_t wrow = (sh ? 0 : (int64_t)e * nb) + (blk < nb ? blk : nb - 1);
    c.sw0 = reinterpret_cast<const float *>(reinterpret_cast<const char *>(sh ? p.sws : p.sw) + wrow * p.ld_sw);
    c.sw1 = MODE == FB_SWIGLU
                ? reinterpret_cast<const float *>(reinterpret_cast<const char *>(sh ? p.sws2 : p.sw2) + wrow * p.ld_sw)
                : c.sw0;
    c.gate = 1.f;
    if (MODE == FB_DOWN && !sh && valid) c.gate = __ldg(p.row_gate + orow);
    c.bias = (!sh && p.bias) ? p.bias + (int64_t)e * p.N_routed : nullptr;
    return c;
}

// Output of one row's 128 sums.
// false: a wait ran out.
template <int MODE>
__device__ __forceinline__ bool finish_row(const Params &p, const RowCtx &c, float (&acc)[128], float (*amax_buf)[BM],
                                           int r_in_tile, uint32_t xch, uint32_t xphase) {
    if (MODE == FB_DOWN) {
        const int col0 = c.nt * BN + c.half * 128;
        __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.out) + c.orow * p.ldo + col0;
#pragma unroll
        for (int u = 0; u < 16; ++u) {
            if (!c.valid || col0 + u * 8 >= c.N) continue;
            uint4 pk;
            __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&pk);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float a = acc[u * 8 + 2 * i], b = acc[u * 8 + 2 * i + 1];
                if (c.bias) {
                    a += __ldg(c.bias + col0 + u * 8 + 2 * i);
                    b += __ldg(c.bias + col0 + u * 8 + 2 * i + 1);
                }
                h[i] = __floats2bfloat162_rn(a * c.gate, b * c.gate);
            }
            *reinterpret_cast<uint4 *>(o + u * 8) = pk;
        }
        return true;
    }
    constexpr int W = MODE == FB_SWIGLU ? 64 : 128;        // hidden values of this thread
    const int col0 = MODE == FB_SWIGLU ? c.nt * 128 + c.half * 64 : c.nt * BN + c.half * 128;
    float amax = 0.f;
    if (MODE == FB_SWIGLU) {
#pragma unroll
        for (int i = 0; i < 64; ++i) {
            acc[i] = silu(acc[i]) * acc[64 + i];
            amax = fmaxf(amax, fabsf(acc[i]));             // columns past N are 0 * 0
        }
        // the block's maximum spans the two halves of the row; an mbarrier,
        // because its wait can be bounded
        amax_buf[c.half][r_in_tile] = amax;
        __syncwarp();
        int ok = 1;
        if ((threadIdx.x & 31) == 0) {
            mbar_arrive(xch);
            ok = mbar_wait(xch, xphase, p.timeout_ns) ? 1 : 0;
        }
        if (!__shfl_sync(0xffffffffu, ok, 0)) return false;
        amax = fmaxf(amax, amax_buf[c.half ^ 1][r_in_tile]);
    } else {
#pragma unroll
        for (int i = 0; i < 128; ++i) {
            const float b = (c.bias && col0 + i < c.N) ? __ldg(c.bias + col0 + i) : 0.f;
            acc[i] = gelu_erf(acc[i] + b);                 // columns past N: gelu(0) = 0
            amax = fmaxf(amax, fabsf(acc[i]));
        }
    }
    amax = fmaxf(amax, 0x1p-100f);
    if (!c.valid) return true;
    const float inv = __fdiv_rn(448.f, amax);
    uint8_t *o = static_cast<uint8_t *>(p.out) + c.orow * p.ldo + col0;
#pragma unroll
    for (int u = 0; u < W / 16; ++u)
        if (col0 + u * 16 < c.N) *reinterpret_cast<uint4 *>(o + u * 16) = codes16(acc + u * 16, inv);
    const int blk = MODE == FB_SWIGLU ? c.nt : c.nt * 2 + c.half;
    if ((MODE != FB_SWIGLU || c.half == 0) && blk * 128 < c.N)
        p.out_scale[c.orow * p.ld_out_scale + blk] = __fdiv_rn(amax, 448.f);
    return true;
}

template <int MODE>
__global__ void __launch_bounds__(kThreads, 1)
fp8_block_gemm(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmAs,
               const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmB2,
               const __grid_constant__ CUtensorMap tmBs, const __grid_constant__ CUtensorMap tmBs2,
               const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (base - raw_addr);
    Tail &s = *reinterpret_cast<Tail *>(smem + STAGES * STAGE_BYTES);
    const uint32_t smA = base;
    const uint32_t smB = base + STAGES * A_BYTES;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int BNO = MODE == FB_SWIGLU ? 128 : 256;     // output columns per tile
    const int G = p.E + (p.has_shared ? 1 : 0);

    if (tid == 0) {
        s.abort_flag = 0;
        for (int i = 0; i < STAGES; ++i) { mbar_init(smem_u32(&s.full[i]), 1); mbar_init(smem_u32(&s.empty[i]), 1); }
        for (int i = 0; i < 2; ++i) { mbar_init(smem_u32(&s.accf[i]), 1); mbar_init(smem_u32(&s.acce[i]), 8); }
        for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&s.xch[i]), 2);
        mbar_init(smem_u32(&s.drain), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) tmem_alloc(smem_u32(&s.tmem_base), TMEM_COLS);
    if (tid == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&tmA) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&tmB) : "memory");
    }
    pdl_wait_then_release();
    if (tid == 0) s.tile_start[0] = 0;
    for (int g = tid; g < G; g += kThreads) {
        const bool sh = g >= p.E;
        int64_t r0 = sh ? 0 : p.offsets[g];
        int64_t rows = sh ? p.T : (int64_t)p.offsets[g + 1] - r0;
        if (!sh && (r0 < 0 || rows < 0 || r0 + rows > p.routed_rows)) {      // not a prefix sum of this many rows
            record_error(p.status, MOE_ERR_DEVICE_BOUNDS, g);
            r0 = rows = 0;
        }
        const int n = sh ? p.N_shared : p.N_routed;
        const int mt = (int)((rows + BM - 1) / BM);
        s.rows[g] = (int)rows;
        s.row0[g] = (int)r0;
        s.mtiles[g] = mt > 0 ? mt : 1;
        s.tile_start[g + 1] = mt * ((n + BNO - 1) / BNO);
    }
    __syncthreads();
    if (warp == 0) {                                       // inclusive scan of the tile counts
        int carry = 0;
        for (int g0 = 0; g0 < G; g0 += 32) {
            const int g = g0 + lane;
            int v = g < G ? s.tile_start[g + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int n = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += n;
            }
            if (g < G) s.tile_start[g + 1] = carry + v;
            carry += __shfl_sync(0xffffffffu, v, 31);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const int total = s.tile_start[G];
    const uint32_t tmem_base = s.tmem_base;

    if (warp == 0) {
        // ================= TMA producer
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0, issued = 0;
            for (int tile = blockIdx.x; tile < total && !aborted(s); tile += gridDim.x) {
                int g, mt, nt;
                decode(s, G, tile, g, mt, nt);
                const bool sh = g >= p.E;
                const int nk = ((sh ? p.K_shared : p.K_routed) + BK - 1) / BK;
                const int a_row = (sh ? (int)p.shared_a_row : s.row0[g]) + mt * BM;
                const CUtensorMap *mA = sh ? &tmAs : &tmA;
                const CUtensorMap *mB = sh ? &tmBs : &tmB;
                const CUtensorMap *mB2 = sh ? &tmBs2 : &tmB2;
                const int e = sh ? 0 : g;
                for (int kb = 0; kb < nk; ++kb) {
                    if (!mbar_wait(smem_u32(&s.empty[stage]), phase ^ 1u, p.timeout_ns)) { fail(s, p, 61); break; }
                    const uint32_t fb = smem_u32(&s.full[stage]);
                    mbar_arrive_expect_tx(fb, STAGE_BYTES);
                    tma_load_2d(smA + stage * A_BYTES, mA, fb, kb * BK, a_row);
                    if (MODE == FB_SWIGLU) {
                        tma_load_3d(smB + stage * B_BYTES, mB, fb, kb * BK, nt * 128, e);
                        tma_load_3d(smB + stage * B_BYTES + B_BYTES / 2, mB2, fb, kb * BK, nt * 128, e);
                    } else {
                        tma_load_3d(smB + stage * B_BYTES, mB, fb, kb * BK, nt * BN, e);
                    }
                    ++issued;
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
            }
            // every copy has landed before the CTA may end: the last use of each stage
            for (uint32_t i = issued > STAGES ? issued - STAGES : 0; i < issued; ++i)
                if (!mbar_wait(smem_u32(&s.full[i % STAGES]), (i / STAGES) & 1u, p.timeout_ns)) fail(s, p, 65);
        }
    } else if (warp == 1) {
        // ================= MMA issuer: one accumulator per K block
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0, cnt = 0;
            for (int tile = blockIdx.x; tile < total && !aborted(s); tile += gridDim.x) {
                // the shared group, when there is one, is the last
                const int nk = ((tile >= s.tile_start[p.E] ? p.K_shared : p.K_routed) + BK - 1) / BK;
                bool ok = true;
                for (int kb = 0; kb < nk; ++kb, ++cnt) {
                    const uint32_t ab = cnt & 1u, aphase = (cnt >> 1) & 1u;
                    if (!mbar_wait(smem_u32(&s.acce[ab]), aphase ^ 1u, p.timeout_ns)) { fail(s, p, 62); ok = false; break; }
                    if (!mbar_wait(smem_u32(&s.full[stage]), phase, p.timeout_ns)) { fail(s, p, 63); ok = false; break; }
                    tc_fence_after();
                    const uint32_t a0 = smA + stage * A_BYTES, b0 = smB + stage * B_BYTES;
#pragma unroll
                    for (int k = 0; k < BK / 32; ++k)
                        mma_e4m3(tmem_base + ab * BN, sdesc(a0 + k * 32), sdesc(b0 + k * 32), kIdesc, k ? 1u : 0u);
                    mma_commit(smem_u32(&s.empty[stage]));
                    mma_commit(smem_u32(&s.accf[ab]));
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
                if (!ok) break;
            }
            if (aborted(s)) {                              // products in flight end before TMEM is freed
                mma_commit(smem_u32(&s.drain));
                if (!mbar_wait(smem_u32(&s.drain), 0, p.timeout_ns)) fail(s, p, 66);
            }
        }
    } else {
        // ================= scaled sums and epilogue: warps 2..9
        const int q = warp & 3, half = (warp - 2) >> 2;
        const int r_in_tile = q * 32 + lane;
        const uint32_t lane_addr = tmem_base + ((uint32_t)(q * 32) << 16);
        // columns of this warp: SwiGLU 64 gate and 64 up columns, else 128 in a row
        const uint32_t c0 = MODE == FB_SWIGLU ? half * 64 : half * 128;
        const uint32_t c1 = MODE == FB_SWIGLU ? 128 + half * 64 : half * 128 + 64;
        uint32_t cnt = 0;
        uint32_t flip = 0;                                 // parity of the tiles this CTA has done
        bool ok = true;
        for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x, flip ^= 1u) {
            int g, mt, nt;
            decode(s, G, tile, g, mt, nt);
            const bool sh = g >= p.E;
            const int grow = mt * BM + r_in_tile;
            const int64_t first = sh ? 0 : (int64_t)s.row0[g];
            const int64_t a_off = sh ? p.shared_a_row : 0, o_off = sh ? p.shared_out_row : 0;
            const RowCtx c = row_ctx<MODE>(p, sh, g, nt, half, a_off + first + grow, a_off + first,
                                           o_off + first + grow, grow < s.rows[g]);
            const int nk = ((sh ? p.K_shared : p.K_routed) + BK - 1) / BK;
            float acc[128];
#pragma unroll
            for (int i = 0; i < 128; ++i) acc[i] = 0.f;
            float ra = __ldg(c.sa), rw0 = __ldg(c.sw0), rw1 = __ldg(c.sw1);
            for (int kb = 0; kb < nk; ++kb, ++cnt) {
                const uint32_t ab = cnt & 1u, aphase = (cnt >> 1) & 1u;
                const uint64_t s0 = both(ra * rw0), s1 = both(ra * rw1);
                if (kb + 1 < nk) {                         // the next block's scales arrive during this one
                    ra = __ldg(c.sa + kb + 1);
                    rw0 = __ldg(c.sw0 + kb + 1);
                    rw1 = MODE == FB_SWIGLU ? __ldg(c.sw1 + kb + 1) : rw0;
                }
                // lane 0 waits, the warp follows its verdict
                int okw = 1;
                if (lane == 0) okw = (!aborted(s) && mbar_wait(smem_u32(&s.accf[ab]), aphase, p.timeout_ns)) ? 1 : 0;
                okw = __shfl_sync(0xffffffffu, okw, 0);
                if (!okw) { if (lane == 0) fail(s, p, 64); ok = false; break; }
                tc_fence_after();
                const uint32_t ta = lane_addr + ab * BN;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t tc = ta + (h ? c1 : c0);
                    const uint64_t sc = h ? s1 : s0;
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        float v[32];
                        tmem_ld32(tc + u * 32, v);
#pragma unroll
                        for (int i = 0; i < 32; i += 2)
                            fma2(acc[h * 64 + u * 32 + i], acc[h * 64 + u * 32 + i + 1], v[i], v[i + 1], sc);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&s.acce[ab]));
            }
            if (!ok) break;
            ok = finish_row<MODE>(p, c, acc, s.amax[flip], r_in_tile, smem_u32(&s.xch[q]), flip);
            if (!ok && lane == 0) fail(s, p, 67);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

template <int MODE>
cudaError_t launch_gemm(const CUtensorMap &A, const CUtensorMap &As, const CUtensorMap &B, const CUtensorMap &B2,
                        const CUtensorMap &Bs, const CUtensorMap &Bs2, const Params &p, int grid, cudaStream_t st,
                        bool pdl) {
    cudaError_t e = cudaFuncSetAttribute(fp8_block_gemm<MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)kSmemBytes);
    if (e != cudaSuccess) return e;
    return launch_kernel(fp8_block_gemm<MODE>, dim3(grid), dim3(kThreads), kSmemBytes, st, pdl, A, As, B, B2, Bs, Bs2, p);
}

}  // namespace

cudaError_t launch_ffn_fp8_block(const FfnFp8BlockArgs &a, cudaStream_t st) {
    const bool swiglu = a.act == MOE_ACT_SWIGLU;
    const bool has_sh = a.S > 0 && a.T > 0;
    if (a.routed_rows == 0 && !has_sh) return cudaSuccess;
    const uint64_t routed = a.routed_rows > 0 ? (uint64_t)a.routed_rows : 1;
    const uint64_t all = (uint64_t)(a.shared_base + (has_sh ? a.T : 0));
    const uint64_t d = a.d, F = a.F, S = a.S;
    const uint32_t box1 = swiglu ? 128 : BN;
    CUtensorMap A1, A1s, B1, B1u, B1s, B1su, A2, A2s, B2, B2s;
    bool ok = make_map(&A1, 2, a.x_perm, d, routed, 1, d, 0, BM, 1) &&
              make_map(&B1, 3, a.W1, d, F, a.E, d, F * d, box1, 1) &&
              make_map(&A2, 2, a.H8, F, all, 1, a.hF, 0, BM, 1) &&
              make_map(&B2, 3, a.W2, F, d, a.E, F, d * F, BN, 1);
    B1u = B1;
    if (ok && swiglu) ok = make_map(&B1u, 3, a.Wu, d, F, a.E, d, F * d, box1, 1);
    A1s = A1; B1s = B1; B1su = B1u; A2s = A2; B2s = B2;
    if (ok && has_sh) {
        ok = make_map(&A1s, 2, a.x, d, a.T, 1, d, 0, BM, 1) && make_map(&B1s, 3, a.Wsg, d, S, 1, d, 0, box1, 1) &&
             make_map(&A2s, 2, a.H8, S, all, 1, a.hF, 0, BM, 1) && make_map(&B2s, 3, a.Wsd, S, d, 1, S, 0, BN, 1);
        B1su = B1s;
        if (ok && swiglu) ok = make_map(&B1su, 3, a.Wsu, d, S, 1, d, 0, box1, 1);
    }
    if (!ok) return cudaErrorInvalidValue;

    Params p{};
    p.offsets = a.offsets;
    p.status = a.status;
    p.E = a.E; p.T = a.T; p.has_shared = has_sh ? 1 : 0;
    p.routed_rows = a.routed_rows;
    p.K_routed = a.d; p.K_shared = a.d; p.N_routed = a.F; p.N_shared = a.S;
    p.sa = a.xs_perm; p.sa_s = a.xs; p.ld_sa = a.ld_xs; p.ld_sa_s = a.ld_xs_shared;
    p.sw = a.W1s; p.sw2 = a.Wus; p.sws = a.Wsgs; p.sws2 = a.Wsus; p.ld_sw = a.sld;
    p.shared_a_row = 0; p.shared_out_row = a.shared_base;
    p.bias = swiglu ? nullptr : a.b1;
    p.out = a.H8; p.ldo = a.hF;
    p.out_scale = a.h_scale; p.ld_out_scale = a.ld_hs / 4;
    p.timeout_ns = 2000000000ull;
    const int grid = a.num_sms;
    cudaError_t e = swiglu ? launch_gemm<FB_SWIGLU>(A1, A1s, B1, B1u, B1s, B1su, p, grid, st, a.pdl)
                           : launch_gemm<FB_GELU>(A1, A1s, B1, B1u, B1s, B1su, p, grid, st, a.pdl);
    if (e != cudaSuccess) return e;

    p.K_routed = a.F; p.K_shared = a.S; p.N_routed = a.d; p.N_shared = a.d;
    p.sa = p.sa_s = a.h_scale; p.ld_sa = p.ld_sa_s = a.ld_hs;
    p.sw = a.W2s; p.sw2 = nullptr; p.sws = a.Wsds; p.sws2 = nullptr;
    p.shared_a_row = a.shared_base;
    p.bias = swiglu ? nullptr : a.b2;
    p.row_gate = a.row_gate;
    p.out = a.y_perm; p.ldo = a.d;
    p.out_scale = nullptr; p.ld_out_scale = 0;
    return launch_gemm<FB_DOWN>(A2, A2s, B2, B2, B2s, B2s, p, grid, st, true);
}

}  // namespace moe
