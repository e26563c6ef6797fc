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
// Persistent CTAs of 384 threads, one to an SM (128 rows x 256 accumulator
// columns, 4 stages of 48 KiB); SwiGLU's columns are 128 of the gate and 128 of the
// up product:
//   warp 0       TMA producer
//   warps 1, 2   TMEM allocator (1) and tcgen05.mma issuers of the even and odd
//                K blocks
//   warp 3       idle: it fills the first warpgroup, which gives its registers away
//   warps 4..11  the scaled sums (two warps per TMEM lane quadrant, 128 columns
//                each: 128 fp32 registers a thread) and the epilogue
// Epilogues: SwiGLU and GELU quantize the hidden row's block of 128 straight
// from the fp32 sums (one rounding), so the second product reads codes and
// scales and no pass over H runs in between; the down projection adds the bias,
// applies the gate and rounds once to bf16.
//
// Per K block the tensor core needs 512 cycles (128 x 256 x 128 products at 8192
// per cycle) and the loop takes about 850, beside the power limit, which holds the
// clock near 1.4 GHz in long runs.  The scaled sums make the difference: in the
// same loop of a CTA pair, at 835 cycles, leaving out the multiply-adds gave 600,
// the TMEM loads too 520, the copies 860.  None of these went below 825: half
// accumulators of 128 columns with barriers of their own, loads of 32 columns
// beside the multiply-adds of the last 32, packed f32x2 multiply-adds.  A library
// product of 8192 x 28672 x 4096 with one scale per tensor, so without the sums,
// takes 757 us where a pair's took 905.
//
// CTA pairs (256-row tiles by cta_group::2, 32 KiB a CTA and K block instead of 48,
// last blocks of 1..128 rows in a launch of their own) are not faster: one expert
// of 8192 rows, 4096 x 14336, 1.55 ms either way, but 16384 tokens of the Qwen3
// shape 945 us against 909, 4096 of the Mixtral shape 1725 against 1672, 8192
// tokens with 128 experts of 7168 x 2048 4.03 ms against 3.74 (each at least three
// runs in turn).
//
// Every mbarrier wait is bounded as in the other tensor-core kernels; a wait
// that runs out records MOE_ERR_TIMEOUT, and the CTA lets its copies and
// products in flight finish before it frees its TMEM.
#include <cudaTypedefs.h>
#include <cuda_fp8.h>

#include <atomic>

#include "common.cuh"
#include "fp8_block.cuh"
#include "kernels.cuh"
#include "sm100.cuh"

namespace moe {

namespace {

constexpr int BM = 128, BN = 256, BK = 128;
constexpr int STAGES = 4;
constexpr int kThreads = 384;                // 3 warpgroups: control, 2 x sums
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

// Barriers and the tile table behind the stages.
struct Tail {
    uint64_t full[STAGES];
    uint64_t empty[STAGES];
    uint64_t accf[2];
    uint64_t acce[2];
    uint64_t drain[2];
    uint64_t xch[4];             // SwiGLU: both halves of a quadrant's rows left their maxima
    uint32_t tmem_base;
    int abort_flag;
    int tile_start[kMaxGroups + 1];
    int mtiles[kMaxGroups];
    int rows[kMaxGroups];
    int row0[kMaxGroups];
    float amax[2][2][BM];        // SwiGLU: the two halves' row maxima, two tiles deep
};
// Output staging: 32 rows of 64 bytes per sums warp.
constexpr uint32_t STG_BYTES = 32 * 64;
constexpr size_t kStgOff = (STAGES * STAGE_BYTES + sizeof(Tail) + 1023) / 1024 * 1024;
constexpr size_t kSmemBytes = 1024 + kStgOff + 8 * STG_BYTES;
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

// One lane of the converged warp, always the same one.
__device__ __forceinline__ bool elect_lane() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}
// A bounded wait of the whole warp with one verdict for all lanes.
__device__ __forceinline__ bool warp_wait(uint32_t addr, uint32_t parity, uint64_t limit_ns) {
    return __all_sync(0xffffffffu, mbar_wait(addr, parity, limit_ns));
}

__device__ __forceinline__ bool aborted(const Tail &s) {
    return *reinterpret_cast<const volatile int *>(&s.abort_flag) != 0;
}
__device__ __forceinline__ void fail(Tail &s, const Params &p, int where) {
    record_error(p.status, MOE_ERR_TIMEOUT, where);
    *reinterpret_cast<volatile int *>(&s.abort_flag) = 1;
}

// The group of tile `tile`, from the group of an earlier one; mt runs fastest
// within a group, so CTAs at work together share weight tiles through L2.
__device__ __forceinline__ void locate(const Tail &s, int tile, int &g, int &mt, int &nt) {
    while (s.tile_start[g + 1] <= tile) ++g;
    const int local = tile - s.tile_start[g], n = s.mtiles[g];
    nt = local / n;
    mt = local - nt * n;
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

// 64 bytes of each of the warp's 32 rows (w: this lane's row) through its staging
// buffer to out + row * ld: four neighbouring lanes store a row's pieces (stores
// by row would touch 32 rows per instruction: 4096 more cycles a tile measured;
// TMA stores need a proxy fence, which waits 500 to 3000 cycles beside the
// loads).  Piece c of row r lies at c ^ ((r / 2) % 4), so both sides are free of
// bank conflicts.  rows: valid rows of the warp; pieces: those below the row's end.
__device__ __forceinline__ void stage_out(uint32_t stg, const uint4 (&w)[4], char *out, int64_t ld, int rows, int pieces) {
    const int lane = threadIdx.x & 31, p = lane & 3;
    __syncwarp();                                          // the last store has read the buffer
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const uint32_t a = stg + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(w[c].x), "r"(w[c].y), "r"(w[c].z),
                     "r"(w[c].w) : "memory");
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + (lane >> 2);
        uint4 v;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"(stg + r * 64 + ((p ^ ((r >> 1) & 3)) << 4)) : "memory");
        if (r < rows && p < pieces) *reinterpret_cast<uint4 *>(out + r * ld + p * 16) = v;
    }
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
                                           int r_in_tile, uint32_t xch, uint32_t xphase, uint32_t stg) {
    const int rows = __popc(__ballot_sync(0xffffffffu, c.valid));     // a prefix of the warp's lanes
    const int64_t row0 = c.orow - (int)(threadIdx.x & 31);
    if (MODE == FB_DOWN) {
        const int col0 = c.nt * BN + c.half * 128;
        if (c.bias) {
#pragma unroll
            for (int i = 0; i < 128; ++i) acc[i] += col0 + i < c.N ? __ldg(c.bias + col0 + i) : 0.f;
        }
        char *o = static_cast<char *>(p.out) + (row0 * p.ldo + col0) * 2;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint4 w[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&w[u]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int n = q * 32 + u * 8 + 2 * i;
                    h[i] = __floats2bfloat162_rn(acc[n] * c.gate, acc[n + 1] * c.gate);
                }
            }
            stage_out(stg, w, o + q * 64, p.ldo * 2, rows, (c.N - col0) / 8 - q * 4);
        }
        return true;
    }
    constexpr int W = MODE == FB_SWIGLU ? 64 : 128;        // hidden values of this thread
    const int col0 = MODE == FB_SWIGLU ? c.nt * 128 + c.half * 64 : c.nt * BN + c.half * 128;
    float amax = 0.f;
    if (MODE == FB_SWIGLU) {
#pragma unroll
        for (int i = 0; i < 64; ++i) {
            acc[i] = fb_silu(acc[i]) * acc[64 + i];
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
        __syncwarp();                                      // lane 0's wait orders memory for the other lanes by this
        amax = fmaxf(amax, amax_buf[c.half ^ 1][r_in_tile]);
    } else {
        if (c.bias) {
#pragma unroll
            for (int i = 0; i < 128; ++i) acc[i] += col0 + i < c.N ? __ldg(c.bias + col0 + i) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 128; i += 2) {
            fb_gelu2(acc[i], acc[i + 1]);                  // columns past N: gelu(0) = 0
            amax = fmaxf(amax, fmaxf(fabsf(acc[i]), fabsf(acc[i + 1])));
        }
    }
    amax = fmaxf(amax, 0x1p-100f);
    const float inv = __fdiv_rn(448.f, amax);
    char *o = static_cast<char *>(p.out) + row0 * p.ldo + col0;
#pragma unroll
    for (int q = 0; q < W / 64; ++q) {
        uint4 w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) w[u] = codes16(acc + q * 64 + u * 16, inv);
        stage_out(stg, w, o + q * 64, p.ldo, rows, (c.N - col0) / 16 - q * 4);
    }
    if (!c.valid) return true;
    const int blk = MODE == FB_SWIGLU ? c.nt : c.nt * 2 + c.half;
    if ((MODE != FB_SWIGLU || c.half == 0) && blk * 128 < c.N)
        p.out_scale[c.orow * p.ld_out_scale + blk] = __fdiv_rn(amax, 448.f);
    return true;
}

// The tile list of a launch from the device-side offsets: groups are the routed
// experts and, last, the shared expert.
template <int BNO>
__device__ __forceinline__ void build_tiles(Tail &s, const Params &p) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = p.E + (p.has_shared ? 1 : 0);
    if (tid == 0) s.tile_start[0] = 0;
    for (int g = tid; g < G; g += kThreads) {
        const bool sh = g >= p.E;
        int64_t r0 = sh ? 0 : p.offsets[g];
        int64_t rows = sh ? p.T : (int64_t)p.offsets[g + 1] - r0;
        if (!sh && (r0 < 0 || rows < 0 || r0 + rows > p.routed_rows)) {      // not a prefix sum of this many rows
            record_error(p.status, MOE_ERR_DEVICE_BOUNDS, g);
            r0 = rows = 0;
        }
        const int mt = (int)((rows + BM - 1) / BM);
        const int n = sh ? p.N_shared : p.N_routed;
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
}

// The work of warps 4..11: two per TMEM lane quadrant, each half of the
// columns.
template <int MODE>
__device__ __forceinline__ void sums_warps(Tail &s, const Params &p, uint32_t tmem_base, uint32_t stg0, int total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int q = warp & 3, half = (warp - 4) >> 2;
    const int r_in_tile = q * 32 + lane;
    const uint32_t stg = stg0 + (uint32_t)(warp - 4) * STG_BYTES;
    const uint32_t lane_addr = tmem_base + ((uint32_t)(q * 32) << 16);
    // columns of this warp: SwiGLU 64 gate and 64 up columns, else 128 in a row
    const uint32_t c0 = MODE == FB_SWIGLU ? half * 64 : half * 128;
    const uint32_t c1 = MODE == FB_SWIGLU ? 128 + half * 64 : half * 128 + 64;
    uint32_t cnt = 0;
    uint32_t flip = 0;                                     // parity of the tiles this CTA has done
    bool ok = true;
    int g = 0;
    for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x, flip ^= 1u) {
        int mt, nt;
        locate(s, tile, g, mt, nt);
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
            const float s0 = ra * rw0, s1 = ra * rw1;
            if (kb + 1 < nk) {                             // the next block's scales arrive during this one
                ra = __ldg(c.sa + kb + 1);
                rw0 = __ldg(c.sw0 + kb + 1);
                rw1 = MODE == FB_SWIGLU ? __ldg(c.sw1 + kb + 1) : rw0;
            }
            if (!warp_wait(smem_u32(&s.accf[ab]), aphase, p.timeout_ns)) { if (lane == 0) fail(s, p, 64); ok = false; break; }
            tc_fence_after();
            const uint32_t ta = lane_addr + ab * BN;
            float v[64];
            tmem_ld32x2(ta + c0, ta + c0 + 32, v);
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = fmaf(v[i], s0, acc[i]);
            tmem_ld32x2(ta + c1, ta + c1 + 32, v);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&s.acce[ab]));     // free: its words are in registers
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[64 + i] = fmaf(v[i], s1, acc[64 + i]);
        }
        if (!ok) break;
        ok = finish_row<MODE>(p, c, acc, s.amax[flip], r_in_tile, smem_u32(&s.xch[q]), flip, stg);
        if (!ok && lane == 0) fail(s, p, 67);
    }
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

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);        // uniform for the compiler too
    constexpr int BNO = MODE == FB_SWIGLU ? 128 : 256;     // output columns per tile
    if (tid == 0) {
        s.abort_flag = 0;
        for (int i = 0; i < STAGES; ++i) { mbar_init(smem_u32(&s.full[i]), 1); mbar_init(smem_u32(&s.empty[i]), 1); }
        for (int i = 0; i < 2; ++i) { mbar_init(smem_u32(&s.accf[i]), 1); mbar_init(smem_u32(&s.acce[i]), 8); }
        for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&s.xch[i]), 2);
        for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&s.drain[i]), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) tmem_alloc(smem_u32(&s.tmem_base), TMEM_COLS);
    if (tid == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&tmA) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&tmB) : "memory");
    }
    pdl_wait_then_release();
    build_tiles<BNO>(s, p);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const int total = s.tile_start[p.E + (p.has_shared ? 1 : 0)];
    const uint32_t tmem_base = s.tmem_base;

    // registers: launched with 168 a thread (3 x 128 x 168), redistributed as
    // 128 x 56 + 256 x 224, the same total (88 and 208 left the sums 64 bytes of
    // spills: 860 instead of 835 cycles a K block)
    if (warp < 4) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
      if (warp == 0) {
        // ================= TMA producer
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0, issued = 0;
            int g = 0;
            for (int tile = blockIdx.x; tile < total && !aborted(s); tile += gridDim.x) {
                int mt, nt;
                locate(s, tile, g, mt, nt);
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
#pragma unroll
                    for (int u = 0; u < 2; ++u)            // SwiGLU: 128 gate, then 128 up rows
                        tma_load_3d(smB + stage * B_BYTES + u * (B_BYTES / 2), MODE == FB_SWIGLU && u ? mB2 : mB, fb,
                                    kb * BK, MODE == FB_SWIGLU ? nt * 128 : nt * BN + u * 128, e);
                    ++issued;
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
            }
            // every copy has landed before the CTA may end: the last use of each stage
            for (uint32_t i = issued > STAGES ? issued - STAGES : 0; i < issued; ++i)
                if (!mbar_wait(smem_u32(&s.full[i % STAGES]), (i / STAGES) & 1u, p.timeout_ns)) fail(s, p, 65);
        }
      } else if (warp < 3) {
        // ================= MMA issuers: one accumulator per K block, warp 1 the
        // even blocks, warp 2 the odd ones, so that one warp's waits and commits
        // pass while the other's products run.  The whole warp runs the loop, so
        // that descriptors stay in uniform registers; one lane issues (with a
        // single-lane loop the issue took 500 cycles per K block beside the busy
        // sums warps, now 70).
        const uint32_t ab = warp - 1;
        const bool leader = elect_lane();
        const uint64_t da0 = sdesc(smA), db0 = sdesc(smB);
        const uint32_t dtm = tmem_base + ab * BN;
        uint32_t cnt = 0;                                  // K blocks before this tile
        bool ok = true;
        for (int tile = blockIdx.x; tile < total && ok && !aborted(s); tile += gridDim.x) {
            // the shared group, when there is one, is the last
            const uint32_t nk = ((tile >= s.tile_start[p.E] ? p.K_shared : p.K_routed) + BK - 1) / BK;
            uint32_t i = cnt + ((cnt ^ ab) & 1u);
            cnt += nk;
            for (; i < cnt; i += 2) {
                const uint32_t stage = i % STAGES, phase = (i / STAGES) & 1u, aphase = (i >> 1) & 1u;
                if (!warp_wait(smem_u32(&s.acce[ab]), aphase ^ 1u, p.timeout_ns)) { if (leader) fail(s, p, 62); ok = false; break; }
                if (!warp_wait(smem_u32(&s.full[stage]), phase, p.timeout_ns)) { if (leader) fail(s, p, 63); ok = false; break; }
                tc_fence_after();
                const uint64_t da = da0 + stage * (A_BYTES >> 4), db = db0 + stage * (B_BYTES >> 4);
                if (leader) {
#pragma unroll
                    for (int k = 0; k < BK / 32; ++k) mma_e4m3(dtm, da + k * 2, db + k * 2, kIdesc, k ? 1u : 0u);
                    mma_commit(smem_u32(&s.accf[ab]));
                    mma_commit(smem_u32(&s.empty[stage]));
                }
                __syncwarp();
            }
        }
        if (aborted(s) && leader) {                        // products in flight end before TMEM is freed
            mma_commit(smem_u32(&s.drain[ab]));
            if (!mbar_wait(smem_u32(&s.drain[ab]), 0, p.timeout_ns)) fail(s, p, 66);
        }
        __syncwarp();
      }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        // ================= scaled sums and epilogue: warps 4..11
        sums_warps<MODE>(s, p, tmem_base, base + (uint32_t)kStgOff, total);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

// Lets `kernel` use its shared memory, once per device.
template <typename K>
cudaError_t allow_smem(std::atomic<bool> (&done)[64], K kernel) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
    if (e == cudaSuccess) done[dev].store(true, std::memory_order_relaxed);
    return e;
}

// Tensor maps of one product: A and weights.
struct Maps {
    CUtensorMap A, As, B, B2, Bs, Bs2;
};

template <int MODE>
cudaError_t launch_product(const Maps &m, const Params &p, int num_sms, cudaStream_t st, bool pdl) {
    static std::atomic<bool> done[64];
    const cudaError_t e = allow_smem(done, fp8_block_gemm<MODE>);
    if (e != cudaSuccess) return e;
    return launch_kernel(fp8_block_gemm<MODE>, dim3(num_sms), dim3(kThreads), kSmemBytes, st, pdl, m.A, m.As, m.B, m.B2, m.Bs,
                         m.Bs2, p);
}

}  // namespace

cudaError_t launch_ffn_fp8_block(const FfnFp8BlockArgs &a, cudaStream_t st) {
    const bool swiglu = a.act == MOE_ACT_SWIGLU;
    const bool has_sh = a.S > 0 && a.T > 0;
    if (a.routed_rows == 0 && !has_sh) return cudaSuccess;
    if (a.T <= kFp8BlockDecodeT) return launch_ffn_fp8_block_decode(a, st);
    const uint64_t routed = a.routed_rows > 0 ? (uint64_t)a.routed_rows : 1;
    const uint64_t all = (uint64_t)(a.shared_base + (has_sh ? a.T : 0));
    const uint64_t d = a.d, F = a.F, S = a.S;
    // weight boxes of 128 rows: half a tile
    auto weights = [](CUtensorMap *m, const uint8_t *w, uint64_t in, uint64_t out, uint64_t n) {
        return make_map(m, 3, w, in, out, n, in, out * in, 128, 1);
    };
    Maps m1, m2;
    bool ok = make_map(&m1.A, 2, a.x_perm, d, routed, 1, d, 0, BM, 1) && weights(&m1.B, a.W1, d, F, a.E) &&
              make_map(&m2.A, 2, a.H8, F, all, 1, a.hF, 0, BM, 1) && weights(&m2.B, a.W2, F, d, a.E);
    m1.B2 = m1.B;
    if (ok && swiglu) ok = weights(&m1.B2, a.Wu, d, F, a.E);
    m1.As = m1.A; m1.Bs = m1.B; m1.Bs2 = m1.B2;
    m2.As = m2.A; m2.B2 = m2.Bs = m2.Bs2 = m2.B;
    if (ok && has_sh) {
        ok = make_map(&m1.As, 2, a.x, d, a.T, 1, d, 0, BM, 1) && weights(&m1.Bs, a.Wsg, d, S, 1) &&
             make_map(&m2.As, 2, a.H8, S, all, 1, a.hF, 0, BM, 1) && weights(&m2.Bs, a.Wsd, S, d, 1);
        m1.Bs2 = m1.Bs;
        m2.Bs2 = m2.Bs;
        if (ok && swiglu) ok = weights(&m1.Bs2, a.Wsu, d, S, 1);
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
    cudaError_t e = swiglu ? launch_product<FB_SWIGLU>(m1, p, a.num_sms, st, a.pdl)
                           : launch_product<FB_GELU>(m1, p, a.num_sms, st, a.pdl);
    if (e != cudaSuccess) return e;

    p.K_routed = a.F; p.K_shared = a.S; p.N_routed = a.d; p.N_shared = a.d;
    p.sa = p.sa_s = a.h_scale; p.ld_sa = p.ld_sa_s = a.ld_hs;
    p.sw = a.W2s; p.sw2 = nullptr; p.sws = a.Wsds; p.sws2 = nullptr;
    p.shared_a_row = a.shared_base;
    p.bias = swiglu ? nullptr : a.b2;
    p.row_gate = a.row_gate;
    p.out = a.y_perm; p.ldo = a.d;
    p.out_scale = nullptr; p.ld_out_scale = 0;
    return launch_product<FB_DOWN>(m2, p, a.num_sms, st, true);
}

}  // namespace moe
