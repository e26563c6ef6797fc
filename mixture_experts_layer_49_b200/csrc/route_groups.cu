// route_groups.cu -- group-limited expert selection from router logits, and
// the gradient of its gates with respect to the logits.
//
// The E experts form n_group equal groups of consecutive ids (the experts of
// one node or GPU); a token may only use experts of its topk_group best
// groups, which bounds how many places its row travels to:
//   s_e     softmax(l)_e or sigmoid(l_e)
//   key_e   l_e + b_e (softmax) or s_e + b_e (sigmoid); b the selection bias
//   group   the sum of its group_top (1 or 2) largest keys
//   choice  the top_k largest keys inside the topk_group largest groups,
//           best first; equal keys and equal groups go to the lower id
//   gate    c s_e (softmax, renorm 0), else c s_e / sum of the chosen s
// Gates, sums and the score sums are fp32.  Keys are compared as their 64-bit
// values: two fp32 sigmoids plus a bias lie within a rounding of each other
// about once in a thousand tokens of a 256-expert router, and then fp32 keys
// would pick by rounding.  Every token is selected with fp32 keys first; a
// token whose decisive differences are all larger than the keys' error bound
// keeps that result, any other repeats the selection in fp64.
//
// One warp per token, lane l holding experts l * EPT .. l * EPT + EPT - 1, so
// a group of 8 * 2^i experts is a power-of-two run of lanes and its best two
// keys meet in a few shuffles.  The floor is the logits read once; the
// selection's instructions bound it (k rounds of redux.sync).
#include "common.cuh"
#include "kernels.cuh"

namespace moe {

namespace {

constexpr int kBlockTok = 32;      // tokens per block: one row of the score sums
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}
__device__ __forceinline__ float warp_min(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fminf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// Order-preserving images of a key: 0 an expert that may not be chosen, 1 a
// NaN key (below every number), else the number's.
__device__ __forceinline__ uint32_t image(float f) {
    if (f != f) return 1u;
    f += 0.f;                                      // -0 and +0 are the same key
    const uint32_t u = __float_as_uint(f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float number(uint32_t u) {
    return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}
__device__ __forceinline__ uint64_t image(double f) {
    if (f != f) return 1ull;
    f += 0.0;
    const uint64_t u = (uint64_t)__double_as_longlong(f);
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

template <typename F>
__device__ __forceinline__ F low() { return (F)(-INFINITY); }

// The best two of two sorted pairs.
template <typename F>
__device__ __forceinline__ void merge2(F &a, F &b, F oa, F ob) {
    const F lo = a < oa ? a : oa;
    a = a < oa ? oa : a;
    b = b < ob ? ob : b;
    b = b < lo ? lo : b;
}

// Which of this lane's experts lie in the topk_group best groups (bit j:
// expert lane * EPT + j).  worst_kept / best_dropped: the two scores that the
// decision lies between.
template <int EPT, typename F>
__device__ __forceinline__ uint32_t kept_experts(const RouteArgs &a, const F (&key)[EPT], F *worst_kept,
                                                 F *best_dropped) {
    const int lane = threadIdx.x & 31;
    const int size = a.E / a.n_group;
    F wk = (F)INFINITY, bd = low<F>();
    uint32_t mask = 0;
    const int lanes = size / EPT;                  // lanes per group when a lane never spans two
    if (size % EPT == 0 && (lanes & (lanes - 1)) == 0) {
        F t1 = low<F>(), t2 = low<F>();
#pragma unroll
        for (int j = 0; j < EPT; ++j) {
            const F v = (lane * EPT + j < a.E && key[j] == key[j]) ? key[j] : low<F>();
            merge2(t1, t2, v, low<F>());
        }
        for (int o = 1; o < lanes; o <<= 1) {
            const F o1 = __shfl_xor_sync(kAll, t1, o), o2 = __shfl_xor_sync(kAll, t2, o);
            merge2(t1, t2, o1, o2);
        }
        F mine = a.group_top == 2 ? t1 + t2 : t1;
        if (mine != mine) mine = low<F>();         // +inf and -inf
        const int g = lane / lanes;
        int rank = 0;
        for (int q = 0; q < a.n_group; ++q) {
            const F s = __shfl_sync(kAll, mine, q * lanes);
            rank += (s > mine || (s == mine && q < g)) ? 1 : 0;
        }
        if (g < a.n_group) {
            if (rank < a.topk_group) { mask = (1u << EPT) - 1u; wk = mine; } else { bd = mine; }
        }
    } else {
        // any size: group by group over the whole warp; lane q % 32 keeps the
        // scores of groups q, q + 32, ... (n_group <= 256)
        F mine[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) mine[i] = low<F>();
        for (int q = 0; q < a.n_group; ++q) {
            F t1 = low<F>(), t2 = low<F>();
#pragma unroll
            for (int j = 0; j < EPT; ++j) {
                const int e = lane * EPT + j;
                if (e >= q * size && e < (q + 1) * size && key[j] == key[j]) merge2(t1, t2, key[j], low<F>());
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const F o1 = __shfl_xor_sync(kAll, t1, o), o2 = __shfl_xor_sync(kAll, t2, o);
                merge2(t1, t2, o1, o2);
            }
            F s = a.group_top == 2 ? t1 + t2 : t1;
            if (s != s) s = low<F>();
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (q == i * 32 + lane) mine[i] = s;
        }
        for (int q = 0; q < a.n_group; ++q) {
            F s = low<F>();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const F v = __shfl_sync(kAll, mine[i], q & 31);
                if (i == (q >> 5)) s = v;
            }
            int rank = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int p = i * 32 + lane;
                if (p < a.n_group && (mine[i] > s || (mine[i] == s && p < q))) ++rank;
            }
            rank = __reduce_add_sync(kAll, rank);
            if (rank < a.topk_group) {
                wk = s < wk ? s : wk;
#pragma unroll
                for (int j = 0; j < EPT; ++j) {
                    const int e = lane * EPT + j;
                    if (e >= q * size && e < (q + 1) * size) mask |= 1u << j;
                }
            } else {
                bd = s > bd ? s : bd;
            }
        }
    }
    *worst_kept = wk;
    *best_dropped = bd;
    return mask;
}

// Compare-exchange and sorting networks for a lane's candidates: key image
// descending, then id ascending (ids ascend within a lane, networks keep the
// order by comparing them).
__device__ __forceinline__ void cex(uint32_t &ka, int &ia, uint32_t &kb, int &ib) {
    const bool sw = ka < kb || (ka == kb && ia > ib);
    const uint32_t tk = sw ? kb : ka;
    kb = sw ? ka : kb;
    ka = tk;
    const int ti = sw ? ib : ia;
    ib = sw ? ia : ib;
    ia = ti;
}
template <int EPT>
__device__ __forceinline__ void lane_sort(uint32_t (&k)[EPT], int (&id)[EPT]) {
#define CEX(i, j) cex(k[i], id[i], k[j], id[j])
    if constexpr (EPT == 2) {
        CEX(0, 1);
    } else if constexpr (EPT == 4) {
        CEX(0, 1); CEX(2, 3); CEX(0, 2); CEX(1, 3); CEX(1, 2);
    } else if constexpr (EPT == 8) {
        CEX(0, 1); CEX(2, 3); CEX(4, 5); CEX(6, 7);
        CEX(0, 2); CEX(1, 3); CEX(4, 6); CEX(5, 7);
        CEX(1, 2); CEX(5, 6);
        CEX(0, 4); CEX(1, 5); CEX(2, 6); CEX(3, 7);
        CEX(2, 4); CEX(3, 5);
        CEX(1, 2); CEX(3, 4); CEX(5, 6);
    }
#undef CEX
}

// Logits of token t, offset included: `splits` partial planes added in order.
template <int EPT>
__device__ __forceinline__ void load_logits(const RouteArgs &a, int t, float (&h)[EPT]) {
    const int lane = threadIdx.x & 31;
    const float *p = a.logits + (size_t)t * a.E + lane * EPT;
    const size_t plane = (size_t)a.T * a.E;
    if (a.vec) {                                   // E % EPT == 0 and aligned: whole vectors
        constexpr int W = EPT < 4 ? EPT : 4;
#pragma unroll
        for (int j = 0; j < EPT; ++j) h[j] = -INFINITY;
        if (lane * EPT < a.E) {
            for (int s = 0; s < a.splits; ++s) {
#pragma unroll
                for (int q = 0; q < EPT; q += W) {
                    float f[4];
                    if constexpr (W == 4) {
                        const float4 v = *reinterpret_cast<const float4 *>(p + q);
                        f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
                    } else if constexpr (W == 2) {
                        const float2 v = *reinterpret_cast<const float2 *>(p + q);
                        f[0] = v.x; f[1] = v.y;
                    } else {
                        f[0] = p[q];
                    }
#pragma unroll
                    for (int j = 0; j < W; ++j) h[q + j] = s == 0 ? f[j] : h[q + j] + f[j];
                }
                p += plane;
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < EPT; ++j) {
            h[j] = -INFINITY;
            if (lane * EPT + j < a.E) {
                h[j] = p[j];
                for (int s = 1; s < a.splits; ++s) h[j] += p[s * plane + j];
            }
        }
    }
}

// The selection with 64-bit keys: k rounds, each the largest key over the
// warp (high word, then low word, then lowest id).  It reads the token's
// logits again, so that the common path keeps its own in registers.
template <int EPT>
__device__ __noinline__ int select_exact(const RouteArgs &a, int t) {
    const int lane = threadIdx.x & 31;
    float h[EPT];
    load_logits<EPT>(a, t, h);
    double key[EPT];
#pragma unroll
    for (int j = 0; j < EPT; ++j) {
        const double l = (double)h[j];
        key[j] = a.score == MOE_SCORE_SOFTMAX ? l : 1.0 / (1.0 + exp(-l));
        if (a.sel_bias && lane * EPT + j < a.E) key[j] += (double)a.sel_bias[lane * EPT + j];
    }
    double wk, bd;
    const uint32_t mask = kept_experts<EPT, double>(a, key, &wk, &bd);
    uint64_t im[EPT];
#pragma unroll
    for (int j = 0; j < EPT; ++j) im[j] = (lane * EPT + j < a.E && (mask >> j & 1u)) ? image(key[j]) : 0ull;
    int my_id = 0;
    for (int r = 0; r < a.k; ++r) {
        uint64_t best = im[0];
        int at = 0;
#pragma unroll
        for (int j = 1; j < EPT; ++j)
            if (im[j] > best) { best = im[j]; at = j; }
        const uint32_t hi = __reduce_max_sync(kAll, (uint32_t)(best >> 32));
        const uint32_t lo = __reduce_max_sync(kAll, (uint32_t)(best >> 32) == hi ? (uint32_t)best : 0u);
        const bool mine = best == ((uint64_t)hi << 32 | lo);
        const uint32_t id = __reduce_min_sync(kAll, mine ? (uint32_t)(lane * EPT + at) : kAll);
        if (lane == r) my_id = (int)id;
#pragma unroll
        for (int j = 0; j < EPT; ++j)
            if ((uint32_t)(lane * EPT + j) == id) im[j] = 0ull;
    }
    return my_id;
}

// Scores of the lane's experts (0 for absent ones) and the factor that makes
// them shares of 1.  A row whose logits are all -inf has no scores: all 0.
template <int EPT>
__device__ __forceinline__ float scores(int score, int E, const float (&h)[EPT], float (&s)[EPT]) {
    const int lane = threadIdx.x & 31;
    float z = 0.f;
    if (score == MOE_SCORE_SOFTMAX) {
        float m = -INFINITY;
#pragma unroll
        for (int j = 0; j < EPT; ++j) m = fmaxf(m, h[j]);
        m = warp_max(m);
        if (m == -INFINITY) m = 0.f;
#pragma unroll
        for (int j = 0; j < EPT; ++j) { s[j] = lane * EPT + j < E ? expf(h[j] - m) : 0.f; z += s[j]; }
    } else {
#pragma unroll
        for (int j = 0; j < EPT; ++j) {
            s[j] = lane * EPT + j < E ? 1.f / (1.f + expf(-h[j])) : 0.f;
            z += s[j];
        }
    }
    z = warp_sum(z);
    return z == 0.f ? 0.f : 1.f / z;
}

// v of expert e (lane e / EPT, register e % EPT) for every lane's own e.
template <int EPT>
__device__ __forceinline__ float of_expert(const float (&v)[EPT], int e) {
    float f = 0.f;
#pragma unroll
    for (int j = 0; j < EPT; ++j) {
        const float t = __shfl_sync(kAll, v[j], (e / EPT) & 31);
        if (e % EPT == j) f = t;
    }
    return f;
}

template <int EPT, int WARPS>
__global__ void __launch_bounds__(WARPS * 32) route_select_kernel(const __grid_constant__ RouteArgs a) {
    pdl_wait_then_release();
    __shared__ float part[WARPS][EPT * 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool softmax = a.score == MOE_SCORE_SOFTMAX;
    float sb[EPT], share[EPT];
#pragma unroll
    for (int j = 0; j < EPT; ++j) {
        sb[j] = (a.sel_bias && lane * EPT + j < a.E) ? __ldg(a.sel_bias + lane * EPT + j) : 0.f;
        share[j] = 0.f;
    }
    for (int i = 0; i < kBlockTok / WARPS; ++i) {
        const int t = blockIdx.x * kBlockTok + warp * (kBlockTok / WARPS) + i;
        if (t >= a.T) break;                       // uniform over the warp
        float h[EPT], s[EPT], key[EPT];
        load_logits<EPT>(a, t, h);
        if (a.logits_out) {
#pragma unroll
            for (int j = 0; j < EPT; ++j)
                if (lane * EPT + j < a.E) a.logits_out[(size_t)t * a.E + lane * EPT + j] = h[j];
        }
        const float inv = scores<EPT>(a.score, a.E, h, s);
        // Error bounds of a key.  Sigmoid: expf within 2 ulp moves s by at most
        // s (1 - s) 2^-22 <= 2^-24, the sum and the quotient round by 2^-24
        // each, so 3 * 2^-24, plus half an ulp of the sum with the bias;
        // softmax: half an ulp of that sum.  Two keys further apart than twice
        // the bound (here taken 2.6 times and 2 times wider) are in order.
        const float tol_abs = softmax ? 0.f : 0x1p-20f;
        const float tol_rel = (softmax && !a.sel_bias) ? 0.f : 0x1p-22f;
#pragma unroll
        for (int j = 0; j < EPT; ++j) {
            share[j] += s[j] * inv;
            if (softmax) s[j] *= inv;
            const float k0 = softmax ? h[j] : s[j];
            key[j] = a.sel_bias ? k0 + sb[j] : k0;
        }
        bool close = false;
        uint32_t mask = kAll;
        if (a.n_group > 1 && a.topk_group < a.n_group) {
            float wk, bd, most = 0.f;
            mask = kept_experts<EPT, float>(a, key, &wk, &bd);
#pragma unroll
            for (int j = 0; j < EPT; ++j)
                if (fabsf(key[j]) < INFINITY) most = fmaxf(most, fabsf(key[j]));
            most = warp_max(most);
            wk = warp_min(wk);
            bd = warp_max(bd);
            // a score sums two keys of at most `most`: per score the bounds of
            // both and a rounding of 2^-24 * 2 most, 2^-21 most for two scores
            close = wk - bd < 2.f * tol_abs + 0x1p-20f * most;
        }
        uint32_t im[EPT];
        int id[EPT];
#pragma unroll
        for (int j = 0; j < EPT; ++j) {
            id[j] = lane * EPT + j;
            im[j] = (id[j] < a.E && (mask >> j & 1u)) ? image(key[j]) : 0u;
        }
        lane_sort<EPT>(im, id);
        int my_id = 0;
        float before = 0.f;
        for (int r = 0; r <= a.k; ++r) {           // round k only looks at the best key left out
            const uint32_t top = __reduce_max_sync(kAll, im[0]);
            if (r > 0 && top > 1u) {
                const float now = number(top);
                close = close || before - now < tol_abs + tol_rel * fmaxf(fabsf(before), fabsf(now));
            }
            if (r == a.k || top == 0u) break;
            before = top == 1u ? -INFINITY : number(top);
            const uint32_t e = __reduce_min_sync(kAll, im[0] == top ? (uint32_t)id[0] : kAll);
            if (lane == r) my_id = (int)e;
            if (im[0] == top && (uint32_t)id[0] == e) {
#pragma unroll
                for (int j = 0; j + 1 < EPT; ++j) { im[j] = im[j + 1]; id[j] = id[j + 1]; }
                im[EPT - 1] = 0u;
                id[EPT - 1] = 0x7fffffff;
            }
        }
        if (close) my_id = select_exact<EPT>(a, t);      // uniform: every lane sees the same keys
        const float g = of_expert<EPT>(s, my_id);
        float f = a.gate_scale;
        if (!softmax || a.renorm) {
            const float sum = warp_sum(lane < a.k ? g : 0.f);
            f = sum == 0.f ? 0.f : g / sum * a.gate_scale;   // no scores left: gates of 0
        } else {
            f = g * a.gate_scale;
        }
        if (lane < a.k) {
            a.idx[(size_t)t * a.k + lane] = my_id;
            a.gate[(size_t)t * a.k + lane] = f;
        }
    }
    if (a.psum == nullptr) return;
#pragma unroll
    for (int j = 0; j < EPT; ++j) part[warp][lane * EPT + j] = share[j];
    __syncthreads();
    for (int e = tid; e < a.E; e += WARPS * 32) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) v += part[w][e];
        a.psum[(size_t)blockIdx.x * a.E + e] = v;
    }
}

// dlogits of ell = sum dgate * gate + alpha * E * sum_e f_e P_e; the choice of
// experts and f_e = counts_e / (T k) carry no gradient.  With ds the gradient
// of the scores: softmax dl = s (ds - <ds, s>), sigmoid dl = ds s (1 - s).
template <int EPT>
__global__ void __launch_bounds__(256) route_bwd_kernel(RouteBwdArgs a) {
    pdl_wait_then_release();
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (t >= a.T) return;
    const bool softmax = a.score == MOE_SCORE_SOFTMAX;
    RouteArgs ra{};
    ra.logits = a.logits; ra.T = a.T; ra.E = a.E; ra.splits = 1; ra.vec = a.vec;
    float h[EPT], s[EPT], ds[EPT];
    load_logits<EPT>(ra, t, h);
    const float inv = scores<EPT>(a.score, a.E, h, s);
    int e = -1;
    float dg = 0.f;
    if (lane < a.k) {
        e = a.idx[(size_t)t * a.k + lane];
        dg = a.dgate[(size_t)t * a.k + lane] * a.gate_scale;
    }
    const bool used = e >= 0 && e < a.E;           // an id out of range carries no gradient
    if (!used) { e = 0; dg = 0.f; }
#pragma unroll
    for (int j = 0; j < EPT; ++j) {
        if (softmax) s[j] *= inv;
        ds[j] = 0.f;
    }
    if (!softmax || a.renorm) {
        const float sv = of_expert<EPT>(s, e);
        const float sum = warp_sum(used ? sv : 0.f);
        const float g = sum == 0.f ? 0.f : sv / sum;
        const float dot = warp_sum(dg * g);
        dg = (used && sum != 0.f) ? (dg - dot) / sum : 0.f;
    }
    for (int r = 0; r < a.k; ++r) {
        const int er = __shfl_sync(kAll, e, r);
        const float v = __shfl_sync(kAll, dg, r);
#pragma unroll
        for (int j = 0; j < EPT; ++j)
            if (er == lane * EPT + j) ds[j] += v;
    }
    if (a.alpha != 0.f) {
        const float c = (float)((double)a.alpha * a.E / a.T / ((double)a.T * a.k));
        float cf[EPT], dot = 0.f;
#pragma unroll
        for (int j = 0; j < EPT; ++j) {
            cf[j] = lane * EPT + j < a.E ? c * (float)__ldg(a.counts + lane * EPT + j) : 0.f;
            dot += cf[j] * s[j];
        }
        if (softmax) {
#pragma unroll
            for (int j = 0; j < EPT; ++j) ds[j] += cf[j];
        } else {
            dot = warp_sum(dot) * inv;
#pragma unroll
            for (int j = 0; j < EPT; ++j) ds[j] += (cf[j] - dot) * inv;
        }
    }
    float dot = 0.f;
    if (softmax) {
#pragma unroll
        for (int j = 0; j < EPT; ++j) dot += ds[j] * s[j];
        dot = warp_sum(dot);
    }
#pragma unroll
    for (int j = 0; j < EPT; ++j) {
        if (softmax) ds[j] = s[j] * (ds[j] - dot);
        else ds[j] *= s[j] * (1.f / (1.f + expf(h[j])));     // 1 - s without its cancellation near s = 1
    }
    float *o = a.dlogits + (size_t)t * a.E + lane * EPT;
    if (EPT >= 4 && a.vec_out) {
        if (lane * EPT < a.E)
#pragma unroll
            for (int q = 0; q + 3 < EPT; q += 4)
                *reinterpret_cast<float4 *>(o + q) = make_float4(ds[q], ds[q + 1], ds[q + 2], ds[q + 3]);
    } else {
#pragma unroll
        for (int j = 0; j < EPT; ++j)
            if (lane * EPT + j < a.E) o[j] = ds[j];
    }
}

constexpr int kSelWarps = 32;

// A row of E fp32 values splits into whole aligned vectors of the lanes.
int vector_rows(const void *p, int E) {
    const int ept = E <= 32 ? 1 : (E <= 64 ? 2 : (E <= 128 ? 4 : 8));
    const int w = ept < 4 ? ept : 4;
    return E % ept == 0 && reinterpret_cast<uintptr_t>(p) % (4 * w) == 0;
}

}  // namespace

cudaError_t launch_route_select(const RouteArgs &in, cudaStream_t st) {
    if (in.T == 0) return cudaSuccess;
    RouteArgs a = in;
    a.vec = vector_rows(a.logits, a.E);
    const dim3 grid((unsigned)((a.T + kBlockTok - 1) / kBlockTok)), block(kSelWarps * 32);
    if (a.E <= 32) return launch_kernel(route_select_kernel<1, kSelWarps>, grid, block, 0, st, a.pdl, a);
    if (a.E <= 64) return launch_kernel(route_select_kernel<2, kSelWarps>, grid, block, 0, st, a.pdl, a);
    if (a.E <= 128) return launch_kernel(route_select_kernel<4, kSelWarps>, grid, block, 0, st, a.pdl, a);
    return launch_kernel(route_select_kernel<8, kSelWarps>, grid, block, 0, st, a.pdl, a);
}

cudaError_t launch_route_bwd(const RouteBwdArgs &in, cudaStream_t st) {
    if (in.T == 0) return cudaSuccess;
    RouteBwdArgs a = in;
    a.vec = vector_rows(a.logits, a.E);
    a.vec_out = vector_rows(a.dlogits, a.E);
    const dim3 grid((unsigned)((a.T + 7) / 8)), block(256);
    if (a.E <= 32) return launch_kernel(route_bwd_kernel<1>, grid, block, 0, st, a.pdl, a);
    if (a.E <= 64) return launch_kernel(route_bwd_kernel<2>, grid, block, 0, st, a.pdl, a);
    if (a.E <= 128) return launch_kernel(route_bwd_kernel<4>, grid, block, 0, st, a.pdl, a);
    return launch_kernel(route_bwd_kernel<8>, grid, block, 0, st, a.pdl, a);
}

}  // namespace moe
