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
// keys meet in a few shuffles.  For the rounds of the choice a candidate is one
// 32-bit word: the upper 24 bits of the fp32 distance of its key from the row's
// largest, then its id, so one redux.sync.min finds the best candidate with the
// lowest id, and a lane's candidates sort with plain minima and maxima.
//
// The floor is the logits read once (2.8 us for 16384 x 256).  What bounds it is
// the latency of a token's serial rounds (8 groups of which 4 are kept, k = 8), with
// 60 % of the issue slots used, at a register limit that keeps 32 warps on an SM:
// 22.0 us there, 13.0 us for 16384 x 128 softmax without groups, 5.6 us for 16 tokens
// of 256.  Rows whose keys all tie, or that choose keys of -inf, repeat the selection
// in 64 bits: 76 us for 16384 x 256 equal sigmoids, 44 for 16384 x 128 equal logits.
// With 85 registers and 24 warps the fp32 path took 22.5 instead of 20.6, 13.9 instead
// of 12.4 and 5.3 instead of 5.5.  Rounds over 64-bit keys took 50 us; the doubtful
// tokens in a pass of their own after the others 23 (14.4 against 7.5 for 1000
// tokens).
#include "common.cuh"
#include "kernels.cuh"

namespace moe {

namespace {

constexpr int kBlockTok = 32;      // tokens per block: one row of the score sums
constexpr unsigned kAll = 0xffffffffu;

// Largest value over the warp (NaN only where every lane holds one).
__device__ __forceinline__ float redux_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// Order-preserving image of a number; NaN counts as +inf.
__device__ __forceinline__ uint32_t ordered(float f) {
    const uint32_t u = __float_as_uint(f != f ? INFINITY : f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
// The same of a key: 0 an expert that may not be chosen, 1 a NaN key (below every
// number), else the number's.
__device__ __forceinline__ uint64_t image(double f) {
    if (f != f) return 1ull;
    f += 0.0;                                      // -0 and +0 are the same key
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

// How far a group's score is off (an infinite one not at all).
template <typename F>
__device__ __forceinline__ F score_error(const RouteArgs &a, F score, F t1, F t2, F abs, F rel) {
    if (!(fabs(score) < (F)INFINITY)) return (F)0;
    return a.group_top == 2 ? (F)2 * abs + rel * (fabs(t1) + fabs(t2)) : abs + rel * fabs(t1);
}

// Which of this lane's experts lie in the topk_group best groups (bit j: expert
// lane * EPT + j).  With keys off by at most abs + rel |key|: *close, whether a
// kept and a dropped group's scores could be in the other order.
template <int EPT, typename F>
__device__ __forceinline__ uint32_t kept_experts(const RouteArgs &a, const F (&key)[EPT], F abs, F rel, bool *close) {
    const int lane = threadIdx.x & 31;
    const int size = a.E / a.n_group;
    F wk = (F)INFINITY, bd = low<F>();             // least kept and greatest dropped score, error taken off and added
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
        const F err = score_error(a, mine, t1, t2, abs, rel);
        const int g = lane / lanes;
        int rank = 0;
        for (int q = 0; q < a.n_group; ++q) {
            const F s = __shfl_sync(kAll, mine, q * lanes);
            rank += (s > mine || (s == mine && q < g)) ? 1 : 0;
        }
        if (g < a.n_group) {
            if (rank < a.topk_group) { mask = (1u << EPT) - 1u; wk = mine - err; } else { bd = mine + err; }
        }
    } else {
        // any size: group by group over the whole warp; lane q % 32 keeps the
        // scores of groups q, q + 32, ... (n_group <= 256)
        F mine[8], err[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) { mine[i] = low<F>(); err[i] = (F)0; }
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
                if (q == i * 32 + lane) {
                    mine[i] = s;
                    err[i] = score_error(a, s, t1, t2, abs, rel);
                }
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
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (q == i * 32 + lane) {
                    if (rank < a.topk_group) wk = mine[i] - err[i] < wk ? mine[i] - err[i] : wk;
                    else bd = mine[i] + err[i] > bd ? mine[i] + err[i] : bd;
                }
            if (rank < a.topk_group)
#pragma unroll
                for (int j = 0; j < EPT; ++j) {
                    const int e = lane * EPT + j;
                    if (e >= q * size && e < (q + 1) * size) mask |= 1u << j;
                }
        }
    }
    *close = false;
    if constexpr (sizeof(F) == 4) {                // fp64 keys decide; a NaN bound (infinite scores) compares false: not close
        uint32_t lo = ordered((float)wk), hi = ordered((float)bd);
        lo = __reduce_min_sync(kAll, lo);
        hi = __reduce_max_sync(kAll, hi);
        // an infinite one may be a sum that passed the fp32 range: 64 bits tell
        *close = lo < hi || lo == ordered(-INFINITY) || hi == ordered(INFINITY);
    }
    return mask;
}

// Ascending sorting networks of a lane's candidates (Batcher's odd-even merge
// sort for 8).
template <int EPT>
__device__ __forceinline__ void lane_sort(uint32_t (&v)[EPT]) {
#define CEX(i, j) { const uint32_t lo = min(v[i], v[j]); v[j] = max(v[i], v[j]); v[i] = lo; }
    if constexpr (EPT == 2) {
        CEX(0, 1)
    } else if constexpr (EPT == 4) {
        CEX(0, 1) CEX(2, 3) CEX(0, 2) CEX(1, 3) CEX(1, 2)
    } else if constexpr (EPT == 8) {
        CEX(0, 1) CEX(2, 3) CEX(4, 5) CEX(6, 7)
        CEX(0, 2) CEX(1, 3) CEX(4, 6) CEX(5, 7)
        CEX(1, 2) CEX(5, 6)
        CEX(0, 4) CEX(1, 5) CEX(2, 6) CEX(3, 7)
        CEX(2, 4) CEX(3, 5)
        CEX(1, 2) CEX(3, 4) CEX(5, 6)
    }
#undef CEX
}

// Logits of token t, offset included: `splits` partial planes added in order.
// FULL: E = 32 EPT and rows of whole aligned vectors, so no lane is short.
template <int EPT, bool FULL>
__device__ __forceinline__ void load_logits(const RouteArgs &a, int t, float (&h)[EPT]) {
    const int lane = threadIdx.x & 31;
    const float *p = a.logits + (size_t)t * a.E + lane * EPT;
    const size_t plane = (size_t)a.T * a.E;
    if (FULL || a.vec) {                           // E % EPT == 0 and aligned: whole vectors
        constexpr int W = EPT < 4 ? EPT : 4;
        if (!FULL)
#pragma unroll
            for (int j = 0; j < EPT; ++j) h[j] = -INFINITY;
        if (FULL || lane * EPT < a.E) {
#pragma unroll
            for (int q = 0; q < EPT; q += W) {
                if constexpr (W == 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(p + q);
                    h[q] = v.x; h[q + 1] = v.y; h[q + 2] = v.z; h[q + 3] = v.w;
                } else if constexpr (W == 2) {
                    const float2 v = *reinterpret_cast<const float2 *>(p + q);
                    h[q] = v.x; h[q + 1] = v.y;
                } else {
                    h[q] = p[q];
                }
            }
            for (int s = 1; s < a.splits; ++s)
#pragma unroll
                for (int j = 0; j < EPT; ++j) h[j] += p[s * plane + j];
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
    load_logits<EPT, false>(a, t, h);
    double key[EPT];
#pragma unroll
    for (int j = 0; j < EPT; ++j) {
        const double l = (double)h[j];
        key[j] = a.score == MOE_SCORE_SOFTMAX ? l : 1.0 / (1.0 + exp(-l));
        if (a.sel_bias && lane * EPT + j < a.E) key[j] += (double)a.sel_bias[lane * EPT + j];
    }
    bool close;
    const uint32_t mask = a.topk_group < a.n_group ? kept_experts<EPT, double>(a, key, 0.0, 0.0, &close) : kAll;
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

// 1 / (1 + exp(-l)) within 7 * 2^-24 of its value (expf 4, the sum 1, the reciprocal
// 2); 0 below -88.72, where exp(-l) passes the largest fp32 number.
__device__ __forceinline__ float sigmoid(float l) {
    float s;
    asm("rcp.approx.f32 %0, %1;" : "=f"(s) : "f"(1.f + expf(-l)));
    return s;
}

// Scores of the lane's experts (0 for absent ones) and the factor that makes
// them shares of 1.  A row whose logits are all -inf has no scores: all 0.
// Sigmoids that are tiny everywhere come times 2^64 (their ratios count), so
// that the factor stays finite.
template <int EPT>
__device__ __forceinline__ float scores(int score, int E, const float (&h)[EPT], float (&s)[EPT]) {
    const int lane = threadIdx.x & 31;
    float z = 0.f;
    if (score == MOE_SCORE_SOFTMAX) {
        float m = -INFINITY;
#pragma unroll
        for (int j = 0; j < EPT; ++j) m = fmaxf(m, h[j]);
        m = redux_max(m);
        if (m == -INFINITY) m = 0.f;
#pragma unroll
        for (int j = 0; j < EPT; ++j) { s[j] = lane * EPT + j < E ? expf(h[j] - m) : 0.f; z += s[j]; }
    } else {
#pragma unroll
        for (int j = 0; j < EPT; ++j) {
            s[j] = lane * EPT + j < E ? sigmoid(h[j]) : 0.f;
            z += s[j];
        }
    }
    z = warp_sum(z);
    if (z < 0x1p-64f && score != MOE_SCORE_SOFTMAX) {
        z *= 0x1p64f;
#pragma unroll
        for (int j = 0; j < EPT; ++j) s[j] *= 0x1p64f;
    }
    return z == 0.f ? 0.f : 1.f / z;
}

// A lane's registers to and from its warp's row in shared memory.
template <int EPT>
__device__ __forceinline__ void put_row(float *row, const float (&v)[EPT]) {
    const int lane = threadIdx.x & 31;
    if constexpr (EPT >= 4) {
#pragma unroll
        for (int j = 0; j < EPT; j += 4)
            *reinterpret_cast<float4 *>(row + lane * EPT + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
    } else {
#pragma unroll
        for (int j = 0; j < EPT; ++j) row[lane * EPT + j] = v[j];
    }
    __syncwarp();
}
template <int EPT>
__device__ __forceinline__ void get_row(const float *row, float (&v)[EPT]) {
    const int lane = threadIdx.x & 31;
    if constexpr (EPT >= 4) {
#pragma unroll
        for (int j = 0; j < EPT; j += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(row + lane * EPT + j);
            v[j] = f.x; v[j + 1] = f.y; v[j + 2] = f.z; v[j + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < EPT; ++j) v[j] = row[lane * EPT + j];
    }
}

// The 64-bit key of a logit.
__device__ __forceinline__ double key64(const RouteArgs &a, float l, int e) {
    const double k = a.score == MOE_SCORE_SOFTMAX ? (double)l : 1.0 / (1.0 + exp(-(double)l));
    return a.sel_bias ? k + (double)a.sel_bias[e] : k;
}
__device__ __forceinline__ float one_logit(const RouteArgs &a, int t, int e) {
    const float *p = a.logits + (size_t)t * a.E + e;
    float h = p[0];
    for (int s = 1; s < a.splits; ++s) h += p[(size_t)s * a.T * a.E];
    return h;
}

// Error bounds.  A sigmoid key: expf is off by 4 * 2^-24 of its value (2 ulp), which
// moves s by s (1 - s) of that, at most 2^-24; the sum is off by 2^-24 and the
// reciprocal by 2 * 2^-24: together at most 4 * 2^-24 (s <= 1); the sum with the bias
// by 2^-24 of it.  A softmax key: the latter alone.  Two distances from the best key
// mx: besides their keys, cut off at 2^-15 of them and one rounding (and 2^-140, what
// the cut takes off a subnormal one).
struct Bounds {
    float abs, rel;                                // of a key
    __device__ __forceinline__ explicit Bounds(const RouteArgs &a)
        : abs(a.score == MOE_SCORE_SOFTMAX ? 0.f : 0x1p-22f),
          rel(a.score == MOE_SCORE_SOFTMAX && !a.sel_bias ? 0.f : 0x1p-23f) {}
    __device__ __forceinline__ float two(float mx) const { return 2.f * abs + 2.f * rel * fabsf(mx) + 0x1p-140f; }
    __device__ __forceinline__ float two_rel() const { return 0x1.2p-14f + 2.f * rel; }
};

// A lane's candidates: 24 bits of the distance from the best key (a NaN key's is
// NaN, above all others), then the id.
template <int EPT, bool FULL>
__device__ __forceinline__ void candidates(const RouteArgs &a, const float (&key)[EPT], float mx, uint32_t (&v)[EPT]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < EPT; ++j) {
        const uint32_t e = lane * EPT + j;
        v[j] = FULL || e < (uint32_t)a.E ? (__float_as_uint(mx - key[j]) & 0x7fffff00u) | e : kAll;
    }
}
__device__ __forceinline__ float distance(uint32_t word) { return __uint_as_float(word & 0x7fffff00u); }

// Takes the best candidate over the warp out of its lane's sorted list.
template <int EPT>
__device__ __forceinline__ uint32_t take_best(uint32_t (&v)[EPT]) {
    const uint32_t top = __reduce_min_sync(kAll, v[0]);
    const bool win = v[0] == top;
#pragma unroll
    for (int j = 0; j + 1 < EPT; ++j) v[j] = win ? v[j + 1] : v[j];
    v[EPT - 1] = win ? kAll : v[EPT - 1];
    return top;
}

// The topk_group best groups where a lane's candidates (sorted, best first) belong
// to one group and a group is `lanes` (a power of two) neighbouring lanes: the sum
// of a group's best distances, its id in the low 8 bits, and one redux per kept
// group.  Whether this lane's group is kept; *close: whether the border is within
// the bounds.
template <int EPT>
__device__ __forceinline__ bool kept_lane(const RouteArgs &a, int lanes, const uint32_t (&v)[EPT], float two,
                                          float two_rel, bool *close) {
    const int lane = threadIdx.x & 31;
    uint32_t t1 = v[0], t2 = EPT > 1 ? v[EPT > 1 ? 1 : 0] : kAll;
    for (int o = 1; o < lanes; o <<= 1) {
        const uint32_t o1 = __shfl_xor_sync(kAll, t1, o), o2 = __shfl_xor_sync(kAll, t2, o);
        t2 = min(max(t1, o1), min(t2, o2));
        t1 = min(t1, o1);
    }
    // a NaN distance (NaN key) counts as +inf, as in the exact selection
    const float d = fminf(distance(t1), INFINITY) + (a.group_top == 2 ? fminf(distance(t2), INFINITY) : 0.f);
    const int g = lane / lanes;
    uint32_t word = g < a.n_group ? (__float_as_uint(d) & 0x7fffff00u) | (uint32_t)g : kAll;
    bool kept = false;
    uint32_t top = kAll;
    for (int r = 0; r < a.topk_group; ++r) {
        top = __reduce_min_sync(kAll, word);
        if (word == top) { kept = true; word = kAll; }
    }
    const float last = distance(top), next = distance(__reduce_min_sync(kAll, word));
    // two keys a score; each distance and the sum cut off at 2^-15
    // (a sum past the fp32 range says nothing beside one near it)
    *close = next < INFINITY ? next - last < 2.f * two + 2.f * two_rel * next : !(last < 0x1p127f);
    return kept;
}

// The best a.k of n <= 31 candidates (lane r < n holds one) by their 64-bit keys:
// lane r's chosen id of rank r.
__device__ __forceinline__ int rank_exact(const RouteArgs &a, int t, uint32_t mine, int n) {
    const int lane = threadIdx.x & 31;
    const int id = lane < n ? (int)(mine & 255u) : 0;
    const uint64_t im = image(key64(a, one_logit(a, t, id), id));
    int rank = 0;
    for (int q = 0; q < n; ++q) {
        const uint64_t o = __shfl_sync(kAll, im, q);
        const int oid = __shfl_sync(kAll, id, q);
        rank += (o > im || (o == im && oid < id)) ? 1 : 0;
    }
    if (lane >= n) rank = 31;
    int chosen = 0;
    for (int q = 0; q < n; ++q) {
        const int r = __shfl_sync(kAll, rank, q), oid = __shfl_sync(kAll, id, q);
        if (r == lane) chosen = oid;
    }
    return lane < a.k ? chosen : 0;
}

// Lanes per group where no lane's experts span two groups and the lanes of a group
// are a power of two, else 0.
template <int EPT>
__device__ __forceinline__ int lanes_per_group(const RouteArgs &a) {
    const int size = a.E / a.n_group;
    return size % EPT == 0 && ((size / EPT) & (size / EPT - 1)) == 0 ? size / EPT : 0;
}

// Gates of the chosen ids (lane r < k holds one) from the scores in `row`.
__device__ __forceinline__ void write_choice(const RouteArgs &a, int t, int my_id, const float *row) {
    const int lane = threadIdx.x & 31;
    const float g = row[my_id];
    float f = g * a.gate_scale;
    if (a.score != MOE_SCORE_SOFTMAX || a.renorm) {
        const float sum = warp_sum(lane < a.k ? g : 0.f);
        f = sum == 0.f ? 0.f : g / sum * a.gate_scale;      // no scores left: gates of 0
    }
    if (lane < a.k) {
        a.idx[(size_t)t * a.k + lane] = my_id;
        a.gate[(size_t)t * a.k + lane] = f;
    }
}

// ALIGNED: every token may use every group, or lanes_per_group is not 0.
template <int EPT, int WARPS, bool FULL, bool ALIGNED>
__global__ void __launch_bounds__(WARPS * 32, 1024 / (WARPS * 32)) route_select_kernel(const __grid_constant__ RouteArgs a) {
    pdl_wait_then_release();
    __shared__ __align__(16) float part[WARPS][EPT * 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool softmax = a.score == MOE_SCORE_SOFTMAX;
    const int lanes = ALIGNED ? lanes_per_group<EPT>(a) : 0;
    const Bounds bounds(a);
    const float two_rel = bounds.two_rel();
    float sb[EPT], share[EPT];
#pragma unroll
    for (int j = 0; j < EPT; ++j) {
        sb[j] = (a.sel_bias && (FULL || lane * EPT + j < a.E)) ? __ldg(a.sel_bias + lane * EPT + j) : 0.f;
        share[j] = 0.f;
    }
    for (int i = 0; i < kBlockTok / WARPS; ++i) {
        const int t = blockIdx.x * kBlockTok + i * WARPS + warp;
        if (t >= a.T) break;                       // uniform over the warp
        float h[EPT], s[EPT], key[EPT];
        load_logits<EPT, FULL>(a, t, h);
        if (a.logits_out) {
#pragma unroll
            for (int j = 0; j < EPT; ++j)
                if (FULL || lane * EPT + j < a.E) a.logits_out[(size_t)t * a.E + lane * EPT + j] = h[j];
        }
        if (softmax) {
            const float inv = scores<EPT>(a.score, a.E, h, s);
#pragma unroll
            for (int j = 0; j < EPT; ++j) {
                s[j] *= inv;
                share[j] += s[j];
                key[j] = h[j] + sb[j];             // absent experts: -inf
            }
        } else {
            float z = 0.f;
#pragma unroll
            for (int j = 0; j < EPT; ++j) {        // absent experts: score 0
                s[j] = sigmoid(h[j]);
                z += s[j];
                key[j] = FULL || lane * EPT + j < a.E ? s[j] + sb[j] : -INFINITY;
            }
            z = warp_sum(z);
            if (z < 0x1p-64f) {                    // gates and shares are ratios: keep 1 / z finite
                z *= 0x1p64f;
#pragma unroll
                for (int j = 0; j < EPT; ++j) s[j] *= 0x1p64f;
            }
            const float inv = z == 0.f ? 0.f : 1.f / z;
#pragma unroll
            for (int j = 0; j < EPT; ++j) share[j] = fmaf(s[j], inv, share[j]);
        }
        put_row<EPT>(part[warp], s);
        float mx = key[0];
#pragma unroll
        for (int j = 1; j < EPT; ++j) mx = fmaxf(mx, key[j]);
        mx = redux_max(mx);
        bool close = !(fabsf(mx) < INFINITY);      // an infinite best key: distances say nothing
        uint32_t v[EPT];
        candidates<EPT, FULL>(a, key, mx, v);
        const float two = bounds.two(mx);
        // two roundings more per score than per key, both within twice rel
        const float score_rel = softmax ? 0x1p-22f : 2.f * bounds.rel;
        bool c = false;
        if (!ALIGNED) {
            const uint32_t mask = kept_experts<EPT, float>(a, key, bounds.abs, score_rel, &c);
#pragma unroll
            for (int j = 0; j < EPT; ++j) v[j] = mask >> j & 1u ? v[j] : kAll;
        }
        lane_sort<EPT>(v);
        if (ALIGNED && a.topk_group < a.n_group) {
            bool kept = kept_lane<EPT>(a, lanes, v, two, two_rel, &c);
            if (c)                                 // too close for cut-off distances: whole fp32 keys
                kept = kept_experts<EPT, float>(a, key, bounds.abs, score_rel, &c) != 0u;
#pragma unroll
            for (int j = 0; j < EPT; ++j) v[j] = kept ? v[j] : kAll;
        }
        uint32_t mine = kAll;                      // lane r: the winner of round r
        for (int r = 0; r < a.k; ++r) {
            const uint32_t top = take_best<EPT>(v);
            mine = lane == r ? top : mine;
        }
        uint32_t next = __reduce_min_sync(kAll, v[0]);
        uint32_t after = __shfl_down_sync(kAll, mine, 1);
        if (lane == a.k - 1) after = next;
        // Where a chosen distance is infinite or NaN (a key of -inf or NaN, or a difference
        // past the fp32 range) the row is selected again; telling -inf apart here took
        // 28 us instead of 69 for 16384 rows that all choose such keys, and 24.7 instead
        // of 22.9 for all others.
        const bool tight = lane < a.k && ((after != kAll && distance(after) - distance(mine) < two + two_rel * distance(after)) ||
                                          !(distance(mine) < INFINITY));
        int my_id = lane < a.k ? (int)(mine & 255u) : 0;
        close = close || c;
        if (!close && __any_sync(kAll, tight)) {
            // the chosen and whatever lies within the bounds behind them, one to a
            // lane, ranked by their 64-bit keys
            const float limit = distance(__shfl_sync(kAll, mine, a.k - 1));
            int n = limit < INFINITY ? a.k : 32;
            while (n < 32 && next != kAll && distance(next) - limit < two + two_rel * distance(next)) {
                take_best<EPT>(v);
                mine = lane == n ? next : mine;
                ++n;
                next = __reduce_min_sync(kAll, v[0]);
            }
            if (n == 32) close = true;             // maybe more than lanes, or no order among the last
            else my_id = rank_exact(a, t, mine, n);
        }
        if (close) my_id = select_exact<EPT>(a, t);
        write_choice(a, t, my_id, part[warp]);
        __syncwarp();
    }
    if (a.psum == nullptr) return;
    put_row<EPT>(part[warp], share);
    __syncthreads();
    for (int e = tid; e < a.E; e += WARPS * 32) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) v += part[w][e];
        a.psum[(size_t)blockIdx.x * a.E + e] = v;
    }
}

// dlogits of ell = sum dgate * gate + alpha * E * sum_e f_e P_e; the choice of
// experts and f_e = counts_e / (T k) carry no gradient.  With v_e the sum over
// the slots of e of
//   c dg s               softmax, renorm 0
//   (c dg - <c dg, g>) g else, g the gates before their factor c
// and cf_e = alpha E f_e / T:
//   softmax  dl = v + s (cf - <cf, s> - sum v)    (sum v is 0 with renorm)
//   sigmoid  dl = (v + q (cf - <cf, q>)) (1 - s), q = s / sum s
// Scores enter as shares alone, so no quotient passes the fp32 range where all
// of a row's, or all chosen, sigmoids are tiny.
template <int EPT>
__global__ void __launch_bounds__(256) route_bwd_kernel(RouteBwdArgs a) {
    pdl_wait_then_release();
    __shared__ __align__(16) float rows[8][EPT * 32];          // a warp's row: scores, then their gradients
    const int lane = threadIdx.x & 31;
    float *row = rows[threadIdx.x >> 5];
    const int t = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (t >= a.T) return;
    const bool softmax = a.score == MOE_SCORE_SOFTMAX;
    RouteArgs ra{};
    ra.logits = a.logits; ra.T = a.T; ra.E = a.E; ra.splits = 1; ra.vec = a.vec;
    float h[EPT], s[EPT], ds[EPT];
    load_logits<EPT, false>(ra, t, h);
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
    put_row<EPT>(row, s);
    const float sv = row[e];
    const bool renorm = !softmax || a.renorm;
    float g = sv;
    if (renorm) {
        const float sum = warp_sum(used ? sv : 0.f);
        g = sum == 0.f ? 0.f : sv / sum;
        dg -= warp_sum(dg * g);
    }
    const float v = used ? dg * g : 0.f;
    // the chosen experts' gradients to their lanes; an id that stands twice shows by
    // the lane numbers of its slots (one of them overwrites the other's)
    __syncwarp();
    put_row<EPT>(row, ds);
    if (used) row[e] = __int_as_float(lane);
    __syncwarp();
    const bool twice = __any_sync(kAll, used && __float_as_int(row[e]) != lane);
    if (used) row[e] = twice ? 0.f : v;
    __syncwarp();
    if (twice)
        for (int r = 0; r < a.k; ++r) {            // slots in order
            if (lane == r && used) row[e] += v;
            __syncwarp();
        }
    get_row<EPT>(row, ds);
    float cf[EPT], dot = renorm ? 0.f : v;
#pragma unroll
    for (int j = 0; j < EPT; ++j) {
        cf[j] = 0.f;
        if (a.alpha != 0.f && lane * EPT + j < a.E) cf[j] = a.balance * (float)__ldg(a.counts + lane * EPT + j);
        dot = fmaf(cf[j], s[j], dot);
    }
    if (!renorm || a.alpha != 0.f) dot = warp_sum(dot);
    if (!softmax) dot *= inv;
#pragma unroll
    for (int j = 0; j < EPT; ++j) {
        if (softmax) ds[j] += s[j] * (cf[j] - dot);
        else ds[j] = (ds[j] + s[j] * inv * (cf[j] - dot)) * (1.f / (1.f + expf(h[j])));     // 1 - s without its cancellation near s = 1
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

constexpr int kSelWarps = 8;

template <int EPT, int W>
cudaError_t launch_select_warps(const RouteArgs &a, cudaStream_t st) {
    const dim3 grid((unsigned)((a.T + kBlockTok - 1) / kBlockTok)), block(W * 32);
    const int size = a.E / a.n_group, lanes = size % EPT == 0 ? size / EPT : 0;
    const bool aligned = a.topk_group == a.n_group || (lanes > 0 && (lanes & (lanes - 1)) == 0);
    if (!aligned) return launch_kernel(route_select_kernel<EPT, W, false, false>, grid, block, 0, st, a.pdl, a);
    if (a.vec && a.E == 32 * EPT) return launch_kernel(route_select_kernel<EPT, W, true, true>, grid, block, 0, st, a.pdl, a);
    return launch_kernel(route_select_kernel<EPT, W, false, true>, grid, block, 0, st, a.pdl, a);
}

// Where all blocks run at once a token has a warp of its own (T = 256: 7.4 us against
// 9.5 with four to a warp, 4000: 7.9 against 10.0); beyond that four tokens share a
// warp's start and its part of the score sums (8000: 12.5 us against 13.5).
template <int EPT>
cudaError_t launch_select(const RouteArgs &a, cudaStream_t st) {
    if ((a.T + kBlockTok - 1) / kBlockTok <= a.num_sms) return launch_select_warps<EPT, 32>(a, st);
    return launch_select_warps<EPT, kSelWarps>(a, st);
}

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
    if (a.E <= 32) return launch_select<1>(a, st);
    if (a.E <= 64) return launch_select<2>(a, st);
    if (a.E <= 128) return launch_select<4>(a, st);
    return launch_select<8>(a, st);
}

cudaError_t launch_route_bwd(const RouteBwdArgs &in, cudaStream_t st) {
    if (in.T == 0) return cudaSuccess;
    RouteBwdArgs a = in;
    a.vec = vector_rows(a.logits, a.E);
    a.vec_out = vector_rows(a.dlogits, a.E);
    a.balance = (float)((double)a.alpha * a.E / a.T / ((double)a.T * a.k));
    const dim3 grid((unsigned)((a.T + 7) / 8)), block(256);
    if (a.E <= 32) return launch_kernel(route_bwd_kernel<1>, grid, block, 0, st, a.pdl, a);
    if (a.E <= 64) return launch_kernel(route_bwd_kernel<2>, grid, block, 0, st, a.pdl, a);
    if (a.E <= 128) return launch_kernel(route_bwd_kernel<4>, grid, block, 0, st, a.pdl, a);
    return launch_kernel(route_bwd_kernel<8>, grid, block, 0, st, a.pdl, a);
}

}  // namespace moe
