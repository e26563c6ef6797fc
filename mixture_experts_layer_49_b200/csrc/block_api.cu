// block_api.cu -- entry points of the operators around the layer that need no
// workspace of it: the RMS norm with the residual's addition and an 8-bit
// output, and the group-limited selection from logits with its gradient.
#include <math.h>

#include "common.cuh"
#include "kernels.cuh"

namespace {

moe_status bad(moe_status s, const char *where, const char *what) {
    moe::set_error_detail(where, what);
    return s;
}
moe_status done(cudaError_t e, const char *where) {
    return e == cudaSuccess ? MOE_OK : bad(MOE_ERR_CUDA, where, cudaGetErrorString(e));
}
bool mis(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

constexpr int kMaxNormWidth = 32768;

moe_status check_norm(const char *where, int32_t dtype, int64_t rows, int32_t d, float eps) {
    if (dtype != MOE_F32 && dtype != MOE_BF16) return bad(MOE_ERR_INVALID_ARG, where, "bad dtype");
    if (rows < 0 || d < 1) return bad(MOE_ERR_INVALID_ARG, where, "negative rows or non-positive d");
    if (d % 8 || d > kMaxNormWidth) return bad(MOE_ERR_UNSUPPORTED, where, "d must be a multiple of 8, at most 32768");
    if (rows >= (int64_t)1 << 31) return bad(MOE_ERR_UNSUPPORTED, where, "2^31 rows or more");
    if (!(eps >= 0.f) || !isfinite(eps)) return bad(MOE_ERR_INVALID_ARG, where, "eps negative or not finite");
    return MOE_OK;
}

size_t bwd_bytes(int64_t rows, int32_t d) {
    return ((size_t)moe::rmsnorm_bwd_parts(rows, d) * (size_t)d * 4 + 256 + 255) / 256 * 256;
}

}  // namespace

extern "C" {

moe_status moe_rmsnorm(int32_t dtype, int64_t rows, int32_t d, const void *x, const void *residual,
                       const float *weight, float eps, void *h, void *y, uint8_t *codes, float *scale,
                       int64_t ld_scale, moe_stream_t stream) {
    const char *where = "moe_rmsnorm";
    moe_status s = check_norm(where, dtype, rows, d, eps);
    if (s != MOE_OK) return s;
    if (rows == 0) return MOE_OK;                  // an empty tensor may have no address
    if ((codes == nullptr) != (scale == nullptr)) return bad(MOE_ERR_INVALID_ARG, where, "codes and scale: both or neither");
    if (!h && !y && !codes) return bad(MOE_ERR_INVALID_ARG, where, "no output: h, y and codes are NULL");
    if (codes && (ld_scale < ((int64_t)d + 127) / 128 * 4 || ld_scale % 4))
        return bad(MOE_ERR_INVALID_ARG, where, "ld_scale below 4 * ceil(d / 128) or not a multiple of 4");
    if (!x || !weight) return bad(MOE_ERR_INVALID_ARG, where, "NULL pointer: x or weight");
    if (mis(x, 16) || mis(residual, 16) || mis(weight, 16) || mis(h, 16) || mis(y, 16) || mis(codes, 8) || mis(scale, 4))
        return bad(MOE_ERR_INVALID_ARG, where, "misaligned pointer (16 bytes; codes 8, scale 4)");
    moe::RmsNormArgs a{};
    a.x = x; a.residual = residual; a.weight = weight; a.h = h; a.y = y; a.codes = codes; a.scale = scale;
    a.ld_scale = ld_scale; a.rows = rows; a.d = d; a.eps = eps;
    return done(moe::launch_rmsnorm(a, dtype == MOE_BF16, reinterpret_cast<cudaStream_t>(stream)), where);
}

size_t moe_rmsnorm_backward_workspace_size(int64_t rows, int32_t d) {
    if (check_norm("moe_rmsnorm_backward_workspace_size", MOE_F32, rows, d, 0.f) != MOE_OK) return 0;
    return bwd_bytes(rows, d);
}

moe_status moe_rmsnorm_backward(int32_t dtype, int64_t rows, int32_t d, const void *h, const float *weight, float eps,
                                const void *dy, const void *dres, void *dh, float *dweight, void *ws,
                                size_t ws_bytes, moe_stream_t stream) {
    const char *where = "moe_rmsnorm_backward";
    moe_status s = check_norm(where, dtype, rows, d, eps);
    if (s != MOE_OK) return s;
    if (!dweight) return bad(MOE_ERR_INVALID_ARG, where, "NULL pointer: dweight");
    if (rows > 0 && (!h || !weight || !dy || !dh)) return bad(MOE_ERR_INVALID_ARG, where, "NULL pointer: h, weight, dy or dh");
    if (mis(h, 16) || mis(weight, 16) || mis(dy, 16) || mis(dres, 16) || mis(dh, 16) || mis(dweight, 4))
        return bad(MOE_ERR_INVALID_ARG, where, "misaligned pointer (16 bytes; dweight 4)");
    if (!ws || mis(ws, 256)) return bad(MOE_ERR_WORKSPACE, where, "workspace NULL or not 256-byte aligned");
    if (ws_bytes < bwd_bytes(rows, d))
        return bad(MOE_ERR_WORKSPACE, where, "workspace smaller than moe_rmsnorm_backward_workspace_size()");
    moe::RmsNormBwdArgs a{};
    a.h = h; a.dy = dy; a.dres = dres; a.weight = weight; a.dh = dh; a.part = static_cast<float *>(ws);
    a.dweight = dweight; a.rows = rows; a.d = d; a.eps = eps; a.num_sms = moe::device_sms();
    return done(moe::launch_rmsnorm_bwd(a, dtype == MOE_BF16, reinterpret_cast<cudaStream_t>(stream)), where);
}

moe_status moe_route_select(const moe_config *cfg, const moe_route_groups *groups, const float *logits,
                            const float *sel_bias, int32_t *idx, float *gate, float *psum, moe_stream_t stream) {
    const char *where = "moe_route_select";
    moe_status s = moe::validate_groups(cfg, groups);
    if (s != MOE_OK) return s;
    if (cfg->T > 0 && (!logits || !idx || !gate)) return bad(MOE_ERR_INVALID_ARG, where, "NULL pointer: logits, idx or gate");
    if (mis(logits, 4) || mis(sel_bias, 4) || mis(idx, 4) || mis(gate, 4) || mis(psum, 4))
        return bad(MOE_ERR_INVALID_ARG, where, "misaligned pointer (4 bytes)");
    moe::RouteArgs a{};
    a.logits = logits; a.sel_bias = sel_bias; a.idx = idx; a.gate = gate; a.psum = psum;
    a.T = cfg->T; a.E = cfg->E; a.k = cfg->top_k; a.score = cfg->score; a.renorm = cfg->renorm; a.splits = 1;
    a.n_group = groups->n_group; a.topk_group = groups->topk_group; a.group_top = groups->group_top;
    a.gate_scale = groups->gate_scale; a.num_sms = moe::device_sms();
    return done(moe::launch_route_select(a, reinterpret_cast<cudaStream_t>(stream)), where);
}

moe_status moe_route_backward(const moe_config *cfg, const moe_route_groups *groups, const float *logits,
                              const int32_t *idx, const float *dgate, const int32_t *counts, float alpha,
                              float *dlogits, moe_stream_t stream) {
    const char *where = "moe_route_backward";
    moe_status s = moe::validate_groups(cfg, groups);
    if (s != MOE_OK) return s;
    if (!isfinite(alpha)) return bad(MOE_ERR_INVALID_ARG, where, "alpha not finite");
    if (cfg->T > 0 && (!logits || !idx || !dgate || !dlogits || (alpha != 0.f && !counts)))
        return bad(MOE_ERR_INVALID_ARG, where, "NULL pointer: logits, idx, dgate, dlogits, or counts with alpha");
    if (mis(logits, 4) || mis(idx, 4) || mis(dgate, 4) || mis(counts, 4) || mis(dlogits, 4))
        return bad(MOE_ERR_INVALID_ARG, where, "misaligned pointer (4 bytes)");
    moe::RouteBwdArgs a{};
    a.logits = logits; a.idx = idx; a.dgate = dgate; a.counts = counts; a.dlogits = dlogits;
    a.T = cfg->T; a.E = cfg->E; a.k = cfg->top_k; a.score = cfg->score; a.renorm = cfg->renorm;
    a.gate_scale = groups->gate_scale; a.alpha = alpha;
    return done(moe::launch_route_bwd(a, reinterpret_cast<cudaStream_t>(stream)), where);
}

}  // extern "C"
