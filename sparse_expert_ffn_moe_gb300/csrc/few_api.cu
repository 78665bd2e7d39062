// few_api.cu -- the entry points of include/moe.h for the layer on a few tokens:
// argument checks and workspace (kernels in few.cu).  Host code only; nothing here
// allocates, frees or synchronises.
#include <stdint.h>

#include "common.cuh"
#include "internal.h"

using namespace moe;

namespace {

moe_status check_few(const moe_shape* shape) {
    const moe_status st = check_shape(shape);
    if (st != MOE_OK) return st;
    return shape->T <= kFewMaxTokens && shape->dtype == MOE_BF16 ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

// what both kinds of call check and enqueue; c has the weights
moe_status run(const moe_shape& s, int fmt, const FewCall& c, void* workspace, size_t ws_bytes,
               void* stream) {
    if (!good(c.x) || !good(c.w_g) || !good(c.y) || !good_or_null(c.residual) ||
        !good_or_null(c.bias, 4))
        return MOE_ERR_INVALID_ARG;
    const bool shared = s.inter_shared > 0;
    const void* routed[] = {c.w_gate, c.w_up, c.w_down};
    const void* ours[] = {c.ws_gate, c.ws_up, c.ws_down};
    for (const void* p : routed)
        if (!good(p)) return MOE_ERR_INVALID_ARG;
    for (const void* p : ours)
        if (shared ? !good(p) : p != nullptr) return MOE_ERR_INVALID_ARG;
    if (fmt) {
        const void* sr[] = {c.s_gate, c.s_up, c.s_down};
        const void* ss[] = {c.ss_gate, c.ss_up, c.ss_down};
        for (const void* p : sr)
            if (!good(p)) return MOE_ERR_INVALID_ARG;
        for (const void* p : ss)
            if (shared && !good(p)) return MOE_ERR_INVALID_ARG;
    }
    const size_t need = few_ws(s, fmt).total;
    if (!good(workspace) || ws_bytes < need) return MOE_ERR_WORKSPACE;
    // What is written lies apart from what is read.  The residual alone may be y: its elements are
    // read where y's are written.
    const uint64_t E = s.E, d = s.d, I = s.inter, Is = s.inter_shared;
    const uint64_t rows = 2 * (uint64_t)s.T * d, size = fmt ? 1 : 2;
    const uint64_t up = fmt == 1 ? 4 * I : I * d / 4096, down = fmt == 1 ? 4 * d : I * d / 4096;
    const uint64_t sup = fmt == 1 ? 4 * Is : Is * d / 4096, sdown = fmt == 1 ? 4 * d : Is * d / 4096;
    const struct {
        const void* p;
        uint64_t bytes;
    } in[] = {{c.x, rows}, {c.residual, rows}, {c.w_g, 2 * E * d}, {c.bias, 4 * E},
              {c.w_gate, E * I * d * size}, {c.w_up, E * I * d * size}, {c.w_down, E * I * d * size},
              {c.ws_gate, Is * d * size}, {c.ws_up, Is * d * size}, {c.ws_down, Is * d * size},
              {c.s_gate, E * up}, {c.s_up, E * up}, {c.s_down, E * down},
              {c.ss_gate, sup}, {c.ss_up, sup}, {c.ss_down, sdown}};
    for (const auto& i : in) {
        if (overlap(workspace, need, i.p, i.bytes)) return MOE_ERR_INVALID_ARG;
        const bool in_place = i.p == c.residual && c.residual == c.y;
        if (!in_place && overlap(c.y, rows, i.p, i.bytes)) return MOE_ERR_INVALID_ARG;
    }
    if (overlap(c.y, rows, workspace, need)) return MOE_ERR_INVALID_ARG;
    if (!tc_available()) return MOE_ERR_UNSUPPORTED;
    return launch_few(s, fmt, c, workspace, (cudaStream_t)stream) == cudaSuccess ? MOE_OK
                                                                                 : MOE_ERR_CUDA;
}

moe_status run_fp8(const moe_shape* shape, int fmt, const void* x, const void* w_g,
                   const float* bias, const moe_fp8_experts* w, const void* residual, void* y,
                   void* workspace, size_t ws_bytes, void* stream) {
    const moe_status st = check_few(shape);
    if (st != MOE_OK) return st;
    const moe_shape& s = *shape;
    if (s.d % 128 || s.inter % 128 || s.inter_shared % 128) return MOE_ERR_UNSUPPORTED;
    if (s.T == 0) return MOE_OK;
    if (!w) return MOE_ERR_INVALID_ARG;
    const FewCall c{x, w_g, residual, bias, w->w_gate, w->w_up, w->w_down, w->ws_gate, w->ws_up,
                    w->ws_down, w->s_gate, w->s_up, w->s_down, w->ss_gate, w->ss_up, w->ss_down, y};
    return run(s, fmt, c, workspace, ws_bytes, stream);
}

}  // namespace

extern "C" {

size_t moe_few_workspace_bytes(const moe_shape* shape) {
    if (check_shape(shape) != MOE_OK || shape->T > kFewMaxTokens) return 0;
    // the larger of the two kinds of weights' needs
    const size_t a = few_ws(*shape, 0).total, b = few_ws(*shape, 1).total;
    return a > b ? a : b;
}

moe_status moe_forward_few(const moe_shape* shape, const void* x, const void* w_g,
                           const float* bias, const void* w_gate, const void* w_up,
                           const void* w_down, const void* ws_gate, const void* ws_up,
                           const void* ws_down, const void* residual, void* y, void* workspace,
                           size_t ws_bytes, void* stream) {
    const moe_status st = check_few(shape);
    if (st != MOE_OK) return st;
    if (shape->T == 0) return MOE_OK;
    FewCall c{};
    c.x = x;
    c.w_g = w_g;
    c.residual = residual;
    c.bias = bias;
    c.w_gate = w_gate;
    c.w_up = w_up;
    c.w_down = w_down;
    c.ws_gate = ws_gate;
    c.ws_up = ws_up;
    c.ws_down = ws_down;
    c.y = y;
    return run(*shape, 0, c, workspace, ws_bytes, stream);
}

moe_status moe_forward_few_fp8(const moe_shape* shape, const void* x, const void* w_g,
                               const float* bias, const moe_fp8_experts* w, const void* residual,
                               void* y, void* workspace, size_t ws_bytes, void* stream) {
    return run_fp8(shape, 1, x, w_g, bias, w, residual, y, workspace, ws_bytes, stream);
}

moe_status moe_forward_few_fp8_blocks(const moe_shape* shape, const void* x, const void* w_g,
                                      const float* bias, const moe_fp8_experts* w,
                                      const void* residual, void* y, void* workspace,
                                      size_t ws_bytes, void* stream) {
    return run_fp8(shape, 2, x, w_g, bias, w, residual, y, workspace, ws_bytes, stream);
}

}  // extern "C"
