// norm_api.cu -- the entry points of include/moe.h for the norm in front of the
// experts: argument checks, workspace and launches (kernels in norm.cu).  Host code
// only; nothing here allocates, frees or synchronises.
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"

using namespace moe;

namespace {

constexpr int64_t kMaxCols = 16384;

moe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

moe_status check_sizes(int64_t rows, int64_t cols) {
    if (rows < 0 || cols <= 0) return MOE_ERR_INVALID_ARG;
    return rows < ((int64_t)1 << 31) && cols <= kMaxCols ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

moe_status check_norm(int64_t rows, int64_t cols, int32_t dtype, float eps) {
    if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || isinf(eps)) return MOE_ERR_INVALID_ARG;
    return check_sizes(rows, cols);
}

}  // namespace

extern "C" {

moe_status moe_rmsnorm(int64_t rows, int64_t cols, int32_t dtype, const void* x,
                       const void* residual, const void* weight, float eps, void* s, void* y,
                       uint8_t* codes, float* scales, void* stream) {
    moe_status st = check_norm(rows, cols, dtype, eps);
    if (st != MOE_OK) return st;
    if (rows == 0) return MOE_OK;
    if (!good(x) || !good(weight) || !good_or_null(residual) || !good_or_null(s) ||
        !good_or_null(y) || !good_or_null(codes) || !good_or_null(scales))
        return MOE_ERR_INVALID_ARG;
    if ((!y && !codes) || !codes != !scales) return MOE_ERR_INVALID_ARG;
    // what is written lies apart from all the rest, but for the rows themselves: s in
    // place of x or of the residual, y in place of x (a row is read before it is written)
    const uint64_t n = (uint64_t)rows * (uint64_t)cols, size = dtype == MOE_BF16 ? 2 : 4;
    struct Buf {
        const void* p;
        uint64_t bytes;
    };
    const Buf in[] = {{x, n * size}, {residual, n * size}, {weight, (uint64_t)cols * size}};
    const Buf out[] = {{s, n * size}, {y, n * size}, {codes, n}, {scales, 4 * (uint64_t)rows}};
    for (const Buf& o : out) {
        for (const Buf& i : in) {
            const bool in_place = o.p == i.p && ((o.p == s && i.p != weight) || (o.p == y && i.p == x));
            if (!in_place && overlap(o.p, o.bytes, i.p, i.bytes)) return MOE_ERR_INVALID_ARG;
        }
        for (const Buf& q : out)
            if (&o != &q && overlap(o.p, o.bytes, q.p, q.bytes)) return MOE_ERR_INVALID_ARG;
    }
    NormArgs a{};
    a.rows = rows;
    a.d = (int)cols;
    a.dtype = dtype;
    a.eps = eps;
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.s = s;
    a.y = y;
    a.codes = codes;
    a.scales = scales;
    return cuda_status(launch_rmsnorm(a, (cudaStream_t)stream));
}

size_t moe_rmsnorm_workspace_bytes(int64_t rows, int64_t cols) {
    if (check_sizes(rows, cols) != MOE_OK) return 0;
    // 0 stands for a refusal: no rows, which are a valid call, get a block's room
    const size_t blocks = rows == 0 ? 1 : (size_t)rmsnorm_backward_blocks(rows, (int)cols);
    return (sizeof(float) * blocks * (size_t)cols + 255) / 256 * 256;
}

moe_status moe_rmsnorm_backward(int64_t rows, int64_t cols, int32_t dtype, const void* d_y,
                                const void* s, const void* weight, float eps, const void* d_s,
                                void* d_x, float* d_weight, void* workspace, size_t ws_bytes,
                                void* stream) {
    moe_status st = check_norm(rows, cols, dtype, eps);
    if (st != MOE_OK) return st;
    if (!good_or_null(d_x) || !good_or_null(d_weight)) return MOE_ERR_INVALID_ARG;
    cudaStream_t cs = (cudaStream_t)stream;
    if (rows == 0)  // arrays without elements may be NULL, d_x among them
        return d_weight ? cuda_status(cudaMemsetAsync(d_weight, 0, sizeof(float) * (size_t)cols, cs))
                        : MOE_OK;
    if (!d_x && !d_weight) return MOE_ERR_INVALID_ARG;
    if (!good(d_y) || !good(s) || !good(weight) || !good_or_null(d_s)) return MOE_ERR_INVALID_ARG;
    const uint64_t n = (uint64_t)rows * (uint64_t)cols * (dtype == MOE_BF16 ? 2 : 4);
    const uint64_t wn = (uint64_t)cols * (dtype == MOE_BF16 ? 2 : 4), dn = 4 * (uint64_t)cols;
    for (const void* p : {d_y, s, d_s}) {
        if (d_x != p && overlap(d_x, n, p, n)) return MOE_ERR_INVALID_ARG;
        if (overlap(d_weight, dn, p, n)) return MOE_ERR_INVALID_ARG;
    }
    if (overlap(d_x, n, weight, wn) || overlap(d_x, n, d_weight, dn) ||
        overlap(d_weight, dn, weight, wn))
        return MOE_ERR_INVALID_ARG;
    if (d_weight) {
        const size_t need = moe_rmsnorm_workspace_bytes(rows, cols);
        if (!good(workspace) || ws_bytes < need) return MOE_ERR_WORKSPACE;
        for (const void* p : {d_y, s, d_s, (const void*)d_x})
            if (overlap(workspace, need, p, n)) return MOE_ERR_INVALID_ARG;
        if (overlap(workspace, need, weight, wn) || overlap(workspace, need, d_weight, dn))
            return MOE_ERR_INVALID_ARG;
    }
    NormArgs a{};
    a.rows = rows;
    a.d = (int)cols;
    a.dtype = dtype;
    a.eps = eps;
    a.x = s;
    a.weight = weight;
    a.d_y = d_y;
    a.d_s = d_s;
    a.d_x = d_x;
    a.d_weight = d_weight;
    a.part = d_weight ? static_cast<float*>(workspace) : nullptr;
    return cuda_status(launch_rmsnorm_backward(a, cs));
}

}  // extern "C"
