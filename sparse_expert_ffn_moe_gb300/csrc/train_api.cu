// train_api.cu -- the entry points of include/moe.h that train a router:
// argument checks, workspace carving and launches (kernels in balance.cu and
// dropout.cu).  Host code only; nothing here allocates, frees or synchronises.
#include <stdint.h>

#include "common.cuh"
#include "internal.h"
#include "philox.cuh"

using namespace moe;

namespace {

constexpr int32_t kMaxSeqs = 1 << 20;

moe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// Error block (the record at its start, the ticket of the last block at
// kTicket), then the shares of the loss and the partial rows.
constexpr size_t kErrBytes = 256, kTicket = 128;

struct BalanceWs {
    size_t shares, part_n, part_bad, part_p, part_c, total;
};

BalanceWs balance_ws(const moe_shape& s, int32_t n_seq) {
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    const size_t blocks = (size_t)balance_blocks(s, n_seq), rows = blocks + (size_t)n_seq;
    const size_t shares = (size_t)n_seq * (size_t)balance_slices(s, n_seq);
    BalanceWs w;
    w.shares = kErrBytes;
    w.part_n = up(w.shares + sizeof(float) * shares);
    w.part_bad = up(w.part_n + sizeof(int32_t) * rows);
    w.part_p = up(w.part_bad + sizeof(int32_t) * blocks);
    w.part_c = up(w.part_p + sizeof(float) * rows * (size_t)s.E);
    w.total = up(w.part_c + sizeof(int32_t) * rows * (size_t)s.E);
    return w;
}

moe_status check_seqs(const int32_t* seq_offsets, int32_t n_seq) {
    if (n_seq < 1 || !aligned(seq_offsets, 4)) return MOE_ERR_INVALID_ARG;
    if (!seq_offsets && n_seq != 1) return MOE_ERR_INVALID_ARG;
    return n_seq <= kMaxSeqs ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

// p in [0, 1] (not NaN), and the generator's words where something is drawn: where
// the rule that the kernels get says so
moe_status check_drop(double p, const uint64_t* rng) {
    if (!(p >= 0.0 && p <= 1.0)) return MOE_ERR_INVALID_ARG;
    if ((drop_rule(p).thr && !rng) || !aligned(rng, 8)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_balance_workspace_bytes(const moe_shape* shape, int32_t n_seq) {
    if (check_shape(shape) != MOE_OK || n_seq < 1 || n_seq > kMaxSeqs) return 0;
    return balance_ws(*shape, n_seq).total;
}

moe_status moe_balance_loss(const moe_shape* shape, const float* logits, const int32_t* topk_idx,
                            const uint8_t* token_mask, const int32_t* seq_offsets, int32_t n_seq,
                            float alpha, int32_t* counts, float* mean_probs, float* loss,
                            void* workspace, size_t ws_bytes, void* stream) {
    moe_status st = check_shape(shape);
    if (st != MOE_OK) return st;
    const moe_shape& s = *shape;
    if ((st = check_seqs(seq_offsets, n_seq)) != MOE_OK) return st;
    if (!good(counts, 4) || !good(mean_probs, 4) || !good(loss, 4)) return MOE_ERR_INVALID_ARG;
    if (s.T > 0 && (!good(logits, 16) || !good(topk_idx, 4))) return MOE_ERR_INVALID_ARG;
    if (!good(workspace, 16)) return MOE_ERR_WORKSPACE;
    const BalanceWs w = balance_ws(s, n_seq);
    if (ws_bytes < w.total) return MOE_ERR_WORKSPACE;
    cudaStream_t cs = (cudaStream_t)stream;
    uint8_t* base = static_cast<uint8_t*>(workspace);
    if (s.T == 0) {
        const size_t n = sizeof(float) * (size_t)n_seq * (size_t)s.E;
        cudaError_t e = cudaMemsetAsync(base, 0, kErrBytes, cs);
        if (e == cudaSuccess) e = cudaMemsetAsync(counts, 0, n, cs);
        if (e == cudaSuccess) e = cudaMemsetAsync(mean_probs, 0, n, cs);
        if (e == cudaSuccess) e = cudaMemsetAsync(loss, 0, sizeof(float), cs);
        return cuda_status(e);
    }
    BalanceArgs a{};
    a.logits = logits;
    a.topk_idx = topk_idx;
    a.mask = token_mask;
    a.cu = seq_offsets;
    a.n_seq = n_seq;
    a.alpha = alpha;
    a.counts = counts;
    a.mean_p = mean_probs;
    a.loss = loss;
    a.part_p = reinterpret_cast<float*>(base + w.part_p);
    a.part_c = reinterpret_cast<int32_t*>(base + w.part_c);
    a.part_n = reinterpret_cast<int32_t*>(base + w.part_n);
    a.part_bad = reinterpret_cast<int32_t*>(base + w.part_bad);
    a.shares = reinterpret_cast<float*>(base + w.shares);
    a.ticket = reinterpret_cast<unsigned int*>(base + kTicket);
    a.err = reinterpret_cast<DevError*>(base);
    return cuda_status(launch_balance_loss(s, a, cs));
}

moe_status moe_route_backward(const moe_shape* shape, const float* logits, const int32_t* topk_idx,
                              const float* d_topk_w, const uint8_t* token_mask,
                              const int32_t* seq_offsets, int32_t n_seq, float alpha,
                              const int32_t* counts, const float* d_loss, float* d_logits,
                              void* stream) {
    moe_status st = check_shape(shape);
    if (st != MOE_OK) return st;
    const moe_shape& s = *shape;
    if ((st = check_seqs(seq_offsets, n_seq)) != MOE_OK) return st;
    if (s.T == 0) return MOE_OK;
    if (!good(logits, 16) || !good(d_logits, 16)) return MOE_ERR_INVALID_ARG;
    // the copies of the scores run ahead of the gradient's rows
    const uintptr_t in = (uintptr_t)logits, out = (uintptr_t)d_logits;
    const uint64_t bytes = sizeof(float) * (uint64_t)s.T * (uint64_t)s.E;
    if (in < out + bytes && out < in + bytes) return MOE_ERR_INVALID_ARG;
    if (!counts && !d_topk_w) return MOE_ERR_INVALID_ARG;
    if (!good_or_null(counts, 4) || !good_or_null(d_topk_w, 4) || !good_or_null(d_loss, 4))
        return MOE_ERR_INVALID_ARG;
    if (d_topk_w ? !good(topk_idx, 4) : !good_or_null(topk_idx, 4)) return MOE_ERR_INVALID_ARG;
    RouteBackwardArgs a{};
    a.logits = logits;
    a.topk_idx = topk_idx;
    a.d_topk_w = d_topk_w;
    a.mask = token_mask;
    a.cu = seq_offsets;
    a.n_seq = n_seq;
    a.alpha = alpha;
    a.counts = counts;
    a.d_loss = d_loss;
    a.d_logits = d_logits;
    return cuda_status(launch_route_backward(s, a, (cudaStream_t)stream));
}

moe_status moe_dropout(int64_t n, int32_t dtype, const void* x, const void* residual, double p,
                       const uint64_t* rng, void* y, void* stream) {
    if (n < 0 || (dtype != MOE_F32 && dtype != MOE_BF16)) return MOE_ERR_INVALID_ARG;
    moe_status st = check_drop(p, rng);
    if (st != MOE_OK) return st;
    if (n == 0) return MOE_OK;
    if (!good(x, 16) || !good(y, 16) || !good_or_null(residual, 16)) return MOE_ERR_INVALID_ARG;
    return cuda_status(launch_dropout(n, dtype, x, residual, p, rng, y, (cudaStream_t)stream));
}

moe_status moe_combine_dropout(const moe_shape* shape, const void* y_perm, const int32_t* inv_perm,
                               const float* topk_w, const void* y_shared, const void* residual,
                               double p, const uint64_t* rng, void* y, void* stream) {
    moe_status st = check_shape(shape);
    if (st != MOE_OK) return st;
    const moe_shape& s = *shape;
    if ((st = check_drop(p, rng)) != MOE_OK) return st;
    if (s.T == 0) return MOE_OK;
    if (!good(y_perm, 16) || !good(inv_perm, 4) || !good(topk_w, 4) || !good(y, 16))
        return MOE_ERR_INVALID_ARG;
    if (!good_or_null(y_shared, 16) || !good_or_null(residual, 16)) return MOE_ERR_INVALID_ARG;
    return cuda_status(launch_combine_dropout(s, y_perm, inv_perm, topk_w, y_shared, residual, p,
                                              rng, y, (cudaStream_t)stream));
}

moe_status moe_combine_backward(const moe_shape* shape, const void* d_y, const void* y_perm,
                                const int32_t* inv_perm, const float* topk_w, double p,
                                const uint64_t* rng, void* d_y_perm, float* d_topk_w,
                                void* d_shared, void* stream) {
    moe_status st = check_shape(shape);
    if (st != MOE_OK) return st;
    const moe_shape& s = *shape;
    if ((st = check_drop(p, rng)) != MOE_OK) return st;
    if (s.T == 0) return MOE_OK;
    if (!d_y_perm && !d_topk_w && !d_shared) return MOE_ERR_INVALID_ARG;
    if (!good(d_y, 16) || !good(inv_perm, 4)) return MOE_ERR_INVALID_ARG;
    if (!good_or_null(y_perm, 16) || !good_or_null(topk_w, 4) || !good_or_null(d_y_perm, 16) ||
        !good_or_null(d_topk_w, 4) || !good_or_null(d_shared, 16))
        return MOE_ERR_INVALID_ARG;
    if ((d_topk_w && !y_perm) || (d_y_perm && !topk_w)) return MOE_ERR_INVALID_ARG;
    return cuda_status(launch_combine_backward(s, d_y, y_perm, inv_perm, topk_w, p, rng, d_y_perm,
                                               d_topk_w, d_shared, (cudaStream_t)stream));
}

}  // extern "C"
