// dropout.cu -- dropout from a counter-based generator, alone and in the
// combine, and the combine's backward pass.
//
//   moe_dropout           y = residual + D(x)
//   moe_combine_dropout   y = residual + D(y_shared + sum_j w_j y_perm[p_j])
//   moe_combine_backward  dz = D(d_y);  d_y_perm[p_j] = w_j dz,
//                         d_w_j = <dz, y_perm[p_j]>,  d_shared = dz
//
// D keeps an element with the chance the rule of philox.cuh gives it and
// divides what stays by that chance.  D is linear with a mask that depends on
// (seed, offset, element) alone, so the backward pass draws it again and
// nothing is stored between the two.
//
// All three are bound by HBM: every row is read once and written once, in
// 16-byte vectors, and the mask costs about 90 integer instructions per eight
// elements.
#include "internal.h"
#include "philox.cuh"

namespace moe {

namespace {

template <typename T>
__global__ void __launch_bounds__(256)
dropout_kernel(const T* x, const T* residual, T* y, int64_t n, DropRule rule,
               const uint64_t* __restrict__ rng) {
    pdl_wait();
    pdl_trigger();
    RngState st = {};
    if (rule.thr) st = load_rng(rng);
    const int64_t groups = n / 8;
    const int64_t stride = (int64_t)gridDim.x * blockDim.x;
    for (int64_t g = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; g < groups; g += stride) {
        float f[8];
        widen(load_unit(x + g * 8), f);
        Unit<T> r;
        if (residual) r = load_unit(residual + g * 8);
        if (rule.thr) drop8(f, (uint64_t)g, st, rule);
        if (residual) {
            float rf[8];
            widen(r, rf);
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] += rf[k];
        }
        store_unit(y + g * 8, f);
    }
    // the last, partial group
    if (blockIdx.x == 0 && threadIdx.x == 0 && n % 8) {
        const int64_t base = groups * 8;
        const int m = (int)(n - base);
        float f[8] = {};
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < m) f[k] = Elem<T>::to_f32(x[base + k]);
        if (rule.thr) drop8(f, (uint64_t)groups, st, rule);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (k >= m) continue;
            if (residual) f[k] += Elem<T>::to_f32(residual[base + k]);
            y[base + k] = Elem<T>::from_f32(f[k]);
        }
    }
}

// A thread owns one group of eight elements of an output row.
template <typename T>
__global__ void __launch_bounds__(256)
combine_dropout_kernel(const T* y_perm, const int32_t* __restrict__ inv_perm,
                       const float* __restrict__ topk_w, const T* y_shared, const T* residual,
                       T* y, int d, int K, int64_t n_rows, DropRule rule,
                       const uint64_t* __restrict__ rng) {
    pdl_wait();
    pdl_trigger();
    const int units = d / 8;
    const int64_t t = blockIdx.x;
    const int u = blockIdx.y * blockDim.x + threadIdx.x;
    if (u >= units) return;
    const int64_t at = t * d + (int64_t)u * 8;
    float acc[8] = {};
    if (y_shared) widen(load_unit(y_shared + at), acc);
    for (int j = 0; j < K; ++j) {
        const int32_t p = inv_perm[t * K + j];
        if (p < 0 || p >= n_rows) continue;  // dropped slot
        const float w = topk_w[t * K + j];
        float f[8];
        widen(load_unit(y_perm + (int64_t)p * d + (int64_t)u * 8), f);
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] = fmaf(w, f[k], acc[k]);
    }
    if (rule.thr) drop8(acc, (uint64_t)(at / 8), load_rng(rng), rule);
    if (residual) {
        float f[8];
        widen(load_unit(residual + at), f);
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] += f[k];
    }
    store_unit(y + at, acc);
}

// One token per block: its threads hold dz in registers (V groups of eight
// elements each) and walk the token's K rows; the K dot products are summed in
// a fixed order (lanes, then warps).
template <typename T, int V>
__global__ void __launch_bounds__(512)
combine_backward_kernel(const T* d_y, const T* y_perm, const int32_t* __restrict__ inv_perm,
                        const float* __restrict__ topk_w, T* d_y_perm, float* d_topk_w, T* d_shared,
                        int d, int K, int64_t n_rows, DropRule rule,
                        const uint64_t* __restrict__ rng) {
    __shared__ float red[16][32];  // [warp][slot]
    pdl_wait();
    pdl_trigger();
    const int units = d / 8;
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    float dz[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int u = threadIdx.x + i * blockDim.x;
#pragma unroll
        for (int k = 0; k < 8; ++k) dz[i][k] = 0.f;
        if (u < units) widen(load_unit(d_y + t * d + (int64_t)u * 8), dz[i]);
    }
    if (rule.thr) {
        const RngState st = load_rng(rng);
#pragma unroll
        for (int i = 0; i < V; ++i)
            drop8(dz[i], (uint64_t)(t * units + threadIdx.x + i * blockDim.x), st, rule);
    }
    if (d_shared) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int u = threadIdx.x + i * blockDim.x;
            if (u < units) store_unit(d_shared + t * d + (int64_t)u * 8, dz[i]);
        }
    }
    for (int j = 0; j < K; ++j) {
        const int32_t p = inv_perm[t * K + j];
        float dot = 0.f;
        if (p >= 0 && p < n_rows) {
            const int64_t row = (int64_t)p * d;
            if (d_topk_w) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int u = threadIdx.x + i * blockDim.x;
                    if (u >= units) continue;
                    float f[8];
                    widen(load_unit(y_perm + row + (int64_t)u * 8), f);
#pragma unroll
                    for (int k = 0; k < 8; ++k) dot = fmaf(dz[i][k], f[k], dot);
                }
            }
            if (d_y_perm) {
                const float w = topk_w[t * K + j];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int u = threadIdx.x + i * blockDim.x;
                    if (u >= units) continue;
                    float f[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) f[k] = w * dz[i][k];
                    store_unit(d_y_perm + row + (int64_t)u * 8, f);
                }
            }
        }
        dot = warp_sum(dot);
        if (lane == 0) red[warp][j] = dot;
    }
    __syncthreads();
    if (d_topk_w && threadIdx.x < K) {
        float s = 0.f;
        for (int w = 0; w < nwarps; ++w) s += red[w][threadIdx.x];
        d_topk_w[t * K + threadIdx.x] = s;
    }
}

template <typename T>
cudaError_t dropout_t(int64_t n, const void* x, const void* residual, DropRule rule,
                      const uint64_t* rng, void* y, cudaStream_t st) {
    const int64_t blocks = ceil_div(n / 8 > 0 ? n / 8 : 1, 256);
    const int64_t most = (int64_t)device_sm_count() * 64;
    return launch_pdl(dropout_kernel<T>, dim3((unsigned)(blocks < most ? blocks : most)), dim3(256),
                      0, st, (const T*)x, (const T*)residual, (T*)y, n, rule, rng);
}

template <typename T>
cudaError_t combine_dropout_t(const moe_shape& s, const void* y_perm, const int32_t* inv_perm,
                              const float* topk_w, const void* y_shared, const void* residual,
                              DropRule rule, const uint64_t* rng, void* y, cudaStream_t st) {
    const dim3 grid((unsigned)s.T, (unsigned)ceil_div(s.d / 8, 256));
    return launch_pdl(combine_dropout_kernel<T>, grid, dim3(256), 0, st, (const T*)y_perm, inv_perm,
                      topk_w, (const T*)y_shared, (const T*)residual, (T*)y, s.d, s.K,
                      (int64_t)s.T * s.K, rule, rng);
}

template <typename T, int V>
cudaError_t combine_backward_v(const moe_shape& s, const void* d_y, const void* y_perm,
                               const int32_t* inv_perm, const float* topk_w, DropRule rule,
                               const uint64_t* rng, void* d_y_perm, float* d_topk_w, void* d_shared,
                               cudaStream_t st) {
    const int threads = (int)ceil_div(ceil_div(s.d / 8, V), 32) * 32;
    return launch_pdl(combine_backward_kernel<T, V>, dim3((unsigned)s.T), dim3((unsigned)threads), 0,
                      st, (const T*)d_y, (const T*)y_perm, inv_perm, topk_w, (T*)d_y_perm, d_topk_w,
                      (T*)d_shared, s.d, s.K, (int64_t)s.T * s.K, rule, rng);
}

template <typename T, typename... Args>
cudaError_t combine_backward_t(const moe_shape& s, Args... args) {
    const int units = s.d / 8;
    if (units > 512) return combine_backward_v<T, 4>(s, args...);
    if (units > 256) return combine_backward_v<T, 2>(s, args...);
    return combine_backward_v<T, 1>(s, args...);
}

}  // namespace

cudaError_t launch_dropout(int64_t n, int dtype, const void* x, const void* residual, double p,
                           const uint64_t* rng, void* y, cudaStream_t st) {
    const DropRule rule = drop_rule(p);
    return dtype == MOE_BF16 ? dropout_t<bf16>(n, x, residual, rule, rng, y, st)
                             : dropout_t<float>(n, x, residual, rule, rng, y, st);
}

cudaError_t launch_combine_dropout(const moe_shape& s, const void* y_perm, const int32_t* inv_perm,
                                   const float* topk_w, const void* y_shared, const void* residual,
                                   double p, const uint64_t* rng, void* y, cudaStream_t st) {
    const DropRule rule = drop_rule(p);
    return s.dtype == MOE_BF16 ? combine_dropout_t<bf16>(s, y_perm, inv_perm, topk_w, y_shared,
                                                         residual, rule, rng, y, st)
                               : combine_dropout_t<float>(s, y_perm, inv_perm, topk_w, y_shared,
                                                          residual, rule, rng, y, st);
}

cudaError_t launch_combine_backward(const moe_shape& s, const void* d_y, const void* y_perm,
                                    const int32_t* inv_perm, const float* topk_w, double p,
                                    const uint64_t* rng, void* d_y_perm, float* d_topk_w,
                                    void* d_shared, cudaStream_t st) {
    const DropRule rule = drop_rule(p);
    return s.dtype == MOE_BF16
               ? combine_backward_t<bf16>(s, d_y, y_perm, inv_perm, topk_w, rule, rng, d_y_perm,
                                          d_topk_w, d_shared, st)
               : combine_backward_t<float>(s, d_y, y_perm, inv_perm, topk_w, rule, rng, d_y_perm,
                                           d_topk_w, d_shared, st);
}

}  // namespace moe
