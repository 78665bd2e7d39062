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
// 16-byte vectors.
#include "internal.h"
#include "philox.cuh"

namespace moe {

namespace {

// A thread takes groups of eight elements, gridDim.x * 256 apart and two at a time,
// and draws their bits while their loads are on their way.  16384 x 7168 bf16 with
// residual takes 102 us (705 MB, 6.9 TB/s; one group at a time 108 us); masks
// gathered into a byte before use took 156 us, the integer work then bounding it.
// Without residual that work, about 140 instructions a group, weighs more: 15920 x
// 3080 takes 35 us (5.5 TB/s; 41 us one at a time).  40 blocks an SM are
// the best of both: 8 to 24 cost fp32 up to a fifth, 64 and more bf16 a tenth.
constexpr int kGroups = 2, kDropoutBlocks = 40;
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
    for (int64_t g0 = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; g0 < groups;
         g0 += kGroups * stride) {
        Unit<T> v[kGroups], r[kGroups];
        Bits8 bits[kGroups] = {};
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int64_t g = g0 + i * stride;
            if (g < groups) {
                v[i] = load_unit(x + g * 8);
                if (residual) r[i] = load_unit(residual + g * 8);
            }
        }
#pragma unroll
        for (int i = 0; i < kGroups; ++i)
            if (rule.thr) bits[i] = draw8((uint64_t)(g0 + i * stride), st);
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int64_t g = g0 + i * stride;
            if (g >= groups) break;
            float f[8];
            widen(v[i], f);
            if (rule.thr) drop8(f, bits[i], rule);
            if (residual) {
                float rf[8];
                widen(r[i], rf);
#pragma unroll
                for (int k = 0; k < 8; ++k) f[k] += rf[k];
            }
            store_unit(y + g * 8, f);
        }
    }
    // the last, partial group
    if (blockIdx.x == 0 && threadIdx.x == 0 && n % 8) {
        const int64_t base = groups * 8;
        const int m = (int)(n - base);
        float f[8] = {};
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < m) f[k] = Elem<T>::to_f32(x[base + k]);
        if (rule.thr) drop8(f, draw8((uint64_t)groups, st), rule);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (k >= m) continue;
            if (residual) f[k] += Elem<T>::to_f32(residual[base + k]);
            y[base + k] = Elem<T>::from_f32(f[k]);
        }
    }
}

// The routed rows of one token, as each of its warps sees them (whole warps work
// on one token): lane j holds slot j's row (-1: dropped) and weight.
struct Slots {
    int32_t p;
    float w;
};
__device__ __forceinline__ Slots load_slots(const int32_t* __restrict__ inv_perm,
                                            const float* __restrict__ topk_w, int64_t t, int K,
                                            int64_t n_rows, bool on) {
    const int lane = threadIdx.x & 31;
    Slots s{-1, 0.f};
    if (on && lane < K) {
        s.p = __ldg(inv_perm + t * K + lane);
        if (s.p >= n_rows) s.p = -1;
        if (topk_w) s.w = __ldg(topk_w + t * K + lane);
    }
    return s;
}

// KB rows from slot j0 on, V groups of eight elements a thread from group u0 on,
// blockDim.x apart; zeros for slots that are dropped or beyond K
template <typename T, int V, int KB>
__device__ __forceinline__ void load_rows(Unit<T> (&row)[KB][V], const T* y_perm, const Slots& s,
                                          int j0, int K, int d, int u0) {
#pragma unroll
    for (int j = 0; j < KB; ++j) {
        const int32_t p = __shfl_sync(0xffffffffu, s.p, (j0 + j) & 31);
        const bool any = j0 + j < K && p >= 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int u = u0 + i * blockDim.x;
            row[j][i] = Unit<T>{};
            if (any && u < d / 8) row[j][i] = load_unit(y_perm + (int64_t)p * d + (int64_t)u * 8);
        }
    }
}

// A warp sums V groups of eight elements a lane of one token's output row, KB
// slots at a time, the next ones asked for as soon as those are used; the mask is
// drawn while the first are on their way.  Bound by HBM.  Warps that depend on
// nothing but themselves, two a block, keep the loads coming: T = 16384, d = 7168,
// K = 8 bf16 with shared expert and residual takes 386 us (6.70 TB/s), blocks of 224
// threads 418 us, four slots at a time 397 us, one group a lane 450 us.  A row of at
// most 32 groups has one a lane, and there four slots at a time take 20 us against
// 22 (T = 32768, d = 256, K = 4).
// (The bound of 256 threads has the compiler spend few enough registers for 20
// and more blocks of 64 an SM: with a bound of 64 the same call takes 400 us.)
template <typename T, int V, int KB>
__global__ void __launch_bounds__(256)
combine_dropout_kernel(const T* y_perm, const int32_t* __restrict__ inv_perm,
                       const float* __restrict__ topk_w, const T* y_shared, const T* residual,
                       T* y, int n_tokens, int d, int K, int64_t n_rows, DropRule rule,
                       const uint64_t* __restrict__ rng) {
    pdl_wait();
    pdl_trigger();
    const int units = d / 8, u0 = blockIdx.y * blockDim.x * V + threadIdx.x;
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool on = t < n_tokens;
    const Slots slots = load_slots(inv_perm, topk_w, t, K, n_rows, on);
    Unit<T> sh[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int u = u0 + i * blockDim.x;
        const int64_t at = t * d + (int64_t)u * 8;
        sh[i] = Unit<T>{};
        if (y_shared && on && u < units) sh[i] = load_unit(y_shared + at);
    }
    Unit<T> row[KB][V];
    load_rows(row, y_perm, slots, 0, K, d, u0);
    Bits8 bits[V] = {};
    if (rule.thr) {
        const RngState st = load_rng(rng);
#pragma unroll
        for (int i = 0; i < V; ++i)
            bits[i] = draw8((uint64_t)(t * units + u0 + i * blockDim.x), st);
    }
    float acc[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) widen(sh[i], acc[i]);
    for (int j0 = 0;;) {
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            const float w = __shfl_sync(0xffffffffu, slots.w, (j0 + j) & 31);
            const bool any =
                __shfl_sync(0xffffffffu, slots.p, (j0 + j) & 31) >= 0 && j0 + j < K;
            if (!any) continue;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float f[8];
                widen(row[j][i], f);
#pragma unroll
                for (int k = 0; k < 8; ++k) acc[i][k] = fmaf(w, f[k], acc[i][k]);
            }
        }
        j0 += KB;
        if (j0 >= K) break;
        load_rows(row, y_perm, slots, j0, K, d, u0);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int u = u0 + i * blockDim.x;
        if (!on || u >= units) continue;
        const int64_t at = t * d + (int64_t)u * 8;
        Unit<T> res;
        if (residual) res = load_unit(residual + at);
        if (rule.thr) drop8(acc[i], bits[i], rule);
        if (residual) {
            float f[8];
            widen(res, f);
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[i][k] += f[k];
        }
        store_unit(y + at, acc[i]);
    }
}

// A token's threads (blockDim.x of them, blockDim.y tokens a block) hold dz in
// registers, V groups of eight elements each, and walk the token's K rows, KB at a
// time and the next ones on their way while the gradients of these are written.
// The K dot products are summed in a fixed order: a thread's elements, lanes,
// warps.  Bound by HBM: T = 16384, d = 7168, K = 8 bf16 takes 615 us for 4.23 GB
// (6.88 TB/s, the measured copy's rate); four groups a thread without the
// look-ahead took 774 us, one row at a time 698 us.  (Four groups a thread, K <= 2, spill 64
// bytes at the 64 registers that the bound of 1024 threads leaves.)
template <typename T, int V, int KB>
__global__ void __launch_bounds__(V == 1 ? 256 : 1024)
combine_backward_kernel(const T* d_y, const T* y_perm, const int32_t* __restrict__ inv_perm,
                        const float* __restrict__ topk_w, T* d_y_perm, float* d_topk_w, T* d_shared,
                        int n_tokens, int d, int K, int64_t n_rows, DropRule rule,
                        const uint64_t* __restrict__ rng) {
    __shared__ float red[32][32];  // [warp of the block][slot]
    pdl_wait();
    pdl_trigger();
    const int units = d / 8;
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int lane = threadIdx.x & 31, nwarps = blockDim.x >> 5;
    const int warp = threadIdx.y * nwarps + (threadIdx.x >> 5);
    const bool on = t < n_tokens;
    const Slots slots = load_slots(inv_perm, d_y_perm ? topk_w : nullptr, t, K, n_rows, on);
    Unit<T> raw[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int u = threadIdx.x + i * blockDim.x;
        raw[i] = Unit<T>{};
        if (on && u < units) raw[i] = load_unit(d_y + t * d + (int64_t)u * 8);
    }
    Unit<T> row[KB][V];
    if (d_topk_w) load_rows(row, y_perm, slots, 0, K, d, threadIdx.x);
    float dz[V][8];
    RngState st = {};
    if (rule.thr) st = load_rng(rng);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        Bits8 bits = {};
        if (rule.thr) bits = draw8((uint64_t)(t * units + threadIdx.x + i * blockDim.x), st);
        widen(raw[i], dz[i]);
        if (rule.thr) drop8(dz[i], bits, rule);
    }
    if (d_shared && on) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int u = threadIdx.x + i * blockDim.x;
            if (u < units) store_unit(d_shared + t * d + (int64_t)u * 8, dz[i]);
        }
    }
    for (int j0 = 0; j0 < K; j0 += KB) {
        if (d_topk_w) {
            float dot[KB];
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                dot[j] = 0.f;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float f[8];
                    widen(row[j][i], f);
#pragma unroll
                    for (int k = 0; k < 8; ++k) dot[j] = fmaf(dz[i][k], f[k], dot[j]);
                }
            }
            if (j0 + KB < K) load_rows(row, y_perm, slots, j0 + KB, K, d, threadIdx.x);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
#pragma unroll
                for (int j = 0; j < KB; ++j) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
#pragma unroll
            for (int j = 0; j < KB; ++j)
                if (lane == 0 && j0 + j < K) red[warp][j0 + j] = dot[j];
        }
        if (d_y_perm) {
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                if (j0 + j >= K) break;
                const int32_t p = __shfl_sync(0xffffffffu, slots.p, j0 + j);
                const float w = __shfl_sync(0xffffffffu, slots.w, j0 + j);
                if (p < 0) continue;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int u = threadIdx.x + i * blockDim.x;
                    if (u >= units) continue;
                    float f[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) f[k] = w * dz[i][k];
                    store_unit(d_y_perm + (int64_t)p * d + (int64_t)u * 8, f);
                }
            }
        }
    }
    __syncthreads();
    if (d_topk_w && on && threadIdx.x < K) {
        float s = 0.f;
        for (int w = 0; w < nwarps; ++w) s += red[threadIdx.y * nwarps + w][threadIdx.x];
        // this lane's slot; a dropped one has 0, whatever dz holds
        d_topk_w[t * K + threadIdx.x] = slots.p >= 0 ? s : 0.f;
    }
}

template <typename T>
cudaError_t dropout_t(int64_t n, const void* x, const void* residual, DropRule rule,
                      const uint64_t* rng, void* y, cudaStream_t st) {
    const int64_t blocks = ceil_div(n / 8 > 0 ? n / 8 : 1, 256);
    const int64_t most = (int64_t)device_sm_count() * kDropoutBlocks;
    return launch_pdl(dropout_kernel<T>, dim3((unsigned)(blocks < most ? blocks : most)), dim3(256),
                      0, st, (const T*)x, (const T*)residual, (T*)y, n, rule, rng);
}

template <typename T, int V, int KB>
cudaError_t combine_dropout_v(const moe_shape& s, const void* y_perm, const int32_t* inv_perm,
                              const float* topk_w, const void* y_shared, const void* residual,
                              DropRule rule, const uint64_t* rng, void* y, cudaStream_t st) {
    const dim3 block(32, 2);
    const dim3 grid((unsigned)ceil_div(s.T, 2), (unsigned)ceil_div(s.d / 8, 32 * V));
    return launch_pdl(combine_dropout_kernel<T, V, KB>, grid, block, 0, st, (const T*)y_perm, inv_perm,
                      topk_w, (const T*)y_shared, (const T*)residual, (T*)y, s.T, s.d, s.K,
                      (int64_t)s.T * s.K, rule, rng);
}

// Two groups a lane, unless that leaves more than an eighth of the lanes' groups
// beyond the row (T = 29639, d = 576, K = 8: 76 us, with two 84 us)
template <typename T, typename... Args>
cudaError_t combine_dropout_t(const moe_shape& s, Args... args) {
    const int64_t units = s.d / 8, held = ceil_div(units, 64) * 64;
    return held * 8 <= units * 9 ? combine_dropout_v<T, 2, 1>(s, args...)
                                 : combine_dropout_v<T, 1, 4>(s, args...);
}

template <typename T, int V, int KB>
cudaError_t combine_backward_v(const moe_shape& s, const void* d_y, const void* y_perm,
                               const int32_t* inv_perm, const float* topk_w, DropRule rule,
                               const uint64_t* rng, void* d_y_perm, float* d_topk_w, void* d_shared,
                               cudaStream_t st) {
    // one token's row in whole warps; several tokens a block of 256 where it is short
    const int x = (int)ceil_div(s.d / 8, V * 32) * 32;
    const dim3 block((unsigned)x, (unsigned)(256 / x > 0 ? 256 / x : 1));
    return launch_pdl(combine_backward_kernel<T, V, KB>, dim3((unsigned)ceil_div(s.T, block.y)), block,
                      0, st, (const T*)d_y, (const T*)y_perm, inv_perm, topk_w, (T*)d_y_perm,
                      d_topk_w, (T*)d_shared, s.T, s.d, s.K, (int64_t)s.T * s.K, rule, rng);
}

// What a thread holds: in bf16 two rows of two groups each where a token has more
// than two rows, else four groups of one row (K = 2, T = 4096, d = 4096: 28 us, two
// groups 32 us; K = 1: 36 and 47 us); in fp32 two groups of one row (two rows spill
// 292 bytes: T = 8192, d = 4096, K = 4 with d_shared 290 us against 201 us).  A row of at most 32 groups has one a thread, and two rows
// (d = 256, K = 4: 28 us against 33 us with one).
template <typename T, typename... Args>
cudaError_t combine_backward_t(const moe_shape& s, Args... args) {
    const int units = s.d / 8;
    if (units <= 32) return combine_backward_v<T, 1, 2>(s, args...);
    if constexpr (sizeof(T) == 2) {
        if (s.K > 2) return combine_backward_v<T, 2, 2>(s, args...);
        if (units >= 128) return combine_backward_v<T, 4, 1>(s, args...);
    }
    return combine_backward_v<T, 2, 1>(s, args...);
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
