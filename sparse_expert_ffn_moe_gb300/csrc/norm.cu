// norm.cu -- root-mean-square norm of the rows in front of the experts, with the
// residual's addition and an 8-bit output, and its backward pass.
//
//   s = x + residual, as the residual stream holds it (rounded to the row type)
//   r = 1 / sqrt(mean(s^2) + eps),  y = (s r) w
//   codes = E4M3 nearest to y / scale, scale = max|y| / 448 of the row
//
// A row is read once and stays in registers between the sums and the stores:
// sum(s^2) and max|s w| come from one reduction (max|y| = r max|s w|), so a row
// costs its bytes and one block barrier.  A row goes to a team of threads: 4 to
// 32 lanes of a warp (rows of at most 128 16-byte vectors), else a whole block.
//
// Rows that no 16-byte vector tiles (width odd, say) are read through the
// aligned vectors that cover them; the two at the ends go by element.
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kTeamThreads = 256;   // block of the variants whose team is part of a warp
constexpr int kBlockThreads = 512;  // most threads of the variants whose team is the block

__device__ __forceinline__ uint4 pack(const float (&f)[4], const float*) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
}
__device__ __forceinline__ uint4 pack(const float (&f)[8], const bf16*) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// Where a lane's vectors of a row lie: vector j is elements at(j) .. at(j) + V - 1 of
// the whole array, of which [a0, a1) belong to the row.
template <typename T, bool AL>
struct Span {
    static constexpr int V = Elem<T>::kPerVec;
    int64_t a0, a1, v0;
    __device__ __forceinline__ Span(int64_t row, int d) {
        a0 = row * d;
        a1 = a0 + d;
        v0 = a0 / V * V;
    }
    __device__ __forceinline__ int64_t at(int i) const { return v0 + (int64_t)i * V; }
    __device__ __forceinline__ bool any(int64_t e) const { return e < a1; }
    __device__ __forceinline__ bool whole(int64_t e) const {
        return AL || (e >= a0 && e + V <= a1);
    }
};

// the vector at element e of p, elements outside the row 0
template <typename T, bool AL>
__device__ __forceinline__ uint4 load_vec(const T* p, const Span<T, AL>& sp, int64_t e) {
    if (sp.whole(e)) return *reinterpret_cast<const uint4*>(p + e);
    float f[Span<T, AL>::V];
#pragma unroll
    for (int k = 0; k < Span<T, AL>::V; ++k)
        f[k] = (e + k >= sp.a0 && e + k < sp.a1) ? Elem<T>::to_f32(p[e + k]) : 0.0f;
    return pack(f, (const T*)nullptr);
}

template <typename T, bool AL>
__device__ __forceinline__ void store_vec(T* p, const Span<T, AL>& sp, int64_t e, const uint4& v) {
    if (sp.whole(e)) {
        *reinterpret_cast<uint4*>(p + e) = v;
        return;
    }
    float f[Span<T, AL>::V];
    unpack(v, f, (const T*)nullptr);
#pragma unroll
    for (int k = 0; k < Span<T, AL>::V; ++k)
        if (e + k >= sp.a0 && e + k < sp.a1) p[e + k] = Elem<T>::from_f32(f[k]);
}

// (sum, max) or (sum, sum) over the team, in every thread.  TEAM 0: the block, through
// `red` (one of two buffers in turn, so that one barrier a row is enough).
template <int TEAM, bool MAX>
__device__ __forceinline__ void team_reduce(float& a, float& b, float2* red) {
    constexpr int W = TEAM ? TEAM : 32;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        const float t = __shfl_xor_sync(0xffffffffu, b, o);
        b = MAX ? fmaxf(b, t) : b + t;
    }
    if constexpr (TEAM == 0) {
        const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
        if (lane == 0) red[threadIdx.x >> 5] = make_float2(a, b);
        __syncthreads();
        const float2 v = lane < warps ? red[lane] : make_float2(0.0f, 0.0f);
        a = v.x;
        b = v.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            const float t = __shfl_xor_sync(0xffffffffu, b, o);
            b = MAX ? fmaxf(b, t) : b + t;
        }
    }
}

// the weights of the vector at element e
template <typename T, bool AL>
__device__ __forceinline__ void load_weight(const T* w, const Span<T, AL>& sp, int64_t e,
                                            float (&f)[Span<T, AL>::V]) {
    if constexpr (AL) {
        if (e < sp.a1) unpack(ld_ro(w + (e - sp.a0)), f, (const T*)nullptr);
        else
#pragma unroll
            for (int k = 0; k < Span<T, AL>::V; ++k) f[k] = 0.0f;
    } else {
#pragma unroll
        for (int k = 0; k < Span<T, AL>::V; ++k)
            f[k] = (e + k >= sp.a0 && e + k < sp.a1) ? Elem<T>::to_f32(__ldg(w + (e + k - sp.a0)))
                                                     : 0.0f;
    }
}

template <typename T, int TEAM, int VPT, bool AL>
__global__ void __launch_bounds__(TEAM ? kTeamThreads : kBlockThreads, VPT <= 4 ? 2 : 1)
rmsnorm_kernel(const T* x, const T* residual, const T* __restrict__ weight, float eps, T* s_out,
               T* y, uint8_t* codes, float* __restrict__ scales, int64_t rows, int d) {
    constexpr int V = Elem<T>::kPerVec;
    __shared__ float2 red[2][32];
    pdl_wait();
    pdl_trigger();
    const int team = TEAM ? TEAM : blockDim.x;
    const int lane = TEAM ? threadIdx.x % (TEAM ? TEAM : 1) : threadIdx.x;
    const int per_block = TEAM ? kTeamThreads / (TEAM ? TEAM : 1) : 1;
    const int64_t stride = (int64_t)gridDim.x * per_block;
    // every team of a block runs as many turns as its first, for the warp-wide shuffles
    const int64_t first = (int64_t)blockIdx.x * per_block;
    const int64_t turns = first < rows ? (rows - first + stride - 1) / stride : 0;
    int64_t row = first + (TEAM ? threadIdx.x / (TEAM ? TEAM : 1) : 0);
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const float inv_d = 1.0f / (float)d;
    for (int64_t it = 0; it < turns; ++it, row += stride) {
        const Span<T, AL> sp(row, d);
        const bool live = row < rows;
        uint4 sv[VPT];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int64_t e = sp.at(lane + j * team);
            sv[j] = live && sp.any(e) ? load_vec<T, AL>(x, sp, e) : zero;
        }
        if (residual) {
            uint4 rv[VPT];
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int64_t e = sp.at(lane + j * team);
                rv[j] = live && sp.any(e) ? load_vec<T, AL>(residual, sp, e) : zero;
            }
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                float f[V], g[V];
                unpack(sv[j], f, (const T*)nullptr);
                unpack(rv[j], g, (const T*)nullptr);
#pragma unroll
                for (int k = 0; k < V; ++k) f[k] += g[k];
                sv[j] = pack(f, (const T*)nullptr);
            }
        }
        float sum = 0.0f, top = 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            float f[V], g[V];
            unpack(sv[j], f, (const T*)nullptr);
#pragma unroll
            for (int k = 0; k < V; ++k) sum = fmaf(f[k], f[k], sum);
            if (codes) {
                load_weight<T, AL>(weight, sp, sp.at(lane + j * team), g);
#pragma unroll
                for (int k = 0; k < V; ++k) top = fmaxf(top, fabsf(f[k] * g[k]));
            }
        }
        team_reduce<TEAM, true>(sum, top, red[it & 1]);
        if (!live) continue;  // the last turn of a block of teams
        const float r = 1.0f / sqrtf(fmaf(sum, inv_d, eps));
        const float most = top * r;
        const float scale = most > 0.0f ? most / 448.0f : 1.0f;
        const float inv_scale = 1.0f / scale;
        if (codes && lane == 0) scales[row] = scale;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int64_t e = sp.at(lane + j * team);
            if (!sp.any(e)) continue;
            float f[V], g[V];
            if (s_out) store_vec<T, AL>(s_out, sp, e, sv[j]);
            unpack(sv[j], f, (const T*)nullptr);
            load_weight<T, AL>(weight, sp, e, g);
#pragma unroll
            for (int k = 0; k < V; ++k) f[k] = f[k] * r * g[k];
            if (y) store_vec<T, AL>(y, sp, e, pack(f, (const T*)nullptr));
            if (codes) {
                uint32_t c[V / 4];
#pragma unroll
                for (int k = 0; k < V / 4; ++k) {
                    const uint32_t lo = __nv_cvt_float2_to_fp8x2(
                        make_float2(f[4 * k] * inv_scale, f[4 * k + 1] * inv_scale), __NV_SATFINITE,
                        __NV_E4M3);
                    const uint32_t hi = __nv_cvt_float2_to_fp8x2(
                        make_float2(f[4 * k + 2] * inv_scale, f[4 * k + 3] * inv_scale),
                        __NV_SATFINITE, __NV_E4M3);
                    c[k] = lo | hi << 16;
                }
                if (sp.whole(e)) {
                    if constexpr (V == 8)
                        *reinterpret_cast<uint2*>(codes + e) = make_uint2(c[0], c[V / 4 - 1]);
                    else
                        *reinterpret_cast<uint32_t*>(codes + e) = c[0];
                } else {
#pragma unroll
                    for (int k = 0; k < V; ++k)
                        if (e + k >= sp.a0 && e + k < sp.a1)
                            codes[e + k] = (uint8_t)(c[k / 4] >> (8 * (k & 3)));
                }
            }
        }
    }
}

// ---------------------------------------------------------------- backward
// g = d_y w, xh = s r:   d_x = d_s + r (g - xh mean(g xh)),   d_w = sum over rows of d_y xh
// From sum(s^2) and sum(g s), one reduction a row.  A thread keeps its columns for all
// of its block's rows, so d_w is summed in registers, once per block over its teams,
// and then by rmsnorm_dw_kernel over the blocks, always in the same order.
// W elements a load: a 16-byte vector, or 1 for rows that vectors do not tile (the
// columns of a thread have to be the same in every row).
template <typename T, int W> struct Raw { using type = uint4; };
template <typename T> struct Raw<T, 1> { using type = T; };

template <typename T, int W>
__device__ __forceinline__ void open(const typename Raw<T, W>::type& v, float (&f)[W]) {
    if constexpr (W == 1) f[0] = Elem<T>::to_f32(v);
    else unpack(v, f, (const T*)nullptr);
}

// block-sized teams: most threads, by the registers that a thread's columns take
template <int W> constexpr int kBackThreads = W == 1 ? 1024 : 512;

template <typename T, int TEAM, int VPT, int W>
__global__ void __launch_bounds__(TEAM ? kTeamThreads : kBackThreads<W>, W > 1 && VPT <= 2 ? 2 : 1)
rmsnorm_backward_kernel(const T* d_y, const T* s, const T* __restrict__ weight, float eps,
                        const T* d_s, T* d_x, float* __restrict__ part, int64_t rows, int d) {
    using R = typename Raw<T, W>::type;
    extern __shared__ float acc_sm[];
    __shared__ float2 red[2][32];
    pdl_wait();
    pdl_trigger();
    const int team = TEAM ? TEAM : blockDim.x;
    const int lane = TEAM ? threadIdx.x % (TEAM ? TEAM : 1) : threadIdx.x;
    const int per_block = TEAM ? kTeamThreads / (TEAM ? TEAM : 1) : 1;
    const int64_t stride = (int64_t)gridDim.x * per_block;
    const int64_t first = (int64_t)blockIdx.x * per_block;
    const int64_t turns = first < rows ? (rows - first + stride - 1) / stride : 0;
    int64_t row = first + (TEAM ? threadIdx.x / (TEAM ? TEAM : 1) : 0);
    float acc[VPT][W];
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int k = 0; k < W; ++k) acc[j][k] = 0.0f;
    const R zero = R{};
    const float inv_d = 1.0f / (float)d;
    for (int64_t it = 0; it < turns; ++it, row += stride) {
        const bool live = row < rows;
        R sv[VPT], yv[VPT];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = (lane + j * team) * W;
            const bool go = live && c < d;
            sv[j] = go ? *reinterpret_cast<const R*>(s + row * d + c) : zero;
            yv[j] = go ? *reinterpret_cast<const R*>(d_y + row * d + c) : zero;
        }
        float sq = 0.0f, gs = 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = (lane + j * team) * W;
            float fs[W], fy[W], fw[W];
            open<T, W>(sv[j], fs);
            open<T, W>(yv[j], fy);
            open<T, W>(c < d ? __ldg(reinterpret_cast<const R*>(weight + c)) : zero, fw);
#pragma unroll
            for (int k = 0; k < W; ++k) {
                sq = fmaf(fs[k], fs[k], sq);
                gs = fmaf(fy[k] * fw[k], fs[k], gs);
            }
        }
        team_reduce<TEAM, false>(sq, gs, red[it & 1]);
        const float r = 1.0f / sqrtf(fmaf(sq, inv_d, eps));
        const float back = gs * inv_d * r * r;  // times s: what the bracket takes off
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = (lane + j * team) * W;
            if (!live || c >= d) continue;
            float fs[W], fy[W], fw[W], fa[W];
            open<T, W>(sv[j], fs);
            open<T, W>(yv[j], fy);
#pragma unroll
            for (int k = 0; k < W; ++k) acc[j][k] = fmaf(fy[k], fs[k] * r, acc[j][k]);
            if (!d_x) continue;
            open<T, W>(__ldg(reinterpret_cast<const R*>(weight + c)), fw);
            open<T, W>(d_s ? *reinterpret_cast<const R*>(d_s + row * d + c) : zero, fa);
#pragma unroll
            for (int k = 0; k < W; ++k)
                fa[k] = fmaf(r, fmaf(-back, fs[k], fy[k] * fw[k]), fa[k]);
            if constexpr (W == 1) d_x[row * d + c] = Elem<T>::from_f32(fa[0]);
            else *reinterpret_cast<uint4*>(d_x + row * d + c) = pack(fa, (const T*)nullptr);
        }
    }
    if (!part) return;
    if constexpr (TEAM == 0) {
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int k = 0; k < W; ++k)
                if ((lane + j * team) * W < d)
                    part[(int64_t)blockIdx.x * d + (lane + j * team) * W + k] = acc[j][k];
    } else {
        // acc_sm[team of the block][columns of a team]
        constexpr int kCols = TEAM * VPT * W;
        const int mine = threadIdx.x / TEAM;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int k = 0; k < W; ++k) acc_sm[mine * kCols + (lane + j * TEAM) * W + k] = acc[j][k];
        __syncthreads();
        for (int c = threadIdx.x; c < d; c += kTeamThreads) {
            float t = 0.0f;
            for (int q = 0; q < kTeamThreads / TEAM; ++q) t += acc_sm[q * kCols + c];
            part[(int64_t)blockIdx.x * d + c] = t;
        }
    }
}

// d_w[c] = sum over the blocks' partial rows: 32 columns a block, 32 strands of rows
__global__ void __launch_bounds__(1024)
rmsnorm_dw_kernel(const float* __restrict__ part, int n, int d, float* __restrict__ d_weight) {
    __shared__ float sm[32][33];
    pdl_wait();
    pdl_trigger();
    const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + cx;
    float t = 0.0f;
    if (c < d) {
#pragma unroll 4
        for (int q = ry; q < n; q += 32) t += part[(int64_t)q * d + c];
    }
    sm[ry][cx] = t;
    __syncthreads();
    // column ry of the block's 32, its strands in the lanes
    float v = warp_sum(sm[cx][ry]);
    if (cx == 0 && blockIdx.x * 32 + ry < d) d_weight[blockIdx.x * 32 + ry] = v;
}

template <typename K>
int blocks_that_fit(K kernel, int threads, size_t smem) {
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem) != cudaSuccess) n = 1;
    return (n > 0 ? n : 1) * device_sm_count();
}

template <typename T, int TEAM, int VPT, bool AL>
cudaError_t go_forward(const NormArgs& a, int threads, cudaStream_t st) {
    auto kernel = rmsnorm_kernel<T, TEAM, VPT, AL>;
    const int per_block = TEAM ? kTeamThreads / (TEAM ? TEAM : 1) : 1;
    const int64_t want = ceil_div(a.rows, per_block);
    const int64_t wave = blocks_that_fit(kernel, threads, 0);
    return launch_pdl(kernel, dim3((unsigned)(want < wave ? want : wave)), dim3(threads), 0, st,
                      (const T*)a.x, (const T*)a.residual, (const T*)a.weight, a.eps, (T*)a.s,
                      (T*)a.y, a.codes, a.scales, a.rows, a.d);
}

template <typename T, bool AL>
cudaError_t pick_forward(const NormArgs& a, cudaStream_t st) {
    // vectors that cover a row, wherever it starts
    const int nv = (int)ceil_div(a.d, Elem<T>::kPerVec) + (AL ? 0 : 1);
    if (nv <= 4) return go_forward<T, 4, 1, AL>(a, kTeamThreads, st);
    if (nv <= 8) return go_forward<T, 8, 1, AL>(a, kTeamThreads, st);
    if (nv <= 16) return go_forward<T, 16, 1, AL>(a, kTeamThreads, st);
    if (nv <= 32) return go_forward<T, 32, 1, AL>(a, kTeamThreads, st);
    if (nv <= 64) return go_forward<T, 32, 2, AL>(a, kTeamThreads, st);
    if (nv <= 128) return go_forward<T, 32, 4, AL>(a, kTeamThreads, st);
    const auto warps = [](int64_t lanes) { return (int)ceil_div(lanes, 32) * 32; };
    if (nv <= 2 * kBlockThreads) return go_forward<T, 0, 2, AL>(a, warps(ceil_div(nv, 2)), st);
    // the widest row (16384 values) has 4096 vectors of fp32 or 2048 of bf16, and one
    // more where it starts within a vector
    if constexpr (Elem<T>::kPerVec == 4) {
        if (nv > 4 * kBlockThreads)
            return go_forward<T, 0, AL ? 8 : 9, AL>(a, warps(ceil_div(nv, AL ? 8 : 9)), st);
        return go_forward<T, 0, 4, AL>(a, warps(ceil_div(nv, 4)), st);
    } else {
        return go_forward<T, 0, AL ? 4 : 5, AL>(a, warps(ceil_div(nv, AL ? 4 : 5)), st);
    }
}

template <typename T, int TEAM, int VPT, int W>
cudaError_t go_backward(const NormArgs& a, int threads, int blocks, cudaStream_t st) {
    auto kernel = rmsnorm_backward_kernel<T, TEAM, VPT, W>;
    const size_t smem = TEAM ? sizeof(float) * kTeamThreads * VPT * W : 0;
    return launch_pdl(kernel, dim3(blocks), dim3(threads), smem, st, (const T*)a.d_y,
                      (const T*)a.x, (const T*)a.weight, a.eps, (const T*)a.d_s, (T*)a.d_x, a.part,
                      a.rows, a.d);
}

// lanes of a team (0: a block of threads) and vectors a lane for rows of nv vectors
struct Team {
    int lanes, vpt, threads;
};

Team team_for(int nv, bool vec) {
    if (nv <= 4) return {4, 1, kTeamThreads};
    if (nv <= 8) return {8, 1, kTeamThreads};
    if (nv <= 16) return {16, 1, kTeamThreads};
    if (nv <= 32) return {32, 1, kTeamThreads};
    if (nv <= 64) return {32, 2, kTeamThreads};
    if (nv <= 128) return {32, 4, kTeamThreads};
    const auto warps = [](int64_t lanes) { return (int)ceil_div(lanes, 32) * 32; };
    const int most = vec ? kBackThreads<8> : kBackThreads<1>;
    if (nv <= 2 * most) return {0, 2, warps(ceil_div(nv, 2))};
    if (nv <= 4 * most) return {0, 4, warps(ceil_div(nv, 4))};
    return vec ? Team{0, 8, warps(ceil_div(nv, 8))} : Team{0, 16, warps(ceil_div(nv, 16))};
}

template <typename T, int W>
cudaError_t pick_backward(const NormArgs& a, const Team& t, int blocks, cudaStream_t st) {
    if (t.lanes == 4) return go_backward<T, 4, 1, W>(a, t.threads, blocks, st);
    if (t.lanes == 8) return go_backward<T, 8, 1, W>(a, t.threads, blocks, st);
    if (t.lanes == 16) return go_backward<T, 16, 1, W>(a, t.threads, blocks, st);
    if (t.lanes == 32 && t.vpt == 1) return go_backward<T, 32, 1, W>(a, t.threads, blocks, st);
    if (t.lanes == 32 && t.vpt == 2) return go_backward<T, 32, 2, W>(a, t.threads, blocks, st);
    if (t.lanes == 32) return go_backward<T, 32, 4, W>(a, t.threads, blocks, st);
    if (t.vpt == 2) return go_backward<T, 0, 2, W>(a, t.threads, blocks, st);
    if (t.vpt == 4) return go_backward<T, 0, 4, W>(a, t.threads, blocks, st);
    if constexpr (W == 8) return cudaErrorInvalidValue;  // 16384 bf16 values: 4 vectors a thread
    else return go_backward<T, 0, W == 1 ? 16 : 8, W>(a, t.threads, blocks, st);
}

// 16-byte vectors tile the rows
bool whole_vectors(int dtype, int d) { return d % (dtype == MOE_BF16 ? 8 : 4) == 0; }

Team backward_team(int dtype, int d) {
    const bool vec = whole_vectors(dtype, d);
    return team_for(vec ? d / (dtype == MOE_BF16 ? 8 : 4) : d, vec);
}

}  // namespace

cudaError_t launch_rmsnorm(const NormArgs& a, cudaStream_t st) {
    const bool al = whole_vectors(a.dtype, a.d);
    if (a.dtype == MOE_BF16)
        return al ? pick_forward<bf16, true>(a, st) : pick_forward<bf16, false>(a, st);
    return al ? pick_forward<float, true>(a, st) : pick_forward<float, false>(a, st);
}

// Partial rows of d_w: counted for 152 SMs, not asked of the device, so that the
// workspace query needs no device and the order of the sums depends on the sizes alone.
int rmsnorm_backward_blocks(int64_t rows, int d) {
    // the larger of the two types' counts (their teams may differ)
    int most = 1;
    for (int dtype : {(int)MOE_F32, (int)MOE_BF16}) {
        const Team t = backward_team(dtype, d);
        const int per_block = t.lanes ? kTeamThreads / t.lanes : 1;
        const int wave = 152 * (t.lanes ? 4 : t.threads > 512 ? 1 : 1024 / t.threads);
        const int64_t want = ceil_div(rows, per_block);
        const int n = (int)(want < wave ? want : wave);
        most = n > most ? n : most;
    }
    return most;
}

cudaError_t launch_rmsnorm_backward(const NormArgs& a, cudaStream_t st) {
    const Team t = backward_team(a.dtype, a.d);
    const int per_block = t.lanes ? kTeamThreads / t.lanes : 1;
    const int wave = 152 * (t.lanes ? 4 : t.threads > 512 ? 1 : 1024 / t.threads);
    const int64_t want = ceil_div(a.rows, per_block);
    const int blocks = (int)(want < wave ? want : wave);
    cudaError_t e;
    const bool vec = whole_vectors(a.dtype, a.d);
    if (a.dtype == MOE_BF16)
        e = vec ? pick_backward<bf16, 8>(a, t, blocks, st) : pick_backward<bf16, 1>(a, t, blocks, st);
    else
        e = vec ? pick_backward<float, 4>(a, t, blocks, st)
                : pick_backward<float, 1>(a, t, blocks, st);
    if (e != cudaSuccess || !a.part) return e;
    return launch_pdl(rmsnorm_dw_kernel, dim3((unsigned)ceil_div(a.d, 32)), dim3(1024), 0, st,
                      (const float*)a.part, blocks, a.d, a.d_weight);
}

}  // namespace moe
