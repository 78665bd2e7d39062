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

constexpr int kTeamVecs = 64;      // widest row of a team, in vectors
constexpr int kTeamThreads = 256;   // block of the variants whose team is part of a warp

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

// E4M3 codes of the values over the scale, four to a word
template <int N>
__device__ __forceinline__ void to_codes(const float (&f)[N], float inv_scale, uint32_t (&c)[N / 4]) {
#pragma unroll
    for (int k = 0; k < N / 4; ++k) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(
            make_float2(f[4 * k] * inv_scale, f[4 * k + 1] * inv_scale), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(
            make_float2(f[4 * k + 2] * inv_scale, f[4 * k + 3] * inv_scale), __NV_SATFINITE, __NV_E4M3);
        c[k] = lo | hi << 16;
    }
}

template <typename T, int TEAM, int VPT, bool AL, bool RES, bool CODES>
__global__ void __launch_bounds__(kTeamThreads)
rmsnorm_kernel(const T* x, const T* residual, const T* __restrict__ weight, float eps, T* s_out,
               T* y, uint8_t* codes, float* __restrict__ scales, int64_t rows, int d) {
    constexpr int V = Elem<T>::kPerVec;
    pdl_wait();
    pdl_trigger();
    constexpr int team = TEAM, per_block = kTeamThreads / TEAM;
    const int lane = threadIdx.x % TEAM;
    const int64_t stride = (int64_t)gridDim.x * per_block;
    // every team of a block runs as many turns as its first, for the warp-wide shuffles
    const int64_t first = (int64_t)blockIdx.x * per_block;
    const int64_t turns = first < rows ? (rows - first + stride - 1) / stride : 0;
    int64_t row = first + threadIdx.x / TEAM;
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
        if constexpr (RES) {
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
            if constexpr (CODES) {
                load_weight<T, AL>(weight, sp, sp.at(lane + j * team), g);
#pragma unroll
                for (int k = 0; k < V; ++k) top = fmaxf(top, fabsf(f[k] * g[k]));
            }
        }
        team_reduce<TEAM, true>(sum, top, nullptr);
        if (!live) continue;  // the last turn of a block of teams
        const float r = 1.0f / sqrtf(fmaf(sum, inv_d, eps));
        const float most = top * r;
        const float scale = most > 0.0f ? most / 448.0f : 1.0f;
        const float inv_scale = 1.0f / scale;
        if (CODES && lane == 0) scales[row] = scale;
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
            if constexpr (CODES) {
                uint32_t c[V / 4];
                to_codes(f, inv_scale, c);
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

// A wide row of whole vectors: a block of its own, which ends with it.  Many small blocks in
// different parts of their rows keep the memory busy; blocks that stayed for many rows, with
// or without a ring of copies ahead, did not (16384 x 7168 bf16 with residual and codes: 178
// and 186 us, this 161).
template <int VPT> constexpr int kBlockThreads = VPT <= 4 ? 256 : 512;

template <typename T, int VPT, bool RES, bool CODES>
__global__ void __launch_bounds__(kBlockThreads<VPT>, VPT <= 4 ? 4 : 1)
rmsnorm_block_kernel(const T* x, const T* residual, const T* __restrict__ weight, float eps, T* s_out,
                     T* y, uint8_t* codes, float* __restrict__ scales, int d) {
    constexpr int V = Elem<T>::kPerVec;
    __shared__ float2 red[32];
    pdl_wait();
    pdl_trigger();
    const int nt = blockDim.x, vecs = d / V;
    const int64_t at = (int64_t)blockIdx.x * d;
    const uint4* px = reinterpret_cast<const uint4*>(x + at);
    const uint4* pr = reinterpret_cast<const uint4*>(residual + at);
    const T* const no = nullptr;
    uint4 sv[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int c = threadIdx.x + j * nt;
        sv[j] = c < vecs ? px[c] : make_uint4(0u, 0u, 0u, 0u);
    }
    if constexpr (RES) {
        uint4 rv[VPT];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = threadIdx.x + j * nt;
            rv[j] = c < vecs ? pr[c] : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            float f[V], g[V];
            unpack(sv[j], f, no);
            unpack(rv[j], g, no);
#pragma unroll
            for (int k = 0; k < V; ++k) f[k] += g[k];
            sv[j] = pack(f, no);
        }
        if (s_out) {  // may be x or the residual: this thread's values, read above
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int c = threadIdx.x + j * nt;
                if (c < vecs) reinterpret_cast<uint4*>(s_out + at)[c] = sv[j];
            }
        }
    }
    float sum = 0.0f, top = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int c = threadIdx.x + j * nt;
        float f[V], g[V];
        unpack(sv[j], f, no);
#pragma unroll
        for (int k = 0; k < V; ++k) sum = fmaf(f[k], f[k], sum);
        if constexpr (CODES) {
            if (c >= vecs) continue;
            unpack(ld_ro(weight + c * V), g, no);
#pragma unroll
            for (int k = 0; k < V; ++k) top = fmaxf(top, fabsf(f[k] * g[k]));
        }
    }
    team_reduce<0, true>(sum, top, red);
    const float r = 1.0f / sqrtf(fmaf(sum, 1.0f / (float)d, eps));
    const float most = top * r;
    const float scale = most > 0.0f ? most / 448.0f : 1.0f;
    const float inv_scale = 1.0f / scale;
    if (CODES && threadIdx.x == 0) scales[blockIdx.x] = scale;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int c = threadIdx.x + j * nt;
        if (c >= vecs) continue;
        float f[V], g[V];
        unpack(sv[j], f, no);
        unpack(ld_ro(weight + c * V), g, no);
#pragma unroll
        for (int k = 0; k < V; ++k) f[k] = f[k] * r * g[k];
        if (!RES && s_out) reinterpret_cast<uint4*>(s_out + at)[c] = sv[j];
        if (y) reinterpret_cast<uint4*>(y + at)[c] = pack(f, no);
        if constexpr (CODES) {
            uint32_t q[V / 4];
            to_codes(f, inv_scale, q);
            if constexpr (V == 8)
                reinterpret_cast<uint2*>(codes + at)[c] = make_uint2(q[0], q[V / 4 - 1]);
            else
                reinterpret_cast<uint32_t*>(codes + at)[c] = q[0];
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

template <typename T, int TEAM, int VPT, int W>
__global__ void __launch_bounds__(kTeamThreads)
rmsnorm_backward_kernel(const T* d_y, const T* s, const T* __restrict__ weight, float eps,
                        const T* d_s, T* d_x, float* __restrict__ part, int64_t rows, int d) {
    using R = typename Raw<T, W>::type;
    extern __shared__ float acc_sm[];
    pdl_wait();
    pdl_trigger();
    constexpr int team = TEAM, per_block = kTeamThreads / TEAM;
    const int lane = threadIdx.x % TEAM;
    const int64_t stride = (int64_t)gridDim.x * per_block;
    const int64_t first = (int64_t)blockIdx.x * per_block;
    const int64_t turns = first < rows ? (rows - first + stride - 1) / stride : 0;
    int64_t row = first + threadIdx.x / TEAM;
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
        team_reduce<TEAM, false>(sq, gs, nullptr);
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
    {
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

// ---------------------------------------------------------------- rings
// Blocks that stay for many rows copy the next ones to shared memory while they work on one
// (cp.async: neither registers nor barriers hold the copies up).  Used where blocks have to
// stay, for the sums of d_w over rows, and for rows that 16-byte vectors do not tile.
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

constexpr int kDepth = 3;  // rows in a ring, or 1 where three do not fit

constexpr int kRingThreads = 512;
constexpr size_t kRingSmem = 220 * 1024;  // of an SM, for the rings of its blocks

// Rows of whole vectors: each thread copies and reads its own.  s and d_y by way of the ring,
// d_s straight to registers, asked for before the row's sums.
template <typename T, int VPT>
__global__ void __launch_bounds__(kRingThreads, VPT <= 2 ? 2 : 1)
rmsnorm_backward_ring_kernel(const T* d_y, const T* s, const T* __restrict__ weight, float eps,
                             const T* d_s, T* d_x, float* __restrict__ part, int64_t rows, int d) {
    constexpr int V = Elem<T>::kPerVec;
    constexpr int D = VPT <= 4 ? kDepth : 1;  // 8 vectors: fp32 rows of more than 8192
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float2 red[2][32];
    pdl_wait();
    pdl_trigger();
    const int nt = blockDim.x, vecs = d / V, row_bytes = vecs * 16;
    const bool add = d_s && d_x;
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(ring);
    const int64_t stride = gridDim.x;
    const T* const no = nullptr;
    auto fetch = [&](int64_t row, int slot) {
        if (row < rows) {
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int c = threadIdx.x + j * nt;
                if (c < vecs) {
                    const uint32_t dst = base + slot * 2 * row_bytes + c * 16;
                    copy_async(dst, s + row * d + c * V);
                    copy_async(dst + row_bytes, d_y + row * d + c * V);
                }
            }
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < D - 1; ++i) fetch(blockIdx.x + i * stride, i);
    float acc[VPT][V];
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int k = 0; k < V; ++k) acc[j][k] = 0.0f;
    const float inv_d = 1.0f / (float)d;
    int slot = 0, turn = 0;
    for (int64_t row = blockIdx.x; row < rows; row += stride, turn ^= 1) {
        uint4 av[VPT];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = threadIdx.x + j * nt;
            av[j] = add && c < vecs ? *reinterpret_cast<const uint4*>(d_s + row * d + c * V)
                                    : make_uint4(0u, 0u, 0u, 0u);
        }
        if constexpr (D == 1) fetch(row, 0);
        copy_wait<D == 1 ? 0 : D - 2>();
        const uint8_t* mine = ring + slot * 2 * row_bytes;
        float sq = 0.0f, gs = 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = threadIdx.x + j * nt;
            if (c >= vecs) continue;
            float fs[V], fy[V], fw[V];
            unpack(*reinterpret_cast<const uint4*>(mine + c * 16), fs, no);
            unpack(*reinterpret_cast<const uint4*>(mine + row_bytes + c * 16), fy, no);
            unpack(ld_ro(weight + c * V), fw, no);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                sq = fmaf(fs[k], fs[k], sq);
                gs = fmaf(fy[k] * fw[k], fs[k], gs);
            }
        }
        team_reduce<0, false>(sq, gs, red[turn]);
        // into the place of the row before this one, used up before the barrier
        if constexpr (D > 1) fetch(row + (D - 1) * stride, slot == 0 ? D - 1 : slot - 1);
        const float r = 1.0f / sqrtf(fmaf(sq, inv_d, eps));
        const float back = gs * inv_d * r * r;  // times s: what the bracket takes off
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = threadIdx.x + j * nt;
            if (c >= vecs) continue;
            float fs[V], fy[V], fw[V], fa[V];
            unpack(*reinterpret_cast<const uint4*>(mine + c * 16), fs, no);
            unpack(*reinterpret_cast<const uint4*>(mine + row_bytes + c * 16), fy, no);
#pragma unroll
            for (int k = 0; k < V; ++k) acc[j][k] = fmaf(fy[k], fs[k] * r, acc[j][k]);
            if (!d_x) continue;
            unpack(ld_ro(weight + c * V), fw, no);
            unpack(av[j], fa, no);
#pragma unroll
            for (int k = 0; k < V; ++k)
                fa[k] = fmaf(r, fmaf(-back, fs[k], fy[k] * fw[k]), fa[k]);
            *reinterpret_cast<uint4*>(d_x + row * d + c * V) = pack(fa, no);
        }
        if (++slot == D) slot = 0;
    }
    copy_wait<0>();
    if (!part) return;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int c = threadIdx.x + j * nt;
        if (c >= vecs) continue;
#pragma unroll
        for (int k = 0; k < V; ++k) part[(int64_t)blockIdx.x * d + c * V + k] = acc[j][k];
    }
}

// Rows that start within a vector: the ring holds the whole vectors that cover a row, and a
// thread reads the elements of its columns, the same in every row.
template <typename T>
struct Window {
    int bytes;  // of a slot's array
    __device__ __forceinline__ explicit Window(int d) : bytes((d * (int)sizeof(T) + 15 + 15) / 16 * 16) {}
    // bytes of the row before its first element
    __device__ __forceinline__ static int skip(int64_t row, int d) {
        return (int)((row * d * (int64_t)sizeof(T)) & 15);
    }
    // copies the vectors; those that reach past the array's end go by element
    __device__ __forceinline__ void fetch(uint32_t dst, uint8_t* to, const T* p, int64_t row, int d,
                                          int64_t rows) const {
        const int64_t b0 = row * d * (int64_t)sizeof(T), from = b0 & ~(int64_t)15;
        const int64_t end = b0 + d * (int64_t)sizeof(T), total = rows * d * (int64_t)sizeof(T);
        const uint8_t* src = reinterpret_cast<const uint8_t*>(p);
        for (int64_t at = from + threadIdx.x * 16; at < end; at += blockDim.x * 16) {
            if (at + 16 <= total) {
                copy_async(dst + (uint32_t)(at - from), src + at);
            } else {
                for (int64_t e = at; e < end; e += sizeof(T))
                    *reinterpret_cast<T*>(to + (e - from)) = *reinterpret_cast<const T*>(src + e);
            }
        }
    }
};

template <typename T, int D>
__global__ void __launch_bounds__(kRingThreads, 2)
rmsnorm_window_kernel(const T* x, const T* residual, const T* __restrict__ weight, float eps, T* s_out,
                      T* y, uint8_t* codes, float* __restrict__ scales, int64_t rows, int d) {
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float2 red[2][32];
    pdl_wait();
    pdl_trigger();
    const Window<T> win(d);
    const int arrays = residual ? 2 : 1;
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(ring);
    const int64_t stride = gridDim.x;
    auto fetch = [&](int64_t row, int slot) {
        if (row < rows) {
            const int at = slot * arrays * win.bytes;
            win.fetch(base + at, ring + at, x, row, d, rows);
            if (residual) win.fetch(base + at + win.bytes, ring + at + win.bytes, residual, row, d, rows);
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < D - 1; ++i) fetch(blockIdx.x + i * stride, i);
    const float inv_d = 1.0f / (float)d;
    int slot = 0, turn = 0;
    for (int64_t row = blockIdx.x; row < rows; row += stride, turn ^= 1) {
        if constexpr (D == 1) {
            __syncthreads();  // everyone is done with the last row
            fetch(row, 0);
            copy_wait<0>();
        } else {
            copy_wait<D - 2>();
        }
        __syncthreads();  // everyone's copies of this row are there (and the last row is done with)
        if constexpr (D > 1) fetch(row + (D - 1) * stride, slot == 0 ? D - 1 : slot - 1);
        const uint8_t* at = ring + slot * arrays * win.bytes + Window<T>::skip(row, d);
        const T* px = reinterpret_cast<const T*>(at);
        const T* pr = reinterpret_cast<const T*>(at + win.bytes);
        const auto value = [&](int c) {  // as the residual stream holds it
            float v = Elem<T>::to_f32(px[c]);
            if (residual) v = Elem<T>::to_f32(Elem<T>::from_f32(v + Elem<T>::to_f32(pr[c])));
            return v;
        };
        float sum = 0.0f, top = 0.0f;
#pragma unroll 4
        for (int c = threadIdx.x; c < d; c += blockDim.x) {
            const float v = value(c);
            sum = fmaf(v, v, sum);
            if (codes) top = fmaxf(top, fabsf(v * Elem<T>::to_f32(__ldg(weight + c))));
        }
        team_reduce<0, true>(sum, top, red[turn]);
        const float r = 1.0f / sqrtf(fmaf(sum, inv_d, eps));
        const float most = top * r;
        const float scale = most > 0.0f ? most / 448.0f : 1.0f;
        const float inv_scale = 1.0f / scale;
        if (codes && threadIdx.x == 0) scales[row] = scale;
        const int64_t e = row * d;
#pragma unroll 4
        for (int c = threadIdx.x; c < d; c += blockDim.x) {
            const float v = value(c);
            if (s_out) s_out[e + c] = Elem<T>::from_f32(v);
            const float o = v * r * Elem<T>::to_f32(__ldg(weight + c));
            if (y) y[e + c] = Elem<T>::from_f32(o);
            if (codes) codes[e + c] = __nv_cvt_float_to_fp8(o * inv_scale, __NV_SATFINITE, __NV_E4M3);
        }
        if (++slot == D) slot = 0;
    }
    copy_wait<0>();
}

template <typename T, int EPT, int D>
__global__ void __launch_bounds__(kRingThreads, EPT <= 16 ? 2 : 1)
rmsnorm_backward_window_kernel(const T* d_y, const T* s, const T* __restrict__ weight, float eps,
                               const T* d_s, T* d_x, float* __restrict__ part, int64_t rows, int d) {
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float2 red[2][32];
    pdl_wait();
    pdl_trigger();
    const Window<T> win(d);
    const bool add = d_s && d_x;
    const int nt = blockDim.x;
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(ring);
    const int64_t stride = gridDim.x;
    auto fetch = [&](int64_t row, int slot) {
        if (row < rows) {
            const int at = slot * 3 * win.bytes;
            win.fetch(base + at, ring + at, s, row, d, rows);
            win.fetch(base + at + win.bytes, ring + at + win.bytes, d_y, row, d, rows);
            if (add)
                win.fetch(base + at + 2 * win.bytes, ring + at + 2 * win.bytes, d_s, row, d, rows);
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < D - 1; ++i) fetch(blockIdx.x + i * stride, i);
    float acc[EPT];
#pragma unroll
    for (int j = 0; j < EPT; ++j) acc[j] = 0.0f;
    const float inv_d = 1.0f / (float)d;
    int slot = 0, turn = 0;
    for (int64_t row = blockIdx.x; row < rows; row += stride, turn ^= 1) {
        if constexpr (D == 1) {
            __syncthreads();  // everyone is done with the last row
            fetch(row, 0);
            copy_wait<0>();
        } else {
            copy_wait<D - 2>();
        }
        __syncthreads();  // everyone's copies of this row are there (and the last row is done with)
        if constexpr (D > 1) fetch(row + (D - 1) * stride, slot == 0 ? D - 1 : slot - 1);
        const uint8_t* at = ring + slot * 3 * win.bytes + Window<T>::skip(row, d);
        const T* ps = reinterpret_cast<const T*>(at);
        const T* py = reinterpret_cast<const T*>(at + win.bytes);
        const T* pa = reinterpret_cast<const T*>(at + 2 * win.bytes);
        float sq = 0.0f, gs = 0.0f;
#pragma unroll
        for (int j = 0; j < EPT; ++j) {
            const int c = threadIdx.x + j * nt;
            if (c >= d) continue;
            const float fs = Elem<T>::to_f32(ps[c]);
            sq = fmaf(fs, fs, sq);
            gs = fmaf(Elem<T>::to_f32(py[c]) * Elem<T>::to_f32(__ldg(weight + c)), fs, gs);
        }
        team_reduce<0, false>(sq, gs, red[turn]);
        const float r = 1.0f / sqrtf(fmaf(sq, inv_d, eps));
        const float back = gs * inv_d * r * r;
#pragma unroll
        for (int j = 0; j < EPT; ++j) {
            const int c = threadIdx.x + j * nt;
            if (c >= d) continue;
            const float fs = Elem<T>::to_f32(ps[c]), fy = Elem<T>::to_f32(py[c]);
            acc[j] = fmaf(fy, fs * r, acc[j]);
            if (!d_x) continue;
            const float g = fy * Elem<T>::to_f32(__ldg(weight + c));
            d_x[row * d + c] = Elem<T>::from_f32(
                fmaf(r, fmaf(-back, fs, g), add ? Elem<T>::to_f32(pa[c]) : 0.0f));
        }
        if (++slot == D) slot = 0;
    }
    copy_wait<0>();
    if (!part) return;
#pragma unroll
    for (int j = 0; j < EPT; ++j) {
        const int c = threadIdx.x + j * nt;
        if (c < d) part[(int64_t)blockIdx.x * d + c] = acc[j];
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

// launches kernel<..., RES, CODES> by what the call wants
#define MOE_NORM_FLAGS(GO)                        \
    do {                                          \
        if (a.residual) {                         \
            if (a.codes) return GO(true, true);   \
            return GO(true, false);               \
        }                                         \
        if (a.codes) return GO(false, true);      \
        return GO(false, false);                  \
    } while (0)

template <typename T, int TEAM, int VPT, bool AL>
cudaError_t go_teams(const NormArgs& a, cudaStream_t st) {
    const auto go = [&](auto kernel) {
        const int64_t want = ceil_div(a.rows, kTeamThreads / TEAM);
        const int64_t wave = blocks_that_fit(kernel, kTeamThreads, 0);
        return launch_pdl(kernel, dim3((unsigned)(want < wave ? want : wave)), dim3(kTeamThreads), 0, st,
                          (const T*)a.x, (const T*)a.residual, (const T*)a.weight, a.eps, (T*)a.s,
                          (T*)a.y, a.codes, a.scales, a.rows, a.d);
    };
#define MOE_GO(RES, CODES) go(rmsnorm_kernel<T, TEAM, VPT, AL, RES, CODES>)
    MOE_NORM_FLAGS(MOE_GO);
#undef MOE_GO
}

template <typename T, int VPT>
cudaError_t go_blocks(const NormArgs& a, cudaStream_t st) {
    const auto go = [&](auto kernel) {
        const int64_t lanes = ceil_div(a.d, Elem<T>::kPerVec * VPT);
        return launch_pdl(kernel, dim3((unsigned)a.rows), dim3((unsigned)ceil_div(lanes, 32) * 32), 0, st,
                          (const T*)a.x, (const T*)a.residual, (const T*)a.weight, a.eps, (T*)a.s,
                          (T*)a.y, a.codes, a.scales, a.d);
    };
#define MOE_GO(RES, CODES) go(rmsnorm_block_kernel<T, VPT, RES, CODES>)
    MOE_NORM_FLAGS(MOE_GO);
#undef MOE_GO
}

template <typename T, bool AL>
cudaError_t teams_for(const NormArgs& a, int nv, cudaStream_t st) {
    if (nv <= 4) return go_teams<T, 4, 1, AL>(a, st);
    if (nv <= 8) return go_teams<T, 8, 1, AL>(a, st);
    if (nv <= 16) return go_teams<T, 16, 1, AL>(a, st);
    if (nv <= 32) return go_teams<T, 32, 1, AL>(a, st);
    return go_teams<T, 32, 2, AL>(a, st);
}

int threads_for(int64_t lanes) { return (int)ceil_div(lanes, 32) * 32; }

// Blocks an SM for a ring of `smem` bytes and blocks of `threads`, by what a GB300's SM has.
int ring_blocks(size_t smem, int threads) {
    const int by_smem = (int)(kRingSmem / smem), by_threads = 1024 / threads;
    const int n = by_smem < by_threads ? by_smem : by_threads;
    return n < 1 ? 1 : n > 16 ? 16 : n;
}

struct RingPlan {
    int per_thread, threads, per_sm, depth;  // per_thread: columns
    size_t smem;
};

// rows that start within vectors, more than 64 of them
RingPlan window_plan(int dtype, int d, int arrays) {
    RingPlan p{};
    const int size = dtype == MOE_BF16 ? 2 : 4;
    p.smem = (size_t)arrays * ((d * size + 30) / 16 * 16);
    p.depth = kDepth * p.smem <= kRingSmem ? kDepth : 1;
    p.smem *= p.depth;
    p.per_thread = 4;
    while (p.per_thread < 32 && d > p.per_thread * 256) p.per_thread *= 2;
    p.threads = threads_for(ceil_div(d, p.per_thread));
    p.per_sm = ring_blocks(p.smem, p.threads);
    return p;
}

template <typename T>
cudaError_t go_window(const NormArgs& a, cudaStream_t st) {
    const RingPlan p = window_plan(a.dtype, a.d, a.residual ? 2 : 1);
    auto kernel = p.depth == 1 ? rmsnorm_window_kernel<T, 1> : rmsnorm_window_kernel<T, kDepth>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)p.smem);
    if (e != cudaSuccess) return e;
    const int64_t wave = blocks_that_fit(kernel, p.threads, p.smem);
    return launch_pdl(kernel, dim3((unsigned)(a.rows < wave ? a.rows : wave)), dim3(p.threads), p.smem,
                      st, (const T*)a.x, (const T*)a.residual, (const T*)a.weight, a.eps, (T*)a.s,
                      (T*)a.y, a.codes, a.scales, a.rows, a.d);
}

template <typename T, int TEAM, int VPT, int W>
cudaError_t go_backward(const NormArgs& a, int threads, int blocks, cudaStream_t st) {
    auto kernel = rmsnorm_backward_kernel<T, TEAM, VPT, W>;
    const size_t smem = TEAM ? sizeof(float) * kTeamThreads * VPT * W : 0;
    return launch_pdl(kernel, dim3(blocks), dim3(threads), smem, st, (const T*)a.d_y,
                      (const T*)a.x, (const T*)a.weight, a.eps, (const T*)a.d_s, (T*)a.d_x, a.part,
                      a.rows, a.d);
}

template <typename T>
cudaError_t forward(const NormArgs& a, cudaStream_t st) {
    constexpr int V = Elem<T>::kPerVec;
    if (a.d % V) {
        const int nv = (int)ceil_div(a.d, V) + 1;  // vectors that cover a row, wherever it starts
        return nv <= kTeamVecs ? teams_for<T, false>(a, nv, st) : go_window<T>(a, st);
    }
    const int nv = a.d / V;
    if (nv <= kTeamVecs) return teams_for<T, true>(a, nv, st);
    if (nv <= 2 * kBlockThreads<2>) return go_blocks<T, 2>(a, st);
    if (nv <= 4 * kBlockThreads<4>) return go_blocks<T, 4>(a, st);
    return go_blocks<T, 8>(a, st);
}

// 16-byte vectors tile the rows
bool whole_vectors(int dtype, int d) { return d % (dtype == MOE_BF16 ? 8 : 4) == 0; }

// How the backward pass runs: teams within a warp (lanes > 0) of `per_thread` vectors (or
// elements, where vectors do not tile the rows) a lane, or a ring a block.
struct BackPlan {
    int lanes, per_thread, threads, blocks, depth;
    size_t smem;
};

// The blocks, and with them the partial rows of d_w, are counted for 152 SMs and not asked of
// the device, whatever gradients are wanted: the workspace query needs no device, and the
// order of the sums depends on the sizes alone.
BackPlan back_plan(int dtype, int64_t rows, int d) {
    BackPlan p{};
    const bool vec = whole_vectors(dtype, d);
    const int nv = vec ? d / (dtype == MOE_BF16 ? 8 : 4) : d;
    int64_t want = rows, wave;
    if (nv <= kTeamVecs) {
        p.lanes = nv <= 4 ? 4 : nv <= 8 ? 8 : nv <= 16 ? 16 : 32;
        p.per_thread = nv <= 32 ? 1 : 2;
        p.threads = kTeamThreads;
        want = ceil_div(rows, kTeamThreads / p.lanes);
        wave = 152 * 4;
    } else if (vec) {
        p.per_thread = nv <= 2 * kRingThreads ? 2 : nv <= 4 * kRingThreads ? 4 : 8;
        p.threads = threads_for(ceil_div(nv, p.per_thread));
        p.smem = (size_t)(p.per_thread <= 4 ? kDepth : 1) * 2 * nv * 16;
        wave = 152 * ring_blocks(p.smem, p.threads);
    } else {
        const RingPlan w = window_plan(dtype, d, 3);
        p.per_thread = w.per_thread;
        p.threads = w.threads;
        p.smem = w.smem;
        p.depth = w.depth;
        wave = 152 * w.per_sm;
    }
    p.blocks = (int)(want < wave ? want : wave);
    return p;
}

template <typename T, int W>
cudaError_t back_teams(const NormArgs& a, const BackPlan& p, cudaStream_t st) {
    if (p.lanes == 4) return go_backward<T, 4, 1, W>(a, p.threads, p.blocks, st);
    if (p.lanes == 8) return go_backward<T, 8, 1, W>(a, p.threads, p.blocks, st);
    if (p.lanes == 16) return go_backward<T, 16, 1, W>(a, p.threads, p.blocks, st);
    if (p.per_thread == 1) return go_backward<T, 32, 1, W>(a, p.threads, p.blocks, st);
    return go_backward<T, 32, 2, W>(a, p.threads, p.blocks, st);
}

template <typename T>
cudaError_t backward(const NormArgs& a, const BackPlan& p, cudaStream_t st) {
    constexpr int V = Elem<T>::kPerVec;
    const bool vec = whole_vectors(a.dtype, a.d);
    if (p.lanes) return vec ? back_teams<T, V>(a, p, st) : back_teams<T, 1>(a, p, st);
    const auto go = [&](auto kernel) {
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)p.smem);
        if (e != cudaSuccess) return e;
        return launch_pdl(kernel, dim3(p.blocks), dim3(p.threads), p.smem, st, (const T*)a.d_y,
                          (const T*)a.x, (const T*)a.weight, a.eps, (const T*)a.d_s, (T*)a.d_x, a.part,
                          a.rows, a.d);
    };
    if (!vec) {
        // up to 4096 columns three rows of three arrays fit
        if (p.per_thread == 4) return go(rmsnorm_backward_window_kernel<T, 4, kDepth>);
        if (p.per_thread == 8) return go(rmsnorm_backward_window_kernel<T, 8, kDepth>);
        if (p.per_thread == 16) return go(rmsnorm_backward_window_kernel<T, 16, kDepth>);
        if (p.depth == 1) return go(rmsnorm_backward_window_kernel<T, 32, 1>);
        return go(rmsnorm_backward_window_kernel<T, 32, kDepth>);
    }
    if (p.per_thread == 2) return go(rmsnorm_backward_ring_kernel<T, 2>);
    if constexpr (V == 4)
        if (p.per_thread == 8) return go(rmsnorm_backward_ring_kernel<T, 8>);
    return go(rmsnorm_backward_ring_kernel<T, 4>);
}

}  // namespace

cudaError_t launch_rmsnorm(const NormArgs& a, cudaStream_t st) {
    return a.dtype == MOE_BF16 ? forward<bf16>(a, st) : forward<float>(a, st);
}

int rmsnorm_backward_blocks(int64_t rows, int d) {
    const int a = back_plan(MOE_F32, rows, d).blocks, b = back_plan(MOE_BF16, rows, d).blocks;
    return a > b ? a : b;
}

cudaError_t launch_rmsnorm_backward(const NormArgs& a, cudaStream_t st) {
    const BackPlan p = back_plan(a.dtype, a.rows, a.d);
    const cudaError_t e = a.dtype == MOE_BF16 ? backward<bf16>(a, p, st) : backward<float>(a, p, st);
    if (e != cudaSuccess || !a.part) return e;
    return launch_pdl(rmsnorm_dw_kernel, dim3((unsigned)ceil_div(a.d, 32)), dim3(1024), 0, st,
                      (const float*)a.part, p.blocks, a.d, a.d_weight);
}

}  // namespace moe
