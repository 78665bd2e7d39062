// norm.cu -- root-mean-square norm of the rows in front of the experts, with the
// residual's addition and an 8-bit output, and its backward pass.
//
//   s = x + residual, as the residual stream holds it (rounded to the row type)
//   r = 1 / sqrt(mean(s^2) + eps),  y = (s r) w
//   codes = E4M3 nearest to y / scale, scale = max|y| / 448 of the row
//
// A row is read once and stays in registers between the sums and the stores:
// sum(s^2) and max|s w| come from one reduction (max|y| = r max|s w|), so a row
// costs its bytes and one block barrier at most.  A row goes to 4 to 32 lanes of a
// warp (rows of at most 32 16-byte vectors), to a warp (128), else to a block.
//
// Rows that no 16-byte vector tiles (width odd, say) are read through the
// aligned vectors that cover them; those at the ends are stored by element, by one
// warp of the row.
//
// Of the instances, eight spill 8 to 56 bytes a thread: those of a warp a row that are held to
// 32 or 40 registers, for the blocks an SM that hides the loads' latency, and the backward
// ring of ragged bf16 rows of 5121 to 16376 elements.
//
// Measured (GB300, a CUDA graph's time a call; floor: the bytes at the measured copy's
// 6788 GB/s): 16384 x 7168 bf16 with residual, both outputs 152 us (floor 156), one array in
// and out 69 (69); 131072 x 512 78 (79); 20011 x 2049 fp32 57 (48), 100000 x 777 bf16 with
// codes 143 (103); 8 x 7168 2.6 (0.07: a launch).  Backward: 16384 x 7168 bf16 140 (138),
// 20011 x 2049 fp32 105 (97), 100000 x 333 bf16 72 (29).
#include <cuda_fp8.h>
#include <float.h>

#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kTeamVecs = 32;      // widest row of a team, in vectors
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

// element k of a vector, as its bits
template <typename T> struct Bits;
template <> struct Bits<float> { using type = uint32_t; };
template <> struct Bits<bf16> { using type = uint16_t; };
template <typename T>
__device__ __forceinline__ typename Bits<T>::type elem_of(const uint4& v, int k) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    if constexpr (sizeof(T) == 4) return u[k];
    else return (uint16_t)(u[k / 2] >> (16 * (k & 1)));
}

// A row that starts `skip` elements into a vector: vector c of the row is elements
// c V - skip .. of it, those outside [0, d) not the row's.
template <typename T, bool AL>
struct Row {
    using B = typename Bits<T>::type;
    static constexpr int V = Elem<T>::kPerVec;
    static constexpr uint32_t kAll = (1u << V) - 1u;
    int64_t at;  // the first vector, in elements of the array; a multiple of V
    int skip, d, vecs;
    __device__ __forceinline__ Row(int64_t row, int d_) : d(d_) {
        const int64_t a = row * d_;
        skip = AL ? 0 : (int)a & (V - 1);
        at = a - skip;
        vecs = AL ? d_ / V : (skip + d_ + V - 1) / V;
    }
    // The i-th of the row's vectors, its ends last: what they cost more is paid by one warp.
    __device__ __forceinline__ int place(int i) const { return AL ? i : i + 1 < vecs ? i + 1 : 0; }
    // The vectors but for the ends: whole, and those of the weight that they cover are too.
    __device__ __forceinline__ bool inner(int c) const {
        return AL || (unsigned)(c - 1) < (unsigned)max(vecs - 3, 0);
    }
    __device__ __forceinline__ bool has(int c, int k) const {
        return AL || (c * V + k >= skip && c * V + k < skip + d);
    }
    // The same as bits.  The forward pass, which asks several times, keeps them (100000 rows of
    // 777 bf16 values with codes 145 us, asking for each element 186); the backward pass, short
    // of registers, does not (20011 x 4097 bf16: 127 us, with bits 133).
    __device__ __forceinline__ uint32_t own(int c) const {
        if (AL) return kAll;
        const int lo = skip - c * V, hi = lo + d;
        return kAll << max(lo, 0) & (hi < V ? (1u << max(hi, 0)) - 1u : kAll);
    }
    // vector c of p, with elements of the rows beside it; `total`: elements of the array
    __device__ __forceinline__ uint4 covering(const T* p, int c, int64_t total) const {
        if (inner(c) || at + c * V + V <= total) return *reinterpret_cast<const uint4*>(p + at + c * V);
        return gather(p + at + c * V, c);  // the array's last vector
    }
    // the row's elements of a vector one by one, 0 for the others
    __device__ __forceinline__ uint4 gather(const T* p, int c) const {
        return gather_if(p, [&](int k) { return has(c, k); });
    }
    template <typename Has>
    __device__ __forceinline__ static uint4 gather_if(const T* p, Has mine) {
        uint32_t u[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const uint32_t e = mine(k) ? *reinterpret_cast<const B*>(p + k) : 0u;
            if constexpr (V == 4) u[k] = e;
            else u[k / 2] |= e << (16 * (k & 1));
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
    // elements that are not the row's 0
    __device__ __forceinline__ uint4 mask(const uint4& v, int c) const {
        if (inner(c)) return v;
        return mask_if(v, [&](int k) { return has(c, k); });
    }
    __device__ __forceinline__ static uint4 mask_own(const uint4& v, uint32_t m) {
        if (AL || m == kAll) return v;
        return mask_if(v, [&](int k) { return (m >> k & 1u) != 0u; });
    }
    template <typename Has>
    __device__ __forceinline__ static uint4 mask_if(const uint4& v, Has mine) {
        uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < V; ++k) {
            if constexpr (V == 4) u[k] = mine(k) ? u[k] : 0u;
            else u[k / 2] &= mine(k) ? 0xffffffffu : k & 1 ? 0xffffu : 0xffff0000u;
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
    __device__ __forceinline__ void store(T* p, int c, const uint4& v) const {
        if (inner(c)) *reinterpret_cast<uint4*>(p + at + c * V) = v;
        else store_if(p + at + c * V, v, [&](int k) { return has(c, k); });
    }
    __device__ __forceinline__ void store_own(T* p, int c, uint32_t m, const uint4& v) const {
        if (AL || m == kAll) *reinterpret_cast<uint4*>(p + at + c * V) = v;
        else store_if(p + at + c * V, v, [&](int k) { return (m >> k & 1u) != 0u; });
    }
    template <typename Has>
    __device__ __forceinline__ static void store_if(T* p, const uint4& v, Has mine) {
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (mine(k)) reinterpret_cast<B*>(p)[k] = elem_of<T>(v, k);
    }
    // the weights of vector c: `skip` elements of the weight's vector before, then the next
    __device__ __forceinline__ uint4 weight(const T* w, int c) const {
        if (AL) return ld_ro(w + c * V);
        if (!inner(c)) return gather(w + c * V - skip, c);
        const uint4 a = ld_ro(w + (c - 1) * V), b = ld_ro(w + c * V);
        if (skip == 0) return b;
        uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        // x from element V - skip on: by two words, one, and half a word of bf16
        const int by = (V - skip) * (int)sizeof(T);  // bytes, 2 .. 14
#pragma unroll
        for (int q = 0; q < 6; ++q) x[q] = by & 8 ? x[q + 2] : x[q];
#pragma unroll
        for (int q = 0; q < 5; ++q) x[q] = by & 4 ? x[q + 1] : x[q];
        if constexpr (sizeof(T) == 2)
#pragma unroll
            for (int q = 0; q < 4; ++q) x[q] = __funnelshift_r(x[q], x[q + 1], (by & 2) * 8);
        return make_uint4(x[0], x[1], x[2], x[3]);
    }
    __device__ __forceinline__ uint4 weight_own(const T* w, int c, uint32_t m) const {
        if (inner(c)) return weight(w, c);
        return gather_if(w + c * V - skip, [&](int k) { return (m >> k & 1u) != 0u; });
    }
};

// What a team sums beside a: nothing, the largest of b, or b.
enum { kAlone, kMax, kSum };
template <int WITH>
__device__ __forceinline__ void fold(float& a, float& b, int o) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    if constexpr (WITH != kAlone) {
        const float t = __shfl_xor_sync(0xffffffffu, b, o);
        b = WITH == kMax ? fmaxf(b, t) : b + t;
    }
}

// Over the team, in every thread.  TEAM 0: the block, through `red` (one of two buffers in
// turn, so that one barrier a row is enough).
template <int TEAM, int WITH>
__device__ __forceinline__ void team_reduce(float& a, float& b, float2* red) {
    constexpr int W = TEAM ? TEAM : 32;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) fold<WITH>(a, b, o);
    if constexpr (TEAM == 0) {
        const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
        if (lane == 0) red[threadIdx.x >> 5] = make_float2(a, b);
        __syncthreads();
        const float2 v = lane < warps ? red[lane] : make_float2(0.0f, 0.0f);
        a = v.x;
        b = v.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) fold<WITH>(a, b, o);
    }
}

// The codes' scale of a row, at least the least normal number, so that its inverse is finite
// (rows of denormal numbers would be NaN otherwise).
__device__ __forceinline__ float row_scale(float most) {
    return most > 0.0f ? fmaxf(most / 448.0f, FLT_MIN) : 1.0f;
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

template <typename T, bool AL>
__device__ __forceinline__ void store_codes(uint8_t* codes, const Row<T, AL>& row, int c, uint32_t m,
                                            const float (&f)[Row<T, AL>::V], float inv_scale) {
    constexpr int V = Row<T, AL>::V;
    uint32_t q[V / 4];
    to_codes(f, inv_scale, q);
    uint8_t* p = codes + row.at + c * V;
    if (AL || m == row.kAll) {
        if constexpr (V == 8) *reinterpret_cast<uint2*>(p) = make_uint2(q[0], q[V / 4 - 1]);
        else *reinterpret_cast<uint32_t*>(p) = q[0];
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (m >> k & 1u) p[k] = (uint8_t)(q[k / 4] >> (8 * (k & 3)));
    }
}

// Narrow rows: a lane a vector, a team of a warp's lanes a row, blocks stay for many.
template <typename T, int TEAM, bool AL, bool RES, bool CODES>
__global__ void __launch_bounds__(kTeamThreads)
rmsnorm_kernel(const T* x, const T* residual, const T* __restrict__ weight, float eps, T* s_out,
               T* y, uint8_t* codes, float* __restrict__ scales, int64_t rows, int d) {
    constexpr int V = Elem<T>::kPerVec, per_block = kTeamThreads / TEAM;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x % TEAM;
    const int64_t stride = (int64_t)gridDim.x * per_block, total = rows * d;
    // every team of a block runs as many turns as its first, for the warp-wide shuffles
    const int64_t first = (int64_t)blockIdx.x * per_block;
    const int64_t turns = first < rows ? (rows - first + stride - 1) / stride : 0;
    int64_t at = first + threadIdx.x / TEAM;
    const T* const no = nullptr;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const float inv_d = 1.0f / (float)d;
    for (int64_t it = 0; it < turns; ++it, at += stride) {
        const Row<T, AL> row(at, d);
        const bool live = at < rows;
        const int c = row.place(lane);
        const uint32_t own = row.own(c);
        const bool mine = live && lane < row.vecs;
        uint4 sv = mine ? row.covering(x, c, total) : zero;
        float f[V], g[V];
        if constexpr (RES) {
            const uint4 rv = mine ? row.covering(residual, c, total) : zero;
            unpack(sv, f, no);
            unpack(rv, g, no);
#pragma unroll
            for (int k = 0; k < V; ++k) f[k] += g[k];
            sv = pack(f, no);
        }
        sv = row.mask_own(sv, own);
        unpack(sv, f, no);
        unpack(lane < row.vecs ? row.weight_own(weight, c, own) : zero, g, no);
        float sum = 0.0f, top = 0.0f;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            sum = fmaf(f[k], f[k], sum);
            if (CODES) top = fmaxf(top, fabsf(f[k] * g[k]));
        }
        team_reduce<TEAM, CODES ? kMax : kAlone>(sum, top, nullptr);
        if (!live) continue;  // the last turn of a block of teams
        const float r = rsqrtf(fmaf(sum, inv_d, eps));
        const float most = top * r;
        const float scale = row_scale(most);
        const float inv_scale = 1.0f / scale;
        if (CODES && lane == 0) scales[at] = scale;
        if (lane >= row.vecs) continue;
        if (s_out) row.store_own(s_out, c, own, sv);
#pragma unroll
        for (int k = 0; k < V; ++k) f[k] = f[k] * r * g[k];
        if (y) row.store_own(y, c, own, pack(f, no));
        if constexpr (CODES) store_codes(codes, row, c, own, f, inv_scale);
    }
}

// A wide row: a block of its own (or, up to kWarpVecs vectors, a warp), which ends with it.  Many
// small blocks in different parts of their rows keep the memory busy; blocks that stayed for many
// rows, with or without a ring of copies ahead, did not (16384 x 7168 bf16 with residual and
// codes: 178 and 186 us, this 153).  AL: whole vectors tile the rows.
constexpr int kBlockThreads = 512;  // most threads of a block
constexpr int kWarpVecs = 128;      // widest row of a warp
constexpr int kWarpRows = 8;        // most rows of a block of such warps

template <typename T, int VPT, bool AL, bool RES, bool CODES, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kWarpRows : kBlockThreads,
                                  WARP ? (VPT <= 2 ? (AL ? 8 : 6) : 4)
                                       : VPT <= 2 ? (AL || sizeof(T) == 4 ? 4 : 3) : VPT <= 4 ? 2 : 1)
rmsnorm_block_kernel(const T* x, const T* residual, const T* __restrict__ weight, float eps, T* s_out,
                     T* y, uint8_t* codes, float* __restrict__ scales, int64_t rows, int d) {
    constexpr int V = Elem<T>::kPerVec;
    __shared__ float2 red[32];
    pdl_wait();
    pdl_trigger();
    const int nt = WARP ? 32 : blockDim.x, tid = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int64_t at = WARP ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    if (WARP && at >= rows) return;
    const int64_t total = rows * d;
    const Row<T, AL> row(at, d);
    const T* const no = nullptr;
    uint4 sv[VPT];
    uint32_t own[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = tid + j * nt, c = row.place(i);
        own[j] = row.own(c);
        sv[j] = i < row.vecs ? row.covering(x, c, total) : make_uint4(0u, 0u, 0u, 0u);
    }
    if constexpr (RES) {
        uint4 rv[VPT];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = tid + j * nt, c = row.place(i);
            rv[j] = i < row.vecs ? row.covering(residual, c, total) : make_uint4(0u, 0u, 0u, 0u);
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
                const int i = tid + j * nt, c = row.place(i);
                if (i < row.vecs) row.store_own(s_out, c, own[j], sv[j]);
            }
        }
    }
    float sum = 0.0f, top = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = tid + j * nt, c = row.place(i);
        float f[V], g[V];
        sv[j] = row.mask_own(sv[j], own[j]);
        unpack(sv[j], f, no);
#pragma unroll
        for (int k = 0; k < V; ++k) sum = fmaf(f[k], f[k], sum);
        if constexpr (CODES) {
            if (i >= row.vecs) continue;
            unpack(row.weight_own(weight, c, own[j]), g, no);
#pragma unroll
            for (int k = 0; k < V; ++k) top = fmaxf(top, fabsf(f[k] * g[k]));
        }
    }
    // A block's reduction carries the maximum even where nobody asks for it: the few steps longer
    // between a row's loads and its stores keep the memory busier (bf16, one array in and one
    // out, 117 M elements: rows of 4608 67.6 us against 72.2, 6144 67.8 and 70.4, 7168 68.4 and
    // 72.8, 10240 68.2 and 73.0; 16384 75.0 and 74.5; narrower rows, fp32 and a residual the same
    // either way).
    team_reduce<WARP ? 32 : 0, CODES || !WARP ? kMax : kAlone>(sum, top, red);
    const float r = rsqrtf(fmaf(sum, 1.0f / (float)d, eps));
    const float most = top * r;
    const float scale = row_scale(most);
    const float inv_scale = 1.0f / scale;
    if (CODES && tid == 0) scales[at] = scale;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = tid + j * nt, c = row.place(i);
        if (i >= row.vecs) continue;
        float f[V], g[V];
        unpack(sv[j], f, no);
        unpack(row.weight_own(weight, c, own[j]), g, no);
#pragma unroll
        for (int k = 0; k < V; ++k) f[k] = f[k] * r * g[k];
        if (!RES && s_out) row.store_own(s_out, c, own[j], sv[j]);
        if (y) row.store_own(y, c, own[j], pack(f, no));
        if constexpr (CODES) {
            store_codes(codes, row, c, own[j], f, inv_scale);
        }
    }
}

// ---------------------------------------------------------------- backward
// g = d_y w, xh = s r:   d_x = d_s + r (g - xh mean(g xh)),   d_w = sum over rows of d_y xh
// From sum(s^2) and sum(g s), one reduction a row.  A thread keeps its columns for all
// of its block's rows, so d_w is summed in registers, once per block over its teams,
// and then by rmsnorm_dw_kernel over the blocks, always in the same order.  Rows that
// start within vectors (AL false) go to teams and blocks by where they start.
template <typename T, int TEAM, bool AL>
__global__ void __launch_bounds__(kTeamThreads, 3)
rmsnorm_backward_kernel(const T* d_y, const T* s, const T* __restrict__ weight, float eps,
                        const T* d_s, T* d_x, float* __restrict__ part, int64_t rows, int d) {
    constexpr int V = Elem<T>::kPerVec, per_block = kTeamThreads / TEAM;
    static_assert(per_block % V == 0, "a team's rows all start at the same place of a vector");
    extern __shared__ float acc_sm[];  // [team of the block][d]
    pdl_wait();
    pdl_trigger();
    const int team = threadIdx.x / TEAM, lane = threadIdx.x % TEAM;
    const int64_t stride = (int64_t)gridDim.x * per_block, total = rows * d;
    const int64_t first = (int64_t)blockIdx.x * per_block;
    const int64_t turns = first < rows ? (rows - first + stride - 1) / stride : 0;
    int64_t row = first + team;
    Row<T, AL> here(row, d);
    const bool mine = lane < here.vecs;
    const int c = here.place(lane);
    const T* const no = nullptr;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const bool add = d_s && d_x;
    const uint4 wv = mine ? here.weight(weight, c) : zero;
    float acc[V];
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.0f;
    uint4 sv, yv, av;
    const auto fetch = [&](const Row<T, AL>& r, bool live) {
        sv = live && mine ? r.covering(s, c, total) : zero;
        yv = live && mine ? r.covering(d_y, c, total) : zero;
        av = live && mine && add ? r.covering(d_s, c, total) : zero;
    };
    fetch(here, row < rows);
    const float inv_d = 1.0f / (float)d;
    for (int64_t it = 0; it < turns; ++it, row += stride) {
        const uint4 ms = here.mask(sv, c), my = here.mask(yv, c), ma = av;
        Row<T, AL> next = here;
        next.at += stride * d;
        if (it + 1 < turns) fetch(next, row + stride < rows);  // in flight over this row
        float fs[V], fy[V], fw[V], fa[V];
        unpack(ms, fs, no);
        unpack(my, fy, no);
        unpack(wv, fw, no);
        float sq = 0.0f, gs = 0.0f;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            sq = fmaf(fs[k], fs[k], sq);
            gs = fmaf(fy[k] * fw[k], fs[k], gs);
        }
        team_reduce<TEAM, kSum>(sq, gs, nullptr);
        const float r = 1.0f / sqrtf(fmaf(sq, inv_d, eps));
        const float back = gs * inv_d * r * r;  // times s: what the bracket takes off
        if (row < rows && mine) {
            unpack(ma, fa, no);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                acc[k] = fmaf(fy[k], fs[k] * r, acc[k]);
                fa[k] = fmaf(r, fmaf(-back, fs[k], fy[k] * fw[k]), fa[k]);
            }
            if (d_x) here.store(d_x, c, pack(fa, no));
        }
        here = next;
    }
    if (!part) return;
    if (mine) {
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (here.has(c, k)) acc_sm[team * d + c * V + k - here.skip] = acc[k];
    }
    __syncthreads();
    for (int col = threadIdx.x; col < d; col += kTeamThreads) {
        float t = 0.0f;
        for (int q = 0; q < per_block; ++q) t += acc_sm[q * d + col];
        part[(int64_t)blockIdx.x * d + col] = t;
    }
}

// ---------------------------------------------------------------- rings
// Blocks that stay for many rows copy the next ones to shared memory while they work on one
// (cp.async: neither registers nor barriers hold the copies up).  Used where blocks have to
// stay, for the sums of d_w over rows, and for rows that 16-byte vectors do not tile.
constexpr int kDepth = 3;  // rows in a ring

constexpr size_t kRingSmem = 220 * 1024;  // of an SM, for the rings of its blocks
constexpr size_t kStaticSmem = 2 * 32 * sizeof(float2);  // beside them, a block's reductions

// s and d_y come by way of the ring, where each thread copies and reads its own; d_s straight
// to registers, asked for before the row's sums.  WARP: rows of up to kWarpVecs / 2 vectors, a
// warp each, with a ring of its own and no barrier.  A thread's columns are the same in every row:
// rows that start within vectors (AL false) go to blocks and warps by where they start (the rows
// of a turn are then a multiple of V, or all rows).
template <int VPT> constexpr int kBackThreads = VPT == 2 ? 320 : 512;

constexpr int kBackWarps = 4;  // of a block of rows of a warp each
constexpr int kBackBlocks = 5;  // such blocks an SM

template <typename T, int VPT, bool AL, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kBackWarps : kBackThreads<VPT>,
                                  WARP ? kBackBlocks : VPT == 2 ? 2 : 1)
rmsnorm_backward_ring_kernel(const T* d_y, const T* s, const T* __restrict__ weight, float eps,
                             const T* d_s, T* d_x, float* __restrict__ part, int64_t rows, int d) {
    constexpr int V = Elem<T>::kPerVec;
    constexpr bool kKeep = VPT <= 4;  // a row's values stay in registers between sums and stores
    extern __shared__ __align__(16) uint8_t rings[];
    __shared__ float2 red[2][32];
    pdl_wait();
    pdl_trigger();
    const int nt = WARP ? 32 : blockDim.x, tid = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int warp = WARP ? threadIdx.x >> 5 : 0, per = WARP ? kBackWarps : 1;
    const int64_t row0 = (int64_t)blockIdx.x * per + warp, stride = (int64_t)gridDim.x * per;
    const int64_t total = rows * d;
    const int room = kDepth * 2 * 16 * (AL ? d / V : (d + V - 1) / V + 1);  // bytes of a ring
    uint8_t* ring = rings + warp * room;
    const Row<T, AL> first(row0, d);
    const int vecs = first.vecs, row_bytes = vecs * 16;
    const bool add = d_s && d_x;
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(ring);
    const T* const no = nullptr;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    auto fetch = [&](int64_t row, int slot) {
        if (row < rows) {
            const int64_t at = row * d - first.skip;
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int i = tid + j * nt, c = first.place(i);
                if (i >= vecs) continue;
                const int to = slot * 2 * row_bytes + c * 16;
                const int64_t e = at + c * V;
                if (first.inner(c) || e + V <= total) {
                    copy_async(base + to, s + e);
                    copy_async(base + to + row_bytes, d_y + e);
                } else {  // the arrays' last vector
                    *reinterpret_cast<uint4*>(ring + to) = first.gather(s + e, c);
                    *reinterpret_cast<uint4*>(ring + to + row_bytes) = first.gather(d_y + e, c);
                }
            }
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) fetch(row0 + i * stride, i);
    float acc[VPT][V];
    uint4 wv[kKeep ? VPT : 1];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
#pragma unroll
        for (int k = 0; k < V; ++k) acc[j][k] = 0.0f;
        const int i = tid + j * nt, c = first.place(i);
        if constexpr (kKeep) wv[j] = i < vecs ? first.weight(weight, c) : zero;
    }
    const float inv_d = 1.0f / (float)d;
    int slot = 0, turn = 0;
    for (int64_t row = row0; row < rows; row += stride, turn ^= 1) {
        Row<T, AL> here = first;
        here.at = row * d - first.skip;
        uint4 av[VPT], sv[kKeep ? VPT : 1], yv[kKeep ? VPT : 1];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = tid + j * nt, c = first.place(i);
            av[j] = add && i < vecs ? here.covering(d_s, c, total) : zero;
        }
        copy_wait<kDepth - 2>();
        const uint8_t* mine = ring + slot * 2 * row_bytes;
        const auto read = [&](int c, bool second) {
            return here.mask(*reinterpret_cast<const uint4*>(mine + (second ? row_bytes : 0) + c * 16), c);
        };
        float sq = 0.0f, gs = 0.0f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = tid + j * nt, c = first.place(i);
            if constexpr (kKeep) sv[j] = yv[j] = zero;
            if (i >= vecs) continue;
            const uint4 a = read(c, false), b = read(c, true);
            if constexpr (kKeep) {
                sv[j] = a;
                yv[j] = b;
            }
            float fs[V], fy[V], fw[V];
            unpack(a, fs, no);
            unpack(b, fy, no);
            unpack(kKeep ? wv[kKeep ? j : 0] : here.weight(weight, c), fw, no);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                sq = fmaf(fs[k], fs[k], sq);
                gs = fmaf(fy[k] * fw[k], fs[k], gs);
            }
        }
        team_reduce<WARP ? 32 : 0, kSum>(sq, gs, red[turn]);
        // into the place of the row before this one, used up before the barrier
        fetch(row + (kDepth - 1) * stride, slot == 0 ? kDepth - 1 : slot - 1);
        const float r = 1.0f / sqrtf(fmaf(sq, inv_d, eps));
        const float back = gs * inv_d * r * r;  // times s: what the bracket takes off
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = tid + j * nt, c = first.place(i);
            if (i >= vecs) continue;
            float fs[V], fy[V], fw[V], fa[V];
            unpack(kKeep ? sv[kKeep ? j : 0] : read(c, false), fs, no);
            unpack(kKeep ? yv[kKeep ? j : 0] : read(c, true), fy, no);
#pragma unroll
            for (int k = 0; k < V; ++k) acc[j][k] = fmaf(fy[k], fs[k] * r, acc[j][k]);
            if (!d_x) continue;
            unpack(kKeep ? wv[kKeep ? j : 0] : here.weight(weight, c), fw, no);
            unpack(av[j], fa, no);
#pragma unroll
            for (int k = 0; k < V; ++k)
                fa[k] = fmaf(r, fmaf(-back, fs[k], fy[k] * fw[k]), fa[k]);
            here.store(d_x, c, pack(fa, no));
        }
        if (++slot == kDepth) slot = 0;
    }
    copy_wait<0>();
    if (!part) return;
    float* sums = part + (int64_t)blockIdx.x * d;
    if constexpr (WARP) {  // the warps' sums in the place of their rings (fewer bytes)
        __syncwarp();
        sums = reinterpret_cast<float*>(ring);
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = tid + j * nt, c = first.place(i);
        if (i >= vecs) continue;
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (first.has(c, k)) sums[c * V + k - first.skip] = acc[j][k];
    }
    if constexpr (WARP) {
        __syncthreads();
        for (int col = threadIdx.x; col < d; col += 32 * kBackWarps) {
            float t = 0.0f;
#pragma unroll
            for (int q = 0; q < kBackWarps; ++q) t += reinterpret_cast<const float*>(rings + q * room)[col];
            part[(int64_t)blockIdx.x * d + col] = t;
        }
    }
}

// W elements a load: a 16-byte vector, or one.
template <typename T, int W> struct Raw { using type = uint4; };
template <typename T> struct Raw<T, 1> { using type = T; };

template <typename T, int W>
__device__ __forceinline__ void open(const typename Raw<T, W>::type& v, float (&f)[W]) {
    if constexpr (W == 1) f[0] = Elem<T>::to_f32(v);
    else unpack(v, f, (const T*)nullptr);
}

// Rows too wide for a ring of three (fp32 rows past 9384 elements): straight from memory, twice
// -- the second time from L2 -- by element where vectors do not tile them.
template <typename T, int W, int EPT>
__global__ void __launch_bounds__(1024)
rmsnorm_backward_wide_kernel(const T* d_y, const T* s, const T* __restrict__ weight, float eps,
                             const T* d_s, T* d_x, float* __restrict__ part, int64_t rows, int d) {
    __shared__ float2 red[2][32];
    pdl_wait();
    pdl_trigger();
    using R = typename Raw<T, W>::type;
    const int nt = blockDim.x;
    float acc[EPT][W];
#pragma unroll
    for (int j = 0; j < EPT; ++j)
#pragma unroll
        for (int k = 0; k < W; ++k) acc[j][k] = 0.0f;
    const float inv_d = 1.0f / (float)d;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, turn ^= 1) {
        float sq = 0.0f, gs = 0.0f;
#pragma unroll 4
        for (int j = 0; j < EPT; ++j) {
            const int c = (threadIdx.x + j * nt) * W;
            if (c >= d) continue;
            float fs[W], fy[W], fw[W];
            open<T, W>(*reinterpret_cast<const R*>(s + row * d + c), fs);
            open<T, W>(*reinterpret_cast<const R*>(d_y + row * d + c), fy);
            open<T, W>(__ldg(reinterpret_cast<const R*>(weight + c)), fw);
#pragma unroll
            for (int k = 0; k < W; ++k) {
                sq = fmaf(fs[k], fs[k], sq);
                gs = fmaf(fy[k] * fw[k], fs[k], gs);
            }
        }
        team_reduce<0, kSum>(sq, gs, red[turn]);
        const float r = 1.0f / sqrtf(fmaf(sq, inv_d, eps));
        const float back = gs * inv_d * r * r;
#pragma unroll
        for (int j = 0; j < EPT; ++j) {
            const int c = (threadIdx.x + j * nt) * W;
            if (c >= d) continue;
            float fs[W], fy[W], fw[W], fa[W];
            open<T, W>(*reinterpret_cast<const R*>(s + row * d + c), fs);
            open<T, W>(*reinterpret_cast<const R*>(d_y + row * d + c), fy);
#pragma unroll
            for (int k = 0; k < W; ++k) acc[j][k] = fmaf(fy[k], fs[k] * r, acc[j][k]);
            if (!d_x) continue;
            open<T, W>(__ldg(reinterpret_cast<const R*>(weight + c)), fw);
            open<T, W>(d_s ? *reinterpret_cast<const R*>(d_s + row * d + c) : R{}, fa);
#pragma unroll
            for (int k = 0; k < W; ++k) fa[k] = fmaf(r, fmaf(-back, fs[k], fy[k] * fw[k]), fa[k]);
            if constexpr (W == 1) d_x[row * d + c] = Elem<T>::from_f32(fa[0]);
            else *reinterpret_cast<uint4*>(d_x + row * d + c) = pack(fa, (const T*)nullptr);
        }
    }
    if (!part) return;
#pragma unroll
    for (int j = 0; j < EPT; ++j) {
        const int c = (threadIdx.x + j * nt) * W;
        if (c >= d) continue;
#pragma unroll
        for (int k = 0; k < W; ++k) part[(int64_t)blockIdx.x * d + c + k] = acc[j][k];
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

int threads_for(int64_t lanes) { return (int)ceil_div(lanes, 32) * 32; }

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

template <typename T, int TEAM, bool AL>
cudaError_t go_teams(const NormArgs& a, cudaStream_t st) {
    const auto go = [&](auto kernel) {
        const int64_t want = ceil_div(a.rows, kTeamThreads / TEAM);
        const int64_t wave = (int64_t)device_sm_count() * (2048 / kTeamThreads);
        return launch_pdl(kernel, dim3((unsigned)(want < wave ? want : wave)), dim3(kTeamThreads), 0, st,
                          (const T*)a.x, (const T*)a.residual, (const T*)a.weight, a.eps, (T*)a.s,
                          (T*)a.y, a.codes, a.scales, a.rows, a.d);
    };
#define MOE_GO(RES, CODES) go(rmsnorm_kernel<T, TEAM, AL, RES, CODES>)
    MOE_NORM_FLAGS(MOE_GO);
#undef MOE_GO
}

template <typename T, int VPT, bool AL, bool WARP = false>
cudaError_t go_blocks(const NormArgs& a, int nv, cudaStream_t st) {
    const auto go = [&](auto kernel) {
        // few rows of a warp each go to as many blocks
        const int64_t per = WARP ? ceil_div(a.rows, 152) : 1, n = per < kWarpRows ? per : kWarpRows;
        const int threads = WARP ? 32 * (int)n : threads_for(ceil_div(nv, VPT));
        return launch_pdl(kernel, dim3((unsigned)ceil_div(a.rows, n)), dim3(threads), 0, st,
                          (const T*)a.x, (const T*)a.residual, (const T*)a.weight, a.eps, (T*)a.s,
                          (T*)a.y, a.codes, a.scales, a.rows, a.d);
    };
#define MOE_GO(RES, CODES) go(rmsnorm_block_kernel<T, VPT, AL, RES, CODES, WARP>)
    MOE_NORM_FLAGS(MOE_GO);
#undef MOE_GO
}

template <typename T, bool AL>
cudaError_t teams_for(const NormArgs& a, int nv, cudaStream_t st) {
    if (nv <= 4) return go_teams<T, 4, AL>(a, st);
    if (nv <= 8) return go_teams<T, 8, AL>(a, st);
    if (nv <= 16) return go_teams<T, 16, AL>(a, st);
    return go_teams<T, 32, AL>(a, st);
}

template <typename T, bool AL>
cudaError_t forward(const NormArgs& a, cudaStream_t st) {
    // vectors that cover a row, wherever it starts
    const int nv = (int)ceil_div(a.d, Elem<T>::kPerVec) + (AL ? 0 : 1);
    if (nv <= kTeamVecs) return teams_for<T, AL>(a, nv, st);
    // A warp a row (131072 x 512 bf16: 78 us, in blocks of 32 threads 133; 100000 x 512 fp32 with
    // codes 67 and 102), but for a few rows, where two warps share the latency (8 x 512 fp32:
    // 2.1 us against 2.5).
    if (nv <= kWarpVecs / 2) return go_blocks<T, 2, AL, true>(a, nv, st);
    if (nv <= kWarpVecs && a.rows > 8 * 152) return go_blocks<T, 4, AL, true>(a, nv, st);
    // Two vectors a thread, so that registers allow four blocks of 512; four a thread where a
    // row is one array in and one out (117 M elements of bf16: rows of 4608 67.6 us against 69.1,
    // 5120 68.0 and 70.3, 7168 68.4 and 74.2, 8192 68.1 and 71.6; 59 M of fp32: 2304 68.5 and
    // 67.0, 2880 68.5 and 69.1, 3584 68.5 and 70.0, 4096 68.4 and 68.3; with a residual 135
    // against 134).
    if (AL && !a.residual && !a.codes && nv > kBlockThreads && nv <= 2 * kBlockThreads)
        return go_blocks<T, 4, AL>(a, nv, st);
    if (nv <= 2 * kBlockThreads) return go_blocks<T, 2, AL>(a, nv, st);
    if constexpr (Elem<T>::kPerVec == 4) {
        // 16384 values that start within a vector: 4097
        if (nv > 4 * kBlockThreads) return go_blocks<T, AL ? 8 : 9, AL>(a, nv, st);
        return go_blocks<T, 4, AL>(a, nv, st);
    } else {
        return go_blocks<T, AL ? 4 : 5, AL>(a, nv, st);
    }
}

// 16-byte vectors tile the rows
bool whole_vectors(int dtype, int d) { return d % (dtype == MOE_BF16 ? 8 : 4) == 0; }

// How the backward pass runs: teams within a warp (lanes > 0) of a vector a lane; a ring a
// warp or a block; or, for rows too wide for a ring, neither (smem 0).
struct BackPlan {
    int lanes, per_thread, threads, blocks;
    bool warps;
    size_t smem;
};

// The blocks, and with them the partial rows of d_w, are counted for 152 SMs and not asked of
// the device, whatever gradients are wanted: the workspace query needs no device, and the
// order of the sums depends on the sizes alone.
BackPlan back_plan(int dtype, int64_t rows, int d) {
    BackPlan p{};
    const bool vec = whole_vectors(dtype, d);
    const int v = dtype == MOE_BF16 ? 8 : 4;
    const int nv = vec ? d / v : (int)ceil_div(d, v) + 1;
    int64_t want = rows, wave;
    if (nv <= kTeamVecs) {
        p.lanes = nv <= 4 ? 4 : nv <= 8 ? 8 : nv <= 16 ? 16 : 32;
        p.threads = kTeamThreads;
        want = ceil_div(rows, kTeamThreads / p.lanes);
        wave = 152 * 3;
    } else if (nv <= kWarpVecs / 2) {  // four vectors a lane spill: 777 bf16 values 231 us, in a block 150
        p.warps = true;
        p.per_thread = 2;
        p.threads = 32 * kBackWarps;
        p.smem = (size_t)kBackWarps * kDepth * 2 * nv * 16;
        want = ceil_div(rows, kBackWarps);
        wave = 152 * kBackBlocks;
    } else if ((size_t)kDepth * 2 * nv * 16 <= kRingSmem) {
        p.per_thread = nv <= 2 * kBackThreads<2> ? 2 : nv <= 4 * kBackThreads<4> ? 4 : 5;
        p.threads = threads_for(ceil_div(nv, p.per_thread));
        p.smem = (size_t)kDepth * 2 * nv * 16;
        // by what a GB300's SM has
        const int by_smem = (int)(kRingSmem / p.smem), by_threads = (p.per_thread == 2 ? 640 : 512) / p.threads;
        const int n = by_smem < by_threads ? by_smem : by_threads;
        wave = 152 * (n < 1 ? 1 : n > 16 ? 16 : n);
    } else {
        p.per_thread = vec ? 4 : 16;
        p.threads = threads_for(ceil_div(vec ? nv : d, p.per_thread));
        wave = 152;
    }
    p.blocks = (int)(want < wave ? want : wave);
    return p;
}

template <typename T, int TEAM, bool AL>
cudaError_t go_back_teams(const NormArgs& a, const BackPlan& p, cudaStream_t st) {
    return launch_pdl(rmsnorm_backward_kernel<T, TEAM, AL>, dim3(p.blocks), dim3(kTeamThreads),
                      sizeof(float) * (kTeamThreads / TEAM) * a.d, st, (const T*)a.d_y, (const T*)a.x,
                      (const T*)a.weight, a.eps, (const T*)a.d_s, (T*)a.d_x, a.part, a.rows, a.d);
}

template <typename T, bool AL>
cudaError_t back_teams(const NormArgs& a, const BackPlan& p, cudaStream_t st) {
    if (p.lanes == 4) return go_back_teams<T, 4, AL>(a, p, st);
    if (p.lanes == 8) return go_back_teams<T, 8, AL>(a, p, st);
    if (p.lanes == 16) return go_back_teams<T, 16, AL>(a, p, st);
    return go_back_teams<T, 32, AL>(a, p, st);
}

template <typename T>
cudaError_t backward(const NormArgs& a, const BackPlan& p, cudaStream_t st) {
    constexpr int V = Elem<T>::kPerVec;
    const bool vec = whole_vectors(a.dtype, a.d);
    if (p.lanes) return vec ? back_teams<T, true>(a, p, st) : back_teams<T, false>(a, p, st);
    const auto go = [&](auto kernel) {
        // A launch has 48 KB without asking, of which static arrays take their part.  What is
        // asked for is the same for every call, so calls of several threads do not undo each
        // other's.
        if (p.smem + kStaticSmem > 48 * 1024) {
            const cudaError_t e = cudaFuncSetAttribute(
                kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRingSmem);
            if (e != cudaSuccess) return e;
        }
        return launch_pdl(kernel, dim3(p.blocks), dim3(p.threads), p.smem, st, (const T*)a.d_y,
                          (const T*)a.x, (const T*)a.weight, a.eps, (const T*)a.d_s, (T*)a.d_x, a.part,
                          a.rows, a.d);
    };
    if constexpr (V == 4) {
        if (p.smem == 0)
            return vec ? go(rmsnorm_backward_wide_kernel<T, V, 4>)
                       : go(rmsnorm_backward_wide_kernel<T, 1, 16>);
    }
#define MOE_RING(AL)                                                                         \
    do {                                                                                     \
        if (p.warps) return go(rmsnorm_backward_ring_kernel<T, 2, AL, true>);                \
        if (p.per_thread == 2) return go(rmsnorm_backward_ring_kernel<T, 2, AL, false>);     \
        /* whole bf16 vectors of the widest row: 2048, four a thread */                      \
        if (p.per_thread == 4 || (AL && V == 8))                                             \
            return go(rmsnorm_backward_ring_kernel<T, 4, AL, false>);                        \
        if constexpr (!(AL && V == 8))                                                       \
            return go(rmsnorm_backward_ring_kernel<T, 5, AL, false>);                        \
    } while (0)
    if (vec) MOE_RING(true);
    MOE_RING(false);
#undef MOE_RING
}

}  // namespace

cudaError_t launch_rmsnorm(const NormArgs& a, cudaStream_t st) {
    const bool vec = whole_vectors(a.dtype, a.d);
    if (a.dtype == MOE_BF16) return vec ? forward<bf16, true>(a, st) : forward<bf16, false>(a, st);
    return vec ? forward<float, true>(a, st) : forward<float, false>(a, st);
}

int rmsnorm_backward_blocks(int64_t rows, int d) {
    const int a = back_plan(MOE_F32, rows, d).blocks, b = back_plan(MOE_BF16, rows, d).blocks;
    return a > b ? a : b;
}

cudaError_t launch_rmsnorm_backward(const NormArgs& args, cudaStream_t st) {
    NormArgs a = args;
    const BackPlan p = back_plan(a.dtype, a.rows, a.d);
    const bool one = p.blocks == 1;  // its partial row is the sum
    if (one && a.part) a.part = a.d_weight;
    const cudaError_t e = a.dtype == MOE_BF16 ? backward<bf16>(a, p, st) : backward<float>(a, p, st);
    if (e != cudaSuccess || !a.part || one) return e;
    return launch_pdl(rmsnorm_dw_kernel, dim3((unsigned)ceil_div(a.d, 32)), dim3(1024), 0, st,
                      (const float*)a.part, p.blocks, a.d, a.d_weight);
}

}  // namespace moe
