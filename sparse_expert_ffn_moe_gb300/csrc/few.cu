// few.cu -- the whole layer for a few tokens (T <= 16) in two launches.
//
//   y = residual + SharedExpert(x) + sum_j w_j Expert_{i_j}(x)
//
// A few tokens read every matrix of every picked expert once, and compute next to
// nothing: the layer is a stream of weights from HBM, bounded by bytes.  What costs
// time beside the stream are the joints between its parts (scores, choice, gate/up,
// down, sum), so the second launch keeps the weights coming across all of them.
//
// Launch 1, few_scores_kernel: partial scores x . w_g^T (a warp per expert and slice
// of d), x as two E4M3 planes for 8-bit experts, and the counters of launch 2 zeroed.
//
// Launch 2, few_experts_kernel: one block an SM.  Every block chooses the experts
// itself (the same sums in the same order everywhere), lists the groups (the shared
// expert, then the picked experts, each once, with the tokens that picked it) and
// cuts all work into units: 64 gate and the same 64 up rows, or 128 down rows, of a
// group, over all of K or, where that would leave blocks idle, a part of it.  Blocks
// take units from one counter in the order gate/up, then down.  A down unit needs its
// group's h, which units before it in that order make: whoever holds those took them
// earlier and is running, so every wait ends whatever part of the grid is resident,
// and two calls on two streams share the GPU safely.
//
// In a block, roles pass work through shared memory as the tensor-core GEMM's do:
// warp 0 takes units and streams weight tiles (TMA, 128-byte swizzle), warp 1 the
// rows that multiply them, warp 2 issues tcgen05 products with the weights as the
// 128-row operand and the tokens as its few columns, warps 4-7 empty the accumulators,
// warps 8-11 count finished parts and join them.  Warp 0 runs ahead by the ring's depth
// (128 or 160 KB an SM) without waiting for h, so the weights of the next part are on
// their way while h is still being finished.
//
// Rows that multiply: every token's x (a group's outputs are kept for its own tokens
// alone, so a column that is not wanted costs nothing and spoils nothing, NaN
// included), and h of the group's tokens.  Precision: bf16 experts take x as it is and
// h as two bf16 planes (hi, remainder: within 2^-16).  8-bit experts take x as two
// E4M3 planes, the second 16 times finer, with a power of two as the row's scale: a bf16
// value of at least 2^-13 of the row's largest is held exactly (its code is a normal number,
// whose remainder the second plane has the bits for), a smaller one to within 2^-21 of the
// row's largest; and h as three such planes with a scale per 128 values (within 2^-12,
// beside a code's own 2^-4).
// Planes are further columns, their sums are joined in fp32.
//
// Sums of parts go to buffers, and whoever finishes a tile's last part adds them in
// their order; the same for the sum over experts.  No floating-point atomics: the same
// bits on every run, whoever takes which unit.
//
// Measured (GB300, a CUDA graph's time a call; floor: the picked experts' bytes at the
// measured copy's 6788 GB/s): 256 experts of 7168 x 2048, K = 8, and a shared one, bf16:
// T = 1 126 us (floor 117), T = 8 603 (617), T = 16 920 (941); E4M3 T = 1 72 (59), T = 8
// 318 (309), T = 16 492 (471); block scales, T = 13 446 (422).  Small layers are a chain of
// joints: eight experts of 2048 x 768 31 us (floor 11), two of 256 x 512 14 us.  Tried and
// slower: units of 16 or 32 rows, which leave the products' other rows empty (T = 1 209 and
// 146 us against 131); units a quarter as long with more parts (T = 1 160); two accumulators
// in turn (+ 2 %); claims of several units at a time (177); the sums' warps counting parts
// themselves.
#include <cuda.h>
#include <cuda_fp8.h>
#include <math.h>
#include <stdlib.h>

#include "common.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace moe {

namespace {

constexpr int kMaxT = kFewMaxTokens;
constexpr int kMaxSlots = kMaxT * 32;      // T * K
constexpr int kMaxGroups = kMaxSlots + 1;  // and the shared expert
constexpr int kScoreWarps = 8;
constexpr int kScoreSplits = 8;
constexpr int kThreads = 384;
constexpr int kBufs = 4;       // accumulator buffers of 128 tensor-memory columns
constexpr int kQueue = 8;      // units between the roles
constexpr int kGateRows = 64;  // gate and up rows of a unit: 128 rows of a product in all
constexpr int kDownRows = 128;
constexpr int kTiles = 2;      // K tiles of a stage
constexpr int kWTile = 16384;  // bytes of a weight tile: 128 rows x 128 bytes
constexpr int kABytes = kTiles * kWTile;
constexpr int kMaxStages = 5;
constexpr int kChunk = 16;     // K tiles whose scales of h are fetched at once
constexpr int kHint = 4096;    // bytes of an L2 prefetch
constexpr int64_t kHintMost = 8 << 20;  // of each of two matrices

// FMT: 0 bf16 weights, 1 E4M3 with a scale a row, 2 E4M3 with a scale per 128 x 128 block.
// NT: columns that tokens take (8 or 16).
template <int FMT, int NT>
struct Cfg {
    static constexpr int kElems = FMT ? 128 : 64;  // K of a tile: 128 bytes
    static constexpr int kHPlanes = FMT ? 3 : 2;   // of h
    // Columns of a product: whole 16s.  Those past the planes multiply whatever follows them
    // in shared memory and are not read.
    static constexpr int kXCols = FMT ? 2 * NT : 16, kHCols = FMT ? 4 : 2;
    static constexpr int kXTile = kXCols * 128;    // bytes beside one weight tile
    // a stage: the weights and the rows beside them (products with h read whole 16s of columns)
    static constexpr int kXStage = kTiles * kXTile;
    static constexpr int kHStage = ((kTiles - 1) * kHPlanes + kHCols) * NT * 128;
    static constexpr int kStage = kABytes + (kXStage > kHStage ? kXStage : kHStage);
    // Fewer in flight cost bandwidth (E4M3, T = 8: 5 stages 323 us, 4 326, 3 333, 2 370), more
    // hold up what the joints wait for (bf16, T = 1, six experts of 1408: 5 stages 42 us, 6 44).
    static constexpr int kStages = kStage <= 40960 ? 5 : 4;
    static_assert(kTiles * kHCols * NT <= 128, "a stage's accumulators fit a buffer");
};

enum { kMapGate, kMapUp, kMapDown, kMapSGate, kMapSUp, kMapSDown, kMapX, kMapH8, kMapHS8, kMapH16,
       kMapHS16, kMaps };

struct FewArgs {
    CUtensorMap maps[kMaps];
    int T, d, E, K, I, Is, sigmoid, splits, test_stall;
    int gp, dp;  // parts that a gate/up and a down tile's K is cut into
    const uint8_t *ws_gate, *ws_up;  // the shared expert's, and their bytes to prefetch
    int64_t hint;
    unsigned long long timeout_ns;
    const float* bias;
    const bf16* residual;
    bf16* y;
    DevError* err;
    int *claim, *ready, *dticket, *gticket;  // units taken; tiles of h done by group; parts done
    float *part, *xs, *gpart, *hs, *hs_s, *yp;
    void *h, *h_s;
    const float *s_gate, *s_up, *s_down, *ss_gate, *ss_up, *ss_down;
};

struct Ctl {
    uint64_t full[kMaxStages], empty[kMaxStages], tfull[kBufs], tempty[kBufs];
    uint64_t qfull[kQueue], qempty[kQueue], summed[kQueue];
    uint32_t tmem;
    int abort_flag;
    int queue[kQueue];
    int last;
    int groups;                   // with the shared expert
    uint32_t present[32];         // experts that a token picked
    uint16_t expert[kMaxGroups];  // of a group
    alignas(4) uint16_t mask[kMaxGroups + 1];  // tokens of a group (set by 32-bit atomics)
    uint16_t row0[kMaxGroups + 1];
    uint16_t pick[kMaxSlots];     // expert, then row, of a slot
    float weight[kMaxSlots];
    float xs[kMaxT];              // scales of x
    float top[4][kMaxT];
    alignas(16) float hscale[2][kChunk * 16];  // of K tiles of h: [tile][token], two chunks in turn
    alignas(16) float strand[4][128];  // read and written as float4
};

struct Unit {
    int down, group, tile, part, k0, n;  // K tiles k0 .. k0 + n - 1
};

// The work as units, the same in every block.
struct Sched {
    int nk, nks, nkr;   // K tiles: gate/up, shared and routed down
    int gs, gr, td;     // tiles of a group: shared and routed gate/up, down
    int u1, u2, u3, u4; // ends of: shared gate/up, routed, shared down, routed down
};

__device__ __forceinline__ Sched make_sched(const FewArgs& a, int groups, int elems) {
    Sched s;
    const int shared = a.Is > 0, routed = groups - shared;
    s.nk = a.d / elems;
    s.nks = a.Is / elems;
    s.nkr = a.I / elems;
    s.gs = a.Is / kGateRows;
    s.gr = a.I / kGateRows;
    s.td = (a.d + kDownRows - 1) / kDownRows;
    s.u1 = s.gs * a.gp;
    s.u2 = s.u1 + routed * s.gr * a.gp;
    s.u3 = s.u2 + shared * s.td * a.dp;
    s.u4 = s.u3 + routed * s.td * a.dp;
    return s;
}

// part p of n K tiles in `parts` parts: whole stages but for the last (a part may be empty)
__device__ __forceinline__ void cut(int n, int parts, int p, int& k0, int& k) {
    const int each = ((n + kTiles - 1) / kTiles + parts - 1) / parts * kTiles;
    k0 = min(n, p * each);
    k = min(each, n - k0);
}

__device__ __forceinline__ Unit unit_at(const FewArgs& a, const Sched& s, int u, int shared) {
    Unit t;
    int n;
    if (u < s.u2) {
        t.down = 0;
        t.part = u % a.gp;
        u /= a.gp;
        t.group = u < s.gs ? 0 : shared + (u - s.gs) / s.gr;
        t.tile = u < s.gs ? u : (u - s.gs) % s.gr;
        n = s.nk;
        cut(n, a.gp, t.part, t.k0, t.n);
    } else {
        u -= s.u2;
        t.down = 1;
        t.part = u % a.dp;
        u /= a.dp;
        t.group = u / s.td;
        t.tile = u % s.td;
        n = t.group < shared ? s.nks : s.nkr;
        cut(n, a.dp, t.part, t.k0, t.n);
    }
    return t;
}

__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, Ctl* ctl,
                                             const FewArgs& a, int where) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = ptx::globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
        if (ptx::mbar_try_wait(bar, parity)) return true;
        if ((it & 63u) == 0) {
            if (*(volatile int*)&ctl->abort_flag) return false;
            if (ptx::globaltimer_ns() - t0 > a.timeout_ns) {
                record_error(a.err, MOE_ERR_TIMEOUT, where);
                *(volatile int*)&ctl->abort_flag = 1;
                return false;
            }
        }
    }
}

// between h's stores, seen by way of an acquired count, and the asynchronous copies of it
__device__ __forceinline__ void fence_proxy_async_global() {
    asm volatile("fence.proxy.async.global;" ::: "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
__device__ __forceinline__ int ld_acquire(const int* p) {
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void tma_load_4d(void* dst, const void* tmap, uint64_t* bar, int32_t c0,
                                            int32_t c1, int32_t c2, int32_t c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(ptx::smem_u32(dst)),
        "l"(tmap), "r"(ptx::smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d(void* dst, const void* tmap, uint64_t* bar, int32_t c0,
                                            int32_t c1, int32_t c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(ptx::smem_u32(dst)),
        "l"(tmap), "r"(ptx::smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
// barrier of the four finishing warps
__device__ __forceinline__ void finish_sync() { asm volatile("bar.sync 2, 128;" ::: "memory"); }

// The least power of two s with amax / s <= 448 (to fp32 rounding), and 1 / s; 1 where
// amax is not positive, NaN where it is infinite (codes saturate: the scale has to show it).
__device__ __forceinline__ void plane_scale(float amax, float& s, float& inv) {
    const uint32_t q = __float_as_uint(amax / 448.0f);
    int e = (int)(q >> 23) + ((q & 0x7FFFFFu) != 0u ? 1 : 0);
    e = amax > 0.0f ? max(1, min(e, 252)) : 127;
    s = isinf(amax) ? amax - amax : __uint_as_float((uint32_t)e << 23);
    inv = __uint_as_float((uint32_t)(254 - e) << 23);
}
__device__ __forceinline__ uint8_t to_code(float v) {
    return __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float of_code(uint8_t c) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

// ------------------------------------------------------------------ launch 1
// Blocks [0, score_blocks): part[split][t][e] = x[t] . w_g[e] over the split's share of d,
// a warp per (chunk of TT tokens, expert, split).  Then, for 8-bit experts, a block per
// token for its planes.  All of them zero a share of the counters.
template <int TT>
__global__ void __launch_bounds__(kScoreWarps * 32)
few_scores_kernel(const bf16* __restrict__ x, const bf16* __restrict__ w_g,
                  float* __restrict__ part, uint8_t* __restrict__ xq, float* __restrict__ xs,
                  int* __restrict__ counters, int n_counters, int T, int d, int E, int splits,
                  int score_blocks) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nvec = d / 8, vps = (nvec + splits - 1) / splits;
    if (blockIdx.x < score_blocks) {
        // a hint for the first unit's weights: nothing is read before the wait
        const int u = blockIdx.x * kScoreWarps + warp, v = u % splits * vps + lane * 8;
        if (u / splits < E && v < nvec && lane * 8 < vps)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(w_g + (int64_t)(u / splits) * d + v * 8));
    }
    pdl_wait();
    pdl_trigger();
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n_counters; i += gridDim.x * blockDim.x)
        counters[i] = 0;
    if (blockIdx.x >= score_blocks) {
        __shared__ float red[kScoreWarps];
        const int t = blockIdx.x - score_blocks;
        const bf16* row = x + (int64_t)t * d;
        float amax = 0.0f;
        for (int v = threadIdx.x; v < nvec; v += blockDim.x) {
            float f[8];
            unpack(ld_ro(row + v * 8), f, (const bf16*)nullptr);
#pragma unroll
            for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(f[k]));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (lane == 0) red[warp] = amax;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kScoreWarps; ++k) amax = fmaxf(amax, red[k]);
        float s, inv;
        plane_scale(amax, s, inv);
        if (threadIdx.x == 0) xs[t] = s;
        for (int v = threadIdx.x; v < nvec; v += blockDim.x) {
            float f[8];
            unpack(ld_ro(row + v * 8), f, (const bf16*)nullptr);
            uint32_t hi[2] = {0u, 0u}, lo[2] = {0u, 0u};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float q = f[k] * inv;
                const uint8_t h = to_code(q);
                const uint8_t l = to_code((q - of_code(h)) * 16.0f);
                hi[k >> 2] |= (uint32_t)h << (8 * (k & 3));
                lo[k >> 2] |= (uint32_t)l << (8 * (k & 3));
            }
            *reinterpret_cast<uint2*>(xq + (int64_t)t * d + v * 8) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2*>(xq + (int64_t)(T + t) * d + v * 8) = make_uint2(lo[0], lo[1]);
        }
        return;
    }
    const int chunks = (T + TT - 1) / TT;
    const int units = chunks * E * splits;
    for (int u = blockIdx.x * kScoreWarps + warp; u < units; u += score_blocks * kScoreWarps) {
        const int s = u % splits, e = (u / splits) % E, t0 = u / (splits * E) * TT;
        const int v0 = s * vps, v1 = min(nvec, v0 + vps);
        float acc[TT];
#pragma unroll
        for (int m = 0; m < TT; ++m) acc[m] = 0.0f;
        const bf16* wrow = w_g + (int64_t)e * d;
        // four vectors a lane at a time, all asked for before the first is used
        for (int vb = v0 + lane; vb < v1; vb += 128) {
            uint4 wv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                wv[i] = vb + 32 * i < v1 ? ld_stream(wrow + (vb + 32 * i) * 8) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float wf[8];
                unpack(wv[i], wf, (const bf16*)nullptr);
                const int v = min(vb + 32 * i, nvec - 1);  // past the share the weights are 0 ...
#pragma unroll
                for (int m = 0; m < TT; ++m) {
                    float xf[8];
                    unpack(ld_ro(x + (int64_t)min(t0 + m, T - 1) * d + v * 8), xf, (const bf16*)nullptr);
                    if (vb + 32 * i < v1)  // ... and x may not be finite
#pragma unroll
                        for (int q = 0; q < 8; ++q) acc[m] = fmaf(wf[q], xf[q], acc[m]);
                }
            }
        }
#pragma unroll
        for (int m = 0; m < TT; ++m) {
            const float r = warp_sum(acc[m]);
            if (lane == 0 && t0 + m < T) part[((int64_t)s * T + t0 + m) * E + e] = r;
        }
    }
}

// ------------------------------------------------------------------ launch 2
__device__ __forceinline__ float score_of(const FewArgs& a, int t, int e) {
    float v[kScoreSplits];
#pragma unroll
    for (int q = 0; q < kScoreSplits; ++q)
        v[q] = q < a.splits ? __ldcg(a.part + ((int64_t)q * a.T + t) * a.E + e) : 0.0f;
    float s = v[0];
#pragma unroll
    for (int q = 1; q < kScoreSplits; ++q)
        if (q < a.splits) s += v[q];
    return s;
}

// A key as an integer of the same order: -0 as +0, and NaN, which a sum makes the one positive
// NaN, above all numbers, so that every pick is one of the experts and none is picked twice.
__device__ __forceinline__ uint32_t ordered(float key) {
    const uint32_t b = __float_as_uint(key + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// The weights of a token's picks, a lane each: a / (sum + 1e-6) or softmax over the keys, as
// numerator and sum.  The lanes that have a pick divide and no others: zeros take the
// division's slow path, whose code has to be fetched (0.6 to 1 us a call).
__device__ __forceinline__ float pick_weight(const FewArgs& a, float s, int e, int lane, float& sum) {
    const float b = a.bias ? __ldg(a.bias + e) : 0.0f;
    const float first = __shfl_sync(0xffffffffu, s + b, 0);
    float w = 0.0f;
    if (lane < a.K) w = a.sigmoid ? 1.0f / (1.0f + expf(-s)) : expf(s + b - first);
    sum = warp_sum(w) + (a.sigmoid ? 1e-6f : 0.0f);
    return w;
}

// A warp's K rounds: lane j gets the j-th pick.  A lane has the experts lane, lane + 32, ...; its
// best one that is not taken (0: none).  The first eight stay in registers, more are read again
// after each pick.
__device__ __forceinline__ int rounds(uint32_t* key, int E, int K, int lane) {
    uint32_t k8[8], best = 0u;
    int at = 0;
#pragma unroll
    for (int m = 0; m < 8; ++m) k8[m] = lane + 32 * m < E ? key[lane + 32 * m] : 0u;
    const auto rescan = [&]() {
        best = 0u;
#pragma unroll
        for (int m = 0; m < 8; ++m)
            if (k8[m] > best) {
                best = k8[m];
                at = lane + 32 * m;
            }
#pragma unroll 4
        for (int e = lane + 256; e < E; e += 32)
            if (key[e] > best) {
                best = key[e];
                at = e;
            }
    };
    rescan();
    int mine = 0;
    for (int j = 0; j < K; ++j) {
        const uint32_t top = __reduce_max_sync(0xffffffffu, best);
        const int e = __reduce_min_sync(0xffffffffu, best == top ? at : 0x7fffffff);
        if (lane == j) mine = e;
        if ((e & 31) == lane) {
#pragma unroll
            for (int m = 0; m < 8; ++m)
                if (e == lane + 32 * m) k8[m] = 0u;
            if (e >= 256) key[e] = 0u;
            rescan();
        }
    }
    return mine;
}

// One token: each pick is a group of its own, and the finishing warps turn the scores in
// ctl->weight into weights.  Up to 128 experts an expert's place is the number of experts before
// it, which all threads count at once (128 experts, K = 8: 31.4 us a call, by rounds 32.5; 256
// experts, E4M3: 75.5, by rounds 73.6).
__device__ __forceinline__ void choose_one(const FewArgs& a, Ctl* ctl, uint32_t* keys,
                                           const float* scores) {
    const int shared = a.Is > 0;
    const auto pick = [&](int j, int e) {
        ctl->expert[shared + j] = (uint16_t)e;
        ctl->weight[j] = scores[e];
    };
    if (a.E <= 128) {
        for (int e = threadIdx.x; e < a.E; e += kThreads) {
            const uint32_t key = keys[e];
            int before = 0;
            // ties go to the lower expert: those below e need only reach its key
#pragma unroll 4
            for (int q = 0; q < a.E / 4; ++q) {
                const uint4 k = reinterpret_cast<const uint4*>(keys)[q];
                const int at = 4 * q;
                before += k.x > key - (at < e) ? 1 : 0;
                before += k.y > key - (at + 1 < e) ? 1 : 0;
                before += k.z > key - (at + 2 < e) ? 1 : 0;
                before += k.w > key - (at + 3 < e) ? 1 : 0;
            }
            for (int o = a.E / 4 * 4; o < a.E; ++o) before += keys[o] > key - (o < e) ? 1 : 0;
            if (before < a.K) pick(before, e);
        }
    } else if (threadIdx.x < 32) {
        const int mine = rounds(keys, a.E, a.K, threadIdx.x);
        if (threadIdx.x < a.K) pick(threadIdx.x, mine);
    }
    const int g = (int)threadIdx.x - 64;
    if (g >= 0 && g < shared + a.K) {
        ctl->mask[g] = 1;
        ctl->row0[g] = (uint16_t)g;
        if (g < shared) ctl->expert[g] = 0;
        else ctl->pick[g - shared] = (uint16_t)g;
    }
    if (threadIdx.x == 128) {
        ctl->groups = shared + a.K;
        if (a.xs) ctl->xs[0] = __ldcg(a.xs);
    }
}

__device__ __forceinline__ void choose_many(const FewArgs& a, Ctl* ctl, uint32_t* keys,
                                            const float* scores) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int shared = a.Is > 0, slots = a.T * a.K;
    for (int t = warp; t < a.T; t += kThreads / 32) {
        const int mine = rounds(keys + t * a.E, a.E, a.K, lane);
        float sum;
        const float w = pick_weight(a, scores[t * a.E + mine], mine, lane, sum);
        if (lane < a.K) {
            ctl->pick[t * a.K + lane] = (uint16_t)mine;
            ctl->weight[t * a.K + lane] = w / sum;
            atomicOr(&ctl->present[mine >> 5], 1u << (mine & 31));
        }
    }
    __syncthreads();
    if (slots <= 32) {
        // a lane a slot; the groups in the order of their first slots
        if (warp == 0) {
            const bool on = lane < slots;
            const int e = on ? ctl->pick[lane] : 0x10000 + lane;
            const uint32_t peers = __match_any_sync(0xffffffffu, e);
            const int leader = __ffs(peers) - 1, t = lane / a.K;
            const uint32_t leaders = __ballot_sync(0xffffffffu, on && leader == lane);
            const int g = shared + __popc(leaders & ((1u << leader) - 1u));
            uint32_t mask = 0;  // tokens of the group: slots t K .. t K + K - 1 are token t's
            for (int q = 0; q < a.T; ++q)
                if (peers >> (q * a.K) & ((2u << (a.K - 1)) - 1u)) mask |= 1u << q;
            int n = on && leader == lane ? __popc(mask) : 0;
            const int own = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, n, o);
                if (lane >= o) n += v;
            }
            const int row0 = __shfl_sync(0xffffffffu, n - own + (shared ? a.T : 0), leader);
            if (on) {
                if (leader == lane) {
                    ctl->expert[g] = (uint16_t)e;
                    ctl->mask[g] = (uint16_t)mask;
                    ctl->row0[g] = (uint16_t)row0;
                }
                ctl->pick[lane] = (uint16_t)(row0 + __popc(mask & ((1u << t) - 1u)));
            }
            if (lane == 0) {
                ctl->groups = shared + __popc(leaders);
                if (shared) {
                    ctl->expert[0] = 0;
                    ctl->mask[0] = (uint16_t)((1u << a.T) - 1u);
                    ctl->row0[0] = 0;
                }
            }
        }
        if (a.xs && threadIdx.x < a.T) ctl->xs[threadIdx.x] = __ldcg(a.xs + threadIdx.x);
        return;
    }
    // picked experts before each 32, in every warp's lanes
    const uint32_t word = ctl->present[lane];
    int before = __popc(word);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
    }
    const int groups = shared + __shfl_sync(0xffffffffu, before, 31);
    before -= __popc(word);
    const auto group_of = [&](int e) {  // by whole warps
        const int w = e >> 5;
        return shared + __shfl_sync(0xffffffffu, before, w) +
               __popc(__shfl_sync(0xffffffffu, word, w) & ((1u << (e & 31)) - 1u));
    };
    // masks are 16-bit halves of words: set with 32-bit atomics
    uint32_t* words = reinterpret_cast<uint32_t*>(ctl->mask);
    if (threadIdx.x == 0) {
        ctl->groups = groups;
        if (shared) {
            ctl->expert[0] = 0;
            atomicOr(&words[0], (1u << a.T) - 1u);
        }
    }
    for (int f0 = warp * 32; f0 < slots; f0 += kThreads) {
        const int f = f0 + lane, e = f < slots ? ctl->pick[f] : 0, g = group_of(e);
        if (f < slots) {
            ctl->expert[g] = (uint16_t)e;
            atomicOr(&words[g >> 1], 1u << (f / a.K + 16 * (g & 1)));
        }
    }
    __syncthreads();
    if (warp == 0) {
        int base = 0;
        for (int g0 = 0; g0 < groups; g0 += 32) {
            const int g = g0 + lane;
            const int own = g < groups ? __popc((uint32_t)ctl->mask[g]) : 0;
            int n = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, n, o);
                if (lane >= o) n += v;
            }
            if (g < groups) ctl->row0[g] = (uint16_t)(base + n - own);
            base += __shfl_sync(0xffffffffu, n, 31);
        }
    }
    __syncthreads();
    for (int f0 = warp * 32; f0 < slots; f0 += kThreads) {
        const int f = f0 + lane, g = group_of(f < slots ? ctl->pick[f] : 0);
        if (f < slots)
            ctl->pick[f] = (uint16_t)(ctl->row0[g] + __popc((uint32_t)ctl->mask[g] &
                                                            ((1u << (f / a.K)) - 1u)));
    }
    if (a.xs && threadIdx.x < a.T) ctl->xs[threadIdx.x] = __ldcg(a.xs + threadIdx.x);
}

// The whole block chooses every token's experts (the rule of moe_route: the K largest keys,
// ties to the lower expert) and lists the groups; the caller's barrier follows.  `keys`,
// `scores`: T * E words each.
template <bool ONE>
__device__ __forceinline__ void choose(const FewArgs& a, Ctl* ctl, uint32_t* keys, float* scores) {
    if constexpr (!ONE) {
        if (threadIdx.x < 32) ctl->present[threadIdx.x] = 0u;
        for (int i = threadIdx.x; i <= kMaxGroups; i += kThreads) ctl->mask[i] = 0;
    }
    for (int i = threadIdx.x; i < a.T * a.E; i += kThreads) {
        const int e = i % a.E;
        const float s = score_of(a, i / a.E, e), b = a.bias ? __ldg(a.bias + e) : 0.0f;
        scores[i] = s;
        // 0 stands for a taken one
        keys[i] = max(ordered(a.sigmoid ? 1.0f / (1.0f + expf(-s)) + b : s + b), 1u);
    }
    __syncthreads();
    if constexpr (ONE) choose_one(a, ctl, keys, scores);
    else choose_many(a, ctl, keys, scores);
}

// y of a tile of 128 columns from every part of every row: the shared expert first, then a
// token's picks in their order.  A warp takes EACH tokens side by side, or a strand of a
// token's parts where there are fewer tokens than warps.
template <int EACH>
__device__ __forceinline__ void join_tokens(const FewArgs& a, Ctl* ctl, int m, int warp, int lane) {
    const int shared = a.Is > 0;
    const int c = m * kDownRows + lane * 4;
    const bool in = c < a.d;
    const int strands = a.T == 1 ? 4 : a.T == 2 ? 2 : 1;
    const int n = (shared + a.K) * a.dp;
    const int t0 = warp / strands, q = warp % strands;  // tokens t0, t0 + 4, ...
    float4 s[EACH];
    uint2 r[EACH];
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
        s[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        // not through the read-only path: y may be the residual itself
        const int t = t0 + 4 * k;
        r[k] = in && a.residual && t < a.T
                   ? *reinterpret_cast<const uint2*>(a.residual + (int64_t)t * a.d + c) : make_uint2(0u, 0u);
    }
    if (in) {
        const float* yp = a.yp + c;
#pragma unroll(8 / EACH)
        for (int i = q; i < n; i += strands) {
            const int e = a.dp == 1 ? i : i / a.dp, j = e - shared, part = i - e * a.dp;
#pragma unroll
            for (int k = 0; k < EACH; ++k) {
                const int t = min(t0 + 4 * k, a.T - 1);  // past the last token: again, not stored
                const int row = j < 0 ? t : ctl->pick[t * a.K + j];
                const float w = j < 0 ? 1.0f : ctl->weight[t * a.K + j];
                const float4 v =
                    __ldcg(reinterpret_cast<const float4*>(yp + ((int64_t)row * a.dp + part) * a.d));
                s[k].x = fmaf(w, v.x, s[k].x);
                s[k].y = fmaf(w, v.y, s[k].y);
                s[k].z = fmaf(w, v.z, s[k].z);
                s[k].w = fmaf(w, v.w, s[k].w);
            }
        }
    }
    if (strands > 1) {
        *reinterpret_cast<float4*>(&ctl->strand[warp][lane * 4]) = s[0];
        finish_sync();
        if (q != 0) return;
        for (int k = 1; k < strands; ++k) {
            const float4 v = *reinterpret_cast<const float4*>(&ctl->strand[warp + k][lane * 4]);
            s[0].x += v.x;
            s[0].y += v.y;
            s[0].z += v.z;
            s[0].w += v.w;
        }
    }
    if (!in) return;
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
        const int t = t0 + 4 * k;
        if (t >= a.T) continue;
        const __nv_bfloat162 lo = __floats2bfloat162_rn(s[k].x + __uint_as_float(r[k].x << 16),
                                                        s[k].y + __uint_as_float(r[k].x & 0xffff0000u));
        const __nv_bfloat162 hi = __floats2bfloat162_rn(s[k].z + __uint_as_float(r[k].y << 16),
                                                        s[k].w + __uint_as_float(r[k].y & 0xffff0000u));
        *reinterpret_cast<uint2*>(a.y + (int64_t)t * a.d + c) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    }
}

template <int NT>
__device__ __forceinline__ void join_tile(const FewArgs& a, Ctl* ctl, int m, int warp, int lane) {
    if constexpr (NT == 16) join_tokens<4>(a, ctl, m, warp, lane);
    else if (a.T <= 4) join_tokens<1>(a, ctl, m, warp, lane);
    else join_tokens<2>(a, ctl, m, warp, lane);
}

// Counts a tile's finished part; true in the four warps of the block that finished the last
// one, which then sees what every part wrote.  The block's own part was written by its sums'
// warps, whose arrival the finishing warps waited for: one thread's fence orders all of it.
__device__ __forceinline__ bool last_part(Ctl* ctl, int* counter, int parts, int tid) {
    if (parts == 1) return true;
    finish_sync();
    if (tid == 0) {
        int old;
        asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;"
                     : "=r"(old)
                     : "l"(counter)
                     : "memory");
        ctl->last = old == parts - 1;
    }
    finish_sync();
    return ctl->last != 0;
}

// Gate and up sums of a row: [tile of the group][part][gate 64, up 64]
__device__ __forceinline__ float* gate_sums(const FewArgs& a, int row, bool sh, int shared, int tile) {
    const int first = shared ? a.T : 0;
    const int64_t at = sh ? (int64_t)row * (a.Is / kGateRows)
                          : (int64_t)first * (a.Is / kGateRows) + (int64_t)(row - first) * (a.I / kGateRows);
    return a.gpart + (at + tile) * a.gp * 2 * kGateRows;
}

// h of row i of a tile from its parts' sums, in their order
__device__ __forceinline__ float h_of(const FewArgs& a, const float* p) {
    float g = 0.0f, u = 0.0f;
#pragma unroll 4
    for (int q = 0; q < a.gp; ++q, p += 2 * kGateRows) {
        g += __ldcg(p);
        u += __ldcg(p + kGateRows);
    }
    return silu_mul(g, u);
}

// h of a finished gate/up tile (bf16) or of two (8-bit: a scale per token and 128 values),
// stored as planes; then the group's count of finished ones.
template <int FMT, int NT>
__device__ __forceinline__ void finish_h(const FewArgs& a, Ctl* ctl, const Unit& u, int r, int shared) {
    using C = Cfg<FMT, NT>;
    const bool sh = u.group < shared;
    const int I = sh ? a.Is : a.I, rows = sh ? a.T : a.T * a.K;
    const int grow0 = ctl->row0[u.group], row0 = grow0 - (sh || !shared ? 0 : a.T);
    const int tokens = __popc((uint32_t)ctl->mask[u.group]);
    if constexpr (FMT == 0) {
        const int i = r % kGateRows;
        bf16* base = reinterpret_cast<bf16*>(sh ? a.h_s : a.h);
        for (int c = r / kGateRows; c < tokens; c += 128 / kGateRows) {
            const float h = h_of(a, gate_sums(a, grow0 + c, sh, shared, u.tile) + i);
            bf16* hp = base + (int64_t)(row0 + c) * I + u.tile * kGateRows + i;
            const bf16 hi = __float2bfloat16_rn(h);
            hp[0] = hi;
            hp[(int64_t)rows * I] = __float2bfloat16_rn(h - __bfloat162float(hi));
        }
    } else {
        const int block = u.tile / 2, i = block * 128 + r;
        uint8_t* base = reinterpret_cast<uint8_t*>(sh ? a.h_s : a.h);
        float* hs = sh ? a.hs_s : a.hs;
        float h[NT];
#pragma unroll
        for (int c = 0; c < NT; ++c) {
            h[c] = 0.0f;
            if (c >= tokens) continue;
            h[c] = h_of(a, gate_sums(a, grow0 + c, sh, shared, i / kGateRows) + i % kGateRows);
            float m = fabsf(h[c]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if ((r & 31) == 0) ctl->top[r >> 5][c] = m;
        }
        finish_sync();
#pragma unroll
        for (int c = 0; c < NT; ++c) {
            if (c >= tokens) continue;
            float s, inv;
            plane_scale(fmaxf(fmaxf(ctl->top[0][c], ctl->top[1][c]),
                              fmaxf(ctl->top[2][c], ctl->top[3][c])), s, inv);
            if (r == 0) hs[(int64_t)(row0 + c) * (I / 128) + block] = s;
            uint8_t* hp = base + (int64_t)(row0 + c) * I + i;
            float q = h[c] * inv;
#pragma unroll
            for (int p = 0; p < C::kHPlanes; ++p) {
                const uint8_t code = to_code(q);
                hp[(int64_t)p * rows * I] = code;
                q = (q - of_code(code)) * 16.0f;
            }
        }
    }
    finish_sync();
    if (r == 0)
        asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(a.ready + u.group) : "memory");
}

// 16 or 32 columns of tensor memory
template <int N>
__device__ __forceinline__ void load_cols(uint32_t at, uint32_t (&v)[N]) {
#pragma unroll
    for (int c = 0; c < N; c += 16) {
        uint32_t (&part)[16] = *reinterpret_cast<uint32_t (*)[16]>(&v[c]);
        ptx::tmem_ld16(at + c, part);
    }
}

// pairs of fp32 values from and to what tensor memory's loads give
__device__ __forceinline__ f2 pack_bits(uint32_t lo, uint32_t hi) {
    return pack2(__uint_as_float(lo), __uint_as_float(hi));
}
template <int N>
__device__ __forceinline__ void unpack_pairs(const f2 (&v)[N / 2], float (&f)[N]) {
#pragma unroll
    for (int t = 0; t < N / 2; ++t) unpack2(v[t], f[2 * t], f[2 * t + 1]);
}

// A down unit's bf16 sums: hi and lo plane, W columns each.
template <int W, int NT>
__device__ __forceinline__ void down_sums(uint32_t at, float (&s)[NT]) {
    uint32_t c[2 * W];
    load_cols(at, c);
    ptx::tmem_ld_wait();
#pragma unroll
    for (int t = 0; t < W; ++t) s[t] = __uint_as_float(c[t]) + __uint_as_float(c[W + t]);
}

// The K tiles of a stage added to a down unit's 8-bit sums: three planes of W columns joined,
// times h's scales (16 a tile) and, FMT 2, the weights'.  For the first N tokens alone: most
// groups have one or two (sums of all 16 in single instructions cost E4M3, T = 16 530 us, these
// 494; block scales, T = 13 470 and 447).  `release`: the
// accumulators are read.
template <int FMT, int W, int N, int NT, typename Release>
__device__ __forceinline__ void add_down(uint32_t at, const float* hs, const float (&bs)[kTiles],
                                         int tiles, f2 (&s)[NT / 2], Release release) {
    uint32_t c[kTiles][W == 16 ? 48 : 32];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) load_cols(at + i * 4 * W, c[i]);
    ptx::tmem_ld_wait();
    release();
    const f2 finer = pack2(0.0625f, 0.0625f);
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
        if (i >= tiles) continue;  // not written
#pragma unroll
        for (int t = 0; t < N / 2; ++t) {
            const float2 q = *reinterpret_cast<const float2*>(hs + 16 * i + 2 * t);
            f2 h = pack2(q.x, q.y);
            if constexpr (FMT == 2) h = mul2(h, pack2(bs[i], bs[i]));
            const f2 mid = fma2(pack_bits(c[i][2 * W + 2 * t], c[i][2 * W + 2 * t + 1]), finer,
                                pack_bits(c[i][W + 2 * t], c[i][W + 2 * t + 1]));
            s[t] = fma2(fma2(mid, finer, pack_bits(c[i][2 * t], c[i][2 * t + 1])), h, s[t]);
        }
    }
}

template <int FMT, int NT, bool ONE>
__global__ void __launch_bounds__(kThreads, 1)
few_experts_kernel(const __grid_constant__ FewArgs a) {
    using C = Cfg<FMT, NT>;
    extern __shared__ uint8_t raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    Ctl* ctl = reinterpret_cast<Ctl*>(ring + C::kStages * C::kStage);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int shared = a.Is > 0;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            ptx::mbar_init(&ctl->full[i], 2);
            ptx::mbar_init(&ctl->empty[i], 1);
        }
        for (int i = 0; i < kBufs; ++i) {
            ptx::mbar_init(&ctl->tfull[i], 1);
            ptx::mbar_init(&ctl->tempty[i], 4);
        }
        for (int i = 0; i < kQueue; ++i) {
            ptx::mbar_init(&ctl->qfull[i], 1);
            ptx::mbar_init(&ctl->qempty[i], 10);
            ptx::mbar_init(&ctl->summed[i], 4);
        }
        ctl->abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 3) {
        ptx::tmem_alloc(&ctl->tmem, 512);
        ptx::tmem_relinquish();
    }
    if (warp == 2 && lane < kMaps) ptx::prefetch_tmap(&a.maps[lane]);
    // The shared expert's weights are wanted whatever is chosen: the first of them go to L2
    // while the scores are computed (a hint: nothing is read before the wait below).
    if (warp == 1) {
        for (int64_t at = ((int64_t)blockIdx.x * 32 + lane) * kHint; at < a.hint;
             at += (int64_t)gridDim.x * 32 * kHint) {
            const uint32_t n = (uint32_t)min((int64_t)kHint, a.hint - at);
            prefetch_l2(a.ws_gate + at, n);
            prefetch_l2(a.ws_up + at, n);
        }
    }
    pdl_wait();
    pdl_trigger();
    // thread 0's first claim: asked for here, answered while the experts are chosen
    int claim = threadIdx.x == 0 ? atomicAdd(a.claim, 1) : 0;
    choose<ONE>(a, ctl, reinterpret_cast<uint32_t*>(ring),
           reinterpret_cast<float*>(ring) + a.T * a.E);
    // the ring held keys: order them before the copies that overwrite them
    ptx::fence_proxy_async_smem();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = ctl->tmem;
    const Sched sc = make_sched(a, ctl->groups, C::kElems);

    if (warp == 0) {
        // -------------------------------------------------- units and their weights
        if (lane == 0 && !a.test_stall) {
            int stage = 0, slot = 0;
            uint32_t phase = 0, qphase = 0;
            bool ok = true;
            const auto post = [&](int u) {
                if (!wait_bounded(&ctl->qempty[slot], qphase ^ 1u, ctl, a, 10)) return false;
                ctl->queue[slot] = u;
                ptx::mbar_arrive(&ctl->qfull[slot]);
                if (++slot == kQueue) { slot = 0; qphase ^= 1u; }
                return true;
            };
            while (ok && claim < sc.u4) {
                const int u = claim;
                claim = atomicAdd(a.claim, 1);  // answered while this unit's copies go out
                if (!post(u)) { ok = false; break; }
                const Unit un = unit_at(a, sc, u, shared);
                const bool sh = un.group < shared;
                const int e = sh ? 0 : ctl->expert[un.group];
                for (int k = un.k0; k < un.k0 + un.n; k += kTiles) {
                    if (!wait_bounded(&ctl->empty[stage], phase ^ 1u, ctl, a, 11)) { ok = false; break; }
                    uint8_t* dst = ring + stage * C::kStage;
                    uint64_t* bar = &ctl->full[stage];
                    if (!un.down) {
                        // a K tile's gate rows, then its up rows
                        const int nk = min(kTiles, un.k0 + un.n - k), row = un.tile * kGateRows;
                        ptx::mbar_arrive_expect_tx(bar, nk * kWTile);
                        for (int i = 0; i < nk; ++i, dst += kWTile) {
                            const int c = (k + i) * C::kElems;
                            tma_load_3d(dst, &a.maps[sh ? kMapSGate : kMapGate], bar, c, row, e);
                            tma_load_3d(dst + kWTile / 2, &a.maps[sh ? kMapSUp : kMapUp], bar, c, row, e);
                        }
                    } else {
                        // K tiles past the end are zero-filled and counted all the same
                        ptx::mbar_arrive_expect_tx(bar, kABytes);
                        tma_load_4d(dst, &a.maps[sh ? kMapSDown : kMapDown], bar, 0,
                                    un.tile * kDownRows, k, e);
                    }
                    if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
                }
            }
            if (ok) post(-1);
        }
    } else if (warp == 1) {
        // -------------------------------------------------- the rows beside the weights
        if (lane == 0 && !a.test_stall) {
        int stage = 0, slot = 0;
        uint32_t phase = 0, qphase = 0;
        bool ok = true;
        while (ok) {
            if (!wait_bounded(&ctl->qfull[slot], qphase, ctl, a, 20)) break;
            const int u = ctl->queue[slot];
            ptx::mbar_arrive(&ctl->qempty[slot]);
            if (++slot == kQueue) { slot = 0; qphase ^= 1u; }
            if (u < 0) break;
            const Unit un = unit_at(a, sc, u, shared);
            const bool sh = un.group < shared;
            const int tokens = __popc((uint32_t)ctl->mask[un.group]);
            const int w = NT == 8 || tokens <= 8 ? 8 : 16;
            const int row0 = ctl->row0[un.group] - (sh || !shared ? 0 : a.T);
            if (un.down) {
                // the group's h: finished tiles are counted by whoever finishes them
                const int tiles = FMT ? (sh ? a.Is : a.I) / 128 : sh ? sc.gs : sc.gr;
                if (ld_acquire(a.ready + un.group) < tiles) {
                    const uint64_t t0 = ptx::globaltimer_ns();
                    while (ld_acquire(a.ready + un.group) < tiles) {
                        __nanosleep(32);
                        if (*(volatile int*)&ctl->abort_flag) { ok = false; break; }
                        if (ptx::globaltimer_ns() - t0 > a.timeout_ns) {
                            record_error(a.err, MOE_ERR_TIMEOUT, 21);
                            *(volatile int*)&ctl->abort_flag = 1;
                            ok = false;
                            break;
                        }
                    }
                    if (!ok) break;
                }
                fence_proxy_async_global();
            }
            const CUtensorMap* map =
                &a.maps[w == 8 ? (sh ? kMapHS8 : kMapH8) : (sh ? kMapHS16 : kMapH16)];
            for (int k = un.k0; k < un.k0 + un.n; k += kTiles) {
                if (!wait_bounded(&ctl->empty[stage], phase ^ 1u, ctl, a, 22)) { ok = false; break; }
                uint8_t* dst = ring + stage * C::kStage + kABytes;
                uint64_t* bar = &ctl->full[stage];
                if (!un.down) {
                    ptx::mbar_arrive_expect_tx(bar, kTiles * C::kXTile);
                    if (FMT) tma_load_4d(dst, &a.maps[kMapX], bar, 0, 0, 0, k);
                    else tma_load_3d(dst, &a.maps[kMapX], bar, 0, 0, k);
                } else {
                    ptx::mbar_arrive_expect_tx(bar, kTiles * C::kHPlanes * w * 128);
                    tma_load_4d(dst, map, bar, 0, row0, 0, k);
                }
                if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
            }
        }
        }
    } else if (warp == 2) {
        // -------------------------------------------------- products
        if (lane == 0) {
            int stage = 0, slot = 0, buf = 0;
            uint32_t phase = 0, qphase = 0, bphase = 0;
            bool ok = true, any = false;
            while (ok) {
                if (!wait_bounded(&ctl->qfull[slot], qphase, ctl, a, 30)) break;
                const int u = ctl->queue[slot];
                ptx::mbar_arrive(&ctl->qempty[slot]);
                if (++slot == kQueue) { slot = 0; qphase ^= 1u; }
                if (u < 0) break;
                const Unit un = unit_at(a, sc, u, shared);
                const int w = NT == 8 || __popc((uint32_t)ctl->mask[un.group]) <= 8 ? 8 : 16;
                const int n = un.down ? C::kHCols * w : C::kXCols;
                const uint32_t idesc = FMT ? ptx::idesc_e4m3_f32(128, n) : ptx::idesc_bf16_f32(128, n);
                const uint32_t btile = un.down ? C::kHPlanes * w * 128 : C::kXTile;
                // an accumulator a K tile, emptied every stage, where the scales change along K
                const bool each = un.down ? FMT != 0 : FMT == 2;
                for (int k = 0; k < un.n; k += kTiles) {
                    if (each || k == 0) {
                        if (!wait_bounded(&ctl->tempty[buf], bphase ^ 1u, ctl, a, 31)) { ok = false; break; }
                    }
                    if (!wait_bounded(&ctl->full[stage], phase, ctl, a, 32)) { ok = false; break; }
                    ptx::tc_fence_after();
                    const uint32_t w0 = ptx::smem_u32(ring + stage * C::kStage), b0 = w0 + kABytes;
                    const uint32_t d0 = tmem + buf * 128;
                    const int nk = min(kTiles, un.n - k);
                    for (int i = 0; i < nk; ++i) {
                        const uint32_t acc = each ? d0 + i * n : d0;
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            const uint64_t wd = ptx::sw128_kmajor_desc(w0 + i * kWTile + kk * 32);
                            const uint64_t bd = ptx::sw128_kmajor_desc(b0 + i * btile + kk * 32);
                            const bool fresh = kk == 0 && (each || (k == 0 && i == 0));
                            if constexpr (FMT) ptx::tc_mma_f8(acc, wd, bd, idesc, fresh ? 0u : 1u);
                            else ptx::tc_mma_f16(acc, wd, bd, idesc, fresh ? 0u : 1u);
                        }
                    }
                    any = true;
                    ptx::tc_commit(&ctl->empty[stage]);
                    if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
                    if (each || k + kTiles >= un.n) {
                        ptx::tc_commit(&ctl->tfull[buf]);
                        if (++buf == kBufs) { buf = 0; bphase ^= 1u; }
                    }
                }
            }
            if (!ok && any) {
                // products in flight read the ring and write tensor memory: let them end
                // (bounded by time: an abort leaves no barrier to count on)
                const uint64_t t0 = ptx::globaltimer_ns();
                while (ptx::globaltimer_ns() - t0 < 2000000ull) {
                }
            }
        }
    } else if (warp >= 4) {
        const bool sums = warp < 8;            // warps 4-7; 8-11 finish
        const int r = (warp & 3) * 32 + lane;  // weight row of the tile
        int slot = 0;
        uint32_t qphase = 0;
        // the four warps of a role stop together: they meet at barriers
        const auto pass = [&](uint64_t* bar, uint32_t parity, int where) {
            const int good = lane == 0 ? (int)wait_bounded(bar, parity, ctl, a, where) : 0;
            return ptx::named_bar_and(sums ? 1 : 2, 128, __shfl_sync(0xffffffffu, good, 0) != 0);
        };
        // a warp's own wait, in loops over stages: its role votes at the ends of units and chunks
        const auto wait = [&](uint64_t* bar, uint32_t parity, int where) {
            const int good = lane == 0 ? (int)wait_bounded(bar, parity, ctl, a, where) : 0;
            __syncwarp();
            return __shfl_sync(0xffffffffu, good, 0) != 0;
        };
        const auto joined = [](const auto& v, int t) {  // x's two planes, tokens 2 t and 2 t + 1
            return fma2(pack_bits(v[NT + 2 * t], v[NT + 2 * t + 1]), pack2(0.0625f, 0.0625f),
                        pack_bits(v[2 * t], v[2 * t + 1]));
        };
        // a K tile's block scale: all of a warp's rows have the same, a lane holds every 32nd
        struct BlockScales {
            const float* p;
            int n, lane;
            float now, next;
            __device__ __forceinline__ float at(int k) const {
                return k + lane < n ? __ldg(p + k + lane) : 0.0f;
            }
            __device__ __forceinline__ BlockScales(const float* p_, int n_, int lane_)
                : p(p_), n(n_), lane(lane_), now(at(0)), next(at(32)) {}
            // of the tiles from k on; every stage in turn
            __device__ __forceinline__ void stage(int k, float (&b)[kTiles]) {
                if (k > 0 && (k & 31) == 0) {
                    now = next;
                    next = at(k + 32);
                }
#pragma unroll
                for (int i = 0; i < kTiles; ++i) b[i] = __shfl_sync(0xffffffffu, now, (k & 31) + i);
            }
        };
        const auto release = [&](uint64_t* bar) {
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar);
        };
        if (sums) {
            // ---------------------------------------------- sums
            const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
            int buf = 0;
            uint32_t bphase = 0;
            bool ok = true;
            while (ok) {
                if (!pass(&ctl->qfull[slot], qphase, 40)) break;
                const int uid = ctl->queue[slot], mine = slot;
                if (++slot == kQueue) { slot = 0; qphase ^= 1u; }
                if (uid < 0) {
                    release(&ctl->summed[mine]);
                    break;
                }
                const Unit un = unit_at(a, sc, uid, shared);
                const bool sh = un.group < shared;
                const int e = sh ? 0 : ctl->expert[un.group];
                const uint32_t mask = ctl->mask[un.group];
                const int row0 = ctl->row0[un.group];
                const int I = sh ? a.Is : a.I;
                if (!un.down) {
                    f2 sums2[NT / 2];
#pragma unroll
                    for (int t = 0; t < NT / 2; ++t) sums2[t] = 0u;
                    const bool up = r >= kGateRows;
                    // the thread's row scale, or its blocks' along K
                    const float* sp = FMT ? (up ? (sh ? a.ss_up : a.s_up) : (sh ? a.ss_gate : a.s_gate))
                                          : nullptr;
                    float rs = 1.0f;
                    if constexpr (FMT == 1)
                        rs = __ldg(sp + (int64_t)e * I + un.tile * kGateRows + r % kGateRows);
                    if constexpr (FMT == 2) {
                        BlockScales scales(sp + ((int64_t)e * (I / 128) + un.tile / 2) * (a.d / 128) + un.k0,
                                           un.n, lane);
                        for (int k = 0; k < un.n; k += kTiles) {
                            if (!wait(&ctl->tfull[buf], bphase, 41)) { ok = false; break; }
                            ptx::tc_fence_after();
                            const uint32_t at = tmem + lanes + buf * 128;
                            uint32_t v[kTiles][C::kXCols];
#pragma unroll
                            for (int i = 0; i < kTiles; ++i) load_cols(at + i * C::kXCols, v[i]);
                            ptx::tmem_ld_wait();
                            ptx::tc_fence_before();
                            release(&ctl->tempty[buf]);
                            if (++buf == kBufs) { buf = 0; bphase ^= 1u; }
                            float bs[kTiles];
                            scales.stage(k, bs);
#pragma unroll
                            for (int i = 0; i < kTiles; ++i) {
                                if (k + i >= un.n) continue;  // not written
#pragma unroll
                                for (int t = 0; t < NT / 2; ++t)
                                    sums2[t] = fma2(joined(v[i], t), pack2(bs[i], bs[i]), sums2[t]);
                            }
                        }
                        ok = ptx::named_bar_and(1, 128, ok);
                    } else if (un.n > 0) {
                        ok = pass(&ctl->tfull[buf], bphase, 41);
                        if (!ok) break;
                        ptx::tc_fence_after();
                        uint32_t v[C::kXCols];
                        load_cols(tmem + lanes + buf * 128, v);
                        ptx::tmem_ld_wait();
                        ptx::tc_fence_before();
                        release(&ctl->tempty[buf]);
                        if (++buf == kBufs) { buf = 0; bphase ^= 1u; }
#pragma unroll
                        for (int t = 0; t < NT / 2; ++t) {
                            if constexpr (FMT) sums2[t] = joined(v, t);
                            else sums2[t] = pack_bits(v[2 * t], v[2 * t + 1]);
                        }
                    }
                    if (!ok) break;
                    float s[NT];
                    unpack_pairs(sums2, s);
                    int c = 0;
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        if (!(mask >> t & 1u)) continue;
                        const float x = FMT ? ctl->xs[t] * rs : 1.0f;
                        __stcg(gate_sums(a, row0 + c, sh, shared, un.tile) + un.part * 2 * kGateRows + r,
                               s[t] * x);
                        ++c;
                    }
                } else {
                    const int tokens = __popc(mask);
                    const int w = NT == 8 || tokens <= 8 ? 8 : 16;
                    const int col = un.tile * kDownRows + r;
                    float s[NT];
                    f2 sums2[NT / 2];
#pragma unroll
                    for (int t = 0; t < NT; ++t) s[t] = 0.0f;
#pragma unroll
                    for (int t = 0; t < NT / 2; ++t) sums2[t] = 0u;
                    float rs = 1.0f;
                    const auto read = [&]() {
                        ptx::tc_fence_before();
                        release(&ctl->tempty[buf]);
                        if (++buf == kBufs) { buf = 0; bphase ^= 1u; }
                    };
                    if constexpr (FMT == 0) {
                        if (un.n > 0) {
                            ok = pass(&ctl->tfull[buf], bphase, 42);
                            if (!ok) break;
                            ptx::tc_fence_after();
                            const uint32_t at = tmem + lanes + buf * 128;
                            if (w == 8) down_sums<8>(at, s);
                            else if constexpr (NT == 16) down_sums<16>(at, s);
                            read();
                        }
                    } else {
                        const float* sp = sh ? a.ss_down : a.s_down;
                        if constexpr (FMT == 1) rs = __ldg(sp + (int64_t)e * a.d + col);  // d a multiple of 128
                        BlockScales scales(FMT == 2 ? sp + ((int64_t)e * (a.d / 128) + un.tile) * (I / 128) + un.k0
                                                    : nullptr,
                                           FMT == 2 ? un.n : 0, lane);
                        // h's scales go through shared memory, a chunk of K tiles at a time, asked
                        // for a chunk ahead (the first once a product shows that h is done)
                        const float* hs = (sh ? a.hs_s : a.hs) + un.k0 +
                                          (int64_t)(row0 - (sh || !shared ? 0 : a.T)) * (I / 128);
                        float hv[kChunk * 16 / 128];
                        const auto ask = [&](int k) {
#pragma unroll
                            for (int q = 0; q < kChunk * 16 / 128; ++q) {
                                const int i = (r + 128 * q) >> 4, c = r & 15;
                                hv[q] = k + i < un.n && c < tokens
                                            ? __ldcg(hs + (int64_t)c * (I / 128) + k + i) : 0.0f;
                            }
                        };
                        for (int k = 0; k < un.n; k += kTiles) {
                            // a warp whose wait ran out goes on to the vote without its sums
                            if (ok) ok = wait(&ctl->tfull[buf], bphase, 42);
                            ptx::tc_fence_after();
                            float* hsc = ctl->hscale[k / kChunk & 1] + k % kChunk * 16;
                            if (k % kChunk == 0) {
                                if (k == 0) ask(0);
#pragma unroll
                                for (int q = 0; q < kChunk * 16 / 128; ++q) hsc[r + 128 * q] = hv[q];
                                ok = ptx::named_bar_and(1, 128, ok);
                                if (!ok) break;
                                if (k + kChunk < un.n) ask(k + kChunk);
                            }
                            if (!ok) continue;
                            float bs[kTiles] = {};
                            if constexpr (FMT == 2) scales.stage(k, bs);
                            const uint32_t at = tmem + lanes + buf * 128;
                            const int tiles = un.n - k;
                            if (tokens <= 2) add_down<FMT, 8, 2, NT>(at, hsc, bs, tiles, sums2, read);
                            else if (w == 8) add_down<FMT, 8, 8, NT>(at, hsc, bs, tiles, sums2, read);
                            else if constexpr (NT == 16)
                                add_down<FMT, 16, 16, NT>(at, hsc, bs, tiles, sums2, read);
                        }
                        ok = ptx::named_bar_and(1, 128, ok);
                    }
                    if (!ok) break;
                    if constexpr (FMT) unpack_pairs(sums2, s);
                    if (col < a.d) {
#pragma unroll
                        for (int t = 0; t < NT; ++t)
                            if (t < tokens)
                                __stcg(a.yp + ((int64_t)(row0 + t) * a.dp + un.part) * a.d + col, s[t] * rs);
                    }
                }
                release(&ctl->summed[mine]);
                release(&ctl->qempty[mine]);
            }
        } else {
            // ---------------------------------------------- finishing
            // Its own warps, so that the fence and the count of a part (microseconds while
            // the memory is busy) hold up neither the sums nor the stream.
            if constexpr (ONE) {
                if (warp == 8) {
                    const bool on = lane < a.K;
                    float sum;
                    const float w = pick_weight(a, on ? ctl->weight[lane] : 0.0f,
                                                on ? ctl->expert[shared + lane] : 0, lane, sum);
                    __syncwarp();
                    if (on) ctl->weight[lane] = w / sum;
                }
                finish_sync();
            }
            while (pass(&ctl->summed[slot], qphase, 50)) {
                const int uid = ctl->queue[slot];
                release(&ctl->qempty[slot]);
                if (++slot == kQueue) { slot = 0; qphase ^= 1u; }
                if (uid < 0) break;
                const Unit un = unit_at(a, sc, uid, shared);
                if (!un.down) {
                    // all parts of the tile; 8-bit: of the two tiles that share h's scales
                    const int tiles = FMT ? max(a.I, a.Is) / 128 : max(sc.gr, sc.gs);
                    int* counter = a.gticket + un.group * tiles + (FMT ? un.tile / 2 : un.tile);
                    if (!last_part(ctl, counter, FMT ? 2 * a.gp : a.gp, r)) continue;
                    finish_h<FMT, NT>(a, ctl, un, r, shared);
                } else if (last_part(ctl, a.dticket + un.tile, ctl->groups * a.dp, r)) {
                    join_tile<NT>(a, ctl, un.tile, warp & 3, lane);
                }
            }
        }
    }
    __syncwarp();
    if (warp == 0 && *(volatile int*)&ctl->abort_flag) {
        // copies in flight write the ring: give them a bounded time before it goes
        const uint64_t t0 = ptx::globaltimer_ns();
        while (ptx::globaltimer_ns() - t0 < 2000000ull) {
        }
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 3) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ host side
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// a map of `rank` dimensions, the first 128 bytes or more of `size`-byte elements; strides in
// bytes, of all but the first
bool make_map(CUtensorMap* m, const void* base, int size, int rank, const int64_t (&dim)[4],
              const int64_t (&stride)[3], const int (&box)[4]) {
    const EncodeTiledFn fn = (EncodeTiledFn)tensor_map_encoder();
    if (!fn) return false;
    cuuint64_t dims[4], strides[3];
    cuuint32_t boxes[4], ones[4] = {1, 1, 1, 1};
    for (int i = 0; i < 4; ++i) {
        dims[i] = (cuuint64_t)dim[i];
        boxes[i] = (cuuint32_t)box[i];
        if (i < 3) strides[i] = (cuuint64_t)stride[i];
    }
    return fn(m, size == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, rank,
              const_cast<void*>(base), dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// gate or up weights [n][rows][cols]: `box` rows of one K tile
bool gate_map(CUtensorMap* m, const void* base, int size, int64_t n, int64_t rows, int64_t cols,
              int box) {
    return make_map(m, base, size, 3, {cols, rows, n, 1}, {cols * size, rows * cols * size, 0},
                    {128 / size, box, 1, 1});
}

// down weights [n][rows][cols]: `box` rows of q K tiles, tile after tile
bool down_map(CUtensorMap* m, const void* base, int size, int64_t n, int64_t rows, int64_t cols,
              int box, int q) {
    return make_map(m, base, size, 4, {128 / size, rows, cols * size / 128, n},
                    {cols * size, 128, rows * cols * size}, {128 / size, box, q, 1});
}

// planes [p][rows][cols] of x or h: `box` rows of every plane, of q K tiles
bool rows_map(CUtensorMap* m, const void* base, int size, int64_t planes, int64_t rows, int64_t cols,
              int box, int q) {
    return make_map(m, base, size, 4, {128 / size, rows, planes, cols * size / 128},
                    {cols * size, rows * cols * size, 128}, {128 / size, box, (int)planes, q});
}

// ONE: T = 1, of its own, for its choice is another and its code is read anew by every call
template <int FMT, int NT, bool ONE = false>
cudaError_t go(const FewArgs& a, cudaStream_t st) {
    using C = Cfg<FMT, NT>;
    constexpr size_t smem = 1024 + (size_t)C::kStages * C::kStage + sizeof(Ctl);
    static_assert(smem <= 232448, "shared memory exceeds the per-block limit");
    static_assert(8u * kMaxT * 1024 <= (size_t)C::kStages * C::kStage, "keys and scores fit the ring");
    static_assert(sizeof(FewArgs) <= 4000, "the arguments fit the launch");
    cudaError_t e = cudaFuncSetAttribute(few_experts_kernel<FMT, NT, ONE>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    // no more blocks than units, were every pick another expert's
    const int64_t groups = a.T * a.K < a.E ? a.T * a.K : a.E;
    const int64_t units = a.gp * (a.Is + groups * a.I) / kGateRows +
                          a.dp * (groups + (a.Is > 0)) * ceil_div(a.d, kDownRows);
    const int sms = device_sm_count();
    return launch_pdl(few_experts_kernel<FMT, NT, ONE>, dim3((unsigned)(units < sms ? units : sms)),
                      dim3(kThreads), smem, st, a);
}

constexpr int kClaimInts = 64;
// Tokens of a warp of launch 1: fewer where that leaves less than these units, for a warp's
// loads and sums are a chain that all wait for (64 experts of 2048, T = 3: a token each 60.3 us a
// call, two 60.7, four 62; 256 experts of 7168, E4M3, T = 8: four 312 us, eight 314).
constexpr int kScoreUnits = 4096;
int score_splits(int d) {
    // a 16-byte vector a lane, or more in rows wider than 2048 (64 experts of 2048, T = 3: 62 us
    // a call, with three vectors 64)
    const int n = d / 8 / 32;
    return n < 1 ? 1 : n > kScoreSplits ? kScoreSplits : n;
}

// Parts that K is cut into: enough that every block gets about this many units, were all
// experts equally likely, with at least this many stages left in each.
constexpr double kGateUnits = 2, kDownUnits = 3;
constexpr int kLeastStages = 8;

int parts_for(double tiles, double units, int64_t k_tiles) {
    const double sms = 152;  // not asked of the device: the workspace query needs none
    int p = 1;
    while (p < 8 && tiles * p < units * sms && k_tiles / kTiles / (p + 1) >= kLeastStages) ++p;
    return p;
}

}  // namespace

FewWs few_ws(const moe_shape& s, int fmt) {
    // fmt 0 bf16 (h as two bf16 planes), else 8-bit (x as two planes, h as three, scales)
    FewWs w{};
    const int64_t T = s.T, K = s.K, d = s.d, I = s.inter, Is = s.inter_shared, n = T * K;
    const int64_t groups = (n < s.E ? n : s.E) + 1;
    const int64_t ti = ceil_div(I, 128), ts = ceil_div(Is, 128), td = ceil_div(d, kDownRows);
    const double routed = s.E * (1.0 - pow(1.0 - (double)K / s.E, (double)T));
    const int elems = fmt ? 128 : 64;
    w.gp = parts_for((routed * I + Is) / kGateRows, kGateUnits, d / elems);
    w.dp = parts_for((routed + (Is > 0)) * td, kDownUnits, (I > Is ? I : Is) / elems);
    w.splits = score_splits(s.d);
    size_t o = 256;  // the error record, then the counters
    auto take = [&](int64_t bytes) {
        const size_t at = o;
        o = (o + (size_t)bytes + 255) / 256 * 256;
        return at;
    };
    // the claims' counter in a cache line of its own
    w.counters = (int)(kClaimInts + groups + td + groups * 2 * (ti > ts ? ti : ts));
    w.claim = take(4 * (int64_t)w.counters);
    w.part = take(4 * (int64_t)w.splits * T * s.E);
    w.xq = take(fmt ? 2 * T * d : 0);
    w.xs = take(fmt ? 4 * T : 0);
    w.gpart = take(8 * (n * I + T * Is) * w.gp);
    w.h = take(fmt ? 3 * n * I : 4 * n * I);
    w.h_s = take(fmt ? 3 * T * Is : 4 * T * Is);
    w.hs = take(fmt ? 4 * n * ti : 0);
    w.hs_s = take(fmt ? 4 * T * ts : 0);
    w.yp = take(4 * (n + (Is ? T : 0)) * d * w.dp);
    w.total = o;
    return w;
}

cudaError_t launch_few(const moe_shape& s, int fmt, const FewCall& c, void* workspace,
                       cudaStream_t st) {
    const FewWs w = few_ws(s, fmt);
    uint8_t* base = static_cast<uint8_t*>(workspace);
    const int64_t T = s.T, d = s.d, E = s.E, I = s.inter, Is = s.inter_shared, n = T * s.K;
    const int size = fmt ? 1 : 2, nt = T <= 8 ? 8 : 16;
    FewArgs a{};
    a.T = s.T; a.d = s.d; a.E = s.E; a.K = s.K; a.I = s.inter; a.Is = s.inter_shared;
    a.sigmoid = s.router == MOE_ROUTER_SIGMOID;
    a.splits = w.splits;
    a.bias = c.bias;
    a.residual = (const bf16*)c.residual;
    a.y = (bf16*)c.y;
    a.err = reinterpret_cast<DevError*>(base);
    a.claim = reinterpret_cast<int*>(base + w.claim);
    const int64_t groups = (n < E ? n : E) + 1;
    a.ready = a.claim + kClaimInts;
    a.dticket = a.ready + groups;
    a.gticket = a.dticket + ceil_div(d, kDownRows);
    a.part = reinterpret_cast<float*>(base + w.part);
    a.xs = fmt ? reinterpret_cast<float*>(base + w.xs) : nullptr;
    a.gpart = reinterpret_cast<float*>(base + w.gpart);
    a.h = base + w.h;
    a.h_s = base + w.h_s;
    a.hs = reinterpret_cast<float*>(base + w.hs);
    a.hs_s = reinterpret_cast<float*>(base + w.hs_s);
    a.yp = reinterpret_cast<float*>(base + w.yp);
    a.s_gate = c.s_gate; a.s_up = c.s_up; a.s_down = c.s_down;
    a.ss_gate = c.ss_gate; a.ss_up = c.ss_up; a.ss_down = c.ss_down;
    a.timeout_ns = tc_timeout_ns();
    a.test_stall = tc_test_stall();
    a.ws_gate = (const uint8_t*)c.ws_gate;
    a.ws_up = (const uint8_t*)c.ws_up;
    a.hint = Is * d * size < kHintMost ? Is * d * size : kHintMost;
    a.gp = w.gp;
    a.dp = w.dp;
    const int elems = 128 / size;
    bool ok = gate_map(&a.maps[kMapGate], c.w_gate, size, E, I, d, kGateRows) &&
              gate_map(&a.maps[kMapUp], c.w_up, size, E, I, d, kGateRows) &&
              down_map(&a.maps[kMapDown], c.w_down, size, E, d, I, kDownRows, kTiles) &&
              rows_map(&a.maps[kMapH8], a.h, size, fmt ? 3 : 2, n, I, 8, kTiles) &&
              rows_map(&a.maps[kMapH16], a.h, size, fmt ? 3 : 2, n, I, nt, kTiles) &&
              (fmt ? rows_map(&a.maps[kMapX], base + w.xq, 1, 2, T, d, nt, kTiles)
                   : make_map(&a.maps[kMapX], c.x, 2, 3, {elems, T, d / elems, 1}, {d * 2, 128, 0},
                              {elems, 16, kTiles, 1}));
    if (Is > 0) {
        ok = ok && gate_map(&a.maps[kMapSGate], c.ws_gate, size, 1, Is, d, kGateRows) &&
             gate_map(&a.maps[kMapSUp], c.ws_up, size, 1, Is, d, kGateRows) &&
             down_map(&a.maps[kMapSDown], c.ws_down, size, 1, d, Is, kDownRows, kTiles) &&
             rows_map(&a.maps[kMapHS8], a.h_s, size, fmt ? 3 : 2, T, Is, 8, kTiles) &&
             rows_map(&a.maps[kMapHS16], a.h_s, size, fmt ? 3 : 2, T, Is, nt, kTiles);
    } else {
        // never loaded from: any valid map
        a.maps[kMapSGate] = a.maps[kMapSUp] = a.maps[kMapGate];
        a.maps[kMapSDown] = a.maps[kMapDown];
        a.maps[kMapHS8] = a.maps[kMapHS16] = a.maps[kMapH8];
    }
    if (!ok) return cudaErrorInvalidValue;

    const auto units_of = [&](int tokens) { return (int)ceil_div(T, tokens) * s.E * w.splits; };
    int tt = T <= 1 ? 1 : T <= 2 ? 2 : T <= 4 ? 4 : 8;
    while (tt > 1 && units_of(tt) < kScoreUnits) tt /= 2;
    const int units = units_of(tt);
    int blocks = (int)ceil_div(units, kScoreWarps);
    const int most = 8 * device_sm_count();
    if (blocks > most) blocks = most;
    const dim3 grid(blocks + (fmt ? s.T : 0)), block(kScoreWarps * 32);
    // the error record is zeroed with the counters
    int* zero = reinterpret_cast<int*>(base);
    const int n_zero = (int)(w.claim / 4) + w.counters;
    cudaError_t e;
#define MOE_SCORES(TT)                                                                           \
    e = launch_pdl(few_scores_kernel<TT>, grid, block, 0, st, (const bf16*)c.x,                  \
                   (const bf16*)c.w_g, a.part, base + w.xq, a.xs, zero, n_zero, s.T, s.d, s.E,   \
                   w.splits, blocks)
    if (tt == 1) MOE_SCORES(1);
    else if (tt == 2) MOE_SCORES(2);
    else if (tt == 4) MOE_SCORES(4);
    else MOE_SCORES(8);
#undef MOE_SCORES
    if (e != cudaSuccess) return e;
    if (T == 1) return fmt == 0 ? go<0, 8, true>(a, st) : fmt == 1 ? go<1, 8, true>(a, st) : go<2, 8, true>(a, st);
    if (fmt == 0) return nt == 8 ? go<0, 8>(a, st) : go<0, 16>(a, st);
    if (fmt == 1) return nt == 8 ? go<1, 8>(a, st) : go<1, 16>(a, st);
    return nt == 8 ? go<2, 8>(a, st) : go<2, 16>(a, st);
}

}  // namespace moe
