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
// cuts all work into units: 128 gate and 128 up rows, or 128 down rows, of a group
// over a run of K.  Blocks take units from one counter in the order gate/up, then
// down.  A down unit needs its group's h, which units before it in that order make:
// whoever holds those took them earlier and is running, so every wait ends whatever
// part of the grid is resident, and two calls on two streams share the GPU safely.
//
// In a block, roles pass work through shared memory as the tensor-core GEMM's do:
// warp 0 takes units and streams weight tiles (TMA, 128-byte swizzle), warp 1 the
// rows that multiply them, warp 2 issues tcgen05 products with the weights as the
// 128-row operand and the tokens as its few columns, warps 4-7 empty the accumulators.
// Warp 0 runs ahead by the ring's depth (160 KB and more an SM) without waiting for h,
// so the weights of the next part are on their way while h is still being finished.
//
// Rows that multiply: every token's x (a group's outputs are kept for its own tokens
// alone, so a column that is not wanted costs nothing and spoils nothing, NaN
// included), and h of the group's tokens.  Precision: bf16 experts take x as it is and
// h as two bf16 planes (hi, remainder: within 2^-16).  8-bit experts take x as two
// E4M3 planes, the second 16 times finer, with a power of two as the row's scale,
// which holds a bf16 value exactly down to 2^-23 of the row's largest; and h as three
// such planes with a scale per 128 values (within 2^-12, beside a code's own 2^-4).
// Planes are further columns, their sums are joined in fp32.
//
// A unit's sums over part of K go to a buffer, and whoever finishes a tile's last part
// adds the parts in their order; the same for the sum over experts.  No floating-point
// atomics: the same bits on every run, whoever takes which unit.
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
constexpr int kThreads = 256;
constexpr int kBufs = 4;       // accumulator buffers of 128 tensor-memory columns
constexpr int kQueue = 4;      // units between the roles
constexpr int kMaxUnit = 32;   // most stages of a unit
constexpr int kABytes = 32768; // weights of a stage: two tiles of 128 rows x 128 bytes
constexpr uint32_t kAcc1 = 64; // columns from a buffer's first accumulator to its second

// FMT: 0 bf16 weights, 1 E4M3 with a scale a row, 2 E4M3 with a scale per 128 x 128 block.
// NT: columns that tokens take (8 or 16).
template <int FMT, int NT>
struct Cfg {
    static constexpr int kElems = FMT ? 128 : 64;    // K of a tile: 128 bytes
    static constexpr int kHPlanes = FMT ? 3 : 2;     // of h
    static constexpr int kHCols = FMT ? 4 : 2;       // the same as columns (a multiple of 16 in all)
    static constexpr int kHTile = kHCols * NT * 128; // bytes of h beside one weight tile
    static constexpr int kXBytes = FMT ? 2 * NT * 128 : 16 * 128;
    static constexpr int kStage = kABytes + 2 * kHTile;
    static constexpr int kStages = kStage > 45000 ? 4 : 5;
};

enum { kMapGate, kMapUp, kMapDown, kMapSGate, kMapSUp, kMapSDown, kMapX, kMapH, kMapHS, kMaps };

struct FewArgs {
    CUtensorMap maps[kMaps];
    int T, d, E, K, I, Is, sigmoid, splits, max_parts, test_stall;
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
    uint64_t full[5], empty[5], tfull[kBufs], tempty[kBufs], qfull[kQueue], qempty[kQueue];
    uint32_t tmem;
    int abort_flag;
    int queue[kQueue];
    int last;
    int groups;                   // with the shared expert
    uint32_t present[32];         // experts that a token picked
    uint16_t before[33];          // how many of them before a word of `present`
    uint16_t expert[kMaxGroups];  // of a group
    alignas(4) uint16_t mask[kMaxGroups + 1];  // tokens of a group (set by 32-bit atomics)
    uint16_t row0[kMaxGroups + 1];
    uint16_t pick[kMaxSlots];     // expert, then row, of a slot
    float weight[kMaxSlots];
    float top[4][kMaxT];
    float hscale[2 * kMaxUnit * kMaxT];
    float wscale[2][2 * kMaxUnit];
    alignas(16) float strand[4][128];  // read and written as float4
};

struct Unit {
    int down, group, tile, part, s0, ns;
};

// Cut of the work into units, the same in every block: a function of the sizes and of the
// number of groups.
struct Sched {
    int nk, nks, nkr;          // stages over K: gate/up, shared and routed down
    int tiles_s, tiles_r, tiles_d;
    int gp, gc, dps, dcs, dpr, dcr;  // parts of a tile and stages of a part
    int u1, u2, u3, u4;        // ends of: shared gate/up, routed, shared down, routed down
};

__device__ __forceinline__ void cut(int n, int want, int most, int& parts, int& stages) {
    parts = min(most, (n + want - 1) / want);
    stages = (n + parts - 1) / parts;
    parts = (n + stages - 1) / stages;
}

__device__ Sched make_sched(const FewArgs& a, int groups, int elems, int blocks) {
    Sched s;
    const int shared = a.Is > 0, routed = groups - shared;
    const auto up = [](int n, int d) { return (n + d - 1) / d; };
    s.nk = up(a.d, elems);
    s.nks = up(a.Is, 2 * elems);
    s.nkr = up(a.I, 2 * elems);
    s.tiles_s = up(a.Is, 128);
    s.tiles_r = up(a.I, 128);
    s.tiles_d = up(a.d, 128);
    const int64_t all = (int64_t)s.nk * (s.tiles_s + routed * s.tiles_r) +
                        (int64_t)s.tiles_d * (s.nks + (int64_t)routed * s.nkr);
    // a block's share in about 16 units, so that the last ones end near each other
    const int want = (int)max((int64_t)1, min((int64_t)kMaxUnit, all / (16 * (int64_t)blocks)));
    cut(s.nk, want, a.max_parts, s.gp, s.gc);
    cut(s.nks > 0 ? s.nks : 1, want, a.max_parts, s.dps, s.dcs);
    cut(s.nkr, want, a.max_parts, s.dpr, s.dcr);
    s.u1 = s.tiles_s * s.gp;
    s.u2 = s.u1 + routed * s.tiles_r * s.gp;
    s.u3 = s.u2 + (shared ? s.tiles_d * s.dps : 0);
    s.u4 = s.u3 + routed * s.tiles_d * s.dpr;
    return s;
}

__device__ __forceinline__ Unit unit_at(const Sched& s, int u, int shared) {
    Unit t;
    int tiles, parts, stages, n;
    if (u < s.u1) {
        t.down = 0; t.group = 0; tiles = s.tiles_s; parts = s.gp; stages = s.gc; n = s.nk;
    } else if (u < s.u2) {
        u -= s.u1;
        t.down = 0; tiles = s.tiles_r; parts = s.gp; stages = s.gc; n = s.nk;
        t.group = shared + u / (tiles * parts);
        u %= tiles * parts;
    } else if (u < s.u3) {
        u -= s.u2;
        t.down = 1; t.group = 0; tiles = s.tiles_d; parts = s.dps; stages = s.dcs; n = s.nks;
    } else {
        u -= s.u3;
        t.down = 1; tiles = s.tiles_d; parts = s.dpr; stages = s.dcr; n = s.nkr;
        t.group = shared + u / (tiles * parts);
        u %= tiles * parts;
    }
    t.tile = u / parts;
    t.part = u % parts;
    t.s0 = t.part * stages;
    t.ns = min(stages, n - t.s0);
    return t;
}

// 128 down rows of a K run with an odd number of tiles: the last stage has one tile
template <int FMT>
__device__ __forceinline__ int tiles_of_stage(const FewArgs& a, const Unit& u, int shared, int i) {
    const int n = (u.group < shared ? a.Is : a.I) / Cfg<FMT, 8>::kElems;
    return min(2, n - 2 * (u.s0 + i));
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

__device__ __forceinline__ void fence_proxy_async_all() {
    asm volatile("fence.proxy.async;" ::: "memory");
}
__device__ __forceinline__ int ld_acquire(const int* p) {
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void tma_load_3d(void* dst, const void* tmap, uint64_t* bar, int32_t c0,
                                            int32_t c1, int32_t c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(ptx::smem_u32(dst)),
        "l"(tmap), "r"(ptx::smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
// barrier of the four accumulator warps
__device__ __forceinline__ void drain_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// The least power of two s with amax / s <= 448 (to fp32 rounding), and 1 / s; 1 where
// amax is not positive.
__device__ __forceinline__ void plane_scale(float amax, float& s, float& inv) {
    const uint32_t q = __float_as_uint(amax / 448.0f);
    int e = (int)(q >> 23) + ((q & 0x7FFFFFu) != 0u ? 1 : 0);
    e = amax > 0.0f ? max(1, min(e, 252)) : 127;
    s = __uint_as_float((uint32_t)e << 23);
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
    pdl_wait();
    pdl_trigger();
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n_counters; i += gridDim.x * blockDim.x)
        counters[i] = 0;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nvec = d / 8;
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
    const int chunks = (T + TT - 1) / TT, vps = (nvec + splits - 1) / splits;
    const int units = chunks * E * splits;
    for (int u = blockIdx.x * kScoreWarps + warp; u < units; u += score_blocks * kScoreWarps) {
        const int s = u % splits, e = (u / splits) % E, t0 = u / (splits * E) * TT;
        const int v0 = s * vps, v1 = min(nvec, v0 + vps);
        float acc[TT];
#pragma unroll
        for (int m = 0; m < TT; ++m) acc[m] = 0.0f;
        const bf16* wrow = w_g + (int64_t)e * d;
#pragma unroll 4
        for (int v = v0 + lane; v < v1; v += 32) {
            float wf[8];
            unpack(ld_stream(wrow + v * 8), wf, (const bf16*)nullptr);
#pragma unroll
            for (int m = 0; m < TT; ++m) {
                float xf[8];
                unpack(ld_ro(x + (int64_t)min(t0 + m, T - 1) * d + v * 8), xf, (const bf16*)nullptr);
#pragma unroll
                for (int q = 0; q < 8; ++q) acc[m] = fmaf(wf[q], xf[q], acc[m]);
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

// The whole block chooses every token's experts (the rule of moe_route: the K largest keys,
// ties to the lower expert) and lists the groups.  `keys`: T * E floats of shared memory.
__device__ void choose(const FewArgs& a, Ctl* ctl, float* keys) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int shared = a.Is > 0;
    if (threadIdx.x < 32) ctl->present[threadIdx.x] = 0u;
    for (int i = threadIdx.x; i <= kMaxGroups; i += kThreads) ctl->mask[i] = 0;
    __syncthreads();
    for (int t = warp; t < a.T; t += kThreads / 32) {
        float* key = keys + t * a.E;
#pragma unroll 2
        for (int e = lane; e < a.E; e += 32) {
            const float s = score_of(a, t, e), b = a.bias ? a.bias[e] : 0.0f;
            key[e] = a.sigmoid ? 1.0f / (1.0f + expf(-s)) + b : s + b;
        }
        __syncwarp();
        uint32_t taken = 0;  // of this lane's experts lane, lane + 32, ...
        int mine = 0;        // lane j: the j-th pick
        float first = 0.0f, mykey = 0.0f;
        for (int j = 0; j < a.K; ++j) {
            float bk = 0.0f;
            int be = -1;
            for (int e = lane, m = 0; e < a.E; e += 32, ++m)
                if (!(taken >> m & 1u) && (be < 0 || key[e] > bk)) {
                    bk = key[e];
                    be = e;
                }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const float k2 = __shfl_xor_sync(0xffffffffu, bk, o);
                const int e2 = __shfl_xor_sync(0xffffffffu, be, o);
                if (e2 >= 0 && (be < 0 || k2 > bk || (k2 == bk && e2 < be))) {
                    bk = k2;
                    be = e2;
                }
            }
            // with NaN keys the lanes may differ: the first one's pick holds
            be = __shfl_sync(0xffffffffu, be, 0);
            bk = __shfl_sync(0xffffffffu, bk, 0);
            if ((be & 31) == lane) taken |= 1u << (be >> 5);
            if (lane == j) {
                mine = be;
                mykey = bk;
            }
            if (j == 0) first = bk;
        }
        float w = 0.0f;
        if (lane < a.K)
            w = a.sigmoid ? 1.0f / (1.0f + expf(-score_of(a, t, mine))) : expf(mykey - first);
        const float sum = warp_sum(w) + (a.sigmoid ? 1e-6f : 0.0f);
        if (lane < a.K) {
            ctl->pick[t * a.K + lane] = (uint16_t)mine;
            ctl->weight[t * a.K + lane] = w / sum;
            atomicOr(&ctl->present[mine >> 5], 1u << (mine & 31));
        }
    }
    __syncthreads();
    if (warp == 0) {
        int n = __popc(ctl->present[lane]);
        const int own = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, n, o);
            if (lane >= o) n += v;
        }
        ctl->before[lane] = (uint16_t)(n - own);
        if (lane == 31) ctl->groups = n + shared;
    }
    __syncthreads();
    const int slots = a.T * a.K;
    const auto group_of = [&](int e) {
        return shared + ctl->before[e >> 5] +
               __popc(ctl->present[e >> 5] & ((1u << (e & 31)) - 1u));
    };
    // masks are 16-bit halves of words: set with 32-bit atomics
    uint32_t* words = reinterpret_cast<uint32_t*>(ctl->mask);
    for (int f = threadIdx.x; f < slots; f += kThreads) {
        const int e = ctl->pick[f], g = group_of(e), t = f / a.K;
        ctl->expert[g] = (uint16_t)e;
        atomicOr(&words[g >> 1], 1u << (t + 16 * (g & 1)));
    }
    if (shared && threadIdx.x == 0) {
        ctl->expert[0] = 0;
        atomicOr(&words[0], (1u << a.T) - 1u);
    }
    __syncthreads();
    if (warp == 0) {
        int base = 0;
        for (int g0 = 0; g0 < ctl->groups; g0 += 32) {
            const int g = g0 + lane;
            const int own = g < ctl->groups ? __popc((uint32_t)ctl->mask[g]) : 0;
            int n = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, n, o);
                if (lane >= o) n += v;
            }
            if (g < ctl->groups) ctl->row0[g] = (uint16_t)(base + n - own);
            base += __shfl_sync(0xffffffffu, n, 31);
        }
        if (lane == 0) ctl->row0[ctl->groups] = (uint16_t)base;
    }
    __syncthreads();
    for (int f = threadIdx.x; f < slots; f += kThreads) {
        const int g = group_of(ctl->pick[f]), t = f / a.K;
        ctl->pick[f] =
            (uint16_t)(ctl->row0[g] + __popc((uint32_t)ctl->mask[g] & ((1u << t) - 1u)));
    }
    __syncthreads();
}

// y of 128 columns (tile m) from every part of every row: the shared expert first, then a
// token's picks in their order.  The four warps take tokens, or strands of a token's rows
// where there are fewer than four.
__device__ void join_tile(const FewArgs& a, const Sched& sc, Ctl* ctl, int m, int warp, int lane) {
    const int shared = a.Is > 0;
    const int c = m * 128 + lane * 4;
    const bool in = c < a.d;
    const int strands = a.T == 1 ? 4 : a.T == 2 ? 2 : 1;
    const int ns = shared ? sc.dps : 0, n = ns + a.K * sc.dpr;
    for (int item = warp; item < a.T * strands; item += 4) {
        const int t = item / strands, q = item % strands;
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (in) {
#pragma unroll 8
            for (int i = q; i < n; i += strands) {
                const bool sh = i < ns;
                const int j = sh ? 0 : (i - ns) / sc.dpr, p = sh ? i : (i - ns) % sc.dpr;
                const int row = sh ? t : ctl->pick[t * a.K + j];
                const float w = sh ? 1.0f : ctl->weight[t * a.K + j];
                const float4 v = __ldcg(reinterpret_cast<const float4*>(
                    a.yp + ((int64_t)row * a.max_parts + p) * a.d + c));
                s.x = fmaf(w, v.x, s.x);
                s.y = fmaf(w, v.y, s.y);
                s.z = fmaf(w, v.z, s.z);
                s.w = fmaf(w, v.w, s.w);
            }
        }
        if (strands > 1) {
            *reinterpret_cast<float4*>(&ctl->strand[item][lane * 4]) = s;
            drain_sync();
            for (int k = 1; k < strands; ++k) {
                const float4 v = *reinterpret_cast<const float4*>(
                    &ctl->strand[(t * strands + k) & 3][lane * 4]);
                if (q == 0) {
                    s.x += v.x;
                    s.y += v.y;
                    s.z += v.z;
                    s.w += v.w;
                }
            }
        }
        if (q != 0 || !in) continue;
        const int64_t at = (int64_t)t * a.d + c;
        if (a.residual) {
            const uint2 r = __ldg(reinterpret_cast<const uint2*>(a.residual + at));
            s.x += __uint_as_float(r.x << 16);
            s.y += __uint_as_float(r.x & 0xffff0000u);
            s.z += __uint_as_float(r.y << 16);
            s.w += __uint_as_float(r.y & 0xffff0000u);
        }
        const __nv_bfloat162 lo = __floats2bfloat162_rn(s.x, s.y), hi = __floats2bfloat162_rn(s.z, s.w);
        *reinterpret_cast<uint2*>(a.y + at) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                                         *reinterpret_cast<const uint32_t*>(&hi));
    }
}

// Thread 0 of the accumulator warps counts the tile's finished parts; true in all four
// warps for the block that finished the last one.  What every part wrote is then visible.
__device__ __forceinline__ bool last_part(Ctl* ctl, int* counter, int parts, int tid) {
    __threadfence();
    drain_sync();
    if (tid == 0) ctl->last = atomicAdd(counter, 1) == parts - 1;
    drain_sync();
    const bool last = ctl->last != 0;
    if (last) __threadfence();
    return last;
}

// h of one finished gate/up tile (thread r: row r), stored as planes; then the group's
// count of finished tiles.
template <int FMT, int NT>
__device__ __forceinline__ void store_h(const FewArgs& a, const Sched& sc, Ctl* ctl, const Unit& u,
                                        float (&h)[NT], int r, int shared) {
    using C = Cfg<FMT, NT>;
    const bool sh = u.group < shared;
    const int I = sh ? a.Is : a.I, rows = sh ? a.T : a.T * a.K;
    const int row0 = ctl->row0[u.group] - (sh || !shared ? 0 : a.T);
    const uint32_t mask = ctl->mask[u.group];
    const int i = u.tile * 128 + r;
    uint8_t* base = (uint8_t*)(sh ? a.h_s : a.h);
    if constexpr (FMT == 0) {
        int c = 0;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (!(mask >> t & 1u)) continue;
            if (i < I) {
                bf16* hp = reinterpret_cast<bf16*>(base) + (int64_t)(row0 + c) * I + i;
                const bf16 hi = __float2bfloat16_rn(h[t]);
                hp[0] = hi;
                hp[(int64_t)rows * I] = __float2bfloat16_rn(h[t] - __bfloat162float(hi));
            }
            ++c;
        }
    } else {
        // a scale per token and 128 values: the largest magnitude over the four warps
        const int warp = r >> 5;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (!(mask >> t & 1u)) continue;
            float m = fabsf(h[t]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if ((r & 31) == 0) ctl->top[warp][t] = m;
        }
        drain_sync();
        float* hs = sh ? a.hs_s : a.hs;
        int c = 0;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (!(mask >> t & 1u)) continue;
            const float m = fmaxf(fmaxf(ctl->top[0][t], ctl->top[1][t]),
                                  fmaxf(ctl->top[2][t], ctl->top[3][t]));
            float s, inv;
            plane_scale(m, s, inv);
            if (r == 0) hs[(int64_t)(row0 + c) * (I / 128) + u.tile] = s;
            uint8_t* hp = base + (int64_t)(row0 + c) * I + i;
            float q = h[t] * inv;
#pragma unroll
            for (int p = 0; p < C::kHPlanes; ++p) {
                const uint8_t code = to_code(q);
                hp[(int64_t)p * rows * I] = code;
                q = (q - of_code(code)) * 16.0f;
            }
            ++c;
        }
    }
    // the copies that read h are of the asynchronous proxy
    fence_proxy_async_all();
    __threadfence();
    drain_sync();
    if (r == 0) {
        __threadfence();
        atomicAdd(a.ready + u.group, 1);
    }
}

template <int FMT, int NT>
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
            ptx::mbar_init(&ctl->qempty[i], 6);
        }
        ctl->abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(&ctl->tmem, 512);
        ptx::tmem_relinquish();
    }
    if (warp == 2 && lane < 9) ptx::prefetch_tmap(&a.maps[lane]);
    pdl_wait();
    pdl_trigger();
    choose(a, ctl, reinterpret_cast<float*>(ring));
    // the ring held keys: order them before the copies that overwrite them
    ptx::fence_proxy_async_smem();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = ctl->tmem;
    const Sched sc = make_sched(a, ctl->groups, C::kElems, gridDim.x);

    if (warp == 0) {
        // -------------------------------------------------- units and their weights
        if (lane == 0 && !a.test_stall) {
            int stage = 0, slot = 0;
            uint32_t phase = 0, qphase = 0;
            bool ok = true;
            int next = atomicAdd(a.claim, 1);
            while (ok) {
                const int u = next < sc.u4 ? next : -1;
                if (!wait_bounded(&ctl->qempty[slot], qphase ^ 1u, ctl, a, 10)) break;
                ctl->queue[slot] = u;
                ptx::mbar_arrive(&ctl->qfull[slot]);
                if (++slot == kQueue) { slot = 0; qphase ^= 1u; }
                if (u < 0) break;
                next = atomicAdd(a.claim, 1);  // answered while this unit's copies go out
                const Unit un = unit_at(sc, u, shared);
                const bool sh = un.group < shared;
                const int e = sh ? 0 : ctl->expert[un.group], row = un.tile * 128;
                for (int i = 0; i < un.ns; ++i) {
                    if (!wait_bounded(&ctl->empty[stage], phase ^ 1u, ctl, a, 11)) { ok = false; break; }
                    uint8_t* dst = ring + stage * C::kStage;
                    if (!un.down) {
                        const int k = (un.s0 + i) * C::kElems;
                        ptx::mbar_arrive_expect_tx(&ctl->full[stage], kABytes);
                        tma_load_3d(dst, &a.maps[sh ? kMapSGate : kMapGate], &ctl->full[stage], k, row, e);
                        tma_load_3d(dst + kABytes / 2, &a.maps[sh ? kMapSUp : kMapUp],
                                    &ctl->full[stage], k, row, e);
                    } else {
                        const int nt = tiles_of_stage<FMT>(a, un, shared, i);
                        const int k = 2 * (un.s0 + i) * C::kElems;
                        ptx::mbar_arrive_expect_tx(&ctl->full[stage], nt * (kABytes / 2));
                        for (int q = 0; q < nt; ++q)
                            tma_load_3d(dst + q * (kABytes / 2), &a.maps[sh ? kMapSDown : kMapDown],
                                        &ctl->full[stage], k + q * C::kElems, row, e);
                    }
                    if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
                }
            }
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
                const Unit un = unit_at(sc, u, shared);
                const bool sh = un.group < shared;
                const int tokens = __popc((uint32_t)ctl->mask[un.group]);
                const int w = NT == 8 || tokens <= 8 ? 8 : 16;
                const int rows = sh ? a.T : a.T * a.K;
                const int row0 = ctl->row0[un.group] - (sh || !shared ? 0 : a.T);
                if (un.down) {
                    // the group's h: finished tiles are counted by whoever finishes them
                    const int tiles = sh ? sc.tiles_s : sc.tiles_r;
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
                    fence_proxy_async_all();
                }
                for (int i = 0; i < un.ns; ++i) {
                    if (!wait_bounded(&ctl->empty[stage], phase ^ 1u, ctl, a, 22)) { ok = false; break; }
                    uint8_t* dst = ring + stage * C::kStage + kABytes;
                    uint64_t* bar = &ctl->full[stage];
                    if (!un.down) {
                        const int k = (un.s0 + i) * C::kElems;
                        ptx::mbar_arrive_expect_tx(bar, C::kXBytes);
                        ptx::tma_load_2d(dst, &a.maps[kMapX], bar, k, 0);
                        if (FMT) ptx::tma_load_2d(dst + NT * 128, &a.maps[kMapX], bar, k, a.T);
                    } else {
                        const int nt = tiles_of_stage<FMT>(a, un, shared, i);
                        const CUtensorMap* map = &a.maps[sh ? kMapHS : kMapH];
                        ptx::mbar_arrive_expect_tx(bar, nt * C::kHPlanes * w * 128);
                        for (int q = 0; q < nt; ++q)
                            for (int p = 0; p < C::kHPlanes; ++p)
                                for (int b = 0; b < w; b += 8)
                                    ptx::tma_load_2d(dst + q * C::kHTile + (p * w + b) * 128, map, bar,
                                                     (2 * (un.s0 + i) + q) * C::kElems,
                                                     p * rows + row0 + b);
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
                const Unit un = unit_at(sc, u, shared);
                const int w = NT == 8 || __popc((uint32_t)ctl->mask[un.group]) <= 8 ? 8 : 16;
                const int n = un.down ? C::kHCols * w : (FMT ? 2 * NT : 16);
                const uint32_t idesc = FMT ? ptx::idesc_e4m3_f32(128, n) : ptx::idesc_bf16_f32(128, n);
                // accumulators emptied every stage where the scales change along K
                const bool each = un.down ? FMT != 0 : FMT == 2;
                for (int i = 0; i < un.ns; ++i) {
                    if (each || i == 0) {
                        if (!wait_bounded(&ctl->tempty[buf], bphase ^ 1u, ctl, a, 31)) { ok = false; break; }
                    }
                    if (!wait_bounded(&ctl->full[stage], phase, ctl, a, 32)) { ok = false; break; }
                    ptx::tc_fence_after();
                    const uint32_t w0 = ptx::smem_u32(ring + stage * C::kStage);
                    const uint32_t b0 = w0 + kABytes;
                    const uint32_t d0 = tmem + buf * 128;
                    const int nt = un.down ? tiles_of_stage<FMT>(a, un, shared, i) : 2;
                    for (int q = 0; q < nt; ++q) {
                        // gate and up rows: two accumulators over the same x; down rows: two K
                        // tiles, into one accumulator or (8-bit h, scaled per 128) two
                        const uint32_t acc = q && (!un.down || FMT) ? d0 + kAcc1 : d0;
                        const uint32_t bq = un.down ? b0 + q * C::kHTile : b0;
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            const uint64_t wd = ptx::sw128_kmajor_desc(w0 + q * (kABytes / 2) + kk * 32);
                            const uint64_t bd = ptx::sw128_kmajor_desc(bq + kk * 32);
                            const bool fresh = kk == 0 && (each || i == 0) &&
                                               !(q && un.down && FMT == 0);
                            if constexpr (FMT) ptx::tc_mma_f8(acc, wd, bd, idesc, fresh ? 0u : 1u);
                            else ptx::tc_mma_f16(acc, wd, bd, idesc, fresh ? 0u : 1u);
                        }
                    }
                    any = true;
                    ptx::tc_commit(&ctl->empty[stage]);
                    if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
                    if (each || i == un.ns - 1) {
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
        // -------------------------------------------------- sums
        const int r = (warp - 4) * 32 + lane;  // weight row of the tile
        const uint32_t lanes = (uint32_t)((warp - 4) * 32) << 16;
        int slot = 0, buf = 0;
        uint32_t qphase = 0, bphase = 0;
        bool ok = true;
        const auto pass = [&](uint64_t* bar, uint32_t parity, int where) {
            const int good = lane == 0 ? (int)wait_bounded(bar, parity, ctl, a, where) : 0;
            // the four warps stop together: they meet at barriers
            return ptx::named_bar_and(1, 128, __shfl_sync(0xffffffffu, good, 0) != 0);
        };
        const auto release = [&](uint64_t* bar) {
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar);
        };
        while (ok) {
            if (!pass(&ctl->qfull[slot], qphase, 40)) break;
            const int uid = ctl->queue[slot];
            release(&ctl->qempty[slot]);
            if (++slot == kQueue) { slot = 0; qphase ^= 1u; }
            if (uid < 0) break;
            const Unit un = unit_at(sc, uid, shared);
            const bool sh = un.group < shared;
            const int e = sh ? 0 : ctl->expert[un.group];
            const uint32_t mask = ctl->mask[un.group];
            const int row0 = ctl->row0[un.group];
            if (!un.down) {
                float sg[NT], su[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t) sg[t] = su[t] = 0.0f;
                const int drains = FMT == 2 ? un.ns : 1;
                const int I = sh ? a.Is : a.I;
                float rg = 1.0f, ru = 1.0f;
                if constexpr (FMT == 1) {
                    const int64_t at = (int64_t)e * I + un.tile * 128 + r;  // I a multiple of 128
                    rg = __ldg((sh ? a.ss_gate : a.s_gate) + at);
                    ru = __ldg((sh ? a.ss_up : a.s_up) + at);
                }
                const int64_t blk = ((int64_t)e * (I / 128) + un.tile) * (a.d / 128) + un.s0;
                for (int k = 0; k < drains; ++k) {
                    if constexpr (FMT == 2) {
                        rg = __ldg((sh ? a.ss_gate : a.s_gate) + blk + k);
                        ru = __ldg((sh ? a.ss_up : a.s_up) + blk + k);
                    }
                    if (!pass(&ctl->tfull[buf], bphase, 41)) { ok = false; break; }
                    ptx::tc_fence_after();
                    const uint32_t at = tmem + lanes + buf * 128;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        float (&s)[NT] = half ? su : sg;
                        const float w = half ? ru : rg;
                        uint32_t v[16], lo[16];
                        ptx::tmem_ld16(at + half * kAcc1, v);
                        if constexpr (FMT && NT == 16) ptx::tmem_ld16(at + half * kAcc1 + 16, lo);
                        ptx::tmem_ld_wait();
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            float x = __uint_as_float(v[t]);
                            if constexpr (FMT)
                                x = fmaf(__uint_as_float(NT == 16 ? lo[t] : v[8 + (t & 7)]), 0.0625f, x);
                            s[t] = FMT == 0 ? x : fmaf(x, w, s[t]);
                        }
                    }
                    ptx::tc_fence_before();
                    release(&ctl->tempty[buf]);
                    if (++buf == kBufs) { buf = 0; bphase ^= 1u; }
                }
                if (!ok) break;
                if constexpr (FMT) {
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const float x = t < a.T ? __ldcg(a.xs + t) : 0.0f;
                        sg[t] *= x;
                        su[t] *= x;
                    }
                }
                if (sc.gp > 1) {
                    // parts of a tile: [row][tile][part][gate 128, up 128]
                    const int tiles = sh ? sc.tiles_s : sc.tiles_r;
                    const int64_t first = sh || !shared
                                              ? (int64_t)row0 * tiles
                                              : (int64_t)a.T * sc.tiles_s + (int64_t)(row0 - a.T) * tiles;
                    float* gp = a.gpart + ((first + un.tile) * a.max_parts) * 256 + r;
                    const int64_t step = (int64_t)tiles * a.max_parts * 256;
                    int c = 0;
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        if (!(mask >> t & 1u)) continue;
                        float* p = gp + c * step + un.part * 256;
                        __stcg(p, sg[t]);
                        __stcg(p + 128, su[t]);
                        ++c;
                    }
                    int* counter = a.gticket + un.group * max(sc.tiles_s, sc.tiles_r) + un.tile;
                    if (!last_part(ctl, counter, sc.gp, r)) continue;
                    c = 0;
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        if (!(mask >> t & 1u)) continue;
                        const float* p = gp + c * step;
                        float g = 0.0f, w = 0.0f;
#pragma unroll 4
                        for (int q = 0; q < sc.gp; ++q) {
                            g += __ldcg(p + q * 256);
                            w += __ldcg(p + q * 256 + 128);
                        }
                        sg[t] = g;
                        su[t] = w;
                        ++c;
                    }
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) sg[t] = silu_mul(sg[t], su[t]);
                store_h<FMT, NT>(a, sc, ctl, un, sg, r, shared);
            } else {
                const int tokens = __popc(mask);
                const int w = NT == 8 || tokens <= 8 ? 8 : 16;
                const int I = sh ? a.Is : a.I;
                const int hrow0 = row0 - (sh || !shared ? 0 : a.T);
                float s[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t) s[t] = 0.0f;
                const int drains = FMT ? un.ns : 1;
                for (int k = 0; k < drains; ++k) {
                    if (!pass(&ctl->tfull[buf], bphase, 42)) { ok = false; break; }
                    ptx::tc_fence_after();
                    if constexpr (FMT) {
                        if (k == 0) {
                            // h's scales of the unit, [K tile][token]; visible once a product of
                            // the unit is: its rows were loaded after the group's h was done
                            const int k0 = 2 * un.s0, nk = min(2 * un.ns, I / 128 - k0);
                            const float* hs = sh ? a.hs_s : a.hs;
                            for (int i = r; i < nk * tokens; i += 128) {
                                const int c = i % tokens, q = i / tokens;
                                ctl->hscale[q * NT + c] =
                                    __ldcg(hs + (int64_t)(hrow0 + c) * (I / 128) + k0 + q);
                            }
                            if constexpr (FMT == 2) {
                                const float* ws = (sh ? a.ss_down : a.s_down) +
                                                  ((int64_t)e * (a.d / 128) + un.tile) * (I / 128) + k0;
                                for (int i = r; i < nk; i += 128) ctl->wscale[0][i] = __ldg(ws + i);
                            }
                            drain_sync();
                        }
                    }
                    const uint32_t at = tmem + lanes + buf * 128;
                    const int nq = FMT ? tiles_of_stage<FMT>(a, un, shared, k) : 1;
                    for (int q = 0; q < nq; ++q) {
                        float v[NT];
#pragma unroll
                        for (int t = 0; t < NT; ++t) v[t] = 0.0f;
                        if (w == 8) {
                            uint32_t p01[16], p23[16];
                            ptx::tmem_ld16(at + q * kAcc1, p01);
                            if constexpr (FMT) ptx::tmem_ld16(at + q * kAcc1 + 16, p23);
                            ptx::tmem_ld_wait();
#pragma unroll
                            for (int t = 0; t < 8; ++t) {
                                const float hi = __uint_as_float(p01[t]), lo = __uint_as_float(p01[8 + t]);
                                if constexpr (FMT)
                                    v[t] = fmaf(fmaf(__uint_as_float(p23[t]), 0.0625f, lo), 0.0625f, hi);
                                else v[t] = hi + lo;
                            }
                        } else if constexpr (NT == 16) {
                            uint32_t p0[16], p1[16], p2[16];
                            ptx::tmem_ld16(at + q * kAcc1, p0);
                            ptx::tmem_ld16(at + q * kAcc1 + 16, p1);
                            if constexpr (FMT) ptx::tmem_ld16(at + q * kAcc1 + 32, p2);
                            ptx::tmem_ld_wait();
#pragma unroll
                            for (int t = 0; t < 16; ++t) {
                                const float hi = __uint_as_float(p0[t]), lo = __uint_as_float(p1[t]);
                                if constexpr (FMT)
                                    v[t] = fmaf(fmaf(__uint_as_float(p2[t]), 0.0625f, lo), 0.0625f, hi);
                                else v[t] = hi + lo;
                            }
                        }
                        const float wsc = FMT == 2 ? ctl->wscale[0][2 * k + q] : 1.0f;
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            if constexpr (FMT) {
                                if (t < tokens)
                                    s[t] = fmaf(v[t], ctl->hscale[(2 * k + q) * NT + t] * wsc, s[t]);
                            } else {
                                s[t] += v[t];
                            }
                        }
                    }
                    ptx::tc_fence_before();
                    release(&ctl->tempty[buf]);
                    if (++buf == kBufs) { buf = 0; bphase ^= 1u; }
                }
                if (!ok) break;
                const int col = un.tile * 128 + r;
                float rs = 1.0f;
                if constexpr (FMT == 1)
                    rs = __ldg((sh ? a.ss_down : a.s_down) + (int64_t)e * a.d + col);  // d a multiple of 128
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    if (t < tokens && col < a.d)
                        __stcg(a.yp + ((int64_t)(row0 + t) * a.max_parts + un.part) * a.d + col, s[t] * rs);
                const int parts = (shared ? sc.dps : 0) + (ctl->groups - shared) * sc.dpr;
                if (last_part(ctl, a.dticket + un.tile, parts, r))
                    join_tile(a, sc, ctl, un.tile, warp - 4, lane);
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
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ host side
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// [n][rows][cols] matrices of `size`-byte elements, box = 128 bytes x box_rows rows of one;
// rank 2 for n = 0 ([rows][cols]).
bool make_map(CUtensorMap* m, const void* base, int64_t n, int64_t rows, int64_t cols, int size,
              int box_rows) {
    const EncodeTiledFn fn = (EncodeTiledFn)tensor_map_encoder();
    if (!fn) return false;
    const cuuint32_t rank = n ? 3 : 2;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)n};
    const cuuint64_t strides[2] = {(cuuint64_t)(cols * size), (cuuint64_t)(rows * cols * size)};
    const cuuint32_t box[3] = {(cuuint32_t)(128 / size), (cuuint32_t)box_rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, size == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, rank,
              const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int FMT, int NT>
cudaError_t go(const FewArgs& a, cudaStream_t st) {
    using C = Cfg<FMT, NT>;
    constexpr size_t smem = 1024 + (size_t)C::kStages * C::kStage + sizeof(Ctl);
    static_assert(smem <= 232448, "shared memory exceeds the per-block limit");
    static_assert(sizeof(float) * kMaxT * 1024 <= (size_t)C::kStages * C::kStage, "keys fit the ring");
    cudaError_t e = cudaFuncSetAttribute(few_experts_kernel<FMT, NT>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(few_experts_kernel<FMT, NT>, dim3(device_sm_count()), dim3(kThreads), smem, st, a);
}

int score_splits(int d) {
    const int n = d / 8 / 96;  // about three 16-byte vectors a lane
    return n < 1 ? 1 : n > kScoreSplits ? kScoreSplits : n;
}

}  // namespace

FewWs few_ws(const moe_shape& s, int fmt) {
    // fmt 0 bf16 (h as two bf16 planes), else 8-bit (x as two planes, h as three, scales)
    FewWs w{};
    const int64_t T = s.T, K = s.K, d = s.d, I = s.inter, Is = s.inter_shared, n = T * K;
    const int64_t groups = (n < s.E ? n : s.E) + 1;
    const int64_t ti = ceil_div(I, 128), ts = ceil_div(Is, 128), td = ceil_div(d, 128);
    w.splits = score_splits(s.d);
    w.max_parts = T <= 4 ? 16 : 8;
    size_t o = 256;  // the error record, then the counters
    auto take = [&](int64_t bytes) {
        const size_t at = o;
        o = (o + (size_t)bytes + 255) / 256 * 256;
        return at;
    };
    w.counters = (int)(1 + groups + td + groups * (ti > ts ? ti : ts));
    w.claim = take(4 * (int64_t)w.counters);
    w.part = take(4 * (int64_t)w.splits * T * s.E);
    w.xq = take(fmt ? 2 * T * d : 0);
    w.xs = take(fmt ? 4 * T : 0);
    w.gpart = take(4 * (n * ti + T * ts) * w.max_parts * 256);
    w.h = take(fmt ? 3 * n * I : 4 * n * I);
    w.h_s = take(fmt ? 3 * T * Is : 4 * T * Is);
    w.hs = take(fmt ? 4 * n * ti : 0);
    w.hs_s = take(fmt ? 4 * T * ts : 0);
    w.yp = take(4 * (n + (Is ? T : 0)) * w.max_parts * d);
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
    a.max_parts = w.max_parts;
    a.bias = c.bias;
    a.residual = (const bf16*)c.residual;
    a.y = (bf16*)c.y;
    a.err = reinterpret_cast<DevError*>(base);
    a.claim = reinterpret_cast<int*>(base + w.claim);
    const int64_t groups = (n < E ? n : E) + 1;
    a.ready = a.claim + 1;
    a.dticket = a.ready + groups;
    a.gticket = a.dticket + ceil_div(d, 128);
    a.part = reinterpret_cast<float*>(base + w.part);
    a.xs = reinterpret_cast<float*>(base + w.xs);
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
    bool ok = make_map(&a.maps[kMapGate], c.w_gate, E, I, d, size, 128) &&
              make_map(&a.maps[kMapUp], c.w_up, E, I, d, size, 128) &&
              make_map(&a.maps[kMapDown], c.w_down, E, d, I, size, 128) &&
              make_map(&a.maps[kMapH], a.h, 0, (fmt ? 3 : 2) * n, I, size, 8) &&
              (fmt ? make_map(&a.maps[kMapX], base + w.xq, 0, 2 * T, d, 1, nt)
                   : make_map(&a.maps[kMapX], c.x, 0, T, d, 2, 16));
    if (Is > 0) {
        ok = ok && make_map(&a.maps[kMapSGate], c.ws_gate, 1, Is, d, size, 128) &&
             make_map(&a.maps[kMapSUp], c.ws_up, 1, Is, d, size, 128) &&
             make_map(&a.maps[kMapSDown], c.ws_down, 1, d, Is, size, 128) &&
             make_map(&a.maps[kMapHS], a.h_s, 0, (fmt ? 3 : 2) * T, Is, size, 8);
    } else {
        // never loaded from: any valid map
        a.maps[kMapSGate] = a.maps[kMapSUp] = a.maps[kMapGate];
        a.maps[kMapSDown] = a.maps[kMapDown];
        a.maps[kMapHS] = a.maps[kMapH];
    }
    if (!ok) return cudaErrorInvalidValue;

    const int tt = T <= 1 ? 1 : T <= 2 ? 2 : T <= 4 ? 4 : 8;
    const int units = (int)ceil_div(T, tt) * s.E * w.splits;
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
    if (fmt == 0) return nt == 8 ? go<0, 8>(a, st) : go<0, 16>(a, st);
    if (fmt == 1) return nt == 8 ? go<1, 8>(a, st) : go<1, 16>(a, st);
    return nt == 8 ? go<2, 8>(a, st) : go<2, 16>(a, st);
}

}  // namespace moe
