// balance.cu -- the router's balance loss with its per-expert counts, and the
// backward pass of the routing.
//
// For the G sequences packed in a batch, over the n_g tokens of sequence g that
// are not masked, with p_te the router's probabilities over all experts
// (softmax of the scores, or sigmoid / sum of sigmoids) and c_ge the number of
// times expert e was picked:
//
//   P_ge = mean_t p_te,   f_ge = E c_ge / (K n_g),
//   loss = alpha / G * sum_g sum_e f_ge P_ge.
//
// Gradient (the counts are constants): a_ge = alpha E c_ge / (G K n_g^2),
//   softmax  dz_te = p_te (a_ge - sum_i p_ti a_gi)
//   sigmoid  dz_te = p_te (1 - sigmoid(z_te)) (a_ge - sum_i p_ti a_gi)
// and the routing weights' part, at the K picked experts:
//   softmax  dz_k = w_k (dw_k - sum_j w_j dw_j)
//   sigmoid  dz_k = a_k (1 - a_k) (dw_k - sum_j w_j dw_j) / (sum_j a_j + 1e-6)
// ("Sparse MoE inference kernels ..." (blog.llmgo.top), section 2.1, names the
// f_i P_i loss; its formula is lost there.)
//
// Both passes are one read of the scores, and the backward pass one write of
// their gradient.  A row of E scores lives in the registers of a group of
// lanes; sums over tokens go lane -> warp -> block in a fixed order, one
// partial row per (block, sequence), and a second small kernel adds the
// partials of each sequence: no floating-point atomics, the same bits each run.
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr float kTinySum = 1e-18f;
constexpr int kStages = 2;  // tiles a warp holds: one at hand, one on its way

// ---- two fp32 values in a 64-bit register: one instruction works on both -----
typedef uint64_t f2;
__device__ __forceinline__ f2 pack2(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ f2 both(float v) { return pack2(v, v); }
__device__ __forceinline__ void unpack2(f2 v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rcp(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// maximum and minimum that are NaN where either value is: a clamp must not turn a score
// that is not a number into one (the same single instruction as without NaN)
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// e^x of two values whose exponentials stay finite (and |x| < 2e38).  t = x
// log2(e) is rounded for the hardware's 2^t; what that took off, d = x - t ln 2
// (ln 2 in two parts: Cody and Waite, "Software Manual for the Elementary Functions",
// 1980), comes back as a factor e^d = 1 + d, so the error stays at
// the hardware's two steps for large |x| too.  Below -87.3 it is 0.
__device__ __forceinline__ f2 exp2x(f2 x) {
    const f2 nt = mul2(x, both(-1.44269504f));  // -t
    const f2 d = fma2(nt, both(-1.90465421e-9f), fma2(nt, both(0.693147182f), x));
    float t0, t1;
    unpack2(nt, t0, t1);
    const f2 y = pack2(ex2(-t0), ex2(-t1));
    return fma2(y, d, y);
}
__device__ __forceinline__ float exp1(float x) {
    float lo, hi;
    unpack2(exp2x(both(x)), lo, hi);
    return lo;
}

constexpr float kFar = 1000.f;     // e^-kFar is 0
constexpr float kOver = 88.7f;     // e^kOver is finite, and 1 / e^kOver rounds to 0

// sigmoid(z) and 1 - sigmoid(z), each with its own relative accuracy (one
// minus the other would lose the small one).  Below z = -87.3, where
// the sigmoid is under fp32's normal range, a is 0 and b unspecified.
__device__ __forceinline__ void sigmoid2(f2 z, f2& a, f2& b) {
    float z0, z1;
    unpack2(z, z0, z1);
    const f2 e = exp2x(pack2(min_nan(-z0, kOver), min_nan(-z1, kOver)));
    float d0, d1;
    unpack2(add2(e, both(1.f)), d0, d1);
    a = pack2(rcp(d0), rcp(d1));
    b = mul2(e, a);
}

// How a row of E scores lies over the lanes of a warp: `kGroup` lanes hold it
// (32 / kGroup rows a warp), kN scores a lane in vectors of kVec, vector i of
// lane l starting at column (i * kGroup + l) * kVec.  In registers a lane's
// scores are kP pairs.  Few lanes with many scores each: a row's sums then take
// few shuffles, and what a row costs beside its scores is shared by 32 / kGroup.
template <int VEC, int N, int G>
struct RowLayout {
    static constexpr int kVec = VEC, kN = N, kGroup = G, kRows = 32 / G, kP = N / 2;
    // A warp's tile (1 to 4 KB): kU rows for each group of lanes.
    static constexpr int kU = N <= 16 ? 2 : 1;
    static constexpr int kTokens = kU * kRows;
    // Rows of a lane group worked on at once: their chains hide each other's latency.
    static constexpr int kV = N <= 8 ? 2 : 1;
    // column of value j of lane l
    __device__ static int col(int j, int l) { return (j / VEC * G + l) * VEC + j % VEC; }
};

// sums and maxima over the lanes of a group, of V rows side by side
template <int G, int V>
__device__ __forceinline__ void group_sum(float (&v)[V]) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}
template <int G, int V>
__device__ __forceinline__ void group_max(float (&v)[V]) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = fmaxf(v[i], __shfl_xor_sync(0xffffffffu, v[i], o));
}

template <int P>
__device__ __forceinline__ float pair_sum(const f2 (&v)[P]) {
    f2 s = v[0];
#pragma unroll
    for (int i = 1; i < P; ++i) s = add2(s, v[i]);
    float lo, hi;
    unpack2(s, lo, hi);
    return lo + hi;
}
template <int P>
__device__ __forceinline__ float pair_max(const f2 (&v)[P]) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        float lo, hi;
        unpack2(v[i], lo, hi);
        m = fmaxf(m, fmaxf(lo, hi));
    }
    return m;
}

// a lane's columns of a row in shared memory; `none` beyond E and where !live
template <typename L>
__device__ __forceinline__ void load_row(const float* row, int E, int l, bool live,
                                         f2 (&z)[L::kP], float none = -INFINITY) {
    if constexpr (L::kVec == 4) {
#pragma unroll
        for (int i = 0; i < L::kN / 4; ++i) {
            const int c = L::col(4 * i, l);
            float4 q = make_float4(none, none, none, none);
            if (live && c < E) q = *reinterpret_cast<const float4*>(row + c);
            z[2 * i] = pack2(q.x, q.y);
            z[2 * i + 1] = pack2(q.z, q.w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < L::kP; ++i) {
            const int c0 = L::col(2 * i, l), c1 = L::col(2 * i + 1, l);
            z[i] = pack2(live && c0 < E ? row[c0] : none, live && c1 < E ? row[c1] : none);
        }
    }
}

// ---- a warp's ring of tiles in shared memory --------------------------------
// Asynchronous copy of the n floats at src + at to dst, by the lanes, as one
// group.  16 bytes at a time: dst takes the place of the multiple of four floats at
// or before src + at (which rows that are whole vectors always start at), and what
// is left behind the last whole vector goes float by float.
template <typename L>
__device__ __forceinline__ void copy_tile(float* dst, const float* src, int64_t at, int n,
                                          int lane) {
    const int head = L::kVec == 4 ? 0 : (int)(at & 3);
    const char* g = reinterpret_cast<const char*>(src + at - head);
    const uint32_t d = ptx::smem_u32(dst);
    const int whole = n > 0 ? (head + n) / 4 : 0;
    auto copy = [&](int i) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d + i * 16), "l"(g + i * 16)
                     : "memory");
    };
    int i = lane;
    for (; i + 96 < whole; i += 128) {
#pragma unroll
        for (int k = 0; k < 4; ++k) copy(i + 32 * k);
    }
#pragma unroll
    for (int k = 0; k < 3; ++k)
        if (i + 32 * k < whole) copy(i + 32 * k);
    if constexpr (L::kVec != 4) {
        const int f = whole * 4 + lane;
        if (n > 0 && f < head + n)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(d + f * 4), "l"(g + f * 4)
                         : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}

// n floats of a tile to dst + at, by the lanes; src is as far from a multiple of 16
// bytes as dst + at is
template <typename L>
__device__ __forceinline__ void store_tile(float* dst, const float* src, int64_t at, int n,
                                           int lane) {
    float* out = dst + at;
    if constexpr (L::kVec != 4) {
        const int head = min(n, (int)(-at & 3));
        if (lane < head) out[lane] = src[lane];
        out += head;
        src += head;
        n -= head;
        const int tail = n & 3;
        if (lane < tail) out[n - tail + lane] = src[n - tail + lane];
    }
    float4* d = reinterpret_cast<float4*>(out) + lane;
    const float4* q = reinterpret_cast<const float4*>(src) + lane;
    int left = n / 4 - lane;
    for (; left > 96; left -= 128, d += 128, q += 128) {
        float4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = q[i * 32];
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i * 32] = v[i];
    }
#pragma unroll
    for (int i = 0; i < 3; ++i)
        if (left > i * 32) d[i * 32] = q[i * 32];
}

// floats of a tile's place in shared memory: its rows, and what lies beside them in
// the vectors of its first and last float
template <typename L>
__host__ __device__ __forceinline__ int tile_floats(int E) {
    return L::kVec == 4 ? L::kTokens * E : (L::kTokens * E + 6) / 4 * 4;
}

// Tile i of a warp holds tokens first + i * stride .. + kTokens - 1, up to
// `last`.  (Tokens are unsigned 32-bit: one past a tile may pass 2^31.)
template <typename L>
struct Ring {
    const float* src;  // the scores, [T][E]
    float* buf;        // kStages places of tile_floats
    uint32_t first, stride, last;
    int E, lane;
    int cur;  // the tile at hand (-1: none yet)

    __device__ __forceinline__ float* slot(int i) const {
        return buf + (i & (kStages - 1)) * tile_floats<L>(E);
    }
    __device__ __forceinline__ void issue(int i) {
        const uint32_t tok = first + i * stride;
        const int n = tok >= last ? 0 : min(last - tok, (uint32_t)L::kTokens);
        copy_tile<L>(slot(i), src, (int64_t)tok * E, n * E, lane);
    }
    __device__ __forceinline__ void start() {
        cur = -1;
#pragma unroll
        for (int i = 0; i < kStages; ++i) issue(i);
    }
    // moves on to tile i >= cur (the warp has done with those before it)
    __device__ __forceinline__ float* get(int i) {
        while (cur < i) {
            if (cur >= 0) {
                __syncwarp();
                issue(cur + kStages);
            }
            ++cur;
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
            __syncwarp();
        }
        return slot(i) + (L::kVec == 4 ? 0 : (int)((int64_t)(first + i * stride) * E & 3));
    }
};

// e^(z - m) of a row in place (m finite), and the sum of a lane's values
template <int P>
__device__ __forceinline__ float exp_row(f2 (&z)[P], float m) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
        float lo, hi;
        unpack2(add2(z[i], both(-m)), lo, hi);
        z[i] = exp2x(pack2(max_nan(lo, -kFar), max_nan(hi, -kFar)));
    }
    return pair_sum(z);
}

// The router's probabilities of V rows, row(v) in shared memory (of none where
// !live[v]), are z times inv; for the sigmoid router s = 1 - sigmoid, the backward
// pass's factor.  Experts with a score of -inf get 0, and a row of them gets all
// zeros; a row with a NaN or +inf gets NaN, by its sum.
template <typename L, bool SIG, int V, typename R>
__device__ __forceinline__ void row_probs(f2 (&z)[V][L::kP], f2 (&s)[V][L::kP], float (&inv)[V],
                                          R&& row, int E, int l, const bool (&live)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) load_row<L>(row(v), E, l, live[v], z[v]);
    if constexpr (SIG) {
        // A row whose sigmoids sum to less than kTinySum has every score below
        // -41, where sigmoid(z) is e^z to fp32's last bit and its share of the
        // sum is the same for scores moved up together: such rows go round once
        // more with their largest score at -18, so that neither they underflow as
        // a whole nor 1 / sum, or its square, overflows.
        for (bool again = false;; again = true) {
            bool tiny = false;
#pragma unroll
            for (int v = 0; v < V; ++v) {
#pragma unroll
                for (int i = 0; i < L::kP; ++i) sigmoid2(z[v][i], z[v][i], s[v][i]);
                inv[v] = pair_sum(z[v]);
            }
            group_sum<L::kGroup>(inv);
#pragma unroll
            for (int v = 0; v < V; ++v) tiny |= live[v] && inv[v] < kTinySum;
            if (again || !__any_sync(0xffffffffu, tiny)) break;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                load_row<L>(row(v), E, l, live[v], z[v]);
                float m[1] = {pair_max(z[v])};
                group_max<L::kGroup>(m);
                const f2 up = both(inv[v] < kTinySum && m[0] != -INFINITY ? -18.f - m[0] : 0.f);
#pragma unroll
                for (int i = 0; i < L::kP; ++i) z[v][i] = add2(z[v][i], up);
            }
        }
    } else {
        float m[V];
#pragma unroll
        for (int v = 0; v < V; ++v) m[v] = pair_max(z[v]);
        group_max<L::kGroup>(m);
#pragma unroll
        for (int v = 0; v < V; ++v) inv[v] = exp_row(z[v], m[v] == -INFINITY ? 0.f : m[v]);
        group_sum<L::kGroup>(inv);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) inv[v] = inv[v] == 0.f ? 0.f : rcp(inv[v]);
}

// Which of a tile's tokens take part: a bit a token, the mask's bytes asked for a
// tile ahead.
template <typename L>
struct LiveBits {
    using Bits = typename std::conditional<(L::kTokens > 32), uint64_t, uint32_t>::type;
    static constexpr int kWords = (L::kTokens + 31) / 32;
    const uint8_t* mask;
    uint32_t last, at;
    uint8_t held[kWords];

    // asks for the bytes of the tile at token `base`
    __device__ __forceinline__ void ask(uint32_t base) {
        at = base;
        if (mask == nullptr) return;
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
            const uint32_t tok = base + w * 32 + (threadIdx.x & 31);
            held[w] = tok < last ? mask[tok] : 0;
        }
    }
    // the tokens [from, to) of the tile at `base` that are not masked
    __device__ __forceinline__ Bits get(uint32_t base, uint32_t from, uint32_t to) {
        Bits b = (Bits)~(Bits)0;
        if (mask != nullptr) {
            if (at != base) ask(base);
            b = 0;
#pragma unroll
            for (int w = 0; w < kWords; ++w)
                b |= (Bits)__ballot_sync(0xffffffffu, held[w] != 0) << (w * 32 % (sizeof(Bits) * 8));
        }
        constexpr int kBits = sizeof(Bits) * 8;
        b &= (Bits)~(Bits)0 << (from - base);
        return b & (Bits)~(Bits)0 >> (kBits - (to - base));
    }
};

// Finds the sequence of a token.  A warp holds a window of kHeld * 32 of the n + 1
// offsets in its registers; all of them, if there are no more, asked for before
// anything else is (behind a block's first copies they would wait as long as
// those).  A token outside the window is searched for in memory, 32 ways at a time,
// and the window moved there.
constexpr int kHeld = 8;
struct SeqFinder {
    const int32_t* cu;
    int n, T;
    int base;  // offset of the window's first
    int32_t held[kHeld];

    __device__ __forceinline__ SeqFinder(const int32_t* __restrict__ cu_, int n_, int T_)
        : cu(cu_), n(n_), T(T_) {
        if (cu != nullptr && n < kHeld * 32) hold(0);
        else base = -1;
    }
    __device__ __forceinline__ void hold(int first) {
        base = first;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int k = first + i * 32 + (int)(threadIdx.x & 31);
            held[i] = k <= n ? cu[k] : 0x7fffffff;
        }
    }
    // The sequence of `token` (-1: none, before the first or after the last), and
    // in `end` the token up to which the answer holds.  Whatever the offsets are,
    // end > token and the answer is below n.
    __device__ __forceinline__ int find(uint32_t token, uint32_t& end) {
        end = T;
        if (cu == nullptr) return 0;
        const int lane = threadIdx.x & 31, t = (int)token;
        for (bool moved = false;; moved = true) {
            if (base >= 0) {
                int before = 0, next = 0x7fffffff;
#pragma unroll
                for (int i = 0; i < kHeld; ++i) {
                    before += held[i] <= t;
                    if (held[i] > t) next = min(next, held[i]);
                }
                before = __reduce_add_sync(0xffffffffu, before);
                next = __reduce_min_sync(0xffffffffu, next);
                // inside the window: an offset on either side, or none there is
                if (moved || ((before > 0 || base == 0) &&
                              (next != 0x7fffffff || base + kHeld * 32 > n))) {
                    if (base + before > n) return -1;
                    end = min(next, T);
                    return base + before - 1;
                }
            }
            int lo = 0, hi = n + 1;  // cu[lo - 1] <= t < cu[hi], where those exist
            while (lo < hi) {
                const int step = (hi - lo + 31) / 32;
                const int i = lo + lane * step;
                const int c = __ffs(~__ballot_sync(0xffffffffu, i < hi && cu[i] <= t)) - 1;
                const int k = c < 0 ? 32 : c;  // lanes up to the first that says no
                if (k == 0) break;
                const int first = lo;
                lo = first + (k - 1) * step + 1;
                hi = min(hi, first + k * step);
            }
            hold(max(lo - 1, 0));
        }
    }
};

__device__ __forceinline__ bool bad_offset(const BalanceArgs& p, int i) {
    return p.cu[i] < 0 || p.cu[i + 1] < p.cu[i] || p.cu[i + 1] > p.T;
}

// Block b takes `chunk` tokens, its warps the tiles in turn.  For each sequence
// g that the chunk touches it writes partial row b + g (along the batch either b
// or g grows from one such pair to the next, so the rows are its own): the sums
// of the probabilities, the counts, and the number of slots counted.  `solo`: the
// only block has all of every sequence, and writes the results itself.
template <typename L, bool SIG>
__global__ void __launch_bounds__(kThreads, 2)
balance_partial_kernel(BalanceArgs p) {
    extern __shared__ __align__(16) float sm[];  // rings, [kWarps][E] sums, [E] counts
    __shared__ int slots, bad;
    constexpr int V = L::kV;
    constexpr uint32_t kStride = kWarps * L::kTokens;
    const int E = p.E, K = p.K;
    float* sums = sm + kWarps * kStages * tile_floats<L>(E);
    int32_t* hist = reinterpret_cast<int32_t*>(sums + kWarps * E);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int l = lane % L::kGroup, r = lane / L::kGroup;
    const uint32_t t0 = blockIdx.x * (uint32_t)p.chunk, t1 = min(t0 + p.chunk, (uint32_t)p.T);
    const uint32_t w0 = t0 + warp * L::kTokens;  // the warp's first tile
    if (threadIdx.x == 0) bad = 0;
    pdl_wait();
    pdl_trigger();
    SeqFinder seqs(p.cu, p.n_seq, p.T);
    // a lane's first pick of the tile that starts at token `next` (slot numbers
    // stay below 2^31)
    auto pick = [&](uint32_t f) { return f < t1 * K ? p.topk_idx[f] : -1; };
    uint32_t next = w0;
    int e_next = next < t1 ? pick(next * K + lane) : -1;
    LiveBits<L> alive{p.mask, t1, 0, {}};
    alive.ask(w0);
    Ring<L> ring{p.logits, sm + warp * kStages * tile_floats<L>(E), w0, kStride, t1, E, lane, -1};
    ring.start();
    float share = 0.f;  // of the loss (solo)
    if (p.solo) {       // sequences without tokens
        for (int i = threadIdx.x; i < p.n_seq * E; i += kThreads) {
            p.mean_p[i] = 0.f;
            p.counts[i] = 0;
        }
        __syncthreads();
    } else if (blockIdx.x == 0 && threadIdx.x == 0) {
        *p.ticket = 0;  // for the kernel that adds the rows
    }
    for (uint32_t t = t0; t < t1;) {
        uint32_t end;
        const int g = seqs.find(t, end);
        end = min(end, t1);
        if (g >= 0) {
            for (int e = threadIdx.x; e < E; e += kThreads) hist[e] = 0;
            if (threadIdx.x == 0) slots = 0;
            __syncthreads();
            int mine = 0;
            f2 acc[L::kP];
#pragma unroll
            for (int j = 0; j < L::kP; ++j) acc[j] = both(0.f);
            // tiles that reach into [t, end)
            int i = (int)((t - t0) / kStride);
            if (w0 + i * kStride + L::kTokens <= t) ++i;
            for (uint32_t base = w0 + i * kStride; base < end; base += kStride, ++i) {
                const float* tile = ring.get(i);
                const uint32_t from = max(t, base), to = min(end, base + L::kTokens);
                const auto on = alive.get(base, from, to);
                alive.ask(base + kStride);
                const bool whole = to - from == L::kTokens && p.mask == nullptr;
                if (next != base) e_next = pick(base * K + lane);
                const int picks = L::kTokens * K;
                auto count = [&](int j, int e) {
                    if (j >= picks || (!whole && !(on >> j / K & 1))) return;
                    if ((uint32_t)e < (uint32_t)E) {
                        atomicAdd(&hist[e], 1);
                        ++mine;
                    } else {
                        bad = 1;
                    }
                };
                count(lane, e_next);
                // (a token has no more than 32) the rest, four asked for at once
                for (int j = lane + 32; L::kTokens > 1 && j < picks; j += 128) {
                    int e[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        e[q] = j + 32 * q < picks ? pick(base * K + j + 32 * q) : -1;
#pragma unroll
                    for (int q = 0; q < 4; ++q) count(j + 32 * q, e[q]);
                }
                next = base + kStride;
                e_next = next < t1 ? pick(next * K + lane) : -1;
#pragma unroll
                for (int h = 0; h < L::kU; h += V) {
                    if (base + h * L::kRows >= to) break;
                    if (base + (h + V) * L::kRows <= from) continue;
                    bool live[V];
#pragma unroll
                    for (int v = 0; v < V; ++v) live[v] = on >> ((h + v) * L::kRows + r) & 1;
                    f2 z[V][L::kP], s[V][L::kP];
                    float inv[V];
                    auto row = [&](int v) { return tile + ((h + v) * L::kRows + r) * E; };
                    row_probs<L, SIG, V>(z, s, inv, row, E, l, live);
#pragma unroll
                    for (int v = 0; v < V; ++v)
#pragma unroll
                        for (int j = 0; j < L::kP; ++j)
                            acc[j] = fma2(z[v][j], both(inv[v]), acc[j]);
                }
            }
            mine = __reduce_add_sync(0xffffffffu, mine);
            if (lane == 0 && mine) atomicAdd(&slots, mine);
#pragma unroll
            for (int j = 0; j < L::kP; ++j) {
                float q[2];
                unpack2(acc[j], q[0], q[1]);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int o = 16; o >= L::kGroup; o >>= 1)
                        q[h] += __shfl_xor_sync(0xffffffffu, q[h], o);
                    const int c = L::col(2 * j + h, l);
                    if (r == 0 && c < E) sums[warp * E + c] = q[h];
                }
            }
            __syncthreads();
            const int64_t at = p.solo ? (int64_t)g * E : ((int64_t)blockIdx.x + g) * E;
            for (int e = threadIdx.x; e < E; e += kThreads) {
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) v += sums[w * E + e];
                if (p.solo) {
                    v = slots > 0 ? v * (float)K / (float)slots : 0.f;
                    p.mean_p[at + e] = v;
                    p.counts[at + e] = hist[e];
                    if (slots > 0) share += v * ((float)hist[e] * ((float)E / (float)slots));
                } else {
                    p.part_p[at + e] = v;
                    p.part_c[at + e] = hist[e];
                }
            }
            if (threadIdx.x == 0 && !p.solo) p.part_n[blockIdx.x + g] = slots;
            __syncthreads();
        }
        t = end;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!p.solo) {
        if (threadIdx.x == 0) p.part_bad[blockIdx.x] = bad;
        return;
    }
    int wrong = bad;
    if (p.cu)
        for (int i = threadIdx.x; i < p.n_seq; i += kThreads) wrong |= bad_offset(p, i);
    wrong = __syncthreads_or(wrong);
    share = warp_sum(share);
    if (lane == 0) sums[warp] = share;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kWarps; ++w) share += sums[w];
        *p.loss = share * (p.alpha / (float)p.n_seq);
        *p.err = DevError{wrong ? MOE_ERR_BOUNDS : MOE_OK, 0, {0, 0}};
    }
}

// sum of f(a), f(a + 1) .. f(b - 1) over a warp's lanes, in every lane
template <typename V, typename F>
__device__ __forceinline__ V warp_sum_over(int64_t a, int64_t b, F&& f) {
    V v = 0;
#pragma unroll 4
    for (int64_t i = a + (threadIdx.x & 31); i < b; i += 32) v += f(i);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Block (g, y) adds sequence g's partial rows over its slices of 32 columns
// (slices y, y + gridDim.y, ...; a warp every `warps`-th row, then the warps in
// order) and writes the counts, mean probabilities and its share of the loss;
// the last block to finish adds the shares in order.  All terms are positive, so
// fp32 sums in a tree keep the loss to a few 2^-24; sums in fp64 took 30 us of a
// block of 1024 threads.  Block (0, 0)'s second warp looks over the offsets and
// the blocks' findings and writes the error record.
__global__ void __launch_bounds__(1024) balance_final_kernel(BalanceArgs p) {
    extern __shared__ float sp[];  // [warps][32] sums, then counts
    pdl_wait();
    pdl_trigger();
    const int g = blockIdx.x, E = p.E;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int* sc = reinterpret_cast<int*>(sp + warps * 32);
    // its partial rows [b0, b1)
    int t0 = 0, t1 = p.T;
    if (p.cu) {
        t0 = max(p.cu[g], 0);
        t1 = min(p.cu[g + 1], p.T);
    }
    const int64_t b0 = t0 / p.chunk + g, b1 = t1 > t0 ? (t1 - 1) / p.chunk + 1 + g : b0;
    int total = 0;
    float share = 0.f;
    for (int e0 = blockIdx.y * 32; e0 < E; e0 += gridDim.y * 32) {
        const int e = e0 + lane;
        float v = 0.f;
        int k = 0;
        if (e < E) {
#pragma unroll 8
            for (int64_t i = b0 + warp; i < b1; i += warps) {
                v += p.part_p[i * E + e];
                k += p.part_c[i * E + e];
            }
        }
        if (warp == 0 && e0 == (int)blockIdx.y * 32)
            total = warp_sum_over<int>(b0, b1, [&](int64_t i) { return p.part_n[i]; });
        if (warp != 0) {
            sp[warp * 32 + lane] = v;
            sc[warp * 32 + lane] = k;
        }
        __syncthreads();
        if (warp == 0) {
#pragma unroll 4
            for (int w = 1; w < warps; ++w) {
                v += sp[w * 32 + lane];
                k += sc[w * 32 + lane];
            }
            if (e < E) {
                const float m = total > 0 ? v * (float)p.K / (float)total : 0.f;
                p.mean_p[(int64_t)g * E + e] = m;
                p.counts[(int64_t)g * E + e] = k;
                if (total > 0) share += m * ((float)k * ((float)E / (float)total));
            }
        }
        if (e0 + (int)gridDim.y * 32 < E) __syncthreads();
    }
    if (warp == 1 && blockIdx.x == 0 && blockIdx.y == 0) {
        int wrong = warp_sum_over<int>(0, p.blocks, [&](int64_t i) { return p.part_bad[i]; });
        if (p.cu)
            wrong += warp_sum_over<int>(0, p.n_seq,
                                        [&](int64_t i) { return (int)bad_offset(p, (int)i); });
        if (lane == 0) *p.err = DevError{wrong ? MOE_ERR_BOUNDS : MOE_OK, 0, {0, 0}};
    }
    if (warp != 0) return;
    share = warp_sum(share);
    const float scale = p.alpha / (float)p.n_seq;
    const unsigned blocks = gridDim.x * gridDim.y;
    if (blocks == 1) {
        if (lane == 0) *p.loss = share * scale;
        return;
    }
    unsigned done = 0;
    if (lane == 0) {
        p.shares[(int64_t)g * gridDim.y + blockIdx.y] = share;
        // this block's share before the count, all blocks' shares after it
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;"
                     : "=r"(done)
                     : "l"(p.ticket)
                     : "memory");
    }
    if (__shfl_sync(0xffffffffu, done, 0) != blocks - 1u) return;
    __syncwarp();  // the shuffle orders no memory: what lane 0 acquired, for the others too
    const float v =
        warp_sum_over<float>(0, blocks, [&](int64_t i) { return __ldcg(p.shares + i); });
    if (lane == 0) *p.loss = v * scale;
}

// A warp takes `chunk` tokens, tile by tile; the coefficients a_ge of the
// sequence at hand stay in shared memory.  The routing weights' part is computed
// with one lane per pick (32 / pw tokens side by side, pw the power of two that
// holds K) and added to the tile's rows, which the gradient has replaced in
// shared memory, before they are written out.
template <typename L, bool SIG>
__global__ void __launch_bounds__(kThreads, 2)
route_backward_kernel(RouteBackwardArgs p) {
    constexpr int V = L::kV;
    extern __shared__ __align__(16) float sm[];  // rings, [kWarps][E] coefficients
    const int E = p.E, K = p.K;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int l = lane % L::kGroup, r = lane / L::kGroup;
    float* coef = sm + kWarps * kStages * tile_floats<L>(E) + warp * E;
    const uint64_t w0 = ((uint64_t)blockIdx.x * kWarps + warp) * p.chunk;
    pdl_wait();
    pdl_trigger();
    if (w0 >= (uint64_t)p.T) return;
    const uint32_t t0 = (uint32_t)w0, t1 = min(t0 + p.chunk, (uint32_t)p.T);
    // What the first tile needs beside its scores is asked for before the ring's
    // copies: behind those (30 MB over all SMs) each would wait 2 to 5 us.
    SeqFinder seqs(p.cu, p.n_seq, p.T);
    const float up = p.counts ? p.alpha / (float)p.n_seq * (p.d_loss ? *p.d_loss : 1.f) : 0.f;
    // The picks, a lane each: a step takes the picks of `per` tokens.  At hand is
    // step `at` with its scores on their way, behind it the next one's experts.
    const int pw = 1 << p.pw_log, pick = lane & (pw - 1), of = lane >> p.pw_log;
    const int per = min(32 >> p.pw_log, L::kTokens);
    uint32_t at = ~0u;
    int e_at = -1, e_next = -1;
    float dw_at = 0.f, dw_next = 0.f, z_at = 0.f;
    auto load_next = [&](uint32_t step) {
        const uint32_t tok = step + of;
        e_next = -1;
        if (of < per && tok < t1 && pick < K) {
            e_next = p.topk_idx[tok * K + pick];  // T * K < 2^31
            dw_next = p.d_topk_w[tok * K + pick];
        }
    };
    auto move_on = [&](uint32_t step) {  // to `step`, whose experts were asked for
        at = step;
        e_at = (uint32_t)e_next < (uint32_t)E ? e_next : -1;
        dw_at = dw_next;
        z_at = e_at >= 0 ? __ldg(p.logits + (int64_t)(step + of) * E + e_at) : -INFINITY;
        load_next(step + per);
    };
    if (p.d_topk_w) load_next(t0);
    LiveBits<L> alive{p.mask, t1, 0, {}};
    alive.ask(t0);
    // the counts of a sequence, a lane's columns: asked for, and made a_ge
    constexpr int kC = (L::kN * L::kGroup + 31) / 32;
    int32_t c_at[kC];
    auto load_counts = [&](int g) {
#pragma unroll
        for (int i = 0; i < kC; ++i)
            c_at[i] = lane + 32 * i < E ? p.counts[(int64_t)g * E + lane + 32 * i] : 0;
    };
    auto make_coef = [&]() {
        int32_t total = 0;  // at most T * K
#pragma unroll
        for (int i = 0; i < kC; ++i) total += c_at[i];
        total = __reduce_add_sync(0xffffffffu, total);
        // a = alpha E c / (G K n^2) with n = total / K
        const float n = (float)total, k = total > 0 ? up * (float)E / n * ((float)K / n) : 0.f;
#pragma unroll
        for (int i = 0; i < kC; ++i)
            if (lane + 32 * i < E) coef[lane + 32 * i] = (float)c_at[i] * k;
        __syncwarp();
    };
    uint32_t end;
    int g = seqs.find(t0, end);
    if (p.counts && g >= 0) load_counts(g);
    if (p.d_topk_w) move_on(t0);
    // without the balance loss no row is read: the ring's copies are empty
    Ring<L> ring{p.logits, sm + warp * kStages * tile_floats<L>(E), t0, L::kTokens,
                 p.counts ? t1 : t0, E, lane, -1};
    ring.start();
    for (uint32_t t = t0; t < t1;) {
        if (t != t0) {
            g = seqs.find(t, end);
            if (p.counts && g >= 0) load_counts(g);
        }
        end = min(end, t1);
        const bool in_seq = g >= 0;
        if (p.counts && in_seq) make_coef();
        int it = (int)((t - t0) / L::kTokens);
        for (uint32_t base = t0 + it * L::kTokens; base < end; base += L::kTokens, ++it) {
            float* tile = ring.get(it);
            const uint32_t from = max(t, base), to = min(end, base + L::kTokens);
            const bool inside = to - from == L::kTokens;
            auto on = alive.get(base, from, to);
            alive.ask(base + L::kTokens);
            if (!in_seq) on = 0;
#pragma unroll
            for (int h = 0; h < L::kU; h += V) {
                if (base + h * L::kRows >= to) break;
                if (base + (h + V) * L::kRows <= from) continue;
                bool in[V], live[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const uint32_t tok = base + (h + v) * L::kRows + r;
                    in[v] = inside || (tok >= from && tok < to);
                    live[v] = on >> (tok - base) & 1;
                }
                auto row = [&](int v) { return tile + ((h + v) * L::kRows + r) * E; };
                f2 z[V][L::kP], s[V][L::kP];
                if (p.counts && in_seq) {
                    float inv[V], dot[V];
                    row_probs<L, SIG, V>(z, s, inv, row, E, l, live);
                    f2 c[L::kP];
                    load_row<L>(coef, E, l, true, c, 0.f);
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        f2 d = mul2(z[v][0], c[0]);
#pragma unroll
                        for (int j = 1; j < L::kP; ++j) d = fma2(z[v][j], c[j], d);
                        float lo, hi;
                        unpack2(d, lo, hi);
                        dot[v] = lo + hi;
                    }
                    group_sum<L::kGroup>(dot);
                    // p (a - sum p a) = z (inv a - inv^2 sum z a)
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const f2 sub = both(-inv[v] * (inv[v] * dot[v]));
#pragma unroll
                        for (int j = 0; j < L::kP; ++j) {
                            z[v][j] = mul2(z[v][j], fma2(c[j], both(inv[v]), sub));
                            if constexpr (SIG) z[v][j] = mul2(z[v][j], s[v][j]);
                        }
                        if (!live[v]) {  // 0 also where a (by d_loss) is not finite
#pragma unroll
                            for (int j = 0; j < L::kP; ++j) z[v][j] = both(0.f);
                        }
                    }
                } else {
#pragma unroll
                    for (int v = 0; v < V; ++v)
#pragma unroll
                        for (int j = 0; j < L::kP; ++j) z[v][j] = both(0.f);
                }
                // each lane puts its columns back where it read them
#pragma unroll
                for (int v = 0; v < V; ++v) {
#pragma unroll
                    for (int j = 0; j < L::kN / L::kVec; ++j) {
                        const int c = L::col(j * L::kVec, l);
                        if (!in[v] || c >= E) continue;
                        if constexpr (L::kVec == 4) {
                            float4 o;
                            unpack2(z[v][2 * j], o.x, o.y);
                            unpack2(z[v][2 * j + 1], o.z, o.w);
                            *reinterpret_cast<float4*>(row(v) + c) = o;
                        } else {
                            float lo, hi;
                            unpack2(z[v][j / 2], lo, hi);
                            row(v)[c] = j % 2 ? hi : lo;
                        }
                    }
                }
            }
            __syncwarp();
            if (p.d_topk_w && in_seq) {
                const int tokens = (int)(to - base);
                for (int i0 = (int)(from - base) / per * per; i0 < tokens; i0 += per) {
                    const uint32_t step = base + i0;
                    if (at != step) {  // a tile that two sequences share, the second time
                        load_next(step);
                        move_on(step);
                    }
                    const int e = of < per && (on >> (i0 + of) & 1) ? e_at : -1;
                    const float dw = dw_at;
                    float a = e >= 0 ? z_at : -INFINITY, b = 1.f;
                    move_on(step + per);
                    if constexpr (SIG) {
                        f2 fa, fb;
                        float x;
                        sigmoid2(both(a), fa, fb);
                        unpack2(fa, a, x);
                        unpack2(fb, b, x);
                    } else {
                        float m = a;
                        for (int o = pw / 2; o > 0; o >>= 1)
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                        a = exp1(max_nan(a - (m == -INFINITY ? 0.f : m), -kFar));
                    }
                    float sum = a, dot = e >= 0 ? a * dw : 0.f;
                    for (int o = pw / 2; o > 0; o >>= 1) {
                        sum += __shfl_xor_sync(0xffffffffu, sum, o);
                        dot += __shfl_xor_sync(0xffffffffu, dot, o);
                    }
                    const float inv = SIG ? rcp(sum + 1e-6f) : sum == 0.f ? 0.f : rcp(sum);
                    float v = a * inv * b * (dw - dot * inv);
                    // picks of the same expert (a top-K gives none) are added in
                    // slot order by the first of them
                    const int i = i0 + of;
                    const unsigned same =
                        __match_any_sync(0xffffffffu, e < 0 ? -1 - lane : i * 1024 + e);
                    if (__any_sync(0xffffffffu, __popc(same) > 1)) {
                        float tot = 0.f;
#pragma unroll 1
                        for (int q = 0; q < 32; ++q) {
                            const float other = __shfl_sync(0xffffffffu, v, q);
                            if (same >> q & 1u) tot += other;
                        }
                        v = tot;
                    }
                    if (e >= 0 && lane == __ffs(same) - 1) tile[i * E + e] += v;
                }
                __syncwarp();
            }
            // the rows of this sequence, contiguous in memory
            store_tile<L>(p.d_logits, tile + (from - base) * E, (int64_t)from * E,
                          (int)(to - from) * E, lane);
        }
        t = end;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// ---- launches ---------------------------------------------------------------

// Calls f with the row layout for E experts, 16 scores a lane where 32 lanes
// allow it (8 and 32 where a row is shorter or longer): 16-byte vectors when rows
// are multiples of 16 bytes.  Measured against 8 scores a lane on twice the lanes
// (E = 256, 131072 tokens, before the blocks were two an SM): the same 39 us for the
// loss, 56 us against 60 us for the gradient.
template <int VEC, typename F>
cudaError_t with_layout_of(int E, F&& f) {
    if (E <= 8) return f(RowLayout<VEC, 8, 1>{});
    if (E <= 16) return f(RowLayout<VEC, 16, 1>{});
    if (E <= 32) return f(RowLayout<VEC, 16, 2>{});
    if (E <= 64) return f(RowLayout<VEC, 16, 4>{});
    if (E <= 128) return f(RowLayout<VEC, 16, 8>{});
    if (E <= 256) return f(RowLayout<VEC, 16, 16>{});
    if (E <= 512) return f(RowLayout<VEC, 16, 32>{});
    return f(RowLayout<VEC, 32, 32>{});
}
template <typename F>
cudaError_t with_layout(int E, F&& f) {
    return E % 4 == 0 ? with_layout_of<4>(E, f) : with_layout_of<1>(E, f);
}

}  // namespace

// The tokens are spread over one wave of blocks, two an SM.  A second, part-filled
// wave is the dearest part of a small kernel; a third block an SM means 80 registers
// a thread, which spill in the backward pass (E = 256, 131072 tokens: 52 us with two
// blocks, 55 us with three; 16384 tokens: 12 us and 16 us), and three tiles a warp in
// place of two gain nothing (52 us).  Above 512 experts the gradient's kernels spill at
// two blocks too, the sigmoid router's 330 to 390 bytes (E = 1024, 32768 tokens: 67 us,
// softmax with 80 to 112 bytes 50 us).
// The SMs are a constant, not the device's: the workspace query needs no device, and the
// order of the sums does not depend on the part of a GPU that a process sees.
constexpr int64_t kWave = 152 * 2;

// Tokens of a block of the forward pass: its share of one wave, in whole steps of
// its warps.  Where sequence and share are both shorter than a step, it is the share
// alone: a block goes through its sequences one after the other (T = 369, E = 64,
// 426 sequences: 14 us, 129 us in whole steps; T = 2048, E = 128, 100 sequences:
// 13 us, 16 us in blocks of an average sequence's length).
int balance_chunk(const moe_shape& s, int n_seq) {
    int chunk = 0;
    with_layout(s.E, [&](auto layout) {
        constexpr int step = decltype(layout)::kRows * kWarps;
        const int64_t per = ceil_div(s.T > 0 ? s.T : 1, kWave), len = ceil_div(s.T, n_seq);
        chunk = (int)(ceil_div(per, step) * step);
        if (per < step && len < step) chunk = (int)per;
        if (chunk < 1) chunk = 1;
        return cudaSuccess;
    });
    return chunk;
}

int64_t balance_blocks(const moe_shape& s, int n_seq) {
    return ceil_div(s.T, balance_chunk(s, n_seq));
}

// Launches `kernel` with dynamic shared memory that may pass the default limit.
// The limit asked for is the same for every call, so calls of several threads do
// not undo each other's.
constexpr int kMaxSmem = 108 * 1024;
template <typename Args>
cudaError_t launch_wide(void (*kernel)(Args), unsigned blocks, size_t smem, cudaStream_t st,
                        const Args& args) {
    if (smem > 48 * 1024) {
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(kernel, dim3(blocks), dim3(kThreads), smem, st, args);
}

// slices of 32 columns, side by side while that leaves at most eight blocks an SM
int balance_slices(const moe_shape& s, int n_seq) {
    const int all = (int)ceil_div(s.E, 32);
    const int fill = (int)ceil_div(152 * 8, n_seq);
    return all < fill ? all : fill;
}

cudaError_t launch_balance_loss(const moe_shape& s, BalanceArgs a, cudaStream_t st) {
    a.T = s.T;
    a.E = s.E;
    a.K = s.K;
    a.chunk = balance_chunk(s, a.n_seq);
    a.blocks = (int)balance_blocks(s, a.n_seq);
    // One block does it all where that takes no longer than a second launch: two
    // tiles a warp (E = 8, T = 64: 3.5 us against 5.3; E = 256: T = 64 5.2 against 6.7,
    // T = 128 7.6 against 6.8).
    with_layout(s.E, [&](auto layout) {
        constexpr int most = 2 * kWarps * decltype(layout)::kTokens;
        a.solo = s.T <= most && a.n_seq <= 4;
        if (a.solo) {
            a.chunk = (int)ceil_div(s.T, kWarps) * kWarps;
            a.blocks = 1;
        }
        return cudaSuccess;
    });
    cudaError_t e = with_layout(s.E, [&](auto layout) {
        using L = decltype(layout);
        const size_t smem = sizeof(float) * (size_t)(kWarps * kStages * tile_floats<L>(s.E) +
                                                     (kWarps + 1) * s.E);
        return launch_wide(s.router == MOE_ROUTER_SIGMOID ? balance_partial_kernel<L, true>
                                                          : balance_partial_kernel<L, false>,
                           (unsigned)a.blocks, smem, st, a);
    });
    if (e != cudaSuccess || a.solo) return e;
    // A block per sequence and slice of columns, a warp for each of the partial rows
    // that a sequence has on average: the longest of ragged ones has several times
    // as many, and all wait for its block.
    const int64_t rows = ceil_div(a.blocks, a.n_seq) + 1;
    int warps = 4;
    while (warps < 32 && warps < rows) warps *= 2;
    return launch_pdl(balance_final_kernel,
                      dim3((unsigned)a.n_seq, (unsigned)balance_slices(s, a.n_seq)),
                      dim3((unsigned)warps * 32), (size_t)warps * 32 * 8, st, a);
}

cudaError_t launch_route_backward(const moe_shape& s, RouteBackwardArgs a, cudaStream_t st) {
    a.T = s.T;
    a.E = s.E;
    a.K = s.K;
    a.pw_log = 0;
    while ((1 << a.pw_log) < s.K) ++a.pw_log;
    return with_layout(s.E, [&](auto layout) {
        using L = decltype(layout);
        // a warp's share of one wave, in whole steps where it is that much (fewer
        // tokens leave lanes idle, but a warp's sequences go one after the other: T = 32,
        // E = 6 in 383 sequences, most of them empty: 4 us, 274 us in whole steps)
        const int64_t per = ceil_div(s.T, kWave * kWarps);
        a.chunk = (int)(per < L::kRows ? per : ceil_div(per, L::kRows) * L::kRows);
        const unsigned blocks = (unsigned)ceil_div(s.T, (int64_t)a.chunk * kWarps);
        const size_t smem =
            sizeof(float) * (size_t)(kWarps * (kStages * tile_floats<L>(s.E) + s.E));
        return launch_wide(s.router == MOE_ROUTER_SIGMOID ? route_backward_kernel<L, true>
                                                          : route_backward_kernel<L, false>,
                           blocks, smem, st, a);
    });
}

}  // namespace moe
