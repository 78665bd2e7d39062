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
#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// How a row of E scores lies over the lanes of a warp: `kGroup` lanes hold it
// (32 / kGroup rows a warp), kNv vectors of kVec scores a lane, vector i of
// lane l starting at column (i * kGroup + l) * kVec.
template <int VEC, int NV, int G>
struct RowLayout {
    static constexpr int kVec = VEC, kNv = NV, kGroup = G, kRows = 32 / G, kN = NV * VEC;
    __device__ static int col(int i, int l) { return (i * G + l) * VEC; }
};

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// a row's scores into registers; -inf beyond E and in rows that take no part
template <typename L>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, int l, bool live,
                                         float (&z)[L::kN]) {
#pragma unroll
    for (int i = 0; i < L::kNv; ++i) {
        const int c = L::col(i, l);
#pragma unroll
        for (int v = 0; v < L::kVec; ++v) z[i * L::kVec + v] = -INFINITY;
        if (live && c < E) {
            if constexpr (L::kVec == 4) {
                const float4 q = *reinterpret_cast<const float4*>(row + c);
                z[i * 4] = q.x; z[i * 4 + 1] = q.y; z[i * 4 + 2] = q.z; z[i * 4 + 3] = q.w;
            } else {
                z[i] = row[c];
            }
        }
    }
}

// sigmoid(z) and 1 - sigmoid(z), each with its own relative accuracy (one
// minus the other would lose the small one)
__device__ __forceinline__ void sigmoid2(float z, float& a, float& b) {
    const float ex = expf(-fabsf(z));
    const float r = __fdividef(1.f, 1.f + ex);
    const float q = ex * r;
    a = z >= 0.f ? r : q;
    b = z >= 0.f ? q : r;
}

// The router's probabilities of one row: p in place of the scores, and for the
// sigmoid router s[i] = 1 - sigmoid (the backward pass's factor).  Experts
// with a score of -inf get 0, and a row of them gets all zeros.
template <typename L, bool SIG>
__device__ __forceinline__ void row_probs(float (&z)[L::kN], float (&s)[L::kN]) {
    if constexpr (SIG) {
        float a[L::kN], sum = 0.f;
#pragma unroll
        for (int i = 0; i < L::kN; ++i) {
            sigmoid2(z[i], a[i], s[i]);
            sum += a[i];
        }
        sum = group_sum<L::kGroup>(sum);
        // below this every score is under -69, where sigmoid(z) = e^z to fp32's
        // last bit: the softmax, which cannot underflow as a whole
        const bool tiny = sum < 1e-30f;
        if (__any_sync(0xffffffffu, tiny)) {
            float m = -INFINITY;
#pragma unroll
            for (int i = 0; i < L::kN; ++i) m = fmaxf(m, z[i]);
            m = group_max<L::kGroup>(m);
            float se = 0.f, e[L::kN];
#pragma unroll
            for (int i = 0; i < L::kN; ++i) {
                e[i] = m == -INFINITY ? 0.f : expf(z[i] - m);
                se += e[i];
            }
            se = group_sum<L::kGroup>(se);
            if (tiny) {
                sum = se > 0.f ? se : 1.f;
#pragma unroll
                for (int i = 0; i < L::kN; ++i) a[i] = e[i];
            }
        }
        const float inv = __fdividef(1.f, sum);
#pragma unroll
        for (int i = 0; i < L::kN; ++i) z[i] = a[i] * inv;
    } else {
        float m = -INFINITY, sum = 0.f;
#pragma unroll
        for (int i = 0; i < L::kN; ++i) m = fmaxf(m, z[i]);
        m = group_max<L::kGroup>(m);
        if (m == -INFINITY) m = 0.f;
#pragma unroll
        for (int i = 0; i < L::kN; ++i) {
            z[i] = expf(z[i] - m);
            sum += z[i];
        }
        sum = group_sum<L::kGroup>(sum);
        const float inv = sum > 0.f ? __fdividef(1.f, sum) : 0.f;
#pragma unroll
        for (int i = 0; i < L::kN; ++i) z[i] *= inv;
    }
}

// The sequence that holds token t, by a 32-way search of the n + 1 offsets by a
// whole warp: [*, end) is the run of tokens from t on with the same answer, and
// -1 is the answer before the first offset and from the last one on.  Whatever
// the offsets hold, end > t.
__device__ __forceinline__ int find_seq(const int32_t* __restrict__ cu, int n, int t, int T,
                                        int& end) {
    if (cu == nullptr) {
        end = T;
        return 0;
    }
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = n + 1;  // cu[lo - 1] <= t < cu[hi], where those exist
    while (lo < hi) {
        const int step = (hi - lo + 31) / 32;
        const int i = lo + lane * step;
        const bool le = i < hi && cu[i] <= t;
        const int c = __ffs(~__ballot_sync(0xffffffffu, le)) - 1;  // leading lanes (-1: all)
        const int k = c < 0 ? 32 : c;
        if (k == 0) break;
        const int first = lo;
        lo = first + (k - 1) * step + 1;
        hi = min(hi, first + k * step);
    }
    end = lo <= n ? min(cu[lo], T) : T;
    return lo <= n ? lo - 1 : -1;
}

// One block per `chunk` tokens.  For each sequence g that the chunk of block b
// touches it writes partial row b + g (along the batch either b or g grows from
// one such pair to the next, so the rows are its own).
template <typename L, bool SIG>
__global__ void __launch_bounds__(kThreads)
balance_partial_kernel(const float* __restrict__ logits, const int32_t* __restrict__ topk_idx,
                       const uint8_t* __restrict__ mask, const int32_t* __restrict__ cu, int n_seq,
                       int T, int E, int K, int chunk, float* __restrict__ part_p,
                       int32_t* __restrict__ part_c, DevError* err) {
    extern __shared__ float sm[];  // [kWarps][E] sums, then [E] counts
    int32_t* hist = reinterpret_cast<int32_t*>(sm + kWarps * E);
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int l = lane % L::kGroup, r = lane / L::kGroup;
    const int64_t first = (int64_t)blockIdx.x * chunk;
    const int t0 = (int)first, t1 = (int)(first + chunk < T ? first + chunk : T);
    for (int t = t0; t < t1;) {
        int end;
        const int g = find_seq(cu, n_seq, t, T, end);
        end = min(end, t1);
        if (g >= 0) {
            float acc[L::kN];
#pragma unroll
            for (int i = 0; i < L::kN; ++i) acc[i] = 0.f;
            for (int e = threadIdx.x; e < E; e += kThreads) hist[e] = 0;
            __syncthreads();
            for (int64_t base = t + warp * L::kRows; base < end; base += kWarps * L::kRows) {
                const int64_t tok = base + r;
                const bool live = tok < end && (mask == nullptr || mask[tok] != 0);
                float z[L::kN], s[L::kN];
                load_row<L>(logits + tok * E, E, l, live, z);
                row_probs<L, SIG>(z, s);
                if (live) {
#pragma unroll
                    for (int i = 0; i < L::kN; ++i) acc[i] += z[i];
                    for (int k = l; k < K; k += L::kGroup) {
                        const int e = topk_idx[tok * K + k];
                        if (e >= 0 && e < E) atomicAdd(&hist[e], 1);
                        else record_error(err, MOE_ERR_BOUNDS, e);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < L::kN; ++i)
#pragma unroll
                for (int o = 16; o >= L::kGroup; o >>= 1)
                    acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
            if (r == 0) {
#pragma unroll
                for (int i = 0; i < L::kNv; ++i)
#pragma unroll
                    for (int v = 0; v < L::kVec; ++v)
                        if (L::col(i, l) + v < E)
                            sm[warp * E + L::col(i, l) + v] = acc[i * L::kVec + v];
            }
            __syncthreads();
            const int64_t row = (int64_t)(blockIdx.x + g) * E;
            for (int e = threadIdx.x; e < E; e += kThreads) {
                float p = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) p += sm[w * E + e];
                part_p[row + e] = p;
                part_c[row + e] = hist[e];
            }
            __syncthreads();
        }
        t = end;
    }
}

constexpr int kFinalThreads = 512;

// sum of v over the block, in every thread (fixed order; buf: one slot a warp)
template <typename V>
__device__ __forceinline__ V block_sum(V v, V* buf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    V s = 0;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) s += buf[w];
    return s;
}

// One block per sequence adds its partial rows and writes its counts, mean
// probabilities and loss; the last block to finish adds the losses in order.
__global__ void __launch_bounds__(kFinalThreads)
balance_final_kernel(const float* __restrict__ part_p, const int32_t* __restrict__ part_c,
                     const int32_t* __restrict__ cu, int n_seq, int T, int E, int K, int chunk,
                     float alpha, int32_t* __restrict__ counts, float* __restrict__ mean_p,
                     float* __restrict__ loss, double* seq_loss, unsigned int* ticket,
                     DevError* err) {
    __shared__ double buf[kFinalThreads / 32];
    __shared__ int ibuf[kFinalThreads / 32];
    __shared__ int last;
    pdl_wait();
    pdl_trigger();
    const int g = blockIdx.x;
    int a = 0, b = T;
    if (cu) {
        a = cu[g];
        b = cu[g + 1];
        if ((a < 0 || b < a || b > T) && threadIdx.x == 0) record_error(err, MOE_ERR_BOUNDS, g);
        a = max(a, 0);
        b = min(b, T);
    }
    const int64_t b0 = a / chunk, b1 = b > a ? (b - 1) / chunk + 1 : b0;  // blocks it lies in
    int total = 0;
    for (int e = threadIdx.x; e < E; e += kFinalThreads) {
        int c = 0;
        for (int64_t i = b0; i < b1; ++i) c += part_c[(i + g) * E + e];
        counts[(int64_t)g * E + e] = c;
        total += c;
    }
    total = block_sum(total, ibuf);
    const float n = (float)total / (float)K;  // tokens that take part
    double sum = 0.0;
    for (int e = threadIdx.x; e < E; e += kFinalThreads) {
        float p = 0.f;
        for (int64_t i = b0; i < b1; ++i) p += part_p[(i + g) * E + e];
        const float m = total > 0 ? p / n : 0.f;
        mean_p[(int64_t)g * E + e] = m;
        if (total > 0)
            sum += (double)m * (double)counts[(int64_t)g * E + e] * (double)E / (double)total;
    }
    sum = block_sum(sum, buf);
    if (threadIdx.x == 0) {
        seq_loss[g] = sum;
        __threadfence();
        last = atomicAdd(ticket, 1u) == (unsigned)n_seq - 1u;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    double v = 0.0;
    for (int i = threadIdx.x; i < n_seq; i += kFinalThreads) v += __ldcg(seq_loss + i);
    v = block_sum(v, buf);
    if (threadIdx.x == 0) *loss = (float)(v * (double)alpha / (double)n_seq);
}

// A warp per `chunk` tokens, kRows of them at a time; the coefficients a_ge of
// the sequence at hand stay in registers.  The routing weights' part is added
// through a row of shared memory per token: lane k scatters pick k's value, and
// every lane reads its columns back.
template <typename L, bool SIG>
__global__ void __launch_bounds__(kThreads)
route_backward_kernel(const float* __restrict__ logits, const int32_t* __restrict__ topk_idx,
                      const float* __restrict__ d_topk_w, const uint8_t* __restrict__ mask,
                      const int32_t* __restrict__ cu, int n_seq, int T, int E, int K, int chunk,
                      float alpha, const int32_t* __restrict__ counts,
                      const float* __restrict__ d_loss, float* __restrict__ d_logits) {
    // K <= min(E, 32) <= kPicks * kGroup
    constexpr int kPicks = L::kVec == 4 ? (32 / L::kGroup < 4 ? 32 / L::kGroup : 4) : 1;
    extern __shared__ float sm[];                 // [kWarps][kRows][E] when d_topk_w
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int l = lane % L::kGroup, r = lane / L::kGroup;
    float* scat = sm + (int64_t)(warp * L::kRows + r) * E;
    if (d_topk_w) {
        for (int e = l; e < E; e += L::kGroup) scat[e] = 0.f;
        __syncwarp();
    }
    const float up = counts ? alpha / (float)n_seq * (d_loss ? *d_loss : 1.f) : 0.f;
    const int64_t first = ((int64_t)blockIdx.x * kWarps + warp) * chunk;
    const int t0 = (int)(first < T ? first : T), t1 = (int)(first + chunk < T ? first + chunk : T);
    for (int t = t0; t < t1;) {
        int end;
        const int g = find_seq(cu, n_seq, t, T, end);
        end = min(end, t1);
        float coef[L::kN];
#pragma unroll
        for (int i = 0; i < L::kN; ++i) coef[i] = 0.f;
        if (counts && g >= 0) {
            float total = 0.f;
#pragma unroll
            for (int i = 0; i < L::kNv; ++i)
#pragma unroll
                for (int v = 0; v < L::kVec; ++v) {
                    const int c = L::col(i, l) + v;
                    if (c < E) coef[i * L::kVec + v] = (float)counts[(int64_t)g * E + c];
                    total += coef[i * L::kVec + v];
                }
            total = group_sum<L::kGroup>(total);
            // a = alpha E c / (G K n^2) with n = total / K
            const float k = total > 0.f ? up * (float)E / total * ((float)K / total) : 0.f;
#pragma unroll
            for (int i = 0; i < L::kN; ++i) coef[i] *= k;
        }
        for (int64_t base = t; base < end; base += L::kRows) {
            const int64_t tok = base + r;
            const bool in = tok < end;
            const bool live = in && g >= 0 && (mask == nullptr || mask[tok] != 0);
            float z[L::kN], s[L::kN];
            if (counts) {
                load_row<L>(logits + tok * E, E, l, live, z);
                row_probs<L, SIG>(z, s);
                float dot = 0.f;
#pragma unroll
                for (int i = 0; i < L::kN; ++i) dot = fmaf(z[i], coef[i], dot);
                dot = group_sum<L::kGroup>(dot);
#pragma unroll
                for (int i = 0; i < L::kN; ++i) {
                    z[i] *= coef[i] - dot;
                    if constexpr (SIG) z[i] *= s[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < L::kN; ++i) z[i] = 0.f;
            }
            if (d_topk_w) {
                int pe[kPicks];
                float dw[kPicks], a[kPicks], b[kPicks];
                float m = -INFINITY, sum = 0.f, dot = 0.f;
#pragma unroll
                for (int i = 0; i < kPicks; ++i) {
                    const int k = i * L::kGroup + l;
                    pe[i] = -1;
                    a[i] = -INFINITY;
                    dw[i] = 0.f;
                    if (live && k < K) {
                        const int e = topk_idx[tok * K + k];
                        if (e >= 0 && e < E) {
                            pe[i] = e;
                            a[i] = logits[tok * E + e];
                            dw[i] = d_topk_w[tok * K + k];
                        }
                    }
                    m = fmaxf(m, a[i]);
                }
                if constexpr (SIG) {
#pragma unroll
                    for (int i = 0; i < kPicks; ++i) {
                        sigmoid2(a[i], a[i], b[i]);
                        sum += a[i];
                    }
                    sum = group_sum<L::kGroup>(sum) + 1e-6f;
                } else {
                    m = group_max<L::kGroup>(m);
                    if (m == -INFINITY) m = 0.f;
#pragma unroll
                    for (int i = 0; i < kPicks; ++i) {
                        a[i] = expf(a[i] - m);
                        b[i] = 1.f;
                        sum += a[i];
                    }
                    sum = group_sum<L::kGroup>(sum);
                    if (!(sum > 0.f)) sum = 1.f;
                }
                const float inv = __fdividef(1.f, sum);
#pragma unroll
                for (int i = 0; i < kPicks; ++i) {
                    a[i] *= inv;  // the routing weight
                    dot = fmaf(a[i], dw[i], dot);
                }
                dot = group_sum<L::kGroup>(dot);
                // picks of the same expert (a top-K gives none) are added in
                // slot order by the first of them
#pragma unroll
                for (int i = 0; i < kPicks; ++i) {
                    const float v = a[i] * b[i] * (dw[i] - dot);
                    const unsigned same =
                        __match_any_sync(0xffffffffu, pe[i] < 0 ? -1 - lane : r * 1024 + pe[i]);
                    float tot = v;
                    if (__any_sync(0xffffffffu, __popc(same) > 1)) {
                        tot = 0.f;
                        for (int q = 0; q < 32; ++q) {
                            const float x = __shfl_sync(0xffffffffu, v, q);
                            if (same >> q & 1u) tot += x;
                        }
                    }
                    if (pe[i] >= 0 && lane == __ffs(same) - 1) scat[pe[i]] += tot;
                    __syncwarp();
                }
#pragma unroll
                for (int i = 0; i < L::kNv; ++i)
#pragma unroll
                    for (int v = 0; v < L::kVec; ++v)
                        if (L::col(i, l) + v < E) z[i * L::kVec + v] += scat[L::col(i, l) + v];
                __syncwarp();
#pragma unroll
                for (int i = 0; i < kPicks; ++i)
                    if (pe[i] >= 0) scat[pe[i]] = 0.f;
                __syncwarp();
            }
            if (in) {
                float* out = d_logits + tok * E;
#pragma unroll
                for (int i = 0; i < L::kNv; ++i) {
                    const int c = L::col(i, l);
                    if (c >= E) continue;
                    if constexpr (L::kVec == 4)
                        *reinterpret_cast<float4*>(out + c) =
                            live ? make_float4(z[i * 4], z[i * 4 + 1], z[i * 4 + 2], z[i * 4 + 3])
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
                    else
                        out[c] = live ? z[i] : 0.f;
                }
            }
        }
        t = end;
    }
}

// ---- launches ---------------------------------------------------------------

// Calls f with the row layout for E experts: 16-byte vectors when rows are
// multiples of 16 bytes, as few lanes as hold a row in one vector each.
template <typename F>
cudaError_t with_layout(int E, F&& f) {
    if (E % 4 == 0) {
        if (E <= 4) return f(RowLayout<4, 1, 1>{});
        if (E <= 8) return f(RowLayout<4, 1, 2>{});
        if (E <= 16) return f(RowLayout<4, 1, 4>{});
        if (E <= 32) return f(RowLayout<4, 1, 8>{});
        if (E <= 64) return f(RowLayout<4, 1, 16>{});
        if (E <= 128) return f(RowLayout<4, 1, 32>{});
        if (E <= 256) return f(RowLayout<4, 2, 32>{});
        if (E <= 512) return f(RowLayout<4, 4, 32>{});
        return f(RowLayout<4, 8, 32>{});
    }
    if (E <= 8) return f(RowLayout<1, 1, 8>{});
    if (E <= 32) return f(RowLayout<1, 1, 32>{});
    if (E <= 64) return f(RowLayout<1, 2, 32>{});
    if (E <= 128) return f(RowLayout<1, 4, 32>{});
    if (E <= 256) return f(RowLayout<1, 8, 32>{});
    if (E <= 512) return f(RowLayout<1, 16, 32>{});
    return f(RowLayout<1, 32, 32>{});
}

}  // namespace

// tokens a block of the forward pass takes: two blocks an SM, and at least one
// step of its warps
int balance_chunk(const moe_shape& s) {
    const int64_t blocks = (int64_t)152 * 2;
    return (int)(ceil_div(s.T > 0 ? s.T : 1, blocks) + 7) / 8 * 8;
}

int64_t balance_partials(const moe_shape& s, int n_seq) {
    return ceil_div(s.T, balance_chunk(s)) + n_seq;
}

cudaError_t launch_balance_loss(const moe_shape& s, const float* logits, const int32_t* topk_idx,
                                const uint8_t* mask, const int32_t* cu, int n_seq, float alpha,
                                int32_t* counts, float* mean_p, float* loss, float* part_p,
                                int32_t* part_c, double* seq_loss, unsigned int* ticket,
                                DevError* err, cudaStream_t st) {
    const int chunk = balance_chunk(s);
    const unsigned blocks = (unsigned)ceil_div(s.T, chunk);
    const size_t smem = sizeof(float) * (size_t)s.E * (kWarps + 1);
    cudaError_t e = with_layout(s.E, [&](auto layout) {
        using L = decltype(layout);
        auto k = s.router == MOE_ROUTER_SIGMOID ? balance_partial_kernel<L, true>
                                                : balance_partial_kernel<L, false>;
        return launch_pdl(k, dim3(blocks), dim3(kThreads), smem, st, logits, topk_idx, mask, cu,
                          n_seq, s.T, s.E, s.K, chunk, part_p, part_c, err);
    });
    if (e != cudaSuccess) return e;
    return launch_pdl(balance_final_kernel, dim3((unsigned)n_seq), dim3(kFinalThreads), 0, st,
                      (const float*)part_p, (const int32_t*)part_c, cu, n_seq, s.T, s.E, s.K, chunk,
                      alpha, counts, mean_p, loss, seq_loss, ticket, err);
}

cudaError_t launch_route_backward(const moe_shape& s, const float* logits, const int32_t* topk_idx,
                                  const float* d_topk_w, const uint8_t* mask, const int32_t* cu,
                                  int n_seq, float alpha, const int32_t* counts,
                                  const float* d_loss, float* d_logits, cudaStream_t st) {
    return with_layout(s.E, [&](auto layout) {
        using L = decltype(layout);
        const int64_t warps = (int64_t)device_sm_count() * 4 * kWarps;
        const int chunk = (int)ceil_div(ceil_div(s.T, warps), L::kRows) * L::kRows;
        const unsigned blocks = (unsigned)ceil_div(s.T, (int64_t)chunk * kWarps);
        const size_t smem = d_topk_w ? sizeof(float) * (size_t)s.E * kWarps * L::kRows : 0;
        auto k = s.router == MOE_ROUTER_SIGMOID ? route_backward_kernel<L, true>
                                                : route_backward_kernel<L, false>;
        return launch_pdl(k, dim3(blocks), dim3(kThreads), smem, st, logits, topk_idx, d_topk_w, mask,
                          cu, n_seq, s.T, s.E, s.K, chunk, alpha, counts, d_loss, d_logits);
    });
}

}  // namespace moe
