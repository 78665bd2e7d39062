// philox.cuh -- the counter-based generator behind dropout, and the rule that
// turns its bits into a mask that is never stored.
//
// Philox4x32-10: J. Salmon, M. Moraes, R. Dror, D. Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", SC 2011.  A 128-bit counter and a 64-bit key
// give 128 random bits through ten rounds of two 32 x 32 -> 64 bit products.
//
// One evaluation serves eight consecutive elements, 16 bits each: element i of
// a tensor takes counter (i / 8, offset) and key seed, and of the four output
// words the half i % 2 of word (i % 8) / 2.  A bit pattern depends on (seed,
// offset, i) alone, so the combine, the plain call and every backward pass see
// the same mask however their threads are laid out.  16 bits an element make
// the drop probability a multiple of 2^-16 (the scale uses that multiple, so
// the expectation is exact) and cost half the products of 32 bits.
#pragma once

#include "common.cuh"

namespace moe {

// What a launch needs to draw a mask.  Of the 65536 values of an element's 16
// bits, thr drop it, and the others are multiplied by scale; `last` is the
// largest dropping value in the upper half of a word, all ones below it, so that
// one comparison of a word (as it is, or shifted up by 16) decides.
struct DropRule {
    uint32_t thr, last;
    float scale;
};

// p in [0, 1]: rounded to the nearest multiple of 2^-16 (the sum in double, so thr is 1
// from the largest p below 2^-17 on)
inline DropRule drop_rule(double p) {
    DropRule r;
    r.thr = (uint32_t)(p * 65536.0 + 0.5);
    r.last = (r.thr << 16) - 1u;
    r.scale = r.thr < 65536u ? (float)(65536.0 / (65536.0 - (double)r.thr)) : 0.f;
    return r;
}

// seed and offset as the caller's device words hold them
struct RngState {
    uint32_t k0, k1, o0, o1;
};

__device__ __forceinline__ RngState load_rng(const uint64_t* rng) {
    const uint64_t seed = rng[0], off = rng[1];
    return {(uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)off, (uint32_t)(off >> 32)};
}

__device__ __forceinline__ void philox4x32_10(uint64_t counter, const RngState& s,
                                              uint32_t (&out)[4]) {
    uint32_t c0 = (uint32_t)counter, c1 = (uint32_t)(counter >> 32), c2 = s.o0, c3 = s.o1;
    uint32_t k0 = s.k0, k1 = s.k1;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)0xD2511F53u * c0;
        const uint64_t b = (uint64_t)0xCD9E8D57u * c2;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)b;
        c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    out[0] = c0;
    out[1] = c1;
    out[2] = c2;
    out[3] = c3;
}

// The bits of the elements 8 * group .. 8 * group + 7.  They depend on no data,
// so a kernel draws them while its loads are on their way.
struct Bits8 {
    uint32_t w[4];
};
__device__ __forceinline__ Bits8 draw8(uint64_t group, const RngState& s) {
    Bits8 b;
    philox4x32_10(group, s, b.w);
    return b;
}

// A dropped element is selected away, not multiplied by zero: it is 0 whatever
// it held.  (Not for thr = 0, where nothing is drawn.)
__device__ __forceinline__ void drop8(float (&v)[8], const Bits8& b, const DropRule& rule) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[2 * j] = (b.w[j] << 16) > rule.last ? v[2 * j] * rule.scale : 0.f;
        v[2 * j + 1] = b.w[j] > rule.last ? v[2 * j + 1] * rule.scale : 0.f;
    }
}

// ---- eight consecutive elements as 16-byte vectors (bf16: one, fp32: two) ----
template <typename T> struct Unit {
    static constexpr int kVecs = 8 / Elem<T>::kPerVec;
    uint4 v[kVecs];
};

// Plain (coherent) loads that skip L1: each element is read once, and the
// output may be the input's own storage.
template <typename T>
__device__ __forceinline__ Unit<T> load_unit(const T* p) {
    Unit<T> u;
#pragma unroll
    for (int i = 0; i < Unit<T>::kVecs; ++i)
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(u.v[i].x), "=r"(u.v[i].y), "=r"(u.v[i].z), "=r"(u.v[i].w)
                     : "l"(reinterpret_cast<const uint4*>(p) + i)
                     : "memory");
    return u;
}

__device__ __forceinline__ void widen(const Unit<float>& u, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        f[4 * i] = __uint_as_float(u.v[i].x);
        f[4 * i + 1] = __uint_as_float(u.v[i].y);
        f[4 * i + 2] = __uint_as_float(u.v[i].z);
        f[4 * i + 3] = __uint_as_float(u.v[i].w);
    }
}
__device__ __forceinline__ void widen(const Unit<bf16>& u, float (&f)[8]) {
    unpack(u.v[0], f, (const bf16*)nullptr);
}

// The only rounding of these operators: fp32 to the stored type, to nearest even.
// Streaming stores: an output of this size is not read again before others have
// passed through L2 (dropout of 16384 x 7168 bf16, one group at a time: 111 us with plain
// ones, 108).
__device__ __forceinline__ void store_unit(float* p, const float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
        __stcs(reinterpret_cast<uint4*>(p) + i,
               make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]),
                          __float_as_uint(f[4 * i + 2]), __float_as_uint(f[4 * i + 3])));
}
__device__ __forceinline__ void store_unit(bf16* p, const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const __nv_bfloat162 b2 = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&b2);
    }
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
}

}  // namespace moe
