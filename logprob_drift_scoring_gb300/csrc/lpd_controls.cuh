// Sampling controls on logits: the arithmetic of one logit, and the block's way
// of finding the few that need it.
//
// For row r and token j with n_all = occurrences of j in the row's history,
// n_gen = those in its generated part, the controlled logit is
//   x1 = n_all > 0 ? (x > 0 ? x / rep : x * rep) : x
//   x2 = n_gen > 0 ? x1 - freq * n_gen - pres    : x1
//   x3 = x2 + sum of the row's biases of token j
//   z  = allowed(j) ? scale * x3 : -inf
// Only the tokens of the history and of the bias list ("touched" tokens) need
// more than the scale and the mask, and they are few: a thousand of a hundred
// thousand.  Seven warps of a block (the scouts) look for them while sixteen
// others stream the row: they mark the touched columns of the unit in a bitmap,
// and with the bitmap's prefix sums a token's rank among the touched ones is a
// look-up and a popcount, so that a second pass over the history counts
// occurrences in a dense array without collisions or empty slots.  The touched
// columns come out in ascending order whatever the order of the marks, and the
// counts are integers, so nothing depends on the order of the shared-memory
// atomics.  The streaming warps see one bit a column.
//
// Masked columns are replaced eight at a time: a 4 KB table in shared memory
// gives the 16-bit lane masks of a byte of bits, and one logical instruction a
// register does the rest (bit tests and selects took a third of the scoring
// kernel's instructions).
#pragma once

#include <cfloat>
#include <cuda_bf16.h>
#include <math_constants.h>

#include "lpd_acc.cuh"
#include "lpd_internal.cuh"
#include "lpd_operators.cuh"

namespace lpd {

constexpr uint32_t kSeen = 0x80000000u;    // count word: the token occurs in the prompt part
constexpr uint32_t kBiased = 0x40000000u;  // the token has a bias entry
constexpr uint32_t kCount = 0x3fffffffu;   // occurrences in the generated part
constexpr int64_t kMaxRange = kCount;      // so a row's range is cut to its last 2^30 - 1 tokens

// The controls of one row: read once a unit by one thread, kept in shared memory.
struct CtlRow {
    int64_t begin, split, end;
    float rep, inv_h, inv_l;  // repetition penalty and 1 / rep as a sum of two floats
    float freq, pres, scale;
    const uint32_t *mask;     // the row's mask words, or nullptr: everything allowed
    bool none;                // a mask row outside the table: nothing allowed
};

__device__ __forceinline__ CtlRow ctl_row(const CtlSide &c, int64_t r, float inv_h, float inv_l, float rep) {
    CtlRow o;
    o.begin = o.split = o.end = 0;
    if (c.counts) {
        const int64_t e = min(max(c.hist_end[r], int64_t{0}), c.n_history);
        const int64_t b = min(max(c.hist_begin[r], e - kMaxRange), e);
        o.end = e;
        o.begin = max(b, int64_t{0});
        o.split = min(max(c.hist_split[r], o.begin), e);
    }
    o.rep = rep;
    o.inv_h = inv_h;
    o.inv_l = inv_l;
    o.freq = c.frequency ? c.frequency[r] : 0.f;
    o.pres = c.presence ? c.presence[r] : 0.f;
    const float s = c.scale ? c.scale[r] : 1.f;
    o.scale = s > 0.f && s <= FLT_MAX ? s : CUDART_NAN_F;
    o.mask = nullptr;
    o.none = false;
    if (c.mask) {
        const int64_t k = c.mask_row ? static_cast<int64_t>(c.mask_row[r]) : r;
        if (k >= c.n_masks) o.none = true;
        else if (k >= 0) o.mask = c.mask + k * c.mask_stride;
    }
    return o;
}

// The same with the reciprocal of the penalty made here.  1 / rep as h + l: h
// is the rounded quotient and l = (1 - rep h) / rep, formed from the exact
// residual of the multiply-add.
__device__ __forceinline__ CtlRow ctl_row(const CtlSide &c, int64_t r) {
    float rep = c.repetition ? c.repetition[r] : 1.f;
    if (!(rep > 0.f && rep <= FLT_MAX)) rep = CUDART_NAN_F;
    const float h = __frcp_rn(rep);
    return ctl_row(c, r, h, __fmul_rn(__fmaf_rn(-rep, h, 1.f), h), rep);
}

// ---- a number as the sum of two floats ---------------------------------------
struct Two {
    float h, l;
};
__device__ __forceinline__ Two two_add(Two a, float b) {
    const float s = __fadd_rn(a.h, b);
    const float t = __fsub_rn(s, a.h);
    const float e = __fadd_rn(__fsub_rn(a.h, __fsub_rn(s, t)), __fsub_rn(b, t));
    return Two{s, __fadd_rn(a.l, e)};
}

// The row's bias entries of one token: the last one's index (-1: none) and how
// many there are.  ids: padded with -1 to a multiple of four, 16-byte aligned.
__device__ __forceinline__ int bias_find(const int4 *ids, int n, int32_t token, int *found) {
    int at = -1, k = 0;
#pragma unroll 2
    for (int e = 0; e < n; e += 4) {
        const int4 v = ids[e >> 2];
        at = v.x == token ? e : at;
        at = v.y == token ? e + 1 : at;
        at = v.z == token ? e + 2 : at;
        at = v.w == token ? e + 3 : at;
        k += (v.x == token) + (v.y == token) + (v.z == token) + (v.w == token);
    }
    *found = k;
    return at;
}
// Their sum as two floats.  Almost always there is one entry; several are added
// in double (at most 1024 terms, so the sum is exact to far below a float's
// step in any order).
__device__ __forceinline__ Two bias_sum(const int32_t *ids, const float *values, int n, int32_t token, int at,
                                        int found) {
    if (found <= 1) return Two{found ? values[at] : 0.f, 0.f};
    double s = 0.0;
    for (int e = 0; e < n; ++e)
        if (ids[e] == token) s += static_cast<double>(values[e]);
    const float h = static_cast<float>(s);
    // an infinite sum (a ban) has no low part
    return Two{h, fabsf(h) <= FLT_MAX ? static_cast<float>(s - static_cast<double>(h)) : 0.f};
}

// x3 of a touched, allowed token with count word w.  Two floats, so that the
// logit's rounding (a step of 1e-6 at a logit of 20) stays out of the logprob
// difference of two sides that nearly agree; `slope` (may be null) receives
// dx3/dx.
__device__ __forceinline__ Two ctl_value(float x, uint32_t w, const CtlRow &o, Two bias, float *slope) {
    Two v{x, 0.f};
    float d = 1.f;
    if ((w & ~kBiased) != 0u) {
        if (x > 0.f) {
            v.h = __fmul_rn(x, o.inv_h);
            v.l = __fmaf_rn(x, o.inv_l, __fmaf_rn(x, o.inv_h, -v.h));
            d = o.inv_h;
        } else {
            v.h = __fmul_rn(x, o.rep);
            v.l = __fmaf_rn(x, o.rep, -v.h);
            d = o.rep;
        }
        const uint32_t n = w & kCount;
        if (n != 0u) {
            const float nf = static_cast<float>(n);
            const float f = __fmul_rn(o.freq, nf);
            v = two_add(v, -f);
            if (fabsf(f) <= FLT_MAX) v = two_add(v, -__fmaf_rn(o.freq, nf, -f));  // (an infinite one has no residual)
            v = two_add(v, -o.pres);
        }
    }
    if (w & kBiased) {
        v = two_add(v, bias.h);
        v = two_add(v, bias.l);
    }
    const float s = __fadd_rn(v.h, v.l);
    // an infinite or NaN logit has no low part
    v = fabsf(s) <= FLT_MAX ? Two{s, __fadd_rn(__fsub_rn(v.h, s), v.l)} : Two{fabsf(v.h) <= FLT_MAX ? s : v.h, 0.f};
    if (slope) *slope = d;
    return v;
}

__device__ __forceinline__ void prefetch_l1(const void *p) { asm volatile("prefetch.global.L1 [%0];" ::"l"(p)); }

// Whether the row's mask lets a token through.
__device__ __forceinline__ bool ctl_allows(const CtlRow &o, int64_t token) {
    if (o.none) return false;
    return !o.mask || (__ldg(o.mask + token / 32) >> (token & 31) & 1u);
}

// ---- eight consecutive columns -----------------------------------------------------
template <bool kBf16>
struct Group8 {
    uint4 w[kBf16 ? 1 : 2];
};

template <bool kBf16>
__device__ __forceinline__ float ctl_elem(const char *row, int64_t j) {
    if constexpr (kBf16)
        return __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const unsigned short *>(row)[j]) << 16);
    else
        return reinterpret_cast<const float *>(row)[j];
}

// Columns [j, j + 8) of a row one by one, those outside [first, end) as 0.
template <bool kBf16>
__device__ __forceinline__ void ctl_gather8(const char *row, int64_t j, int64_t first, int64_t end, Group8<kBf16> &g) {
    uint32_t w[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const bool in = j + q >= first && j + q < end;
        if constexpr (kBf16) {
            const uint32_t b = in ? reinterpret_cast<const unsigned short *>(row)[j + q] : 0u;
            if (q & 1) w[q >> 1] |= b << 16;
            else w[q >> 1] = b;
        } else {
            w[q] = in ? reinterpret_cast<const uint32_t *>(row)[j + q] : 0u;
        }
    }
    g.w[0] = make_uint4(w[0], w[1], w[2], w[3]);
    if constexpr (!kBf16) g.w[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// Eight columns from shared memory at byte offset `at` of a stage.  kAligned:
// `at` is a multiple of 16.  Otherwise the 16-byte words around them, shifted:
// by two words, one word, half a word, as the offset's bits say (the same for
// every thread).
template <bool kBf16, bool kAligned>
__device__ __forceinline__ void ctl_shared8(const char *stage, uint32_t at, Group8<kBf16> &g) {
    constexpr int kHi = kBf16 ? 0 : 1;
    const uint4 *p = reinterpret_cast<const uint4 *>(stage + (at & ~15u));
    if constexpr (kAligned) {
        g.w[0] = p[0];
        if constexpr (!kBf16) g.w[kHi] = p[1];
        return;
    }
    constexpr int kN = kBf16 ? 4 : 8;  // words wanted
    uint32_t w[kN + 4];
#pragma unroll
    for (int q = 0; q < kN / 4 + 1; ++q) {
        const uint4 v = p[q];
        w[4 * q] = v.x;
        w[4 * q + 1] = v.y;
        w[4 * q + 2] = v.z;
        w[4 * q + 3] = v.w;
    }
    if (at & 8u) {
#pragma unroll
        for (int q = 0; q < kN + 2; ++q) w[q] = w[q + 2];
    }
    if (at & 4u) {
#pragma unroll
        for (int q = 0; q < kN + 1; ++q) w[q] = w[q + 1];
    }
    if (kBf16 && (at & 2u)) {
#pragma unroll
        for (int q = 0; q < kN; ++q) w[q] = __funnelshift_r(w[q], w[q + 1], 16);
    }
    g.w[0] = make_uint4(w[0], w[1], w[2], w[3]);
    if constexpr (!kBf16) g.w[kHi] = make_uint4(w[4], w[5], w[6], w[7]);
}

template <bool kBf16>
__device__ __forceinline__ void ctl_unpack8(const Group8<kBf16> &g, float *x) {
    if constexpr (kBf16) {
        const uint32_t ws[4] = {g.w[0].x, g.w[0].y, g.w[0].z, g.w[0].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            x[2 * q] = __uint_as_float(ws[q] << 16);
            x[2 * q + 1] = __uint_as_float(ws[q] & 0xffff0000u);
        }
    } else {
        const uint32_t ws[8] = {g.w[0].x, g.w[0].y, g.w[0].z, g.w[0].w, g.w[1].x, g.w[1].y, g.w[1].z, g.w[1].w};
#pragma unroll
        for (int q = 0; q < 8; ++q) x[q] = __uint_as_float(ws[q]);
    }
}

// Eight values as the words of an output group, each rounded once to its type.
template <bool kBf16>
__device__ __forceinline__ void ctl_pack8(const float *v, Group8<kBf16> &g) {
    uint32_t w[8];
    if constexpr (kBf16) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * q], v[2 * q + 1]);
            w[q] = *reinterpret_cast<const uint32_t *>(&h);
        }
        g.w[0] = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) w[q] = __float_as_uint(v[q]);
        g.w[0] = make_uint4(w[0], w[1], w[2], w[3]);
        g.w[kBf16 ? 0 : 1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// Entry b of the mask table: the 16-bit lanes of the columns whose bit is set.
__device__ __forceinline__ uint4 ctl_lanes(uint32_t b) {
    auto two = [&](int p) { return (b >> (2 * p) & 1u ? 0xffffu : 0u) | (b >> (2 * p + 1) & 1u ? 0xffff0000u : 0u); };
    return make_uint4(two(0), two(1), two(2), two(3));
}

// The group's columns whose bit is set replaced by the 16-bit pattern `fill`
// (of a float32 column: its upper half; the lower half becomes 0).
template <bool kBf16, uint32_t kFill>
__device__ __forceinline__ void ctl_fill8(Group8<kBf16> &g, const uint4 &m) {
    constexpr uint32_t k2 = kFill | kFill << 16, k1 = kFill << 16;
    if constexpr (kBf16) {
        g.w[0].x = (g.w[0].x & ~m.x) | (k2 & m.x);
        g.w[0].y = (g.w[0].y & ~m.y) | (k2 & m.y);
        g.w[0].z = (g.w[0].z & ~m.z) | (k2 & m.z);
        g.w[0].w = (g.w[0].w & ~m.w) | (k2 & m.w);
    } else {
        auto put = [&](uint32_t &w, uint32_t lane) { w = (w & ~lane) | (k1 & lane); };
        constexpr int kHi = kBf16 ? 0 : 1;
        put(g.w[0].x, __byte_perm(m.x, 0, 0x1010));
        put(g.w[0].y, __byte_perm(m.x, 0, 0x3232));
        put(g.w[0].z, __byte_perm(m.y, 0, 0x1010));
        put(g.w[0].w, __byte_perm(m.y, 0, 0x3232));
        put(g.w[kHi].x, __byte_perm(m.z, 0, 0x1010));
        put(g.w[kHi].y, __byte_perm(m.z, 0, 0x3232));
        put(g.w[kHi].z, __byte_perm(m.w, 0, 0x1010));
        put(g.w[kHi].w, __byte_perm(m.w, 0, 0x3232));
    }
}

// The columns of mask `m` taken from `from`, bit for bit.
template <bool kBf16>
__device__ __forceinline__ void ctl_keep8(Group8<kBf16> &g, const Group8<kBf16> &from, const uint4 &m) {
    auto put = [](uint32_t &w, uint32_t f, uint32_t lanes) { w = (w & ~lanes) | (f & lanes); };
    if constexpr (kBf16) {
        put(g.w[0].x, from.w[0].x, m.x);
        put(g.w[0].y, from.w[0].y, m.y);
        put(g.w[0].z, from.w[0].z, m.z);
        put(g.w[0].w, from.w[0].w, m.w);
    } else {
        auto wide = [](uint32_t two, int half) { return __byte_perm(two, 0, half ? 0x3232 : 0x1010); };
        constexpr int kHi = kBf16 ? 0 : 1;
        put(g.w[0].x, from.w[0].x, wide(m.x, 0));
        put(g.w[0].y, from.w[0].y, wide(m.x, 1));
        put(g.w[0].z, from.w[0].z, wide(m.y, 0));
        put(g.w[0].w, from.w[0].w, wide(m.y, 1));
        put(g.w[kHi].x, from.w[kHi].x, wide(m.z, 0));
        put(g.w[kHi].y, from.w[kHi].y, wide(m.z, 1));
        put(g.w[kHi].z, from.w[kHi].z, wide(m.w, 0));
        put(g.w[kHi].w, from.w[kHi].w, wide(m.w, 1));
    }
}

// Columns [j, j + 8) of an output row on a 16-byte boundary.
template <bool kBf16>
__device__ __forceinline__ void ctl_store8(char *row, int64_t j, const Group8<kBf16> &g) {
    uint4 *p = reinterpret_cast<uint4 *>(row + j * (kBf16 ? 2 : 4));
    __stcs(p, g.w[0]);
    if constexpr (!kBf16) __stcs(p + 1, g.w[kBf16 ? 0 : 1]);
}

// Those of columns [j, j + 8) that lie in [first, end), one by one.
template <bool kBf16>
__device__ __forceinline__ void ctl_scatter8(char *row, int64_t j, int64_t first, int64_t end, const Group8<kBf16> &g) {
    constexpr int kHi = kBf16 ? 0 : 1;
    const uint32_t w[8] = {g.w[0].x,   g.w[0].y,   g.w[0].z,   g.w[0].w,
                           g.w[kHi].x, g.w[kHi].y, g.w[kHi].z, g.w[kHi].w};
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        if (j + q >= first && j + q < end) {
            if constexpr (kBf16)
                reinterpret_cast<unsigned short *>(row)[j + q] = static_cast<unsigned short>(w[q >> 1] >> (16 * (q & 1)));
            else
                reinterpret_cast<uint32_t *>(row)[j + q] = w[q];
        }
    }
}

template <bool kBf16>
__device__ __forceinline__ void ctl_store1(char *row, int64_t j, float v) {
    if constexpr (kBf16) reinterpret_cast<__nv_bfloat16 *>(row)[j] = __float2bfloat16_rn(v);
    else reinterpret_cast<float *>(row)[j] = v;
}

}  // namespace lpd
