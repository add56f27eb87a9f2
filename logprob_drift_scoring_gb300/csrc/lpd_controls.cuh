// Sampling controls on logits: what the three control kernels (apply, score,
// gradient) share.
//
// For row r and token j with n_all = occurrences of j in the row's history,
// n_gen = those in its generated part, the controlled logit is
//   x1 = n_all > 0 ? (x > 0 ? x / rep : x * rep) : x
//   x2 = n_gen > 0 ? x1 - freq * n_gen - pres    : x1
//   x3 = x2 + sum of the row's biases of token j
//   z  = allowed(j) ? scale * x3 : -inf
// Only the tokens of the history and of the bias list ("touched" tokens) need
// more than the scale and the mask, and they are few: a thousand of a hundred
// thousand.  A block therefore takes a chunk of one row, marks the touched
// columns of the chunk in a bitmap, lists them in column order, and works on
// the list with all lanes busy: a touched token is some 80 instructions, which
// a branch in the streaming loop would spend for a whole warp each time.  The
// streaming loop sees one bit a column.
//
// The occurrence counts live in a table of one word a column of the chunk.  The
// table is zero between units: whoever consumes a touched entry zeroes it, so
// the chunk is cleared once a block and not once a unit.
//
// Masked columns are replaced eight at a time: a 4 KB table in shared memory
// gives the 16-bit lane masks of a byte of bits, and one logical instruction a
// register does the rest (bit tests and selects were 100 instructions a thread
// and 16 columns, a third of the scoring kernel's).
//
// The list is made from the bitmap by a prefix sum over its words, never in the
// order of arrival, and the counts are integers, so nothing depends on the
// order of the shared-memory atomics.
#pragma once

#include <cuda_bf16.h>
#include <math_constants.h>

#include "lpd_acc.cuh"
#include "lpd_internal.cuh"

namespace lpd {

constexpr int kCtlThreads = 256;
constexpr int kCtlWarps = kCtlThreads / 32;
constexpr uint32_t kSeen = 0x80000000u;    // table: the token occurs in the prompt part
constexpr uint32_t kBiased = 0x40000000u;  // table: the token has a bias entry
constexpr uint32_t kCount = 0x3fffffffu;   // table: occurrences in the generated part
constexpr int64_t kMaxRange = kCount;      // so a row's range is cut to its last 2^30 - 1 tokens

// The controls of one row: read once a unit by one thread, kept in shared
// memory (in registers, two of them spilled a quarter of the scoring kernel's).
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

// Sum of the row's bias entries of one token, in double (at most 1024 terms,
// so the sum is exact to far below a float's step in any order).
__device__ __forceinline__ double bias_sum(const CtlSide &c, int64_t r, int64_t token) {
    const int32_t *ids = c.bias_ids + r * c.n_bias;
    const float *v = c.bias + r * c.n_bias;
    double s = 0.0;
#pragma unroll 8
    for (int e = 0; e < c.n_bias; ++e)
        if (ids[e] == token) s += static_cast<double>(v[e]);
    return s;
}

// x3 of a touched, allowed token with table word w.  Two floats, so that the
// logit's rounding (a step of 1e-6 at a logit of 20) stays out of the logprob
// difference of two sides that nearly agree; `slope` (may be null) receives
// dx3/dx.
__device__ __forceinline__ Two ctl_value(float x, uint32_t w, const CtlSide &c, const CtlRow &o, int64_t r,
                                         int64_t token, float *slope) {
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
            v = two_add(v, -__fmaf_rn(o.freq, nf, -f));
            v = two_add(v, -o.pres);
        }
    }
    if (w & kBiased) {
        const double b = bias_sum(c, r, token);
        const float bh = static_cast<float>(b);
        v = two_add(v, bh);
        v = two_add(v, static_cast<float>(b - static_cast<double>(bh)));
    }
    const float s = __fadd_rn(v.h, v.l);
    // an infinite or NaN logit has no low part
    v = fabsf(s) <= FLT_MAX ? Two{s, __fadd_rn(__fsub_rn(v.h, s), v.l)} : Two{fabsf(v.h) <= FLT_MAX ? s : v.h, 0.f};
    if (slope) *slope = d;
    return v;
}

// ---- the unit: one chunk of one row ----------------------------------------------
// Marks the chunk's touched columns: table words and bitmap bits.  `id_word`
// (shared, may be null) collects the word of token `id` over the whole row.
__device__ __forceinline__ void ctl_mark(const CtlSide &c, const CtlRow &o, int64_t r, int64_t c0, uint32_t len,
                                         volatile uint32_t *vtable, volatile uint32_t *vtouched, int64_t id, uint32_t *id_word) {
    uint32_t *const table = const_cast<uint32_t *>(vtable), *const touched = const_cast<uint32_t *>(vtouched);
    auto take = [&](int32_t tok, bool gen) {
        const uint64_t j = static_cast<uint64_t>(static_cast<int64_t>(tok) - c0);
        if (j < len) {
            if (gen) atomicAdd(&table[j], 1u);
            else if (!(vtable[j] & kSeen)) atomicOr(&table[j], kSeen);  // (a text's frequent tokens come often)
            const uint32_t bit = 1u << (j & 31);
            if (!(vtouched[j >> 5] & bit)) atomicOr(&touched[j >> 5], bit);
        }
        if (id_word && tok == id) {
            if (gen) atomicAdd(id_word, 1u);
            else atomicOr(id_word, kSeen);
        }
    };
    constexpr int kU = 4;  // independent loads in flight
    int64_t k = o.begin + threadIdx.x;
    for (; k + (kU - 1) * kCtlThreads < o.end; k += kU * kCtlThreads) {
        int32_t t[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) t[u] = __ldg(c.history + k + u * kCtlThreads);
#pragma unroll
        for (int u = 0; u < kU; ++u) take(t[u], k + u * kCtlThreads >= o.split);
    }
    for (; k < o.end; k += kCtlThreads) take(__ldg(c.history + k), k >= o.split);
    for (int e = threadIdx.x; e < c.n_bias; e += kCtlThreads) {
        const int32_t tok = __ldg(c.bias_ids + r * c.n_bias + e);
        const uint64_t j = static_cast<uint64_t>(static_cast<int64_t>(tok) - c0);
        if (j < len) {
            atomicOr(&table[j], kBiased);
            atomicOr(&touched[j >> 5], 1u << (j & 31));
        }
        if (id_word && tok == id) atomicOr(id_word, kBiased);
    }
}

// Word w of the row's allowed bits for the chunk at column c0 (a multiple of
// 32), columns from the vocabulary's end on not allowed.
__device__ __forceinline__ uint32_t ctl_allowed(const CtlRow &o, int64_t c0, int w, int64_t vocab) {
    const int64_t first = c0 + 32 * static_cast<int64_t>(w);
    if (first >= vocab || o.none) return 0u;
    const uint32_t bits = o.mask ? __ldg(o.mask + first / 32) : 0xffffffffu;
    const int64_t left = vocab - first;
    return left >= 32 ? bits : bits & ((1u << left) - 1u);
}

// The touched columns in ascending order: thread t holds word t of the bitmap
// (0 behind the chunk's words).  Returns their number; the list is visible
// after the caller's next __syncthreads.
__device__ __forceinline__ int ctl_list(uint32_t bits, uint16_t *list, int *warp_sum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n = __popc(bits);
    int incl = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += y;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int base = 0, total = 0;
#pragma unroll
    for (int k = 0; k < kCtlWarps; ++k) {
        const int s = warp_sum[k];
        base += k < warp ? s : 0;
        total += s;
    }
    int pos = base + incl - n;
    while (bits) {
        const int b = __ffs(bits) - 1;
        bits &= bits - 1;
        list[pos++] = static_cast<uint16_t>(threadIdx.x * 32 + b);
    }
    return total;
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

// Columns [j, j + 8) of a row as raw words, columns from `vocab` on as 0.
// kVec: rows start on 16-byte boundaries.
template <bool kBf16, bool kVec>
__device__ __forceinline__ void ctl_load8(const char *row, int64_t j, int64_t vocab, Group8<kBf16> &g) {
    if (kVec && j + 8 <= vocab) {
        const uint4 *p = reinterpret_cast<const uint4 *>(row + j * (kBf16 ? 2 : 4));
        g.w[0] = __ldcs(p);
        if constexpr (!kBf16) g.w[1] = __ldcs(p + 1);
        return;
    }
    uint32_t w[kBf16 ? 4 : 8];
    if constexpr (kBf16) {
        // inside the row: whole words, shifted by half a word where the row
        // starts on an odd element
        const uintptr_t at = reinterpret_cast<uintptr_t>(row + 2 * j);
        if (j > 0 && j + 9 <= vocab) {
            const uint32_t *p = reinterpret_cast<const uint32_t *>(at & ~uintptr_t{3});
            if (at & 2) {
                uint32_t v[5];
#pragma unroll
                for (int q = 0; q < 5; ++q) v[q] = p[q];
#pragma unroll
                for (int q = 0; q < 4; ++q) w[q] = __funnelshift_r(v[q], v[q + 1], 16);
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) w[q] = p[q];
            }
            g.w[0] = make_uint4(w[0], w[1], w[2], w[3]);
            return;
        }
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        if constexpr (kBf16) {
            const uint32_t b = j + q < vocab ? reinterpret_cast<const unsigned short *>(row)[j + q] : 0u;
            if (q & 1) w[q >> 1] |= b << 16;
            else w[q >> 1] = b;
        } else {
            w[q] = j + q < vocab ? reinterpret_cast<const uint32_t *>(row)[j + q] : 0u;
        }
    }
    g.w[0] = make_uint4(w[0], w[1], w[2], w[3]);
    if constexpr (!kBf16) g.w[1] = make_uint4(w[4], w[5], w[6], w[7]);
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

// Columns [j, j + 8) of an output row.
template <bool kBf16, bool kVec>
__device__ __forceinline__ void ctl_store8(char *row, int64_t j, int64_t vocab, const Group8<kBf16> &g) {
    constexpr int kHi = kBf16 ? 0 : 1;
    if (kVec && j + 8 <= vocab) {
        uint4 *p = reinterpret_cast<uint4 *>(row + j * (kBf16 ? 2 : 4));
        __stcs(p, g.w[0]);
        if constexpr (!kBf16) __stcs(p + 1, g.w[kHi]);
        return;
    }
    const uint32_t w[8] = {g.w[0].x,   g.w[0].y,   g.w[0].z,   g.w[0].w,
                           g.w[kHi].x, g.w[kHi].y, g.w[kHi].z, g.w[kHi].w};
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        if (j + q < vocab) {
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
