// Token sampling under temperature, min-p, top-k and top-p, and the kept sets of
// such filters as bit masks.
//
// For a row with z = scale x the filters leave a set that is always a prefix of
// the row in descending order (ties by index), so it is described by the key T of
// its last value and by how many of the tokens at T belong to it.  T is the
// border of a weighted selection: the k-th largest value, or the first value at
// which the mass in front of it reaches top_p of the whole.  A draw is the first
// kept token, in index order, whose running mass passes u W.
//
// Masses are whole numbers (lpd_weights.cuh), so neither the order of the atomics nor the
// number of CTAs that share a row changes a bit of the answer; three ways to it exist:
//
// - Few rows: a cluster of CTAs a row, each holding a slice in shared memory, so that the
//   row is read once and all of its tokens are at hand (cluster_row).  A row whose border is
//   in the list takes five barriers of the cluster, and then one CTA's selections (pick: one
//   for a top-k, one for a top-p, one for the draw, each up to four turns of five barriers
//   for some hundred entries), a row alone all of them one after the other: one row of
//   128256 float32 takes 13.5 us for the mask of a top-k, 17 for a draw under it, 18.5 under
//   a top-p too.
// - Many rows: a CTA a row, the row streamed (row_kernel).  Under a small top-k or a
//   min-p the largest tokens are collected against a value that a sample of the row gave:
//   4096 rows (3687 of them active) x 151936 bf16 in 293 us, 4.1 TB/s of 6.8; the pass
//   over the row takes three quarters of that, with 48 warps a multiprocessor and 96 KB
//   in flight, the selections behind it the rest.  A bf16 row under any other filter is
//   counted by value (counted_row).  Rows of 151936 go in rounds of 304, two a
//   multiprocessor: 304 take 92 us under a temperature and 57 under a top-p, 305 take 135
//   and 81, a row alone 61 and 41.  A row's passes follow one another: the counting (24 us
//   alone, an atomic in shared memory a token), the bins, and the list's or, for a draw from
//   many tokens, a table look-up a token.  A float32 row of which all is kept is weighed
//   token by token (plain_row), 30 operations each.
// - What is left of many rows (a nucleus beyond the list in float32, ties without end)
//   goes to clusters behind them.
//
// In every way the border is found by bins: tokens (or their mass) added up in 256 bins
// over the range of their keys, the bin that holds the border cut in 256 again, until it
// holds one key.
#include <algorithm>
#include <cfloat>
#include <cooperative_groups.h>
#include <type_traits>
#include <cuda_bf16.h>
#include <math_constants.h>

#include "lpd_internal.cuh"
#include "lpd_operators.cuh"
#include "lpd_weights.cuh"

namespace cg = cooperative_groups;

namespace lpd {
namespace {

constexpr int kBins = 256;
constexpr int kList = 512;          // candidates a CTA of a cluster keeps
constexpr int kReach = 512;         // thread maxima of a cluster that a nucleus's candidates go down to
constexpr int kMaxWarps = 32;
constexpr float kPreciseOctaves = 8.f;  // tokens within this of the top are weighed more exactly

// 2^(i / 256), by the series of exp around 0 (the argument is below 0.7).
constexpr double series_exp(double x) {
    double term = 1, sum = 1;
    for (int n = 1; n < 24; ++n) {
        term *= x / n;
        sum += term;
    }
    return sum;
}
struct Tables {
    uint64_t precise[kUnits];
    WeightEntry rough[kUnits];
};
constexpr Tables make_tables() {
    Tables t{};
    for (int i = 0; i < kUnits; ++i) {
        const double v = series_exp(kLn2Unit * i);
        t.precise[i] = static_cast<uint64_t>(v * 4611686018427387904.0);
        t.rough[i].whole = static_cast<uint32_t>(v * 1073741824.0 + 0.5);
        t.rough[i].part = static_cast<float>(v * 1073741824.0);
    }
    return t;
}
__device__ constexpr Tables kTables = make_tables();

// From so many rows on a CTA takes a row alone (and clusters what it leaves).  64 x 151936
// bf16 under any filters take 83 us so and 97 us with clusters, 32 take 74 and 41; 152
// of float32 146 and 148 (under a top-k 40 and 112), 64 take 139 and 76.  On the two sides
// of the rule, under a temperature / a top-k of 50: 63 and 64 rows of 1024 bf16 19 and 21 /
// 26 and 17 us, of 37984 31 and 32 / 17 and 18; 127 and 128 of 1024 float32 15 and 13 / 13
// and 16, of 37984 38 and 29 / 21 and 18, of 151936 133 and 73 / 78 and 28.
constexpr int kAloneBf16 = 64, kAloneF32 = 128;
constexpr int kTopList = 2048;      // candidates of a row that a CTA has alone
constexpr int kTopMost = 512;       // the largest top-k that such a CTA takes
constexpr float kListShare = 48.f;  // the sampled tokens that a list goes down to without a top-k

// What finding a border takes: bins, and the CTA's sums.
struct Scratch {
    uint32_t cnt[2][kBins], mass_lo[2][kBins], mass_hi[2][kBins], far[2][kBins];
    uint64_t red64[2][kMaxWarps];
    uint32_t red32[2][kMaxWarps];
    uint64_t found_mass, found_excl_mass;
    uint32_t found_bin, found_cnt, found_excl, found_far, found_before;
    double log_min_p;
    float base;
};

// Keys in the order of the values; -0 and +0 share one.  bf16 rows have 16-bit keys.
template <bool kBf16>
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = __float_as_uint(__fadd_rn(x, 0.f));
    const uint32_t k = u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
    return kBf16 ? k >> 16 : k;
}
template <bool kBf16>
__device__ __forceinline__ float value_of(uint32_t key) {
    if (kBf16) {
        const uint32_t u = (key & 0x8000u) ? key ^ 0x8000u : key ^ 0xffffu;
        return __uint_as_float(u << 16);
    }
    return __uint_as_float((key & 0x80000000u) ? key ^ 0x80000000u : ~key);
}

template <bool kBf16>
__device__ __forceinline__ void unpack(const uint4 &c, float *v) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if constexpr (kBf16) {
            v[2 * q] = __uint_as_float(w[q] << 16);
            v[2 * q + 1] = __uint_as_float(w[q] & 0xffff0000u);
        } else {
            v[q] = __uint_as_float(w[q]);
        }
    }
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint32_t max_nan2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// The largest value of a chunk, NaN if one is.
template <bool kBf16>
__device__ __forceinline__ float chunk_max(const uint4 &c) {
    if constexpr (kBf16) {
        const uint32_t m = max_nan2(max_nan2(c.x, c.y), max_nan2(c.z, c.w));
        return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
    } else {
        return max_nan(max_nan(__uint_as_float(c.x), __uint_as_float(c.y)), max_nan(__uint_as_float(c.z), __uint_as_float(c.w)));
    }
}

template <class T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ void add_mass(Scratch &sh, int buf, uint32_t b, uint64_t w) {
    const uint32_t lo = static_cast<uint32_t>(w), old = atomicAdd(&sh.mass_lo[buf][b], lo);
    const uint32_t hi = static_cast<uint32_t>(w >> 32) + (old + lo < old);
    if (hi) atomicAdd(&sh.mass_hi[buf][b], hi);
}
// Two masses and a number summed over the CTA, for every thread.
template <int kThreads>
__device__ __forceinline__ void block_sums(Scratch &sh, uint64_t &v, uint64_t &w, uint32_t &c) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    v = warp_sum(v);
    w = warp_sum(w);
    c = __reduce_add_sync(0xffffffffu, c);
    __syncthreads();
    if (lane == 0) {
        sh.red64[0][warp] = v;
        sh.red64[1][warp] = w;
        sh.red32[0][warp] = c;
    }
    __syncthreads();
    v = w = 0;
    c = 0;
#pragma unroll
    for (int q = 0; q < kThreads / 32; ++q) {
        v += sh.red64[0][q];
        w += sh.red64[1][q];
        c += sh.red32[0][q];
    }
}

// Chunk e of a row whose elements [lead, end) are its own: the others read as -inf
// (nothing is read outside the row's memory).
template <bool kBf16>
__device__ __forceinline__ uint4 edge_chunk(const uint4 *from, int e, int lead, int end) {
    constexpr int kPer = kBf16 ? 8 : 4;
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
        const int j = e * kPer + q;
        const bool in = j >= lead && j < end;
        if constexpr (kBf16) {
            const uint32_t b = in ? reinterpret_cast<const unsigned short *>(from)[j] : 0xff80u;
            if (q & 1) w[q >> 1] |= b << 16;
            else w[q >> 1] = b;
        } else {
            w[q] = in ? reinterpret_cast<const uint32_t *>(from)[j] : 0xff800000u;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

struct SampleArgs {
    const char *x;
    int64_t x_stride;  // bytes
    int64_t n_rows;
    int vocab, slice, chunk_room;
    FilterParams f;
    const float *uniform;
    int32_t *ids;
    float *logp;
    const int32_t *keep;
    const uint8_t *active;
    uint32_t *mask;
    int64_t mask_stride;
    float *lse;
    int32_t *kept;
    int after_rows;    // the row kernel has been there: only what it left is to do
};
// What the row kernel puts into a row's first word of output where it leaves
// the row to the other kernel (a mask that begins like this is found a second time).
constexpr int32_t kLeftId = -2;
constexpr uint32_t kLeftMask = 0xa5a5c3c3u;

// One row's parameters.
struct RowFilter {
    float scale, min_p, top_p;
    int top_k;
    bool active, valid, use_k, use_p;
};
__device__ __forceinline__ RowFilter filter_of(const SampleArgs &a, int64_t row) {
    RowFilter f;
    f.active = !a.active || a.active[row] != 0;
    f.scale = a.f.scale ? a.f.scale[row] : 1.f;
    f.min_p = a.f.min_p ? a.f.min_p[row] : 0.f;
    f.top_p = a.f.top_p ? a.f.top_p[row] : 1.f;
    f.top_k = a.f.top_k ? a.f.top_k[row] : 0;
    f.valid = f.scale > 0.f && f.scale <= FLT_MAX && f.min_p == f.min_p && f.top_p == f.top_p;
    f.use_k = f.top_k > 0 && f.top_k < a.vocab;
    f.use_p = f.top_p < 1.f;
    return f;
}
// A row without an answer.
template <bool kMask>
__device__ __forceinline__ void no_answer(const SampleArgs &a, int64_t row, float value) {
    if (a.kept) a.kept[row] = 0;
    if constexpr (kMask) {
        if (a.lse) a.lse[row] = value;
    } else {
        a.ids[row] = -1;
        if (a.logp) a.logp[row] = value;
    }
}

// What min-p leaves: x >= base, the smallest value with (x - top) scale >= log(min_p).
// (Doubles are slow here: one thread's work; its logarithm was taken under the loads.)
template <bool kBf16>
__device__ __forceinline__ float base_of(Scratch &sh, const RowFilter &f, float top) {
    float base = -FLT_MAX;
    if (f.min_p > 0.f) {
        if (threadIdx.x == 0) {
            const double lp = sh.log_min_p, s = f.scale, tp = top;
            float v = static_cast<float>(fmax(tp + lp / s, -static_cast<double>(FLT_MAX)));
            for (int i = 0; i < 4 && !((static_cast<double>(v) - tp) * s >= lp); ++i) v = nextafterf(v, CUDART_INF_F);
            for (int i = 0; i < 4; ++i) {
                const float g = nextafterf(v, -CUDART_INF_F);
                if (!((static_cast<double>(g) - tp) * s >= lp) || !(g >= -FLT_MAX)) break;
                v = g;
            }
            sh.base = fminf(v, top);
        }
        __syncthreads();
        base = sh.base;
    }
    if constexpr (kBf16) {  // up to a bf16 value, so that its key is its own
        const float down = __uint_as_float(__float_as_uint(base) & 0xffff0000u);
        base = down < base ? __uint_as_float((__float_as_uint(base) & 0xffff0000u) + 0x10000u) : down;
    }
    return base;
}
template <bool kBf16>
__device__ __forceinline__ float floor_of(uint32_t key) {
    return key == 0xffffffffu ? CUDART_INF_F : key <= key_of<kBf16>(-FLT_MAX) ? -FLT_MAX : value_of<kBf16>(key);
}

// The row's weights: those near the top more exactly (in wide rows all).
struct Weigh {
    WeightScale ws;
    float top, precise_from;
    const WeightEntry *table;
    __device__ __forceinline__ Weigh(float scale, float row_top, const WeightEntry *t) : ws(weight_scale(scale, row_top)), top(row_top), table(t) {
        precise_from = ws.wide ? -FLT_MAX : top - __fdiv_rn(kPreciseOctaves * kUnits, ws.ch);
    }
    __device__ __forceinline__ uint64_t operator()(float x) const {
        if (x >= precise_from) return weight_precise(x, ws, top, kTables.precise);
        return x > ws.cut ? weight_rough(x, ws, table) : 0;
    }
    // log of the share that the token x has of the mass.  (Of more than a half it comes
    // from what the others have: a token alone has 0, and next to 1 nothing cancels.)
    __device__ __forceinline__ double logp(float x, uint64_t mass, float scale) const {
        const uint64_t own = (*this)(x);
        if (own > mass / 2) return -log1p(static_cast<double>(mass - own) / static_cast<double>(own));
        return static_cast<double>(x) * scale - lse(mass, scale);
    }
    // log of the sum that the mass stands for
    __device__ __forceinline__ double lse(uint64_t mass, float scale) const {
        const double origin = ws.wide ? static_cast<double>(top) * scale : ws.origin * kLn2Unit;
        return origin + log(static_cast<double>(mass) * (1.0 / static_cast<double>(uint64_t{1} << kWeightOne)));
    }
};
// The least mass that is top_p of the whole, at least 1.
__device__ __forceinline__ uint64_t share_of(float top_p, uint64_t whole) {
    const double want = ceil(fmax(static_cast<double>(top_p), 0.0) * static_cast<double>(whole));
    return min(max(static_cast<uint64_t>(want), static_cast<uint64_t>(1)), whole);
}
// Whether the draw is the first or the last kept token.  That goes by their number: a kept token
// may weigh less than a step and so nothing.
__device__ __forceinline__ bool at_an_end(float u) { return !(u > 0.f) || u >= 1.f; }
__device__ __forceinline__ uint64_t end_of(float u, uint64_t kept_n) { return u > 0.f ? kept_n - 1 : 0; }
// The draw's place in the running mass: the first token that passes it.
__device__ __forceinline__ uint64_t place_of(float u, uint64_t mass) {
    const uint64_t at = u > 0.f ? static_cast<uint64_t>(static_cast<double>(fminf(u, 1.f)) * static_cast<double>(mass)) : 0;
    return min(at, mass - 1);
}

// ---------------------------------------------------------------- rows whose border is in a list
struct Picked {
    uint32_t at, cnt;
    uint64_t under_n, under_mass, mass;
};
// The first position, from `lo` on, at which the entries' number (or mass) reaches
// `target`; place(i, &position) says whether entry i counts.  A CTA's work.
template <int kThreads, class Place>
__device__ Picked pick(Scratch &sh, const uint64_t *w_of, uint32_t total, Place place, uint32_t lo, uint32_t hi, bool by_mass, uint64_t target) {
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    Picked got{};
#pragma unroll 1
    for (int turn = 0;; ++turn) {  // (32 bits of range are four turns)
        const int shift = max(0, 24 - __clz((hi - lo) | 1u));
        for (int b = t; b < kBins; b += kThreads) sh.cnt[0][b] = sh.mass_lo[0][b] = sh.mass_hi[0][b] = 0;
        __syncthreads();
        for (uint32_t i = t; i < total; i += kThreads) {
            uint32_t at;
            if (place(i, &at) && at >= lo && at <= hi) {
                const uint32_t b = (at - lo) >> shift;
                atomicAdd(&sh.cnt[0][b], 1u);
                sh.far[0][b] = at;  // (read where it is the only one)
                add_mass(sh, 0, b, w_of[i]);
            }
        }
        __syncthreads();
        uint32_t up_n = 0;
        uint64_t up_mass = 0, mass = 0;
        uint32_t cnt = 0;
        if (t < kBins) {
            up_n = cnt = sh.cnt[0][t];
            up_mass = mass = static_cast<uint64_t>(sh.mass_hi[0][t]) << 32 | sh.mass_lo[0][t];
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t pn = __shfl_up_sync(0xffffffffu, up_n, o);
            const uint64_t pm = __shfl_up_sync(0xffffffffu, up_mass, o);
            if (lane >= o) {
                up_n += pn;
                up_mass += pm;
            }
        }
        if (lane == 31) {
            sh.red32[0][warp] = up_n;
            sh.red64[0][warp] = up_mass;
        }
        __syncthreads();
        if (t < kBins) {
            for (int w = 0; w < warp; ++w) {
                up_n += sh.red32[0][w];
                up_mass += sh.red64[0][w];
            }
            const uint64_t upto = by_mass ? got.under_mass + up_mass : got.under_n + up_n;
            const uint64_t under = upto - (by_mass ? mass : cnt);
            if (under < target && upto >= target) {
                sh.found_bin = t;
                sh.found_cnt = cnt;
                sh.found_mass = mass;
                sh.found_excl = up_n - cnt;
                sh.found_excl_mass = up_mass - mass;
            }
        }
        __syncthreads();
        const uint32_t fb = sh.found_bin;
        got.under_n += sh.found_excl;
        got.under_mass += sh.found_excl_mass;
        got.cnt = sh.found_cnt;
        got.mass = sh.found_mass;
        if (shift == 0 || got.cnt == 1 || turn == 4) {
            got.at = shift == 0 ? lo + fb : sh.far[0][fb];
            __syncthreads();
            return got;
        }
        lo += fb << shift;
        hi = min(hi, lo + ((1u << shift) - 1));
        __syncthreads();
    }
}

// The answer from the list, once the border is known: kept are the entries whose `far`
// lies below the border's, and the first `ties` of the `ties_all` tokens at it.
template <bool kBf16, bool kMask, int kThreads>
__device__ __forceinline__ void answer_list(const SampleArgs &a, int64_t row, const RowFilter &f, Scratch &sh, const Weigh &weight, uint32_t top_key, float cand,
                            uint32_t total, const uint64_t *w_of, const uint32_t *far_of, const uint32_t *id_of, uint32_t border,
                            uint32_t ties, uint32_t ties_all, uint64_t kept_n, uint64_t kept_mass) {
    const int t = threadIdx.x;
    uint32_t last_id = 0xffffffffu;  // the last token at the border that is kept
    if (ties < ties_all) {
        const auto at_border = [&](uint32_t i, uint32_t *p) {
            *p = id_of[i];
            return far_of[i] == border;
        };
        last_id = pick<kThreads>(sh, w_of, total, at_border, 0, a.vocab - 1, false, ties).at;
    }
    const auto is_kept = [&](uint32_t far, uint32_t id) { return far < border || (far == border && id <= last_id); };
    if constexpr (kMask) {
        uint32_t *const words_of = a.mask + row * a.mask_stride;
        for (uint32_t i = t; i < total; i += kThreads)
            if (is_kept(far_of[i], id_of[i])) atomicOr(words_of + id_of[i] / 32, 1u << (id_of[i] % 32));
        if (t == 0) {
            const int64_t id = a.keep ? a.keep[row] : -1;
            if (id >= 0 && id < a.vocab) {
                const char *from = a.x + row * a.x_stride + id * (kBf16 ? 2 : 4);
                const float x = kBf16 ? __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const unsigned short *>(from)) << 16)
                                      : *reinterpret_cast<const float *>(from);
                // (below the list's values, or at -inf, it is not kept by the filter)
                if (x >= -FLT_MAX && !(x >= cand && is_kept(top_key - key_of<kBf16>(x), static_cast<uint32_t>(id)))) {
                    kept_n += 1;
                    kept_mass += weight(x);
                    atomicOr(words_of + id / 32, 1u << (id % 32));
                }
            }
            if (a.kept) a.kept[row] = static_cast<int32_t>(kept_n);
            if (a.lse) a.lse[row] = static_cast<float>(weight.lse(kept_mass, f.scale));
        }
    } else {
        const float u = a.uniform[row];
        const auto at_kept = [&](uint32_t i, uint32_t *p) {
            *p = id_of[i];
            return is_kept(far_of[i], id_of[i]);
        };
        const bool end = at_an_end(u);
        const uint32_t id = pick<kThreads>(sh, w_of, total, at_kept, 0, a.vocab - 1, !end, (end ? end_of(u, kept_n) : place_of(u, kept_mass)) + 1).at;
        for (uint32_t i = t; i < total; i += kThreads)
            if (id_of[i] == id) {
                const float x = value_of<kBf16>(top_key - far_of[i]);
                const bool drawn = u == u;
                a.ids[row] = drawn ? static_cast<int32_t>(id) : -1;
                if (a.logp) a.logp[row] = drawn ? static_cast<float>(weight.logp(x, kept_mass, f.scale)) : CUDART_NAN_F;
                if (a.kept) a.kept[row] = static_cast<int32_t>(kept_n);
            }
    }
}

// The filter and its answer from a list of the row's candidates: w_of, far_of (how far
// their keys lie below the top's) and id_of (tokens), all of the tokens at `cand` and above.
// all_mass: what min-p leaves (not needed under a top-k).
template <bool kBf16, bool kMask, int kThreads>
__device__ void finish_list(const SampleArgs &a, int64_t row, const RowFilter &f, Scratch &sh, const Weigh &weight, uint32_t top_key, float cand,
                            uint32_t total, const uint64_t *w_of, const uint32_t *far_of, const uint32_t *id_of, uint64_t list_mass, uint64_t all_mass) {
    const int t = threadIdx.x;
    uint32_t border = 0xffffffffu;
    uint64_t kept_n = total, kept_mass = 0;
    uint32_t ties = 0, ties_all = 0;
    const uint32_t deepest = top_key - key_of<kBf16>(fminf(cand, weight.top));
    const auto at_far = [&](uint32_t i, uint32_t *p) {
        *p = far_of[i];
        return true;
    };
    uint64_t whole_mass = list_mass;
    if (f.use_k && total <= static_cast<uint32_t>(f.top_k)) {  // nothing to leave out
        uint64_t none = 0;
        uint32_t c = 0;
        for (uint32_t i = t; i < total; i += kThreads) whole_mass += w_of[i];
        block_sums<kThreads>(sh, whole_mass, none, c);
    }
    if (f.use_k && total > static_cast<uint32_t>(f.top_k)) {
        const Picked p = pick<kThreads>(sh, w_of, total, at_far, 0, deepest, false, f.top_k);
        border = p.at;
        ties = static_cast<uint32_t>(f.top_k - p.under_n);
        ties_all = p.cnt;
        kept_n = f.top_k;
        kept_mass = p.under_mass + ties * (p.mass / p.cnt);  // (one weight p.cnt times)
    }
    if (f.use_p) {
        const uint64_t target = share_of(f.top_p, !f.use_k ? all_mass : ties_all ? kept_mass : whole_mass);
        const Picked p = pick<kThreads>(sh, w_of, total, at_far, 0, min(border, deepest), true, target);
        const uint64_t one = p.mass / p.cnt;
        border = p.at;
        ties = static_cast<uint32_t>((target - p.under_mass + one - 1) / one);
        ties_all = p.cnt;
        kept_n = p.under_n + ties;
        kept_mass = p.under_mass + ties * one;
    }
    if (ties_all == 0) kept_mass = whole_mass;
    answer_list<kBf16, kMask, kThreads>(a, row, f, sh, weight, top_key, cand, total, w_of, far_of, id_of, border, ties, ties_all, kept_n, kept_mass);
}

// ------------------------------------------------------------------ many rows, a CTA each
// Bins of a bf16 row, one for each value of 24 octaves and both signs, in descending
// order: +2^14 down to +2^-10, what lies between 2^-10 and 0 (a bin of several values),
// 0 itself, the same below 0, and the finite values from -2^14 down (another).
constexpr int kOctaves = 24, kLowest = 117;             // octaves, and the first one's exponent field
constexpr int kSide = kOctaves * 128;
constexpr int kTinyUp = kSide, kZero = kSide + 1, kTinyDown = kSide + 2, kDown = kSide + 3, kLow = 2 * kSide + 3;
constexpr int kValues = 2 * kSide + 4;
constexpr int kTinyRoom = 1024;
__device__ __forceinline__ float bin_value(int b) {  // of a bin of one value
    const uint32_t up = static_cast<uint32_t>(kSide - 1 - b + (kLowest << 7)) << 16;
    const uint32_t down = static_cast<uint32_t>(b - kDown + (kLowest << 7)) << 16 | 0x80000000u;
    return b == kZero ? 0.f : __uint_as_float(b < kSide ? up : down);
}

constexpr int kRowThreads = 512;
constexpr int kOwnBins = (kValues + kRowThreads - 1) / kRowThreads | 1;  // a thread's (odd: no bank conflicts)
struct RowShared {
    Scratch scratch;
    WeightEntry table[kUnits];
    uint4 edge[2];
    union {
        uint32_t bins[kOwnBins * kRowThreads];
        struct {
            uint64_t w[kTopList];
            uint32_t key[kTopList], at[kTopList];
        } list;
        uint64_t value_w[kValues];     // the weights of the bins' values, 0 where they are not kept
    };
    uint16_t tiny[kTinyRoom];          // the bits of values within 2^-10 of 0
    uint64_t part[kMaxWarps];
    uint32_t list_n, floor_key, tiny_n;
    int leave, at;
    // the border
    uint64_t above_mass, one;
    uint32_t above_n, ties_all, border;
};

// The chunks of a row that a CTA has alone.
template <bool kBf16>
struct RowChunks {
    static constexpr int kElt = kBf16 ? 2 : 4, kPer = 16 / kElt, kAhead = 4;
    const uint4 *from;
    const uint4 *edge;
    int lead, end, n, c0, c1;  // whole chunks: [c0, c1)
    __device__ __forceinline__ RowChunks(const SampleArgs &a, int64_t row, uint4 *edges) {
        const char *const src = a.x + row * a.x_stride;
        lead = static_cast<int>((reinterpret_cast<uintptr_t>(src) & 15u) / kElt);  // elements of the first chunk in front of the row
        end = lead + a.vocab;
        n = (end + kPer - 1) / kPer;
        from = reinterpret_cast<const uint4 *>(src - lead * kElt);
        c0 = lead > 0 ? 1 : 0;
        c1 = max(c0, end / kPer);
        edge = edges;
        if (threadIdx.x < 2) edges[threadIdx.x] = edge_chunk<kBf16>(from, threadIdx.x == 0 ? 0 : n - 1, lead, end);
    }
    // whether thread 0 (1) has the first (last) chunk to itself, being a part of it only
    __device__ __forceinline__ bool has_edge() const {
        return (threadIdx.x == 0 && c0 == 1) || (threadIdx.x == 1 && n > c1 && n - 1 >= c0);
    }
    __device__ __forceinline__ uint4 at(int i) const { return i >= c0 && i < c1 ? __ldg(from + i) : edge[i == 0 ? 0 : 1]; }
    template <class G>
    __device__ __forceinline__ void each(G g) const {  // g(chunk, its number), the CTA side by side
        int i = c0 + threadIdx.x;
        for (; i + (kAhead - 1) * kRowThreads < c1; i += kAhead * kRowThreads) {
            uint4 c[kAhead];
#pragma unroll
            for (int q = 0; q < kAhead; ++q) c[q] = __ldg(from + i + q * kRowThreads);
#pragma unroll
            for (int q = 0; q < kAhead; ++q) g(c[q], i + q * kRowThreads);
        }
        for (; i < c1; i += kRowThreads) g(__ldg(from + i), i);
        if (has_edge()) g(edge[threadIdx.x], threadIdx.x == 0 ? 0 : n - 1);
    }
    template <class G>
    __device__ __forceinline__ void each_of_warp(int per_warp, G g) const {  // the warp's part of the row, its lanes side by side
        const int warp = threadIdx.x >> 5, last = min(n, (warp + 1) * per_warp);
        int i = warp * per_warp + (threadIdx.x & 31);
        for (; i + (kAhead - 1) * 32 < last; i += kAhead * 32) {
            uint4 c[kAhead];
#pragma unroll
            for (int q = 0; q < kAhead; ++q) c[q] = at(i + q * 32);
#pragma unroll
            for (int q = 0; q < kAhead; ++q) g(c[q], i + q * 32);
        }
        for (; i < last; i += 32) g(at(i), i);
    }
    __device__ __forceinline__ float value(int e) const {
        return kBf16 ? __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const unsigned short *>(from)[e]) << 16)
                     : reinterpret_cast<const float *>(from)[e];
    }
};

// The first element of the row whose running sum of g(element, value) passes `target`;
// of_chunk(chunk, its number) is g's sum over a chunk.
// (`known`: the sums of the warps' parts are in sh.part.)
template <bool kBf16, class H, class G>
__device__ int find_in_row(const RowChunks<kBf16> &c, RowShared &sh, H of_chunk, G g, uint64_t target, bool known = false) {
    constexpr int kPer = RowChunks<kBf16>::kPer, kWarps = kRowThreads / 32;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, per_warp = (c.n + kWarps - 1) / kWarps;
    uint64_t s = 0;
    if (!known) {
        c.each_of_warp(per_warp, [&](const uint4 &u, int i) { s += of_chunk(u, i); });
        s = warp_sum(s);
        if (lane == 0) sh.part[warp] = s;
    }
    if (t == 0) sh.at = -1;
    __syncthreads();
    int w = 0;
    for (; w < kWarps - 1 && target >= sh.part[w]; ++w) target -= sh.part[w];
    const int b0 = w * per_warp, b1 = min(c.n, b0 + per_warp), per = (per_warp + kRowThreads - 1) / kRowThreads;
    s = 0;
    for (int i = b0 + t * per; i < min(b1, b0 + (t + 1) * per); ++i) s += of_chunk(c.at(i), i);
    uint64_t up = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t p = __shfl_up_sync(0xffffffffu, up, o);
        if (lane >= o) up += p;
    }
    __syncthreads();
    if (lane == 31) sh.part[warp] = up;
    __syncthreads();
    for (int q = 0; q < warp; ++q) up += sh.part[q];
    if (up - s <= target && target < up) {
        uint64_t left = target - (up - s);
        for (int e = max((b0 + t * per) * kPer, c.lead), last = min(min(b1, b0 + (t + 1) * per) * kPer, c.end); e < last; ++e) {
            const uint64_t y = g(e, c.value(e));
            if (left < y) {
                sh.at = e;
                break;
            }
            left -= y;
        }
    }
    __syncthreads();
    const int e = sh.at;
    __syncthreads();
    return e;
}

// The weights of a list's tokens (formed as they are found they take a warp's whole way
// for each: 154 us instead of 95 for 256 rows with 1000 kept tokens).
template <bool kBf16>
__device__ __forceinline__ void weigh_list(RowShared &sh, const Weigh &weight, uint32_t top_key, uint32_t total) {
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < min(total, static_cast<uint32_t>(kTopList)); i += kRowThreads)
        sh.list.w[i] = weight(value_of<kBf16>(top_key - sh.list.key[i]));
    __syncthreads();
}

// The answers that a pass over the row gives, is_kept(element, value) being known.
template <bool kBf16, class K>
__device__ __forceinline__ void mask_of_row(const SampleArgs &a, int64_t row, const RowFilter &f, const RowChunks<kBf16> &c, const Weigh &weight,
                                            K is_kept, uint32_t set_n, uint64_t set_mass) {
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    uint32_t *const words_of = a.mask + row * a.mask_stride;
    const int64_t id = a.keep ? a.keep[row] : -1;
    const int forced = id >= 0 && id < a.vocab ? static_cast<int>(id) : -1;
    for (int w = warp; w < (a.vocab + 31) / 32; w += kRowThreads / 32) {
        const int j = w * 32 + lane;
        bool k = false;
        if (j < a.vocab) {
            const float x = c.value(c.lead + j);
            k = is_kept(c.lead + j, x) || (j == forced && x >= -FLT_MAX);
        }
        const uint32_t word = __ballot_sync(0xffffffffu, k);
        if (lane == 0) words_of[w] = word;
    }
    if (t == 0) {
        if (forced >= 0) {
            const float x = c.value(c.lead + forced);
            if (x >= -FLT_MAX && !is_kept(c.lead + forced, x)) {
                set_n += 1;
                set_mass += weight(x);
            }
        }
        if (a.kept) a.kept[row] = static_cast<int32_t>(set_n);
        if (a.lse) a.lse[row] = static_cast<float>(weight.lse(set_mass, f.scale));
    }
}
template <bool kBf16>
__device__ __forceinline__ void draw_of_row(const SampleArgs &a, int64_t row, const RowFilter &f, const RowChunks<kBf16> &c, const Weigh &weight,
                                            int e, float u, uint32_t set_n, uint64_t set_mass) {
    if (threadIdx.x != 0) return;
    if (e < 0) return no_answer<false>(a, row, CUDART_NAN_F);  // (the logits changed under the call)
    const float x = c.value(e);
    const bool drawn = u == u;
    a.ids[row] = drawn ? e - c.lead : -1;
    if (a.logp) a.logp[row] = drawn ? static_cast<float>(weight.logp(x, set_mass, f.scale)) : CUDART_NAN_F;
    if (a.kept) a.kept[row] = static_cast<int32_t>(set_n);
}

// A list of the largest tokens.  A sample of the row (one turn in `every`) gives a value
// that about `share` of the sample's tokens reach and some more, the pass over the whole
// row collects what reaches it and the top, and the border is found among those: of a
// top-k, of what min-p leaves, or of a nucleus (whose other tokens are weighed in a second
// pass).  False where they are too few after all, or too many for the list.
template <bool kBf16, bool kMask>
__device__ bool list_row(const SampleArgs &a, int64_t row, const RowFilter &f, const RowChunks<kBf16> &row_chunks, RowShared &sh) {
    constexpr int kPer = RowChunks<kBf16>::kPer, kThreads = kRowThreads, kWarps = kThreads / 32, kAhead = 4;
    Scratch &sc = sh.scratch;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const uint4 *const from = row_chunks.from;
    const int c0 = row_chunks.c0, c1 = row_chunks.c1, lead = row_chunks.lead;
    // ---- the sample
    const int turn = kThreads * kAhead, turns = (c1 - c0) / turn;
    const int every = turns >= 16 ? 8 : turns >= 6 ? 4 : turns >= 2 ? 2 : 1;
    float tmax = -CUDART_INF_F;
    for (int u = 0; u < turns; u += every) {
        uint4 c[kAhead];
#pragma unroll
        for (int q = 0; q < kAhead; ++q) c[q] = __ldg(from + c0 + u * turn + q * kThreads + t);
#pragma unroll
        for (int q = 0; q < kAhead; ++q) tmax = fmaxf(tmax, chunk_max<kBf16>(c[q]));
    }
    if (every == 1) {
        for (int i = c0 + turns * turn + t; i < c1; i += kThreads) tmax = fmaxf(tmax, chunk_max<kBf16>(__ldg(from + i)));
        if (row_chunks.has_edge()) tmax = fmaxf(tmax, chunk_max<kBf16>(sh.edge[t]));
    }
    // Each warp's R-th largest thread maximum, R being the warp's part of the share (of a
    // top-k the sample's, and five standard deviations); the median of the warps'.
    {
        const float share = f.use_k ? static_cast<float>(f.top_k) / every : kListShare;
        const int reach = min(32, (static_cast<int>(share + 5.f * sqrtf(share) + 8.f) + kWarps - 1) / kWarps);
        const uint32_t key = key_of<kBf16>(tmax), key16 = kBf16 ? key : key >> 16;
        uint32_t prefix = 0;
#pragma unroll
        for (uint32_t bit = 0x8000u; bit; bit >>= 1)
            if (__popc(__ballot_sync(0xffffffffu, key16 >= (prefix | bit))) >= reach) prefix |= bit;
        if (lane == 0) sc.red32[0][warp] = kBf16 ? prefix : prefix << 16;
        __syncthreads();
        if (warp == 0) {
            const uint32_t mine = lane < kWarps ? sc.red32[0][lane] : 0xffffffffu;
            int under = 0;
#pragma unroll
            for (int q = 0; q < kWarps; ++q) under += __shfl_sync(0xffffffffu, mine, q) < mine;
            const uint32_t mid = __reduce_max_sync(0xffffffffu, lane < kWarps && under <= (kWarps - 1) / 2 ? mine : 0u);
            if (lane == 0) {
                sh.floor_key = mid;
                sh.list_n = 0;
            }
        }
        __syncthreads();
    }
    // ---- the row
    const float floor_x = floor_of<kBf16>(sh.floor_key);
    tmax = -CUDART_INF_F;
    const auto take = [&](const uint4 &c, int i) {
        const float m = chunk_max<kBf16>(c);
        tmax = max_nan(tmax, m);
        if (m >= floor_x) {
            float v[kPer];
            unpack<kBf16>(c, v);
#pragma unroll
            for (int q = 0; q < kPer; ++q)
                if (v[q] >= floor_x) {
                    const uint32_t at = atomicAdd(&sh.list_n, 1u);
                    if (at < kTopList) {
                        sh.list.key[at] = key_of<kBf16>(v[q]);
                        sh.list.at[at] = i * kPer + q - lead;
                    }
                }
        }
    };
    row_chunks.each(take);
    const bool nan = tmax != tmax;
    const uint32_t wm = __reduce_max_sync(0xffffffffu, nan ? 0u : key_of<kBf16>(tmax));
    if (lane == 0) sc.red32[1][warp] = wm;
    const bool bad = __syncthreads_or(nan);
    uint32_t top_key = 0;
#pragma unroll
    for (int q = 0; q < kWarps; ++q) top_key = max(top_key, sc.red32[1][q]);
    const float top = value_of<kBf16>(top_key);
    if (bad || !(fabsf(top) <= FLT_MAX)) {  // NaN, +inf, or nothing above -inf: no distribution
        if (t == 0) no_answer<kMask>(a, row, CUDART_NAN_F);
        return true;
    }
    // ---- what min-p takes leaves the list
    const float base = base_of<kBf16>(sc, f, top);
    uint32_t total = sh.list_n;
    if (base > floor_x && total <= kTopList) {
        constexpr int kOwn = kTopList / kThreads;
        const uint32_t lowest = key_of<kBf16>(base);
        uint32_t keys[kOwn], ids[kOwn];
#pragma unroll
        for (int q = 0; q < kOwn; ++q) {
            const uint32_t i = q * kThreads + t;
            keys[q] = i < total ? sh.list.key[i] : 0;
            ids[q] = i < total ? sh.list.at[i] : 0;
        }
        __syncthreads();
        if (t == 0) sh.list_n = 0;
        __syncthreads();
#pragma unroll
        for (int q = 0; q < kOwn; ++q)
            if (keys[q] >= lowest) {
                const uint32_t at = atomicAdd(&sh.list_n, 1u);
                sh.list.key[at] = keys[q];
                sh.list.at[at] = ids[q];
            }
        __syncthreads();
        total = sh.list_n;
    }
    const float cand = fmaxf(floor_x, base);
    const bool complete = cand <= base;  // the list is all that min-p leaves
    if (total > kTopList || (!complete && (f.use_k ? total < static_cast<uint32_t>(f.top_k) : !f.use_p))) return false;
    const Weigh weight(f.scale, top, sh.table);
    uint64_t mass = 0, rest = 0;
    uint32_t none = 0;
    for (uint32_t i = t; i < total; i += kThreads) {
        const uint32_t key = sh.list.key[i];
        const uint64_t w = weight(value_of<kBf16>(key));
        sh.list.w[i] = w;
        sh.list.key[i] = top_key - key;
        mass += w;
    }
    if (!f.use_k) {
        if (!complete) {
            const float least = fmaxf(weight.ws.cut, nextafterf(base, -CUDART_INF_F));
            const bool light = cand <= weight.precise_from;  // (mostly)
            row_chunks.each([&](const uint4 &c, int) {
                float v[kPer];
                unpack<kBf16>(c, v);
                if (light) {
#pragma unroll
                    for (int q = 0; q < kPer; ++q) rest += v[q] > least && v[q] < cand ? weight_rough(v[q], weight.ws, sh.table) : 0;
                } else {
#pragma unroll 1
                    for (int q = 0; q < kPer; ++q) rest += v[q] >= base && v[q] < cand ? weight(v[q]) : 0;
                }
            });
        }
        block_sums<kThreads>(sc, mass, rest, none);
        if (f.use_p && mass < share_of(f.top_p, mass + rest)) return false;
    }
    __syncthreads();
    finish_list<kBf16, kMask, kThreads>(a, row, f, sc, weight, top_key, cand, total, sh.list.w, sh.list.key, sh.list.at, f.use_k ? 0 : mass, mass + rest);
    return true;
}

// Any filter on a bf16 row: how often each value occurs, counted in one pass, is all that
// the border needs, and a weight is formed once a value and not once a token (a weight a
// token made 509 rows of 151936 take 278 us).  A second pass collects the kept tokens, or
// where they are many finds the draw's place.  False where the border lies among values
// that share a bin, or the row's top does.
template <bool kMask>
__device__ bool counted_row(const SampleArgs &a, int64_t row, const RowFilter &f, const RowChunks<true> &c, RowShared &sh) {
    constexpr int kPer = 8, kThreads = kRowThreads, kWarps = kThreads / 32;
    Scratch &sc = sh.scratch;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    __syncthreads();  // (what another way has left of the row)
    for (int b = t; b < kOwnBins * kThreads; b += kThreads) sh.bins[b] = 0;
    if (t == 0) {
        sh.tiny_n = sh.list_n = 0;
        sh.leave = 0;
    }
    __syncthreads();
    bool bad = false;
    const auto count = [&](uint32_t bits) {  // of a value, not -inf, without a bin of its own
        if ((bits & 0x7fffu) >= 0x7f80u) {
            bad = true;
        } else if ((bits & 0x7fffu) == 0) {
            atomicAdd(&sh.bins[kZero], 1u);
        } else if ((bits & 0x7fffu) < (kLowest << 7)) {
            atomicAdd(&sh.bins[(bits & 0x8000u) ? kTinyDown : kTinyUp], 1u);
            const uint32_t at = atomicAdd(&sh.tiny_n, 1u);
            if (at < kTinyRoom) sh.tiny[at] = static_cast<uint16_t>(bits);
        } else if (bits & 0x8000u) {
            atomicAdd(&sh.bins[kLow], 1u);
        } else {
            sh.leave = 1;
        }
    };
    c.each([&](const uint4 &u, int) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        uint32_t odd = 0;
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
            const uint32_t bits = (q & 1) ? w[q >> 1] >> 16 : w[q >> 1] & 0xffffu, m = (bits & 0x7fffu) - (kLowest << 7);
            if (m < static_cast<uint32_t>(kSide)) atomicAdd(&sh.bins[(bits & 0x8000u) ? kDown + m : kSide - 1 - m], 1u);
            else if (bits != 0xff80u) odd |= 1u << q;
        }
#pragma unroll 1
        for (; odd; odd &= odd - 1) {
            const int q = __ffs(odd) - 1;
            const uint32_t pair = q < 4 ? (q < 2 ? w[0] : w[1]) : (q < 6 ? w[2] : w[3]);
            count((q & 1) ? pair >> 16 : pair & 0xffffu);
        }
    });
    if (__syncthreads_or(bad)) {
        if (t == 0) no_answer<kMask>(a, row, CUDART_NAN_F);
        return true;
    }
    // ---- the top: the first bin that is not empty
    uint32_t *const own = &sh.bins[t * kOwnBins];
    uint32_t lowest = 0xffffffffu;
#pragma unroll 1
    for (int i = kOwnBins - 1; i >= 0; --i)
        if (own[i]) lowest = t * kOwnBins + i;
    lowest = __reduce_min_sync(0xffffffffu, lowest);
    if (lane == 0) sc.red32[0][warp] = lowest;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kWarps; ++q) lowest = min(lowest, sc.red32[0][q]);
    if (sh.leave || sh.tiny_n > kTinyRoom) return false;
    if (lowest == 0xffffffffu) {  // nothing above -inf
        if (t == 0) no_answer<kMask>(a, row, CUDART_NAN_F);
        return true;
    }
    if (lowest == kTinyUp || lowest == kTinyDown || lowest == kLow) return false;
    const float top = bin_value(static_cast<int>(lowest));
    const uint32_t top_key = key_of<true>(top);
    const Weigh weight(f.scale, top, sh.table);
    const float base = base_of<true>(sc, f, top);
    // (the finite values from -2^14 down have to weigh nothing, and a bin of several values lies on one side of min-p:
    // that one wholly below it, or min-p leaves the lowest of all)
    constexpr float kTiny = 9.765625e-4f;  // 2^-10
    constexpr float kLeast = -3.3895313892515355e38f;  // of bf16's finite values
    if (sh.bins[kLow] && (weight.ws.wide || weight.ws.cut < -16384.f || (base > kLeast && base <= -16384.f))) return false;
    if (sh.tiny_n && base > -kTiny && base < kTiny && base != 0.f) return false;
    const bool low_in = base <= kLeast, up_in = base <= 0.f, down_in = base <= -kTiny;
    // ---- numbers and masses of the thread's bins
    uint64_t tiny_up = 0, tiny_down = 0;
    uint32_t none = 0;
    if (sh.tiny_n) {
        for (uint32_t i = t; i < sh.tiny_n; i += kThreads) {
            const uint32_t bits = sh.tiny[i];
            const uint64_t w = weight(__uint_as_float(bits << 16));
            if (bits & 0x8000u) tiny_down += w;
            else tiny_up += w;
        }
        block_sums<kThreads>(sc, tiny_up, tiny_down, none);
    }
    const auto bin_of = [&](int i, uint32_t *n, uint64_t *one) -> uint64_t {  // the mass of own bin i, its number and a token's weight
        const int b = t * kOwnBins + i;
        *n = own[i];
        *one = 0;
        if (*n == 0) return 0;
        if (b == kTinyUp || b == kTinyDown || b == kLow) {
            if (!(b == kTinyUp ? up_in : b == kTinyDown ? down_in : low_in)) *n = 0;
            return *n == 0 || b == kLow ? 0 : b == kTinyUp ? tiny_up : tiny_down;
        }
        const float x = bin_value(b);
        if (!(x >= base)) {
            *n = 0;
            return 0;
        }
        *one = weight(x);
        return *n * *one;
    };
    uint32_t n = 0;
    uint64_t mass = 0;
#pragma unroll 1
    for (int i = 0; i < kOwnBins; ++i) {
        uint32_t m;
        uint64_t one;
        mass += bin_of(i, &m, &one);
        n += m;
    }
    uint32_t up_n = n;
    uint64_t up_mass = mass;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t pn = __shfl_up_sync(0xffffffffu, up_n, o);
        const uint64_t pm = __shfl_up_sync(0xffffffffu, up_mass, o);
        if (lane >= o) {
            up_n += pn;
            up_mass += pm;
        }
    }
    __syncthreads();
    if (lane == 31) {
        sc.red32[0][warp] = up_n;
        sc.red64[0][warp] = up_mass;
    }
    __syncthreads();
    uint32_t set_n = 0;
    uint64_t set_mass = 0;
#pragma unroll
    for (int q = 0; q < kWarps; ++q) {
        if (q == warp) {
            up_n += set_n;
            up_mass += set_mass;
        }
        set_n += sc.red32[0][q];
        set_mass += sc.red64[0][q];
    }
    // ---- the border: the bin at which the number, or the mass, reaches `target`
    uint32_t ties = 0;
    const auto descend = [&](bool by_mass, uint64_t target) -> bool {
        const uint64_t upto = by_mass ? up_mass : up_n, under = upto - (by_mass ? mass : n);
        if (under < target && upto >= target) {
            uint32_t an = up_n - n, m = 0;
            uint64_t am = up_mass - mass, one = 0;
            int i = 0;
#pragma unroll 1
            for (; i < kOwnBins; ++i) {
                const uint64_t x = bin_of(i, &m, &one);
                if (by_mass ? am + x >= target : an + m >= target) break;
                an += m;
                am += x;
            }
            sh.border = t * kOwnBins + i;
            sh.above_n = an;
            sh.above_mass = am;
            sh.ties_all = m;
            sh.one = one;
        }
        __syncthreads();
        const uint32_t b = sh.border;
        const uint64_t left = target - (by_mass ? sh.above_mass : sh.above_n);
        if (b == kTinyUp || b == kTinyDown || b == kLow) return false;
        ties = static_cast<uint32_t>(by_mass ? (left + sh.one - 1) / sh.one : left);
        set_n = sh.above_n + ties;
        set_mass = sh.above_mass + ties * sh.one;
        return true;
    };
    bool whole = true;
    if (f.use_k && static_cast<uint32_t>(f.top_k) < set_n) {
        if (!descend(false, f.top_k)) return false;
        whole = false;
        __syncthreads();
    }
    if (f.use_p) {
        if (!descend(true, share_of(f.top_p, set_mass))) return false;
        whole = false;
    }
    const uint32_t ties_all = whole ? 0 : sh.ties_all;
    const float border_x = whole ? base : bin_value(static_cast<int>(sh.border));
    const uint32_t border_far = whole ? 0xffffffffu : top_key - key_of<true>(border_x);
    const uint32_t reach = whole ? set_n : sh.above_n + ties_all;  // tokens at the border and above
    __syncthreads();
    if (reach <= kTopList) {
        // ---- few tokens: they are collected
        c.each([&](const uint4 &u, int i) {
            if (chunk_max<true>(u) >= border_x) {
                float v[kPer];
                unpack<true>(u, v);
#pragma unroll
                for (int q = 0; q < kPer; ++q)
                    if (v[q] >= border_x) {
                        const uint32_t at = atomicAdd(&sh.list_n, 1u);
                        if (at < kTopList) {
                            sh.list.key[at] = top_key - key_of<true>(v[q]);
                            sh.list.at[at] = i * kPer + q - c.lead;
                        }
                    }
            }
        });
        weigh_list<true>(sh, weight, top_key, reach);
        answer_list<true, kMask, kThreads>(a, row, f, sc, weight, top_key, border_x, min(sh.list_n, static_cast<uint32_t>(kTopList)), sh.list.w,
                                           sh.list.key, sh.list.at, border_far, ties, ties_all, set_n, set_mass);
        return true;
    }
    // ---- many: the row itself
    int tie_last = INT32_MAX;
    if (ties < ties_all) {
        const auto at_border = [&](int, float x) -> uint64_t { return x == border_x; };
        const auto of_chunk = [&](const uint4 &u, int) -> uint64_t {
            float v[kPer];
            unpack<true>(u, v);
            uint32_t n = 0;
#pragma unroll
            for (int q = 0; q < kPer; ++q) n += v[q] == border_x;
            return n;
        };
        tie_last = find_in_row<true>(c, sh, of_chunk, at_border, ties - 1);
    }
    const auto is_kept = [&](int e, float x) { return x > border_x || (x == border_x && e <= tie_last); };
    if constexpr (kMask) {
        mask_of_row<true>(a, row, f, c, weight, is_kept, set_n, set_mass);
    } else {
        // (a weight looked up: 10 operations a token, formed anew it takes 30)
        const float u = a.uniform[row];
        const bool end = at_an_end(u);
        for (int b = t; b < kValues; b += kThreads) {
            const float x = bin_value(b);
            sh.value_w[b] = b != kTinyUp && b != kTinyDown && b != kLow && x >= border_x && x <= top ? end ? 1 : weight(x) : 0;
        }
        __syncthreads();
        const auto mass_of = [&](int i, float x) -> uint64_t { return is_kept(i, x) ? end ? 1 : weight(x) : 0; };
        const uint32_t border_bits = __float_as_uint(border_x) >> 16;
        const auto of_chunk = [&](const uint4 &c4, int i) -> uint64_t {
            const uint32_t w[4] = {c4.x, c4.y, c4.z, c4.w};
            uint64_t s = 0;
            uint32_t odd = 0;  // values without a bin of their own
#pragma unroll
            for (int q = 0; q < kPer; ++q) {
                const uint32_t bits = (q & 1) ? w[q >> 1] >> 16 : w[q >> 1] & 0xffffu, m = (bits & 0x7fffu) - (kLowest << 7);
                const bool in = m < static_cast<uint32_t>(kSide);
                const bool out = !in || (bits == border_bits && i * kPer + q > tie_last);
                s += sh.value_w[out ? kLow : (bits & 0x8000u) ? kDown + m : kSide - 1 - m];
                odd |= (!in && bits != 0xff80u ? 1u : 0u) << q;
            }
#pragma unroll 1
            for (; odd; odd &= odd - 1) {
                const int e = i * kPer + __ffs(odd) - 1;
                if (e >= c.lead && e < c.end) s += mass_of(e, c.value(e));
            }
            return s;
        };
        const int e = find_in_row<true>(c, sh, of_chunk, mass_of, end ? end_of(u, set_n) : place_of(u, set_mass));
        draw_of_row<true>(a, row, f, c, weight, e, u, set_n, set_mass);
    }
    return true;
}

// A float32 row of which all is kept, or what min-p leaves: a pass for the top, one for the
// masses of the warps' parts, and a look into the part that the draw falls into.
template <bool kBf16, bool kMask>
__device__ void plain_row(const SampleArgs &a, int64_t row, const RowFilter &f, const RowChunks<kBf16> &c, RowShared &sh) {
    constexpr int kPer = RowChunks<kBf16>::kPer, kThreads = kRowThreads, kWarps = kThreads / 32;
    Scratch &sc = sh.scratch;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    __syncthreads();  // (what another way has left of the row)
    float tmax = -CUDART_INF_F;
    c.each([&](const uint4 &u, int) { tmax = max_nan(tmax, chunk_max<kBf16>(u)); });
    const bool nan = tmax != tmax;
    const uint32_t wm = __reduce_max_sync(0xffffffffu, nan ? 0u : key_of<kBf16>(tmax));
    if (lane == 0) sc.red32[1][warp] = wm;
    const bool bad = __syncthreads_or(nan);
    uint32_t top_key = 0;
#pragma unroll
    for (int q = 0; q < kWarps; ++q) top_key = max(top_key, sc.red32[1][q]);
    const float top = value_of<kBf16>(top_key);
    if (bad || !(fabsf(top) <= FLT_MAX)) {  // NaN, +inf, or nothing above -inf: no distribution
        if (t == 0) no_answer<kMask>(a, row, CUDART_NAN_F);
        return;
    }
    const Weigh weight(f.scale, top, sh.table);
    const float base = base_of<kBf16>(sc, f, top);
    uint64_t set_mass = 0, none = 0;
    uint32_t set_n = 0;
    c.each_of_warp((c.n + kWarps - 1) / kWarps, [&](const uint4 &u, int) {
        if (!(chunk_max<kBf16>(u) >= base)) return;
        float v[kPer];
        unpack<kBf16>(u, v);
#pragma unroll
        for (int q = 0; q < kPer; ++q)
            if (v[q] >= base) {
                set_mass += weight(v[q]);
                ++set_n;
            }
    });
    const uint64_t part = warp_sum(set_mass);
    if (lane == 0) sh.part[warp] = part;
    block_sums<kThreads>(sc, set_mass, none, set_n);
    const auto is_kept = [&](int, float x) { return x >= base; };
    if constexpr (kMask) {
        mask_of_row<kBf16>(a, row, f, c, weight, is_kept, set_n, set_mass);
    } else {
        const float u = a.uniform[row];
        const bool end = at_an_end(u);
        const auto mass_of = [&](int i, float x) -> uint64_t { return is_kept(i, x) ? end ? 1 : weight(x) : 0; };
        const auto of_chunk = [&](const uint4 &c4, int i) -> uint64_t {
            uint64_t s = 0;
            if (!(chunk_max<kBf16>(c4) >= base)) return s;
            float v[kPer];
            unpack<kBf16>(c4, v);
#pragma unroll
            for (int q = 0; q < kPer; ++q) s += mass_of(i * kPer + q, v[q]);
            return s;
        };
        const int e = find_in_row<kBf16>(c, sh, of_chunk, mass_of, end ? end_of(u, set_n) : place_of(u, set_mass), !end);
        draw_of_row<kBf16>(a, row, f, c, weight, e, u, set_n, set_mass);
    }
}

// (Two CTAs a multiprocessor; three where the row's bytes are what counts, masks of bf16
// rows: 4096 rows in 293 us instead of 334.  Registers then spill, which costs draws 5 to
// 10 %, and float32 masks 8 %.)
template <bool kBf16, bool kMask>
__global__ void __launch_bounds__(kRowThreads, kBf16 && kMask ? 3 : 2) row_kernel(const __grid_constant__ SampleArgs a) {
    extern __shared__ __align__(16) char smem[];
    RowShared &sh = *reinterpret_cast<RowShared *>(smem);
    const int64_t row = blockIdx.x;
    const int t = threadIdx.x;
    const RowFilter f = filter_of(a, row);
    if constexpr (kMask) {
        uint32_t *const words = a.mask + row * a.mask_stride;
        for (int w = t; w < (a.vocab + 31) / 32; w += kRowThreads) words[w] = 0;
    }
    if (!f.active || !f.valid) {
        if (t == 0) no_answer<kMask>(a, row, f.active ? CUDART_NAN_F : 0.f);
        return;
    }
    if (f.min_p > 0.f && t == kRowThreads - 1) sh.scratch.log_min_p = log(fmin(static_cast<double>(f.min_p), 1.0));
    const RowChunks<kBf16> c(a, row, sh.edge);
    for (int i = t; i < kUnits; i += kRowThreads) sh.table[i] = kTables.rough[i];
    __syncthreads();
    bool done = false;
    const bool few = f.use_k ? f.top_k <= kTopMost : f.min_p >= 0.01f || (!kBf16 && f.use_p);
    if (few) done = list_row<kBf16, kMask>(a, row, f, c, sh);
    if constexpr (kBf16) {
        if (!done) done = counted_row<kMask>(a, row, f, c, sh);
    } else if (!done && !f.use_k && !f.use_p) {
        plain_row<kBf16, kMask>(a, row, f, c, sh);
        done = true;
    }
    if (!done && t == 0) {
        if constexpr (kMask) a.mask[row * a.mask_stride] = kLeftMask;
        else a.ids[row] = kLeftId;
    }
}

// ------------------------------------------------------------- any row, a cluster's work
struct Shared {
    Scratch scratch;
    WeightEntry table[kUnits];
    uint64_t list_w[kList];
    uint32_t list[kList];
    uint16_t list_in[kList];           // elements of the slice
    uint64_t part[kMaxWarps];          // sums of the warps' parts of the slice
    int at;
    // read by the cluster's other CTAs, as the bins are
    uint64_t list_mass, rest_mass, kept_mass;
    uint32_t list_n, rest_n;
    uint32_t top, floor_key, key_min, key_max;
    int bad;
};

template <bool kBf16, bool kMask, int kThreads>
__device__ void cluster_row(const SampleArgs &a, int64_t row, const RowFilter &f, const cg::cluster_group &cluster, uint4 *chunks, char *smem) {
    constexpr int kElt = kBf16 ? 2 : 4, kPer = 16 / kElt, kWarps = kThreads / 32, kAhead = 4;
    Shared &sh = *reinterpret_cast<Shared *>(smem + static_cast<size_t>(a.chunk_room) * 16);
    Scratch &sc = sh.scratch;
    const int ranks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int first = rank * a.slice;                                   // the slice's first token
    const int n = max(0, min(a.slice, a.vocab - first));                // and its tokens
    const int words = (n + 31) / 32;
    uint32_t *const mask_row = kMask ? a.mask + row * a.mask_stride + first / 32 : nullptr;
    // The mask starts empty: where the border is found in the list, rank 0 adds its bits.
    if constexpr (kMask)
        for (int w = t; w < words; w += kThreads) mask_row[w] = 0;
    if (!f.active || !f.valid) {
        if (rank == 0 && t == 0) no_answer<kMask>(a, row, f.active ? CUDART_NAN_F : 0.f);
        return;
    }
    const float scale = f.scale;
    const bool use_k = f.use_k, use_p = f.use_p;
    if (f.min_p > 0.f && t == kThreads - 1) sc.log_min_p = log(fmin(static_cast<double>(f.min_p), 1.0));

    // ------------------------------------------------------------------ the slice, and each thread's maximum
    const char *const src = a.x + row * a.x_stride + static_cast<int64_t>(first) * kElt;
    const int lead = static_cast<int>((reinterpret_cast<uintptr_t>(src) & 15u) / kElt);  // elements of the first chunk in front of it
    const int end = lead + n, n_chunks = n > 0 ? (end + kPer - 1) / kPer : 0;
    const uint4 *const from = reinterpret_cast<const uint4 *>(src - lead * kElt);
    const int c0 = lead > 0 ? 1 : 0, c1 = max(c0, end / kPer);  // whole chunks: [c0, c1)
    for (int i = t; i < kUnits; i += kThreads) sh.table[i] = kTables.rough[i];
    float tmax = -CUDART_INF_F;
    {
        int i = c0 + t;
        for (; i + (kAhead - 1) * kThreads < c1; i += kAhead * kThreads) {
            uint4 c[kAhead];
#pragma unroll
            for (int q = 0; q < kAhead; ++q) c[q] = __ldcs(from + i + q * kThreads);
#pragma unroll
            for (int q = 0; q < kAhead; ++q) {
                chunks[i + q * kThreads] = c[q];
                tmax = max_nan(tmax, chunk_max<kBf16>(c[q]));
            }
        }
        for (; i < c1; i += kThreads) {
            const uint4 c = __ldcs(from + i);
            chunks[i] = c;
            tmax = max_nan(tmax, chunk_max<kBf16>(c));
        }
        // the first and the last chunk where they hold others' elements too
        const int e = t == 0 ? 0 : n_chunks - 1;
        if (t < 2 && n_chunks > 0 && (t == 0 ? c0 == 1 : n_chunks > c1 && n_chunks - 1 >= c0)) {
            const uint4 c = edge_chunk<kBf16>(from, e, lead, end);
            chunks[e] = c;
            tmax = max_nan(tmax, chunk_max<kBf16>(c));
        }
    }
    const auto each_chunk = [&](auto g) {  // g(chunk, its number)
        for (int i = t; i < n_chunks; i += kThreads) g(chunks[i], i);
    };
    const auto each = [&](auto g) {  // g(value)
        each_chunk([&](const uint4 &c, int) {
            float v[kPer];
            unpack<kBf16>(c, v);
#pragma unroll
            for (int q = 0; q < kPer; ++q) g(v[q]);
        });
    };

    // --------------------------------------------- the row's top, and a value that enough tokens reach
    // Each warp's R-th largest thread maximum, R = k / (warps of the cluster): the
    // smallest of them is reached by k tokens at least.  Above 32 there is no such
    // value and the list stays empty.
    const int reach = ((use_k ? f.top_k : kReach) + ranks * kWarps - 1) / (ranks * kWarps);
    {
        const bool nan = tmax != tmax;
        const uint32_t key = nan ? 0u : key_of<kBf16>(tmax), key16 = kBf16 ? key : key >> 16;
        uint32_t prefix = 0;
        if (reach <= 32) {
#pragma unroll
            for (uint32_t bit = 0x8000u; bit; bit >>= 1)
                if (__popc(__ballot_sync(0xffffffffu, key16 >= (prefix | bit))) >= reach) prefix |= bit;
        }
        const uint32_t wm = __reduce_max_sync(0xffffffffu, key);
        if (lane == 0) {
            sc.red32[0][warp] = wm;
            sc.red32[1][warp] = kBf16 ? prefix : prefix << 16;
        }
        const int any_nan = __syncthreads_or(nan);
        if (warp == 0) {
            const uint32_t m = __reduce_max_sync(0xffffffffu, lane < kWarps ? sc.red32[0][lane] : 0u);
            const uint32_t l = __reduce_min_sync(0xffffffffu, lane < kWarps ? sc.red32[1][lane] : 0xffffffffu);
            if (lane == 0) {
                sh.top = n > 0 ? m : 0;
                sh.floor_key = n > 0 && reach <= 32 ? l : 0xffffffffu;
                sh.bad = any_nan;
                sh.list_n = 0;
            }
        }
        cluster.sync();
    }
    // (a lane reads one CTA's words; a cluster has 8 at most)
    const auto peer_of = [&](int r) -> const Shared * { return cluster.map_shared_rank(&sh, r); };
    const Shared *const peer = peer_of(lane < ranks ? lane : 0);
    const uint32_t top_key = __reduce_max_sync(0xffffffffu, peer->top);
    const uint32_t floor_key = __reduce_min_sync(0xffffffffu, peer->floor_key);
    const bool bad = __any_sync(0xffffffffu, peer->bad != 0);
    const float top = value_of<kBf16>(top_key);
    if (bad || !(fabsf(top) <= FLT_MAX)) {  // NaN, +inf, or nothing above -inf: no distribution
        if (rank == 0 && t == 0) no_answer<kMask>(a, row, CUDART_NAN_F);
        return;
    }
    const Weigh weight(scale, top, sh.table);
    const WeightScale &ws = weight.ws;
    const float base = base_of<kBf16>(sc, f, top);
    const bool listed = floor_key != 0xffffffffu;
    const float cand = fmaxf(floor_of<kBf16>(floor_key), base);

    // ------------------------------------------------------------- candidates, and the mass of the others
    const auto push = [&](float x, int e) {
        const uint32_t at = atomicAdd(&sh.list_n, 1u);
        if (at < kList) {
            sh.list[at] = key_of<kBf16>(x);
            sh.list_in[at] = static_cast<uint16_t>(e);
        }
    };
    uint64_t rest = 0;
    uint32_t rest_n = 0;
    if (use_k) {
        each_chunk([&](const uint4 &c, int i) {
            if (chunk_max<kBf16>(c) >= cand) {
                float v[kPer];
                unpack<kBf16>(c, v);
#pragma unroll
                for (int q = 0; q < kPer; ++q)
                    if (v[q] >= cand) push(v[q], i * kPer + q);
            }
        });
    } else {
        const auto others = [&](auto count, auto light_only) {
            const float least = fmaxf(ws.cut, nextafterf(base, -CUDART_INF_F));
            each_chunk([&](const uint4 &c, int i) {
                float v[kPer];
                unpack<kBf16>(c, v);
#pragma unroll
                for (int q = 0; q < kPer; ++q) {
                    if (v[q] >= cand) {
                        push(v[q], i * kPer + q);
                    } else {
                        if constexpr (light_only.value) rest += v[q] > least ? weight_rough(v[q], ws, sh.table) : 0;
                        else rest += v[q] >= base ? weight(v[q]) : 0;
                        if constexpr (count.value) rest_n += v[q] >= base;
                    }
                }
            });
        };
        // (mostly no token below the candidates is near the top; a nucleus's size is counted in the list)
        if (!(cand <= weight.precise_from)) others(std::true_type{}, std::false_type{});
        else if (use_p) others(std::false_type{}, std::true_type{});
        else others(std::true_type{}, std::true_type{});
    }
    __syncthreads();
    const uint32_t own_n = sh.list_n, in_list = min(own_n, static_cast<uint32_t>(kList));
    // (under a top-k only the number counts here, and the list's masses are rank 0's work)
    uint64_t own_list_mass = 0, own_rest_mass = rest;
    uint32_t own_rest_n = rest_n;
    if (!use_k) {
        for (uint32_t i = t; i < in_list; i += kThreads) {
            const uint64_t w = weight(value_of<kBf16>(sh.list[i]));
            sh.list_w[i] = w;
            own_list_mass += w;
        }
        if (own_n > kList) {  // the list does not hold them all: their mass is the slice's
            own_list_mass = 0;
            each([&](float x) {
                if (x >= cand) own_list_mass += weight(x);
            });
        }
        block_sums<kThreads>(sc, own_list_mass, own_rest_mass, own_rest_n);
        if (t == 0) {
            sh.list_mass = own_list_mass;
            sh.rest_mass = own_rest_mass;
            sh.rest_n = own_rest_n;
        }
    }
    cluster.sync();
    const uint32_t peer_n = lane < ranks ? peer->list_n : 0;
    const uint32_t all_list_n = __reduce_add_sync(0xffffffffu, min(peer_n, 1u << 24));
    const bool overflow = __any_sync(0xffffffffu, peer_n > kList);
    uint64_t all_list_mass = 0, all_rest_mass = 0;
    uint32_t all_rest_n = 0;
    if (!use_k) {
        all_list_mass = warp_sum(lane < ranks ? peer->list_mass : 0);
        all_rest_mass = warp_sum(lane < ranks ? peer->rest_mass : 0);
        all_rest_n = __reduce_add_sync(0xffffffffu, lane < ranks ? peer->rest_n : 0u);
    }
    const uint32_t base_key = key_of<kBf16>(base);
    const bool complete = listed && !overflow && cand <= base;  // the list is all that min-p leaves
    const uint64_t all_mass = all_list_mass + all_rest_mass;

    const bool on_list = listed && !overflow && all_list_n <= static_cast<uint32_t>(a.chunk_room) &&
                         (complete || (use_k ? all_list_n >= static_cast<uint32_t>(f.top_k)
                                             : use_p && all_list_mass >= share_of(f.top_p, all_mass)));
    if (on_list) {
        // every CTA brings its list into rank 0's slice, which nothing needs any more
        char *const home = rank == 0 ? smem : cluster.map_shared_rank(smem, 0);
        uint64_t *const w_of = reinterpret_cast<uint64_t *>(home);
        uint32_t *const far_of = reinterpret_cast<uint32_t *>(w_of + a.chunk_room), *const id_of = far_of + a.chunk_room;
        const uint32_t before = __reduce_add_sync(0xffffffffu, lane < rank ? peer_n : 0u);
        for (uint32_t i = t; i < own_n; i += kThreads) {
            w_of[before + i] = use_k ? weight(value_of<kBf16>(sh.list[i])) : sh.list_w[i];
            far_of[before + i] = top_key - sh.list[i];
            id_of[before + i] = first + sh.list_in[i] - lead;
        }
        cluster.sync();  // (and the masks' zeros are there)
        if (rank == 0)
            finish_list<kBf16, kMask, kThreads>(a, row, f, sc, weight, top_key, cand, all_list_n, w_of, far_of, id_of, all_list_mass, all_mass);
        return;
    }

    // ------------------------------------------------ the others: the border by rounds over the slices
    // Kept: keys above `border`, and the first `ties` of the tokens at it.
    uint32_t border = base_key, ties = 0xffffffffu, ties_before = 0, ties_own = 0;
    uint64_t above_mass = 0, above_n = 0, tie_weight = 0;
    bool whole = true;  // everything from `base` on is kept
    int round = 0;
    // Adds up a round's bins (in buffer `buf`) over the cluster and finds the first, from the
    // last one down, at which the tokens (or their mass) reach `target`.
    uint64_t over_mass = 0, over_n = 0, own_over = 0;  // own_over: this CTA's part of the mass above, a thread's bins
    const auto descend = [&](int buf, bool by_mass, uint64_t target) -> uint32_t {
        if (t == 0) sc.found_bin = kBins;
        cluster.sync();
        uint32_t cnt = 0, before = 0, largest = 0;
        uint64_t mass = 0, own_bin = 0;
        const int bin = kBins - 1 - t;
        if (t < kBins) {
            for (int r = 0; r < ranks; ++r) {
                const Shared *o = peer_of(r);
                const uint32_t c = o->scratch.cnt[buf][bin];
                if (r < rank) before += c;
                cnt += c;
                if (c) {
                    const uint64_t m = static_cast<uint64_t>(o->scratch.mass_hi[buf][bin]) << 32 | o->scratch.mass_lo[buf][bin];
                    if (r == rank) own_bin = m;
                    mass += m;
                    largest = max(largest, o->scratch.far[buf][bin]);
                }
            }
        }
        uint32_t up_n = cnt;
        uint64_t up_mass = mass;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t pn = __shfl_up_sync(0xffffffffu, up_n, o);
            const uint64_t pm = __shfl_up_sync(0xffffffffu, up_mass, o);
            if (lane >= o) {
                up_n += pn;
                up_mass += pm;
            }
        }
        if (lane == 31) {
            sc.red32[0][warp] = up_n;
            sc.red64[0][warp] = up_mass;
        }
        __syncthreads();
        if (t < kBins) {
            for (int w = 0; w < warp; ++w) {
                up_n += sc.red32[0][w];
                up_mass += sc.red64[0][w];
            }
            const uint64_t upto = by_mass ? over_mass + up_mass : over_n + up_n;
            const uint64_t under = upto - (by_mass ? mass : cnt);
            if (under < target && upto >= target) {
                sc.found_bin = bin;
                sc.found_cnt = cnt;
                sc.found_mass = mass;
                sc.found_excl = up_n - cnt;
                sc.found_excl_mass = up_mass - mass;
                sc.found_far = largest;
                sc.found_before = before;
            }
        }
        __syncthreads();
        ++round;  // (others may still read this round's bins: the next takes the other buffer)
        if (bin > static_cast<int>(sc.found_bin)) own_over += own_bin;
        return sc.found_bin;
    };
    const auto clear = [&](int buf) {
        for (int b = t; b < kBins; b += kThreads) sc.cnt[buf][b] = sc.mass_lo[buf][b] = sc.mass_hi[buf][b] = sc.far[buf][b] = 0;
        __syncthreads();
    };
    // The first key, from the top down to `lo`, at which the tokens (or their mass) reach
    // `target`; false if they don't.  The first round's bins are cut evenly between the
    // top and where weights end (keys would crowd: half of them lie within 2^-64 of 0).
    const float last_x = fmaxf(base, ws.wide ? top - __fdiv_rn(46.f, fmaxf(scale, FLT_MIN)) : ws.cut);
    const float per_bin = __fdiv_rn(kBins - 1.f, fmaxf(top - last_x, FLT_MIN));
    const auto coarse = [&](float x) { return kBins - 1 - static_cast<uint32_t>(fminf(__fmul_rn(__fsub_rn(top, x), per_bin), kBins - 1.f)); };
    const auto select = [&](bool by_mass, uint64_t target, uint32_t lo) -> bool {
        over_mass = over_n = own_over = 0;
        clear(round & 1);
        {
            const int buf = round & 1;
            each([&](float x) {
                if (key_of<kBf16>(x) >= lo) {
                    const uint32_t b = coarse(x);
                    atomicAdd(&sc.cnt[buf][b], 1u);
                    add_mass(sc, buf, b, weight(x));
                }
            });
            const uint32_t fb = descend(buf, by_mass, target);
            if (fb == kBins) return false;
            over_n += sc.found_excl;
            over_mass += sc.found_excl_mass;
            // the keys that the bin holds
            uint32_t least = 0xffffffffu, most = 0;
            each([&](float x) {
                const uint32_t key = key_of<kBf16>(x);
                if (key >= lo && coarse(x) == fb) {
                    least = min(least, key);
                    most = max(most, key);
                }
            });
            least = __reduce_min_sync(0xffffffffu, least);
            most = __reduce_max_sync(0xffffffffu, most);
            if (lane == 0) {
                sc.red32[0][warp] = least;
                sc.red32[1][warp] = most;
            }
            __syncthreads();
            if (t == 0) {
                for (int w = 1; w < kWarps; ++w) {
                    least = min(least, sc.red32[0][w]);
                    most = max(most, sc.red32[1][w]);
                }
                sh.key_min = least;
                sh.key_max = most;
            }
            cluster.sync();
        }
        uint32_t hi = 0;
        lo = 0xffffffffu;
        for (int r = 0; r < ranks; ++r) {
            const Shared *o = peer_of(r);
            lo = min(lo, o->key_min);
            hi = max(hi, o->key_max);
        }
#pragma unroll 1
        for (int turn = 0;; ++turn) {  // (32 bits of range are four turns)
            const int buf = round & 1;
            const int shift = max(0, 24 - __clz((hi - lo) | 1u));
            clear(buf);
            each([&](float x) {
                const uint32_t key = key_of<kBf16>(x);
                if (key >= lo && key <= hi) {
                    const uint32_t b = (key - lo) >> shift;
                    atomicAdd(&sc.cnt[buf][b], 1u);
                    sc.far[buf][b] = key;  // (read where it is the only one)
                    add_mass(sc, buf, b, weight(x));
                }
            });
            const uint32_t fb = descend(buf, by_mass, target);
            over_n += sc.found_excl;
            over_mass += sc.found_excl_mass;
            const uint32_t fc = sc.found_cnt;
            if (shift == 0 || fc == 1 || turn == 4) {
                border = shift == 0 ? lo + fb : sc.found_far;
                above_n = over_n;
                above_mass = over_mass;
                tie_weight = sc.found_mass / fc;  // (one weight fc times)
                ties_before = sc.found_before;
                ties_own = sc.cnt[buf][fb];
                const uint64_t left = target - (by_mass ? over_mass : over_n);
                ties = static_cast<uint32_t>(by_mass ? (left + tie_weight - 1) / tie_weight : left);
                whole = false;
                __syncthreads();
                return true;
            }
            lo += fb << shift;
            hi = lo + min(hi - lo, (1u << shift) - 1);  // (lo and a bin's width may pass 2^32)
            __syncthreads();
        }
    };
    uint64_t kept_n = all_list_n + all_rest_n, kept_mass = all_mass;
    {
        uint32_t lo = base_key;
        if (use_k) {
            if (select(false, f.top_k, base_key)) {
                kept_n = f.top_k;
                kept_mass = above_mass + ties * tie_weight;
                lo = border;
            } else {  // fewer than top_k are left: the slices' whole
                uint64_t m = 0, none = 0;
                uint32_t c = 0;
                each([&](float x) {
                    if (x >= base) {
                        m += weight(x);
                        ++c;
                    }
                });
                block_sums<kThreads>(sc, m, none, c);
                if (t == 0) {
                    sh.rest_mass = m;
                    sh.rest_n = c;
                }
                own_list_mass = 0;
                own_rest_mass = m;
                cluster.sync();
                kept_n = kept_mass = 0;
                for (int r = 0; r < ranks; ++r) {
                    const Shared *o = peer_of(r);
                    kept_mass += o->rest_mass;
                    kept_n += o->rest_n;
                }
            }
        }
        if (use_p) {
            select(true, share_of(f.top_p, kept_mass), lo);  // (of a top-k's tied tokens it takes no more than that did)
            kept_n = above_n + ties;
            kept_mass = above_mass + ties * tie_weight;
        }
    }
    // this CTA's share of the tied tokens: all of them, none, or the first few
    const uint32_t own_ties = whole ? 0 : ties <= ties_before ? 0 : min(ties - ties_before, ties_own);

    // The first element of the slice whose running sum of f(element, value) passes `target`.
    const auto value_at = [&](int e) {
        return kBf16 ? __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const unsigned short *>(chunks)[e]) << 16)
                     : reinterpret_cast<const float *>(chunks)[e];
    };
    const auto find = [&](auto g, uint64_t target) -> int {
        const int per_warp = (n_chunks + kWarps - 1) / kWarps;
        {
            uint64_t s = 0;
            for (int i = warp * per_warp + lane; i < min(n_chunks, (warp + 1) * per_warp); i += 32) {
                float v[kPer];
                unpack<kBf16>(chunks[i], v);
#pragma unroll
                for (int q = 0; q < kPer; ++q) s += g(i * kPer + q, v[q]);
            }
            s = warp_sum(s);
            if (lane == 0) sh.part[warp] = s;
        }
        if (t == 0) sh.at = -1;
        __syncthreads();
        int w = 0;
        for (; w < kWarps - 1 && target >= sh.part[w]; ++w) target -= sh.part[w];
        const int c0 = w * per_warp, c1 = min(n_chunks, c0 + per_warp);
        const int per = (per_warp + kThreads - 1) / kThreads;
        uint64_t s = 0;
        for (int i = c0 + t * per; i < min(c1, c0 + (t + 1) * per); ++i) {
            float v[kPer];
            unpack<kBf16>(chunks[i], v);
#pragma unroll
            for (int q = 0; q < kPer; ++q) s += g(i * kPer + q, v[q]);
        }
        uint64_t up = s;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t p = __shfl_up_sync(0xffffffffu, up, o);
            if (lane >= o) up += p;
        }
        __syncthreads();
        if (lane == 31) sc.red64[0][warp] = up;
        __syncthreads();
        for (int q = 0; q < warp; ++q) up += sc.red64[0][q];
        if (up - s <= target && target < up) {
            uint64_t left = target - (up - s);
            for (int e = (c0 + t * per) * kPer, last = min(c1, c0 + (t + 1) * per) * kPer; e < last; ++e) {
                if (e < lead || e >= end) continue;
                const uint64_t y = g(e, value_at(e));
                if (left < y) {
                    sh.at = e;
                    break;
                }
                left -= y;
            }
        }
        __syncthreads();
        const int e = sh.at;
        __syncthreads();
        return e;
    };
    // the last tied element of the slice that is kept
    int tie_last = own_ties == 0 ? -1 : INT32_MAX;
    if (own_ties > 0 && own_ties < ties_own)
        tie_last = find([&](int, float x) -> uint64_t { return key_of<kBf16>(x) == border; }, own_ties - 1);
    const auto is_kept = [&](int e, float x) {
        if (whole) return x >= base;
        const uint32_t key = key_of<kBf16>(x);
        return key > border || (key == border && e <= tie_last);
    };

    if constexpr (kMask) {
        cluster.barrier_arrive();
        const int64_t id = a.keep ? a.keep[row] : -1;
        const bool mine = id >= first && id < first + n, forced_in = id >= 0 && id < a.vocab;
        const int forced = mine ? static_cast<int>(id - first) : -1;
        for (int w = warp; w < words; w += kWarps) {
            const int j = w * 32 + lane;
            bool k = false;
            if (j < n) {
                const float x = value_at(lead + j);
                k = is_kept(lead + j, x) || (j == forced && x >= -FLT_MAX);
            }
            const uint32_t word = __ballot_sync(0xffffffffu, k);
            if (lane == 0) mask_row[w] = word;
        }
        if (t == 0 && (forced_in ? mine : rank == 0)) {
            if (mine) {
                const float x = value_at(lead + forced);
                if (x >= -FLT_MAX && !is_kept(lead + forced, x)) {
                    kept_n += 1;
                    kept_mass += weight(x);
                }
            }
            if (a.kept) a.kept[row] = static_cast<int32_t>(kept_n);
            if (a.lse) a.lse[row] = static_cast<float>(weight.lse(kept_mass, scale));
        }
        cluster.barrier_wait();
    } else {
        // ------------------------------------------------------------------------------ the draw
        uint64_t own = own_list_mass + own_rest_mass, none = 0;
        if (!whole) {
            uint32_t c = 0;
            own = own_over;
            block_sums<kThreads>(sc, own, none, c);
            own += own_ties * tie_weight;
        }
        const float u = a.uniform[row];
        const bool end = at_an_end(u);
        if (end) {
            uint32_t c = 0;
            own = none = 0;
            each_chunk([&](const uint4 &c4, int i) {
                float v[kPer];
                unpack<kBf16>(c4, v);
#pragma unroll
                for (int q = 0; q < kPer; ++q) own += is_kept(i * kPer + q, v[q]);
            });
            block_sums<kThreads>(sc, own, none, c);
        }
        if (t == 0) sh.kept_mass = own;
        cluster.sync();
        const uint64_t target = end ? end_of(u, kept_n) : place_of(u, kept_mass);
        uint64_t in_front = 0;
        for (int r = 0; r < rank; ++r) in_front += peer_of(r)->kept_mass;
        cluster.barrier_arrive();
        if (target >= in_front && target - in_front < own) {
            const int e = find([&](int e, float x) -> uint64_t { return is_kept(e, x) ? end ? 1 : weight(x) : 0; }, target - in_front);
            if (t == 0 && e < 0) no_answer<false>(a, row, CUDART_NAN_F);  // (the logits changed under the call)
            if (t == 0 && e >= 0) {
                const float x = value_at(e);
                const bool drawn = u == u;
                a.ids[row] = drawn ? first + e - lead : -1;
                if (a.logp) a.logp[row] = drawn ? static_cast<float>(weight.logp(x, kept_mass, scale)) : CUDART_NAN_F;
                if (a.kept) a.kept[row] = static_cast<int32_t>(kept_n);
            }
        }
        cluster.barrier_wait();
    }
}

// Clusters go from row to row; a warp looks at 32 rows at a time for those that are its
// cluster's to answer.
template <bool kBf16, bool kMask, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) cluster_kernel(const __grid_constant__ SampleArgs a) {
    extern __shared__ __align__(16) char smem[];
    const cg::cluster_group cluster = cg::this_cluster();
    const int64_t step = gridDim.x / cluster.num_blocks();
    for (int64_t at = blockIdx.x / cluster.num_blocks(); at < a.n_rows; at += 32 * step) {
        const int64_t mine = at + (threadIdx.x & 31) * step;
        bool todo = mine < a.n_rows;
        if (todo && a.after_rows) todo = kMask ? a.mask[mine * a.mask_stride] == kLeftMask : a.ids[mine] == kLeftId;
        // (no row of these is answered before every warp of the cluster has its answer here)
        uint32_t rows = __ballot_sync(0xffffffffu, todo);
        cluster.sync();
        for (; rows; rows &= rows - 1) {
            const int64_t row = at + (__ffs(rows) - 1) * step;
            cluster_row<kBf16, kMask, kThreads>(a, row, filter_of(a, row), cluster, reinterpret_cast<uint4 *>(smem), smem);
            cluster.sync();  // (the others may still read this CTA's words)
        }
    }
}

template <bool kBf16, bool kMask, int kThreads>
cudaError_t launch_clusters(const SampleArgs &a, int ranks, size_t smem, cudaStream_t stream) {
    static std::atomic<uint64_t> configured{0};
    cudaError_t e = set_smem_max_once(cluster_kernel<kBf16, kMask, kThreads>, configured);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    // (Float32 nuclei beyond a list are left over.  Of bf16 rows few are, and clusters that find
    // nothing cost time, so a cluster has 32 rows; a row with more than kTinyRoom values within
    // 2^-10 of 0 is one, and where all are, as with flat logits of a deviation below 0.1, those 32
    // follow one another: 64 rows of 151936 take 1.9 ms then, 0.07 otherwise.)
    const int64_t each = !a.after_rows ? 1 : kBf16 ? 32 : a.n_rows <= 512 ? 1 : 2;
    cfg.gridDim = dim3(static_cast<unsigned>((a.n_rows + each - 1) / each * ranks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(ranks);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, cluster_kernel<kBf16, kMask, kThreads>, a);
}

template <bool kBf16, bool kMask>
cudaError_t launch_typed(const SampleArgs &a, int ranks, cudaStream_t stream) {
    constexpr int kElt = kBf16 ? 2 : 4;
    if (a.after_rows) {
        static std::atomic<uint64_t> configured{0};
        cudaError_t e = set_smem_once(row_kernel<kBf16, kMask>, sizeof(RowShared), configured);
        if (e != cudaSuccess) return e;
        row_kernel<kBf16, kMask><<<static_cast<unsigned>(a.n_rows), kRowThreads, sizeof(RowShared), stream>>>(a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    const size_t smem = static_cast<size_t>(a.chunk_room) * 16 + sizeof(Shared);
    const bool alone = a.n_rows * ranks <= device_sm_count();
    return a.slice * kElt <= 49152 && !(alone && a.slice >= 8192) ? launch_clusters<kBf16, kMask, 256>(a, ranks, smem, stream)
                                                                  : launch_clusters<kBf16, kMask, 512>(a, ranks, smem, stream);
}

}  // namespace

// A cluster's slices have at most 40 KB where 8 CTAs can hold the row so: three CTAs of 256
// threads a multiprocessor (a slice and 18.5 KB beside it each; four up to 37 KB), of which one
// loads while others count.  Shorter rows go to fewer CTAs, one at last, unless rows are so few
// that multiprocessors would stand idle.  Slices beyond 48 KB (float32 rows of a large
// vocabulary) have twice the threads, and so have those of 8192 tokens and more that have a
// multiprocessor to themselves (8 rows of 151936 bf16, all kinds of filters: 41 us with 256,
// 33 with 512; of 37984 under top-k and top-p 19 and 21, of 1024 41 and 43).
cudaError_t launch_sample(const SampleCall &c, cudaStream_t stream) {
    if (c.n_rows == 0) return cudaSuccess;
    const bool bf16 = c.dtype == LPD_BF16, mask = c.mask != nullptr;
    const int64_t elt = bf16 ? 2 : 4;
    int ranks = 1;
    while (ranks < 8 && c.vocab * elt > ranks * int64_t{40960}) ranks *= 2;
    while (ranks < 8 && c.n_rows * ranks < device_sm_count() && c.vocab > ranks * int64_t{4096}) ranks *= 2;
    SampleArgs a{};
    a.x = static_cast<const char *>(c.x);
    a.x_stride = c.x_stride_elems * elt;
    a.n_rows = c.n_rows;
    a.vocab = static_cast<int>(c.vocab);
    a.slice = static_cast<int>(((c.vocab + ranks - 1) / ranks + 63) / 64 * 64);
    a.chunk_room = static_cast<int>(std::max<int64_t>((a.slice * elt + 15) / 16 + 1, 1024));  // (also the cluster's lists)
    a.f = c.f;
    a.uniform = c.uniform;
    a.ids = c.ids;
    a.logp = c.logp;
    a.keep = c.keep;
    a.active = c.active;
    a.mask = c.mask;
    a.mask_stride = c.mask_stride;
    a.lse = c.lse;
    a.kept = c.kept;
    a.after_rows = c.n_rows >= (bf16 ? kAloneBf16 : kAloneF32) ? 1 : 0;
    if (bf16) return mask ? launch_typed<true, true>(a, ranks, stream) : launch_typed<true, false>(a, ranks, stream);
    return mask ? launch_typed<false, true>(a, ranks, stream) : launch_typed<false, false>(a, ranks, stream);
}

}  // namespace lpd
