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
// A cluster of C CTAs takes a row; each CTA holds a slice of it in shared memory,
// so the row is read from memory once.  Each thread keeps the maximum of what it
// loads; the R-th largest of a CTA's thread maxima is a value that at least R of
// its tokens reach, so with R = k / C the tokens at or above the smallest of the
// C values are few and hold the top k (and mostly the nucleus).  They go into a
// list, and the border is found among them by histograms of 256 bins over the
// range of their keys, added up over the cluster through distributed shared
// memory.  Where the border lies below the list (a flat row, a large k, ties
// without end) the same histograms run over the slices.  Masses are whole numbers
// (lpd_weights.cuh), so neither the order of the atomics nor the cut into slices
// changes a bit.
#include <cfloat>
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <math_constants.h>

#include "lpd_internal.cuh"
#include "lpd_operators.cuh"
#include "lpd_weights.cuh"

namespace cg = cooperative_groups;

namespace lpd {
namespace {

constexpr int kBins = 256;
constexpr int kList = 512;          // candidates a CTA keeps
constexpr int kReach = 96;          // thread maxima that a nucleus's candidates go down to
constexpr int kMaxWarps = 32;
constexpr float kPreciseOctaves = 10.f;  // candidates within this of the top are weighed in double

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
    double precise[kUnits];
    WeightEntry rough[kUnits];
};
constexpr Tables make_tables() {
    Tables t{};
    for (int i = 0; i < kUnits; ++i) {
        const double v = series_exp(kLn2Unit * i);
        t.precise[i] = v;
        t.rough[i].whole = static_cast<uint32_t>(v * 1073741824.0 + 0.5);
        t.rough[i].part = static_cast<float>(v * 1073741824.0);
    }
    return t;
}
__device__ constexpr Tables kTables = make_tables();

struct Shared {
    WeightEntry table[kUnits];
    uint64_t list_w[kList];
    uint64_t mass[2][kBins];
    uint32_t cnt[2][kBins];
    uint32_t kmax[2][kBins];
    uint32_t list[kList];
    // read by the cluster's other CTAs
    uint64_t list_mass, rest_mass, kept_mass;
    uint32_t list_n, rest_n;
    uint32_t top, floor_key;
    int bad;
    // the CTA's own
    uint64_t red64[kMaxWarps];
    uint32_t red32[kMaxWarps];
    uint64_t found_mass, found_excl_mass;
    uint32_t found_bin, found_cnt, found_excl;
    int at;
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

struct SampleArgs {
    const char *x;
    int64_t x_stride;  // bytes
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
};

template <bool kBf16, bool kMask, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) sample_kernel(const __grid_constant__ SampleArgs a) {
    constexpr int kElt = kBf16 ? 2 : 4, kPer = 16 / kElt, kWarps = kThreads / 32;
    extern __shared__ __align__(16) char smem[];
    uint4 *const chunks = reinterpret_cast<uint4 *>(smem);
    Shared &sh = *reinterpret_cast<Shared *>(smem + static_cast<size_t>(a.chunk_room) * 16);
    const cg::cluster_group cluster = cg::this_cluster();
    const int ranks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int64_t row = blockIdx.x / ranks;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int first = rank * a.slice;                                   // the slice's first token
    const int n = max(0, min(a.slice, a.vocab - first));                // and its tokens
    const int words = (n + 31) / 32;
    uint32_t *const mask_row = kMask ? a.mask + row * a.mask_stride + first / 32 : nullptr;

    const float scale = a.f.scale ? a.f.scale[row] : 1.f, min_p = a.f.min_p ? a.f.min_p[row] : 0.f;
    const float top_p = a.f.top_p ? a.f.top_p[row] : 1.f;
    const int top_k = a.f.top_k ? a.f.top_k[row] : 0;
    const auto nothing = [&](float value) {  // a row without an answer
        if constexpr (kMask)
            for (int w = t; w < words; w += kThreads) mask_row[w] = 0;
        if (rank == 0 && t == 0) {
            if (a.kept) a.kept[row] = 0;
            if constexpr (kMask) {
                if (a.lse) a.lse[row] = value;
            } else {
                a.ids[row] = -1;
                if (a.logp) a.logp[row] = value;
            }
        }
    };
    if (kMask && a.active && a.active[row] == 0) return nothing(0.f);
    if (!(scale > 0.f && scale <= FLT_MAX) || min_p != min_p || top_p != top_p) return nothing(CUDART_NAN_F);
    const bool use_k = top_k > 0 && top_k < a.vocab, use_p = top_p < 1.f;

    // ------------------------------------------------------------------ the slice, and each thread's maximum
    const char *const src = a.x + row * a.x_stride + static_cast<int64_t>(first) * kElt;
    const int lead = static_cast<int>((reinterpret_cast<uintptr_t>(src) & 15u) / kElt);  // elements of the first chunk in front of it
    const int end = lead + n, n_chunks = n > 0 ? (end + kPer - 1) / kPer : 0;
    float tmax = -CUDART_INF_F;
    {
        const uint4 *const from = reinterpret_cast<const uint4 *>(src - lead * kElt);
        const int c0 = lead > 0 ? 1 : 0, c1 = end / kPer;  // whole chunks
        constexpr int kAhead = 4;
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
        // the first and the last chunk where they hold others' elements too:
        // those read as -inf (a chunk is never read outside the slice)
        if (t < 2) {
            const int e = t == 0 ? 0 : n_chunks - 1;
            if (e >= 0 && e < n_chunks && (t == 0 ? c0 == 1 || c1 == 0 : e > 0 && e >= c1)) {
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
                const uint4 c = make_uint4(w[0], w[1], w[2], w[3]);
                chunks[e] = c;
                tmax = max_nan(tmax, chunk_max<kBf16>(c));
            }
        }
        for (int i = t; i < kUnits; i += kThreads) sh.table[i] = kTables.rough[i];
    }

    // --------------------------------------------- the row's top, and a value that enough tokens reach
    // R thread maxima a CTA; above the threads' number there is no such value
    // and the list stays empty.
    const int reach = use_k ? (top_k + ranks - 1) / ranks : kReach;
    uint32_t floor_key = 0xffffffffu;
    {
        const bool bad = tmax != tmax;
        const uint32_t key = bad ? 0u : key_of<kBf16>(tmax), key16 = kBf16 ? key : key >> 16;
        if (t == 0) sh.bad = 0;
        const uint32_t wm = __reduce_max_sync(0xffffffffu, key);
        if (lane == 0) sh.red32[warp] = wm;
        const int any_bad = __syncthreads_or(bad);
        if (n > 0 && reach <= kThreads) {
            uint32_t prefix = 0;
#pragma unroll 1
            for (uint32_t bit = 0x8000u; bit; bit >>= 1)
                if (__syncthreads_count(key16 >= (prefix | bit)) >= reach) prefix |= bit;
            floor_key = kBf16 ? prefix : prefix << 16;
        }
        if (t == 0) {
            uint32_t m = 0;
            for (int w = 0; w < kWarps; ++w) m = max(m, sh.red32[w]);
            sh.top = n > 0 ? m : 0;
            sh.floor_key = floor_key;
            sh.bad = any_bad;
        }
        cluster.sync();
    }
    uint32_t top_key = 0;
    int bad = 0;
    for (int r = 0; r < ranks; ++r) {
        const Shared *o = cluster.map_shared_rank(&sh, r);
        top_key = max(top_key, o->top);
        floor_key = min(floor_key, o->floor_key);
        bad |= o->bad;
    }
    const float top = value_of<kBf16>(top_key);
    if (bad || !(fabsf(top) <= FLT_MAX)) {  // NaN, +inf, or nothing above -inf: no distribution
        cluster.sync();  // (the others may still be reading)
        return nothing(CUDART_NAN_F);
    }

    const WeightScale ws = weight_scale(scale, top);
    // What min-p leaves: x >= base, the smallest float with (x - top) scale >= log(min_p).
    float base = -FLT_MAX;
    if (min_p > 0.f) {
        const double lp = log(fmin(static_cast<double>(min_p), 1.0)), s = scale, tp = top;
        float f = static_cast<float>(fmax(tp + lp / s, -static_cast<double>(FLT_MAX)));
        for (int i = 0; i < 4 && !((static_cast<double>(f) - tp) * s >= lp); ++i) f = nextafterf(f, CUDART_INF_F);
        for (int i = 0; i < 4; ++i) {
            const float g = nextafterf(f, -CUDART_INF_F);
            if (!((static_cast<double>(g) - tp) * s >= lp) || !(g >= -FLT_MAX)) break;
            f = g;
        }
        base = fminf(f, top);
    }
    if constexpr (kBf16) {  // up to a bf16 value, so that its key is its own
        const float down = __uint_as_float(__float_as_uint(base) & 0xffff0000u);
        base = down < base ? __uint_as_float((__float_as_uint(base) & 0xffff0000u) + 0x10000u) : down;
    }
    const bool listed = floor_key != 0xffffffffu;
    const float floor_x = !listed ? CUDART_INF_F : floor_key <= key_of<kBf16>(-FLT_MAX) ? -FLT_MAX : value_of<kBf16>(floor_key);
    const float cand = fmaxf(floor_x, base);
    // the heaviest candidates are weighed in double, in wide rows every token
    const float precise_from = ws.wide ? -FLT_MAX : fmaxf(floor_x, static_cast<float>(top - kPreciseOctaves * kUnits / ws.c));
    const auto weight = [&](float x) -> uint64_t {
        if (x >= precise_from) return weight_precise(x, ws, top, kTables.precise);
        return x > ws.cut ? weight_rough(x, ws, sh.table) : 0;
    };

    // ------------------------------------------------------------- candidates, and the mass of the others
    if (t == 0) sh.list_n = 0;
    __syncthreads();
    const auto push = [&](float x) {
        const uint32_t at = atomicAdd(&sh.list_n, 1u);
        if (at < kList) sh.list[at] = key_of<kBf16>(x);
    };
    uint64_t rest = 0;
    uint32_t rest_n = 0;
    if (use_k) {
        for (int i = t; i < n_chunks; i += kThreads) {
            const uint4 c = chunks[i];
            if (chunk_max<kBf16>(c) >= cand) {
                float v[kPer];
                unpack<kBf16>(c, v);
#pragma unroll
                for (int q = 0; q < kPer; ++q)
                    if (v[q] >= cand) push(v[q]);
            }
        }
    } else {
        for (int i = t; i < n_chunks; i += kThreads) {
            float v[kPer];
            unpack<kBf16>(chunks[i], v);
#pragma unroll
            for (int q = 0; q < kPer; ++q) {
                if (v[q] >= cand) {
                    push(v[q]);
                } else if (v[q] >= base) {
                    rest += weight(v[q]);
                    ++rest_n;
                }
            }
        }
    }
    __syncthreads();
    const uint32_t own_n = sh.list_n, in_list = min(own_n, static_cast<uint32_t>(kList));
    uint64_t list_mass = 0;
    for (uint32_t i = t; i < in_list; i += kThreads) {
        const uint64_t w = weight(value_of<kBf16>(sh.list[i]));
        sh.list_w[i] = w;
        list_mass += w;
    }
    if (own_n > kList) {  // the list does not hold them all: their mass is the slice's
        list_mass = 0;
        for (int i = t; i < n_chunks; i += kThreads) {
            float v[kPer];
            unpack<kBf16>(chunks[i], v);
#pragma unroll
            for (int q = 0; q < kPer; ++q)
                if (v[q] >= cand) list_mass += weight(v[q]);
        }
    }
    // sums over the CTA into thread 0's `v`
    const auto block_sum = [&](uint64_t v) -> uint64_t {
        v = warp_sum(v);
        __syncthreads();
        if (lane == 0) sh.red64[warp] = v;
        __syncthreads();
        v = 0;
        for (int w = 0; w < kWarps; ++w) v += sh.red64[w];
        return v;
    };
    const uint64_t own_list_mass = block_sum(list_mass), own_rest_mass = block_sum(rest);
    const uint32_t own_rest_n = static_cast<uint32_t>(block_sum(rest_n));
    if (t == 0) {
        sh.list_mass = own_list_mass;
        sh.rest_mass = own_rest_mass;
        sh.rest_n = own_rest_n;
    }
    cluster.sync();
    uint64_t all_list_mass = 0, all_rest_mass = 0, all_list_n = 0, all_rest_n = 0;
    bool overflow = false;
    for (int r = 0; r < ranks; ++r) {
        const Shared *o = cluster.map_shared_rank(&sh, r);
        all_list_mass += o->list_mass;
        all_rest_mass += o->rest_mass;
        all_list_n += o->list_n;
        all_rest_n += o->rest_n;
        overflow |= o->list_n > kList;
    }

    // ------------------------------------------------------------------------------ the border
    // Kept: keys above `border`, and the first `ties` of the tokens at it.
    uint32_t border = key_of<kBf16>(base), ties = 0xffffffffu, ties_before = 0, ties_own = 0, ties_all = 0;
    uint64_t above_mass = 0, above_n = 0, tie_weight = 0;
    bool whole = true, from_list = false;  // `whole`: everything from `base` on is kept
    int round = 0;
    // The first key, going down from the top to `lo`, at which the tokens (or
    // their mass) reach `target`; false if they don't.
    const auto select = [&](bool by_mass, uint64_t target, uint32_t lo, bool list) -> bool {
        uint32_t hi = top_key;
        uint64_t over_mass = 0, over_n = 0;
#pragma unroll 1
        for (;; ++round) {
            const int buf = round & 1;
            const uint32_t span = hi - lo;
            const int shift = max(0, 24 - __clz(span | 1u));
            for (int b = t; b < kBins; b += kThreads) {
                sh.cnt[buf][b] = 0;
                sh.kmax[buf][b] = 0;
                sh.mass[buf][b] = 0;
            }
            __syncthreads();
            const auto add = [&](uint32_t key, uint64_t w) {
                const uint32_t b = (key - lo) >> shift;
                atomicAdd(&sh.cnt[buf][b], 1u);
                atomicMax(&sh.kmax[buf][b], key);
                if (w) atomicAdd(reinterpret_cast<unsigned long long *>(&sh.mass[buf][b]), static_cast<unsigned long long>(w));
            };
            if (list) {
                for (uint32_t i = t; i < in_list; i += kThreads) {
                    const uint32_t key = sh.list[i];
                    if (key >= lo && key <= hi) add(key, sh.list_w[i]);
                }
            } else {
                for (int i = t; i < n_chunks; i += kThreads) {
                    float v[kPer];
                    unpack<kBf16>(chunks[i], v);
#pragma unroll
                    for (int q = 0; q < kPer; ++q) {
                        const uint32_t key = key_of<kBf16>(v[q]);
                        if (key >= lo && key <= hi) add(key, weight(v[q]));
                    }
                }
            }
            if (t == 0) sh.found_bin = kBins;
            cluster.sync();
            // thread b: bin 255 - b of the whole row, then what lies above it
            uint32_t cnt = 0, before = 0, largest = 0;
            uint64_t mass = 0;
            const int bin = kBins - 1 - t;
            if (t < kBins) {
                for (int r = 0; r < ranks; ++r) {
                    const Shared *o = cluster.map_shared_rank(&sh, r);
                    const uint32_t c = o->cnt[buf][bin];
                    if (r < rank) before += c;
                    cnt += c;
                    if (c) {
                        mass += o->mass[buf][bin];
                        largest = max(largest, o->kmax[buf][bin]);
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
                sh.red32[warp] = up_n;
                sh.red64[warp] = up_mass;
            }
            __syncthreads();
            if (t < kBins) {
                for (int w = 0; w < warp; ++w) {
                    up_n += sh.red32[w];
                    up_mass += sh.red64[w];
                }
                const uint64_t upto = by_mass ? over_mass + up_mass : over_n + up_n;
                const uint64_t under = by_mass ? upto - mass : upto - cnt;
                if (under < target && upto >= target) {
                    sh.found_bin = bin;
                    sh.found_cnt = cnt;
                    sh.found_mass = mass;
                    sh.found_excl = up_n - cnt;
                    sh.found_excl_mass = up_mass - mass;
                    sh.at = static_cast<int>(largest);
                    sh.red32[kMaxWarps - 1] = before;
                }
            }
            __syncthreads();
            const uint32_t fb = sh.found_bin;
            if (fb == kBins) {  // (only in the first round: `lo` is reached)
                ++round;  // (others may still read this round's bins)
                return false;
            }
            over_n += sh.found_excl;
            over_mass += sh.found_excl_mass;
            const uint32_t fc = sh.found_cnt;
            if (shift == 0 || fc == 1) {
                border = shift == 0 ? lo + fb : static_cast<uint32_t>(sh.at);
                above_n = over_n;
                above_mass = over_mass;
                ties_all = fc;
                tie_weight = sh.found_mass / fc;  // (one weight fc times)
                ties_before = sh.red32[kMaxWarps - 1];
                ties_own = sh.cnt[buf][fb];
                const uint64_t left = target - (by_mass ? over_mass : over_n);
                ties = static_cast<uint32_t>(by_mass ? (left + tie_weight - 1) / tie_weight : left);
                whole = false;
                from_list = list;
                __syncthreads();  // (the results were read; the next round may write them)
                ++round;
                return true;
            }
            lo += fb << shift;
            hi = min(hi, lo + ((1u << shift) - 1));
            __syncthreads();
        }
    };
    const uint32_t base_key = key_of<kBf16>(base), cand_key = key_of<kBf16>(fminf(cand, top));
    uint64_t kept_n, kept_mass;
    {
        bool complete = listed && !overflow && cand <= base;  // the list is all that min-p leaves
        uint64_t set_n = all_list_n + all_rest_n, set_mass = all_list_mass + all_rest_mass;
        bool list_ok = listed && !overflow;
        uint32_t lo = base_key;
        if (use_k) {
            const bool on_list = list_ok && all_list_n >= static_cast<uint64_t>(top_k);
            bool some = false;
            if (on_list) some = select(false, top_k, cand_key, true);
            else if (!complete) some = select(false, top_k, base_key, false);
            if (some) {
                set_n = above_n + ties;
                set_mass = above_mass + ties * tie_weight;
                lo = border;
                list_ok = on_list;
            } else if (!complete) {  // fewer than top_k are left: the slices' whole
                uint64_t m = 0, c = 0;
                for (int i = t; i < n_chunks; i += kThreads) {
                    float v[kPer];
                    unpack<kBf16>(chunks[i], v);
#pragma unroll
                    for (int q = 0; q < kPer; ++q)
                        if (v[q] >= base) {
                            m += weight(v[q]);
                            ++c;
                        }
                }
                m = block_sum(m);
                c = block_sum(c);
                if (t == 0) {
                    sh.rest_mass = m;
                    sh.rest_n = static_cast<uint32_t>(c);
                }
                cluster.sync();
                set_n = set_mass = 0;
                for (int r = 0; r < ranks; ++r) {
                    const Shared *o = cluster.map_shared_rank(&sh, r);
                    set_mass += o->rest_mass;
                    set_n += o->rest_n;
                }
                list_ok = false;
            }
        } else if (list_ok && !complete && use_p) {
            // the nucleus's border lies in the list only if the list's mass reaches it
            list_ok = static_cast<double>(all_list_mass) >= ceil(static_cast<double>(top_p) * static_cast<double>(set_mass));
            if (list_ok) lo = cand_key;
        }
        kept_n = set_n;
        kept_mass = set_mass;
        if (use_p) {
            const double want = ceil(fmax(static_cast<double>(top_p), 0.0) * static_cast<double>(set_mass));
            const uint64_t target = min(max(static_cast<uint64_t>(want), static_cast<uint64_t>(1)), set_mass);
            const uint32_t most = use_k && !whole ? ties : 0xffffffffu, at = border;
            if (select(true, target, lo, list_ok)) {
                if (most != 0xffffffffu && border == at) ties = min(ties, most);
                kept_n = above_n + ties;
                kept_mass = above_mass + ties * tie_weight;
            }
        }
    }
    // this CTA's share of the tied tokens: all of them, none, or the first few
    const uint32_t own_ties = whole ? 0 : ties <= ties_before ? 0 : min(ties - ties_before, ties_own);

    // The first element of the slice whose running sum of f(element, value) passes `target`.
    const auto find = [&](auto f, uint64_t target) -> int {
        const int per_warp = (n_chunks + kWarps - 1) / kWarps;
        uint64_t s = 0;
        for (int i = warp * per_warp + lane; i < min(n_chunks, (warp + 1) * per_warp); i += 32) {
            float v[kPer];
            unpack<kBf16>(chunks[i], v);
#pragma unroll
            for (int q = 0; q < kPer; ++q) s += f(i * kPer + q, v[q]);
        }
        s = warp_sum(s);
        __syncthreads();
        if (lane == 0) sh.red64[warp] = s;
        if (t == 0) sh.at = -1;
        __syncthreads();
        int w = 0;
        for (; w < kWarps - 1 && target >= sh.red64[w]; ++w) target -= sh.red64[w];
        const int c0 = w * per_warp, c1 = min(n_chunks, c0 + per_warp);
        const int per = (per_warp + kThreads - 1) / kThreads;
        s = 0;
        for (int i = c0 + t * per; i < min(c1, c0 + (t + 1) * per); ++i) {
            float v[kPer];
            unpack<kBf16>(chunks[i], v);
#pragma unroll
            for (int q = 0; q < kPer; ++q) s += f(i * kPer + q, v[q]);
        }
        uint64_t up = s;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t p = __shfl_up_sync(0xffffffffu, up, o);
            if (lane >= o) up += p;
        }
        __syncthreads();
        if (lane == 31) sh.red64[warp] = up;
        __syncthreads();
        for (int q = 0; q < warp; ++q) up += sh.red64[q];
        if (up - s <= target && target < up) {
            uint64_t left = target - (up - s);
            for (int e = (c0 + t * per) * kPer, last = min(c1, c0 + (t + 1) * per) * kPer; e < last; ++e) {
                const float x = kBf16 ? __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const unsigned short *>(chunks)[e]) << 16)
                                      : reinterpret_cast<const float *>(chunks)[e];
                const uint64_t y = f(e, x);
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
    const double origin = ws.wide ? static_cast<double>(top) * scale : ws.origin * kLn2Unit;
    const auto lse_of = [&](uint64_t m) {
        return origin + log(static_cast<double>(m) * (1.0 / static_cast<double>(uint64_t{1} << kWeightOne)));
    };

    if constexpr (kMask) {
        cluster.barrier_arrive();
        const auto at = [&](int e) {
            return kBf16 ? __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const unsigned short *>(chunks)[e]) << 16)
                         : reinterpret_cast<const float *>(chunks)[e];
        };
        const int64_t id = a.keep ? a.keep[row] : -1;
        const bool mine = id >= first && id < first + n, forced_in = id >= 0 && id < a.vocab;
        const int forced = mine ? static_cast<int>(id - first) : -1;
        for (int w = warp; w < words; w += kWarps) {
            const int j = w * 32 + lane;
            bool k = false;
            if (j < n) {
                const float x = at(lead + j);
                k = is_kept(lead + j, x) || (j == forced && x >= -FLT_MAX);
            }
            const uint32_t word = __ballot_sync(0xffffffffu, k);
            if (lane == 0) mask_row[w] = word;
        }
        if (t == 0 && (forced_in ? mine : rank == 0)) {
            if (mine) {
                const float x = at(lead + forced);
                if (x >= -FLT_MAX && !is_kept(lead + forced, x)) {
                    kept_n += 1;
                    kept_mass += weight(x);
                }
            }
            if (a.kept) a.kept[row] = static_cast<int32_t>(kept_n);
            if (a.lse) a.lse[row] = static_cast<float>(lse_of(kept_mass));
        }
        cluster.barrier_wait();
    } else {
        // ------------------------------------------------------------------------------ the draw
        uint64_t own = 0;
        if (whole && !(use_k && !(listed && !overflow && cand <= base))) {
            own = own_list_mass + own_rest_mass;
        } else if (whole) {
            own = sh.rest_mass;
        } else {
            if (from_list) {
                for (uint32_t i = t; i < in_list; i += kThreads)
                    if (sh.list[i] > border) own += sh.list_w[i];
            } else {
                for (int i = t; i < n_chunks; i += kThreads) {
                    float v[kPer];
                    unpack<kBf16>(chunks[i], v);
#pragma unroll
                    for (int q = 0; q < kPer; ++q)
                        if (key_of<kBf16>(v[q]) > border) own += weight(v[q]);
                }
            }
            own = block_sum(own) + own_ties * tie_weight;
        }
        if (t == 0) sh.kept_mass = own;
        cluster.sync();
        const float u = a.uniform[row];
        uint64_t target = u > 0.f ? static_cast<uint64_t>(static_cast<double>(fminf(u, 1.f)) * static_cast<double>(kept_mass)) : 0;
        target = min(target, kept_mass - 1);
        uint64_t in_front = 0;
        for (int r = 0; r < rank; ++r) in_front += cluster.map_shared_rank(&sh, r)->kept_mass;
        cluster.barrier_arrive();
        if (target >= in_front && target - in_front < own) {
            const int e = find([&](int e, float x) -> uint64_t { return is_kept(e, x) ? weight(x) : 0; }, target - in_front);
            if (t == 0) {
                const float x = kBf16 ? __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const unsigned short *>(chunks)[e]) << 16)
                                      : reinterpret_cast<const float *>(chunks)[e];
                const bool drawn = u == u;
                a.ids[row] = drawn ? first + e - lead : -1;
                if (a.logp) a.logp[row] = drawn ? static_cast<float>(static_cast<double>(x) * scale - lse_of(kept_mass)) : CUDART_NAN_F;
                if (a.kept) a.kept[row] = static_cast<int32_t>(kept_n);
            }
        }
        cluster.barrier_wait();
    }
}

template <bool kBf16, bool kMask, int kThreads>
cudaError_t launch_typed(const SampleArgs &a, int64_t n_rows, int ranks, size_t smem, cudaStream_t stream) {
    static std::atomic<uint64_t> configured{0};
    cudaError_t e = set_smem_max_once(sample_kernel<kBf16, kMask, kThreads>, configured);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(n_rows * ranks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(ranks);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sample_kernel<kBf16, kMask, kThreads>, a);
}

}  // namespace

// Slices of at most 40 KB leave four CTAs a multiprocessor, one loading while
// others count; rows of fewer than that go to one CTA unless rows are so few that
// the multiprocessors would stand idle.  Larger slices (float32 rows of a large
// vocabulary) have twice the threads.
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
    a.vocab = static_cast<int>(c.vocab);
    a.slice = static_cast<int>(((c.vocab + ranks - 1) / ranks + 63) / 64 * 64);
    a.chunk_room = static_cast<int>((a.slice * elt + 15) / 16 + 1);
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
    const size_t smem = static_cast<size_t>(a.chunk_room) * 16 + sizeof(Shared);
    if (a.slice * elt <= 49152) {
        if (bf16) return mask ? launch_typed<true, true, 256>(a, c.n_rows, ranks, smem, stream) : launch_typed<true, false, 256>(a, c.n_rows, ranks, smem, stream);
        return mask ? launch_typed<false, true, 256>(a, c.n_rows, ranks, smem, stream) : launch_typed<false, false, 256>(a, c.n_rows, ranks, smem, stream);
    }
    if (bf16) return mask ? launch_typed<true, true, 512>(a, c.n_rows, ranks, smem, stream) : launch_typed<true, false, 512>(a, c.n_rows, ranks, smem, stream);
    return mask ? launch_typed<false, true, 512>(a, c.n_rows, ranks, smem, stream) : launch_typed<false, false, 512>(a, c.n_rows, ranks, smem, stream);
}

}  // namespace lpd
