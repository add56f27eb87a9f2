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
constexpr int kList = 512;          // candidates a CTA keeps
constexpr int kReach = 512;         // thread maxima of a cluster that a nucleus's candidates go down to
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
    uint32_t list[kList];
    uint16_t list_at[kList];           // elements of the slice
    uint32_t cnt[2][kBins], mass_lo[2][kBins], mass_hi[2][kBins], far[2][kBins];
    // read by the cluster's other CTAs
    uint64_t list_mass, rest_mass, kept_mass;
    uint32_t list_n, rest_n;
    uint32_t top, floor_key, key_min, key_max;
    int bad;
    // the CTA's own
    uint64_t red64[2][kMaxWarps];
    uint32_t red32[2][kMaxWarps];
    uint64_t found_mass, found_excl_mass;
    uint32_t found_bin, found_cnt, found_excl, found_far, found_before;
    double log_min_p;
    float base;
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
    // The mask starts empty: where the border is found in the list, rank 0 adds its bits.
    if constexpr (kMask)
        for (int w = t; w < words; w += kThreads) mask_row[w] = 0;
    const auto nothing = [&](float value) {  // a row without an answer
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
    // (doubles are slow here: one thread's work, under the loads)
    if (min_p > 0.f && t == kThreads - 1) sh.log_min_p = log(fmin(static_cast<double>(min_p), 1.0));

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
    // Each warp's R-th largest thread maximum, R = k / (warps of the cluster):
    // the smallest of them is reached by k tokens at least.  Above 32 there is
    // no such value and the list stays empty.
    const int reach = ((use_k ? top_k : kReach) + ranks * kWarps - 1) / (ranks * kWarps);
    uint32_t floor_key = 0xffffffffu;
    {
        const bool bad = tmax != tmax;
        const uint32_t key = bad ? 0u : key_of<kBf16>(tmax), key16 = kBf16 ? key : key >> 16;
        uint32_t prefix = 0;
        if (reach <= 32) {
#pragma unroll
            for (uint32_t bit = 0x8000u; bit; bit >>= 1)
                if (__popc(__ballot_sync(0xffffffffu, key16 >= (prefix | bit))) >= reach) prefix |= bit;
        }
        const uint32_t wm = __reduce_max_sync(0xffffffffu, key);
        if (lane == 0) {
            sh.red32[0][warp] = wm;
            sh.red32[1][warp] = kBf16 ? prefix : prefix << 16;
        }
        const int any_bad = __syncthreads_or(bad);
        if (warp == 0) {
            const uint32_t m = __reduce_max_sync(0xffffffffu, lane < kWarps ? sh.red32[0][lane] : 0u);
            const uint32_t f = __reduce_min_sync(0xffffffffu, lane < kWarps ? sh.red32[1][lane] : 0xffffffffu);
            if (lane == 0) {
                sh.top = n > 0 ? m : 0;
                sh.floor_key = n > 0 && reach <= 32 ? f : 0xffffffffu;
                sh.bad = any_bad;
                sh.list_n = 0;
            }
        }
        cluster.sync();
    }
    // (a lane reads one CTA's words; a cluster has 8 at most)
    const Shared *const peer = cluster.map_shared_rank(&sh, lane < ranks ? lane : 0);
    const uint32_t top_key = __reduce_max_sync(0xffffffffu, peer->top);
    floor_key = __reduce_min_sync(0xffffffffu, peer->floor_key);
    const bool bad = __any_sync(0xffffffffu, peer->bad != 0);
    const float top = value_of<kBf16>(top_key);
    if (bad || !(fabsf(top) <= FLT_MAX)) {  // NaN, +inf, or nothing above -inf: no distribution
        cluster.sync();  // (the others may still be reading)
        return nothing(CUDART_NAN_F);
    }

    const WeightScale ws = weight_scale(scale, top);
    // What min-p leaves: x >= base, the smallest value with (x - top) scale >= log(min_p).
    float base = -FLT_MAX;
    if (min_p > 0.f) {
        if (t == 0) {
            const double lp = sh.log_min_p, s = scale, tp = top;
            float f = static_cast<float>(fmax(tp + lp / s, -static_cast<double>(FLT_MAX)));
            for (int i = 0; i < 4 && !((static_cast<double>(f) - tp) * s >= lp); ++i) f = nextafterf(f, CUDART_INF_F);
            for (int i = 0; i < 4; ++i) {
                const float g = nextafterf(f, -CUDART_INF_F);
                if (!((static_cast<double>(g) - tp) * s >= lp) || !(g >= -FLT_MAX)) break;
                f = g;
            }
            sh.base = fminf(f, top);
        }
        __syncthreads();
        base = sh.base;
    }
    if constexpr (kBf16) {  // up to a bf16 value, so that its key is its own
        const float down = __uint_as_float(__float_as_uint(base) & 0xffff0000u);
        base = down < base ? __uint_as_float((__float_as_uint(base) & 0xffff0000u) + 0x10000u) : down;
    }
    const bool listed = floor_key != 0xffffffffu;
    const float floor_x = !listed ? CUDART_INF_F : floor_key <= key_of<kBf16>(-FLT_MAX) ? -FLT_MAX : value_of<kBf16>(floor_key);
    const float cand = fmaxf(floor_x, base);
    // the heaviest candidates are weighed in double, in wide rows every token
    const float precise_from = ws.wide ? -FLT_MAX : fmaxf(floor_x, top - __fdiv_rn(kPreciseOctaves * kUnits, ws.ch));
    const auto weight = [&](float x) -> uint64_t {
        if (x >= precise_from) return weight_precise(x, ws, top, kTables.precise);
        return x > ws.cut ? weight_rough(x, ws, sh.table) : 0;
    };

    // ------------------------------------------------------------- candidates, and the mass of the others
    const auto push = [&](float x, int e) {
        const uint32_t at = atomicAdd(&sh.list_n, 1u);
        if (at < kList) {
            sh.list[at] = key_of<kBf16>(x);
            sh.list_at[at] = static_cast<uint16_t>(e);
        }
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
                    if (v[q] >= cand) push(v[q], i * kPer + q);
            }
        }
    } else {
        // (what is no candidate is lighter than any that is weighed in double)
        const auto others = [&](auto count, auto wide) {
            const float light = fmaxf(ws.cut, nextafterf(base, -CUDART_INF_F));
            for (int i = t; i < n_chunks; i += kThreads) {
                float v[kPer];
                unpack<kBf16>(chunks[i], v);
#pragma unroll
                for (int q = 0; q < kPer; ++q) {
                    if (v[q] >= cand) {
                        push(v[q], i * kPer + q);
                    } else {
                        if constexpr (wide.value) rest += v[q] >= base ? weight(v[q]) : 0;
                        else rest += v[q] > light ? weight_rough(v[q], ws, sh.table) : 0;
                        if constexpr (count.value) rest_n += v[q] >= base;
                    }
                }
            }
        };
        if (ws.wide) others(std::true_type{}, std::true_type{});
        else if (use_p) others(std::false_type{}, std::false_type{});  // (the nucleus's size is counted in the list)
        else others(std::true_type{}, std::false_type{});
    }
    __syncthreads();
    const uint32_t own_n = sh.list_n, in_list = min(own_n, static_cast<uint32_t>(kList));
    // two masses and a number summed over the CTA, for every thread
    const auto block_sums = [&](uint64_t &v, uint64_t &w, uint32_t &c) {
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
        for (int q = 0; q < kWarps; ++q) {
            v += sh.red64[0][q];
            w += sh.red64[1][q];
            c += sh.red32[0][q];
        }
    };
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
            for (int i = t; i < n_chunks; i += kThreads) {
                float v[kPer];
                unpack<kBf16>(chunks[i], v);
#pragma unroll
                for (int q = 0; q < kPer; ++q)
                    if (v[q] >= cand) own_list_mass += weight(v[q]);
            }
        }
        block_sums(own_list_mass, own_rest_mass, own_rest_n);
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
    const auto share_of = [&](uint64_t whole) {  // the least mass that is top_p of the whole, at least 1
        const double want = ceil(fmax(static_cast<double>(top_p), 0.0) * static_cast<double>(whole));
        return min(max(static_cast<uint64_t>(want), static_cast<uint64_t>(1)), whole);
    };
    const auto lse_of = [&](uint64_t m) {
        const double origin = ws.wide ? static_cast<double>(top) * scale : ws.origin * kLn2Unit;
        return origin + log(static_cast<double>(m) * (1.0 / static_cast<double>(uint64_t{1} << kWeightOne)));
    };
    // The draw's place in the running mass: the first token that passes it.
    const auto place_of = [&](float u, uint64_t mass) {
        const uint64_t at = u > 0.f ? static_cast<uint64_t>(static_cast<double>(fminf(u, 1.f)) * static_cast<double>(mass)) : 0;
        return min(at, mass - 1);
    };
    const auto add_mass = [&](int buf, uint32_t b, uint64_t w) {
        const uint32_t lo = static_cast<uint32_t>(w), old = atomicAdd(&sh.mass_lo[buf][b], lo);
        const uint32_t hi = static_cast<uint32_t>(w >> 32) + (old + lo < old);
        if (hi) atomicAdd(&sh.mass_hi[buf][b], hi);
    };

    // ------------------------------------------------------- rows whose border is in the list: rank 0's
    const bool on_list = listed && !overflow && all_list_n <= static_cast<uint32_t>(a.chunk_room) &&
                         (complete || (use_k ? all_list_n >= static_cast<uint32_t>(top_k)
                                             : use_p && all_list_mass >= share_of(all_mass)));
    if (on_list) {
        // every CTA brings its list into rank 0's slice, which nothing needs any more
        const uint32_t total = all_list_n;
        char *const home = rank == 0 ? smem : cluster.map_shared_rank(smem, 0);
        uint64_t *const w_of = reinterpret_cast<uint64_t *>(home);
        uint32_t *const far_of = reinterpret_cast<uint32_t *>(w_of + a.chunk_room), *const id_of = far_of + a.chunk_room;
        const uint32_t before = __reduce_add_sync(0xffffffffu, lane < rank ? peer_n : 0u);
        for (uint32_t i = t; i < own_n; i += kThreads) {
            w_of[before + i] = use_k ? weight(value_of<kBf16>(sh.list[i])) : sh.list_w[i];
            far_of[before + i] = top_key - sh.list[i];  // how far below the top
            id_of[before + i] = first + sh.list_at[i] - lead;
        }
        cluster.sync();  // (and the masks' zeros are there)
        if (rank != 0) return;
        // The first position, from `lo` on, at which the entries' number (or mass) reaches
        // `target`; place(i, &position) says whether entry i counts.
        struct Picked {
            uint32_t at, cnt;
            uint64_t under_n, under_mass, mass;
        };
        const auto pick = [&](auto place, uint32_t lo, uint32_t hi, bool by_mass, uint64_t target) {
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
                        add_mass(0, b, w_of[i]);
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
        };
        // Kept: `far` below the border's, and at the border the tokens up to `last_id`.
        uint32_t border = 0xffffffffu, last_id = 0xffffffffu;
        uint64_t kept_n = total, kept_mass = 0;
        uint32_t ties = 0, ties_all = 0;
        const uint32_t deepest = top_key - key_of<kBf16>(fminf(cand, top));
        const auto at_far = [&](uint32_t i, uint32_t *p) {
            *p = far_of[i];
            return true;
        };
        uint64_t whole_mass = all_list_mass;
        if (use_k && total <= static_cast<uint32_t>(top_k)) {  // nothing to leave out
            uint64_t none = 0;
            uint32_t c = 0;
            for (uint32_t i = t; i < total; i += kThreads) whole_mass += w_of[i];
            block_sums(whole_mass, none, c);
        }
        if (use_k && total > static_cast<uint32_t>(top_k)) {
            const Picked p = pick(at_far, 0, deepest, false, top_k);
            border = p.at;
            ties = static_cast<uint32_t>(top_k - p.under_n);
            ties_all = p.cnt;
            kept_n = top_k;
            kept_mass = p.under_mass + ties * (p.mass / p.cnt);  // (one weight p.cnt times)
        }
        if (use_p) {
            const uint64_t target = share_of(!use_k ? all_mass : ties_all ? kept_mass : whole_mass);
            const Picked p = pick(at_far, 0, min(border, deepest), true, target);
            const uint64_t one = p.mass / p.cnt;
            border = p.at;
            ties = static_cast<uint32_t>((target - p.under_mass + one - 1) / one);
            ties_all = p.cnt;
            kept_n = p.under_n + ties;
            kept_mass = p.under_mass + ties * one;
        }
        if (ties_all == 0) kept_mass = whole_mass;
        if (ties < ties_all) {
            const auto at_border = [&](uint32_t i, uint32_t *p) {
                *p = id_of[i];
                return far_of[i] == border;
            };
            last_id = pick(at_border, 0, a.vocab - 1, false, ties).at;
        }
        const auto is_kept = [&](uint32_t far, uint32_t id) { return far < border || (far == border && id <= last_id); };
        if constexpr (kMask) {
            uint32_t *const words_of = a.mask + row * a.mask_stride;
            for (uint32_t i = t; i < total; i += kThreads)
                if (is_kept(far_of[i], id_of[i])) atomicOr(words_of + id_of[i] / 32, 1u << (id_of[i] % 32));
            if (t == 0) {
                const int64_t id = a.keep ? a.keep[row] : -1;
                if (id >= 0 && id < a.vocab) {
                    const char *from = a.x + row * a.x_stride + id * kElt;
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
                if (a.lse) a.lse[row] = static_cast<float>(lse_of(kept_mass));
            }
        } else {
            const float u = a.uniform[row];
            const auto at_kept = [&](uint32_t i, uint32_t *p) {
                *p = id_of[i];
                return is_kept(far_of[i], id_of[i]);
            };
            const uint32_t id = pick(at_kept, 0, a.vocab - 1, true, place_of(u, kept_mass) + 1).at;
            for (uint32_t i = t; i < total; i += kThreads)
                if (id_of[i] == id) {
                    const float x = value_of<kBf16>(top_key - far_of[i]);
                    const bool drawn = u == u;
                    a.ids[row] = drawn ? static_cast<int32_t>(id) : -1;
                    if (a.logp) a.logp[row] = drawn ? static_cast<float>(static_cast<double>(x) * scale - lse_of(kept_mass)) : CUDART_NAN_F;
                    if (a.kept) a.kept[row] = static_cast<int32_t>(kept_n);
                }
        }
        return;
    }

    // ------------------------------------------------ the others: the border by rounds over the slices
    // Kept: keys above `border`, and the first `ties` of the tokens at it.
    uint32_t border = base_key, ties = 0xffffffffu, ties_before = 0, ties_own = 0;
    uint64_t above_mass = 0, above_n = 0, tie_weight = 0;
    bool whole = true;  // everything from `base` on is kept
    int round = 0;
    const auto each = [&](auto f) {  // f(value) for the slice's values
        for (int i = t; i < n_chunks; i += kThreads) {
            float v[kPer];
            unpack<kBf16>(chunks[i], v);
#pragma unroll
            for (int q = 0; q < kPer; ++q) f(v[q]);
        }
    };
    // Adds up a round's bins (in buffer `buf`) over the cluster and finds the first, from the
    // last one down, at which the tokens (or their mass) reach `target`.
    uint64_t over_mass = 0, over_n = 0;
    const auto descend = [&](int buf, bool by_mass, uint64_t target) -> uint32_t {
        if (t == 0) sh.found_bin = kBins;
        cluster.sync();
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
                    mass += static_cast<uint64_t>(o->mass_hi[buf][bin]) << 32 | o->mass_lo[buf][bin];
                    largest = max(largest, o->far[buf][bin]);
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
            sh.red32[0][warp] = up_n;
            sh.red64[0][warp] = up_mass;
        }
        __syncthreads();
        if (t < kBins) {
            for (int w = 0; w < warp; ++w) {
                up_n += sh.red32[0][w];
                up_mass += sh.red64[0][w];
            }
            const uint64_t upto = by_mass ? over_mass + up_mass : over_n + up_n;
            const uint64_t under = upto - (by_mass ? mass : cnt);
            if (under < target && upto >= target) {
                sh.found_bin = bin;
                sh.found_cnt = cnt;
                sh.found_mass = mass;
                sh.found_excl = up_n - cnt;
                sh.found_excl_mass = up_mass - mass;
                sh.found_far = largest;
                sh.found_before = before;
            }
        }
        __syncthreads();
        ++round;  // (others may still read this round's bins: the next takes the other buffer)
        return sh.found_bin;
    };
    const auto clear = [&](int buf) {
        for (int b = t; b < kBins; b += kThreads) sh.cnt[buf][b] = sh.mass_lo[buf][b] = sh.mass_hi[buf][b] = sh.far[buf][b] = 0;
        __syncthreads();
    };
    // The first key, from the top down to `lo`, at which the tokens (or their mass) reach
    // `target`; false if they don't.  The first round's bins are cut evenly between the
    // top and where weights end (keys would crowd: half of them lie within 2^-64 of 0).
    const float last_x = fmaxf(base, ws.wide ? top - __fdiv_rn(46.f, fmaxf(scale, FLT_MIN)) : ws.cut);
    const float per_bin = __fdiv_rn(kBins - 1.f, fmaxf(top - last_x, FLT_MIN));
    const auto coarse = [&](float x) { return kBins - 1 - static_cast<uint32_t>(fminf(__fmul_rn(__fsub_rn(top, x), per_bin), kBins - 1.f)); };
    const auto select = [&](bool by_mass, uint64_t target, uint32_t lo) -> bool {
        over_mass = over_n = 0;
        clear(round & 1);
        {
            const int buf = round & 1;
            each([&](float x) {
                if (key_of<kBf16>(x) >= lo) {
                    const uint32_t b = coarse(x);
                    atomicAdd(&sh.cnt[buf][b], 1u);
                    add_mass(buf, b, weight(x));
                }
            });
            const uint32_t fb = descend(buf, by_mass, target);
            if (fb == kBins) return false;
            over_n += sh.found_excl;
            over_mass += sh.found_excl_mass;
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
                sh.red32[0][warp] = least;
                sh.red32[1][warp] = most;
            }
            __syncthreads();
            if (t == 0) {
                for (int w = 1; w < kWarps; ++w) {
                    least = min(least, sh.red32[0][w]);
                    most = max(most, sh.red32[1][w]);
                }
                sh.key_min = least;
                sh.key_max = most;
            }
            cluster.sync();
        }
        uint32_t hi = 0;
        lo = 0xffffffffu;
        for (int r = 0; r < ranks; ++r) {
            const Shared *o = cluster.map_shared_rank(&sh, r);
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
                    atomicAdd(&sh.cnt[buf][b], 1u);
                    sh.far[buf][b] = key;  // (read where it is the only one)
                    add_mass(buf, b, weight(x));
                }
            });
            const uint32_t fb = descend(buf, by_mass, target);
            over_n += sh.found_excl;
            over_mass += sh.found_excl_mass;
            const uint32_t fc = sh.found_cnt;
            if (shift == 0 || fc == 1 || turn == 4) {
                border = shift == 0 ? lo + fb : sh.found_far;
                above_n = over_n;
                above_mass = over_mass;
                tie_weight = sh.found_mass / fc;  // (one weight fc times)
                ties_before = sh.found_before;
                ties_own = sh.cnt[buf][fb];
                const uint64_t left = target - (by_mass ? over_mass : over_n);
                ties = static_cast<uint32_t>(by_mass ? (left + tie_weight - 1) / tie_weight : left);
                whole = false;
                __syncthreads();
                return true;
            }
            lo += fb << shift;
            hi = min(hi, lo + ((1u << shift) - 1));
            __syncthreads();
        }
    };
    uint64_t kept_n = all_list_n + all_rest_n, kept_mass = all_mass;
    {
        uint32_t lo = base_key;
        if (use_k) {
            if (select(false, top_k, base_key)) {
                kept_n = top_k;
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
                block_sums(m, none, c);
                if (t == 0) {
                    sh.rest_mass = m;
                    sh.rest_n = c;
                }
                own_list_mass = 0;
                own_rest_mass = m;
                cluster.sync();
                kept_n = kept_mass = 0;
                for (int r = 0; r < ranks; ++r) {
                    const Shared *o = cluster.map_shared_rank(&sh, r);
                    kept_mass += o->rest_mass;
                    kept_n += o->rest_n;
                }
            }
        }
        if (use_p) {
            select(true, share_of(kept_mass), lo);  // (of a top-k's tied tokens it takes no more than that did)
            kept_n = above_n + ties;
            kept_mass = above_mass + ties * tie_weight;
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
        if (lane == 0) sh.red64[0][warp] = s;
        if (t == 0) sh.at = -1;
        __syncthreads();
        int w = 0;
        for (; w < kWarps - 1 && target >= sh.red64[0][w]; ++w) target -= sh.red64[0][w];
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
        if (lane == 31) sh.red64[0][warp] = up;
        __syncthreads();
        for (int q = 0; q < warp; ++q) up += sh.red64[0][q];
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
        uint64_t own = own_list_mass + own_rest_mass, none = 0;
        if (!whole) {
            uint32_t c = 0;
            own = 0;
            each([&](float x) {
                if (key_of<kBf16>(x) > border) own += weight(x);
            });
            block_sums(own, none, c);
            own += own_ties * tie_weight;
        }
        if (t == 0) sh.kept_mass = own;
        cluster.sync();
        const float u = a.uniform[row];
        const uint64_t target = place_of(u, kept_mass);
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
    const size_t smem = static_cast<size_t>(a.chunk_room) * 16 + sizeof(Shared);
    if (a.slice * elt <= 49152) {
        if (bf16) return mask ? launch_typed<true, true, 256>(a, c.n_rows, ranks, smem, stream) : launch_typed<true, false, 256>(a, c.n_rows, ranks, smem, stream);
        return mask ? launch_typed<false, true, 256>(a, c.n_rows, ranks, smem, stream) : launch_typed<false, false, 256>(a, c.n_rows, ranks, smem, stream);
    }
    if (bf16) return mask ? launch_typed<true, true, 512>(a, c.n_rows, ranks, smem, stream) : launch_typed<true, false, 512>(a, c.n_rows, ranks, smem, stream);
    return mask ? launch_typed<false, true, 512>(a, c.n_rows, ranks, smem, stream) : launch_typed<false, false, 512>(a, c.n_rows, ranks, smem, stream);
}

}  // namespace lpd
