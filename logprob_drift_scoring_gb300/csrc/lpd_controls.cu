// Sampling controls on logits: penalties for repeated tokens, biases, grammar
// masks and the request's temperature, in three forms.
//   apply_kernel     writes the controlled logits (what a sampler reads);
//   score_kernel     the log-sum-exp of both sides' controlled logits in one
//                    read of each row, never written to memory;
//   gradient_kernel  the selected-token logprob's gradient with respect to the
//                    raw logits.
// The mathematics of a row and the block's way of working on a chunk of it are
// described in lpd_controls.cuh.
//
// Method: "WS2 Cross-Config Logprob Drift Contract", "Measurement Contract":
// the rollout's tokens are scored under the distribution that they were
// sampled from.
//
// Bound: HBM.  Units of (row, 8192 columns) go to persistent blocks of 256
// threads, three or four a multiprocessor, so that one block's history scan
// and list run under another's loads; each block issues its unit's first loads
// before the scan.
#include <cfloat>

#include "lpd_controls.cuh"

namespace lpd {
namespace {

constexpr int kChunk = 8192;       // columns of a unit: one bitmap word a thread
constexpr int kSmallChunk = 2048;  // of the elementwise forms when few rows leave multiprocessors idle

// Shared memory of a block: `tables` count tables, the list, the bitmaps, and
// the mask table.
template <int kCols>
struct Shared {
    static constexpr int kWords = kCols / 32;
    uint32_t *table;
    uint4 *lanes;
    uint16_t *list;
    uint32_t *touched, *allow_t, *allow_r, *skip_t, *skip_r;
    static constexpr size_t bytes(int tables) {
        return static_cast<size_t>(kCols) * (4 * tables + 2) + 256 * sizeof(uint4) + kWords * 4 * 5;
    }
    __device__ Shared(char *p, int tables) {
        table = reinterpret_cast<uint32_t *>(p);
        p += static_cast<size_t>(kCols) * 4 * tables;
        lanes = reinterpret_cast<uint4 *>(p);
        p += 256 * sizeof(uint4);
        list = reinterpret_cast<uint16_t *>(p);
        p += kCols * 2;
        touched = reinterpret_cast<uint32_t *>(p);
        allow_t = touched + kWords;
        allow_r = allow_t + kWords;
        skip_t = allow_r + kWords;
        skip_r = skip_t + kWords;
    }
    __device__ void init(int n_table_words) const {
        for (int j = threadIdx.x; j < n_table_words; j += kCtlThreads) table[j] = 0;
        lanes[threadIdx.x] = ctl_lanes(threadIdx.x);
    }
};
static_assert(kCtlThreads == 256, "one mask table entry a thread");

// the byte of bits for the eight columns of group g
__device__ __forceinline__ uint32_t group_bits(const uint32_t *words, int g) {
    return reinterpret_cast<const uint8_t *>(words)[g];
}

struct ApplyArgs {
    CtlSide c;
    const char *x;
    char *out;
    int64_t x_stride, out_stride;  // bytes
    int64_t n_rows, vocab;
    int n_chunks, per_unit;        // chunks a row, chunks a unit
};

// Unit u of `n_units` a row: the row, and which of its units.  Consecutive
// units belong to one row; each row starts at another of its units, because a
// tokenizer's frequent tokens sit in the first columns: with a grid that is a
// multiple of n_units, the same blocks would otherwise get every row's first
// unit (measured: 428 us instead of 131 us on 256 rows of long histories).
__device__ __forceinline__ void unit_of(int64_t u, int n_units, int64_t &row, int &k) {
    row = u / n_units;
    k = static_cast<int>((u - row * n_units + row) % n_units);
}

template <bool kXBf16, bool kOBf16, bool kVec, int kCols>
__global__ void __launch_bounds__(kCtlThreads, 4) apply_kernel(const __grid_constant__ ApplyArgs a) {
    extern __shared__ __align__(16) char smem[];
    __shared__ int warp_sum[kCtlWarps];
    __shared__ CtlRow o;
    const Shared<kCols> sh(smem, 1);
    constexpr int kGroups = kCols / 8 / kCtlThreads;
    const int t = threadIdx.x;
    const bool marks = a.c.counts || a.c.n_bias > 0;
    sh.init(marks ? kCols : 0);
    if (t < Shared<kCols>::kWords) sh.touched[t] = 0;
    const int n_units = (a.n_chunks + a.per_unit - 1) / a.per_unit;
    const int64_t units = a.n_rows * n_units;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        int64_t r;
        int k;
        unit_of(u, n_units, r, k);
        const char *xrow = a.x + r * a.x_stride;
        char *orow = a.out + r * a.out_stride;
        __syncthreads();  // the last unit's row is done with
        if (t == 0) o = ctl_row(a.c, r);
        const int ch1 = min(a.n_chunks, (k + 1) * a.per_unit);
        for (int ch = k * a.per_unit; ch < ch1; ++ch) {
            const int64_t c0 = static_cast<int64_t>(ch) * kCols;
            Group8<kXBf16> raw[kGroups];
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                const int64_t j = c0 + 8 * (t + g * kCtlThreads);
                if (j < a.vocab) ctl_load8<kXBf16, kVec>(xrow, j, a.vocab, raw[g]);
            }
            __syncthreads();  // the table and the bitmaps are free again
            int n = 0;
            if (marks) {
                const uint32_t len = static_cast<uint32_t>(min(static_cast<int64_t>(kCols), a.vocab - c0));
                ctl_mark(a.c, o, r, c0, len, sh.table, sh.touched, -1, nullptr);
                __syncthreads();
            }
            uint32_t bits = 0;
            if (t < Shared<kCols>::kWords) {
                bits = sh.touched[t];
                sh.touched[t] = 0;
                sh.allow_t[t] = ctl_allowed(o, c0, t, a.vocab);
            }
            if (marks) n = ctl_list(bits, sh.list, warp_sum);
            __syncthreads();
            const float scale = o.scale;
            // the touched tokens' logits replace their table words
            for (int i = t; i < n; i += kCtlThreads) {
                const int j = sh.list[i];
                const uint32_t w = sh.table[j];
                float z = -INFINITY;
                if (sh.allow_t[j >> 5] >> (j & 31) & 1u) {
                    const Two v = ctl_value(ctl_elem<kXBf16>(xrow, c0 + j), w, a.c, o, r, c0 + j, nullptr);
                    z = __fmaf_rn(v.h, scale, __fmul_rn(v.l, scale));
                }
                sh.table[j] = __float_as_uint(z);
            }
            if (n && a.x == a.out) __syncthreads();  // in place: read before the stream overwrites
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                const int gi = t + g * kCtlThreads;
                const int64_t j = c0 + 8 * static_cast<int64_t>(gi);
                if (j >= a.vocab) continue;
                float v[8];
                ctl_unpack8<kXBf16>(raw[g], v);
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] = __fmul_rn(v[q], scale);
                Group8<kOBf16> w;
                ctl_pack8<kOBf16>(v, w);
                const uint32_t skip = group_bits(sh.allow_t, gi) ^ 0xffu;
                if (skip) ctl_fill8<kOBf16, 0xff80u>(w, sh.lanes[skip]);  // -inf
                ctl_store8<kOBf16, kVec>(orow, j, a.vocab, w);
            }
            if (n) {
                __syncthreads();  // the stream's stores come first
                for (int i = t; i < n; i += kCtlThreads) {
                    const int j = sh.list[i];
                    ctl_store1<kOBf16>(orow, c0 + j, __uint_as_float(sh.table[j]));
                    sh.table[j] = 0;
                }
            }
        }
    }
}

struct GradArgs {
    CtlSide c;
    const char *x;
    char *out;
    int64_t x_stride, out_stride;  // bytes
    int64_t n_rows, vocab;
    int n_chunks, per_unit;
    const int32_t *ids;
    const uint8_t *mask;
    const float *logp, *grad;
};

// d(g logp)/dx_j = g scale (1[j = id] - p_j) dx3/dx, p_j = 2^(z_j log2 e - lse
// log2 e) with lse = z[id] - logp from the forward's own output (as the plain
// gradient does).  Its base-2 form is kept as two floats; the low one enters as
// a factor, so the stream spends one multiply-add, one exponential and one
// product a column.  The selected token is always on the list, so the stream
// has no one-hot term.
template <bool kXBf16, bool kOBf16, bool kVec, int kCols>
__global__ void __launch_bounds__(kCtlThreads, 4) gradient_kernel(const __grid_constant__ GradArgs a) {
    extern __shared__ __align__(16) char smem[];
    __shared__ int warp_sum[kCtlWarps];
    __shared__ uint32_t id_word;
    __shared__ float lse2[2];
    __shared__ CtlRow o;
    const Shared<kCols> sh(smem, 1);
    constexpr int kGroups = kCols / 8 / kCtlThreads;
    const int t = threadIdx.x;
    const bool marks = a.c.counts || a.c.n_bias > 0;
    sh.init(kCols);
    if (t < Shared<kCols>::kWords) sh.touched[t] = 0;
    const int n_units = (a.n_chunks + a.per_unit - 1) / a.per_unit;
    const int64_t units = a.n_rows * n_units;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        int64_t r;
        int k;
        unit_of(u, n_units, r, k);
        const char *xrow = a.x + r * a.x_stride;
        char *orow = a.out + r * a.out_stride;
        const int ch0 = k * a.per_unit, ch1 = min(a.n_chunks, ch0 + a.per_unit);
        const bool active = a.mask[r] != 0;
        const int64_t id = active ? a.ids[r] : 0;
        if (!(active && id >= 0 && id < a.vocab)) {
            // inactive rows: 0; an active row with an out-of-range id: NaN
            float v[8];
            Group8<kOBf16> w;
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = active ? CUDART_NAN_F : 0.f;
            ctl_pack8<kOBf16>(v, w);
            const int64_t end = min(static_cast<int64_t>(ch1) * kCols, a.vocab);
            for (int64_t j = static_cast<int64_t>(ch0) * kCols + 8 * t; j < end; j += 8 * kCtlThreads)
                ctl_store8<kOBf16, kVec>(orow, j, a.vocab, w);
            continue;
        }
        __syncthreads();  // the last unit's row is done with
        if (t == 0) o = ctl_row(a.c, r);
        float gs = a.grad[r], f = 0.f, lh = 0.f, ll = 0.f, gl = 0.f;
        for (int ch = ch0; ch < ch1; ++ch) {
            const int64_t c0 = static_cast<int64_t>(ch) * kCols;
            Group8<kXBf16> raw[kGroups];
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                const int64_t j = c0 + 8 * (t + g * kCtlThreads);
                if (j < a.vocab) ctl_load8<kXBf16, kVec>(xrow, j, a.vocab, raw[g]);
            }
            if (t == 0) id_word = 0;
            __syncthreads();  // the table and the bitmaps are free again
            const bool first = ch == ch0;
            if (marks) {
                const uint32_t len = static_cast<uint32_t>(min(static_cast<int64_t>(kCols), a.vocab - c0));
                ctl_mark(a.c, o, r, c0, len, sh.table, sh.touched, first ? id : -1, first ? &id_word : nullptr);
                __syncthreads();
            }
            uint32_t bits = 0;
            if (t < Shared<kCols>::kWords) {
                bits = sh.touched[t];
                sh.touched[t] = 0;
                sh.allow_t[t] = ctl_allowed(o, c0, t, a.vocab);
                if ((id - c0) >> 5 == t) bits |= 1u << (id & 31);
            }
            const int n = ctl_list(bits, sh.list, warp_sum);
            if (first && t == kCtlThreads - 1) {
                const uint32_t word = o.mask ? __ldg(o.mask + id / 32) : 0xffffffffu;
                double z = -CUDART_INF;
                if (!o.none && (word >> (id & 31) & 1u)) {
                    const Two v = ctl_value(ctl_elem<kXBf16>(xrow, id), id_word, a.c, o, r, id, nullptr);
                    z = (static_cast<double>(v.h) + static_cast<double>(v.l)) * static_cast<double>(o.scale);
                }
                const double l2 = (z - static_cast<double>(a.logp[r])) * 1.4426950408889634;
                lse2[0] = static_cast<float>(l2);
                lse2[1] = static_cast<float>(l2 - static_cast<double>(lse2[0]));
            }
            __syncthreads();
            if (first) {
                gs = __fmul_rn(gs, o.scale);
                f = __fmul_rn(o.scale, kLog2e);
                lh = lse2[0];
                ll = lse2[1];
                gl = __fmul_rn(-gs, ex2(-ll));
            }
            for (int i = t; i < n; i += kCtlThreads) {
                const int j = sh.list[i];
                const uint32_t w = sh.table[j];
                float d = 0.f;
                if (sh.allow_t[j >> 5] >> (j & 31) & 1u) {
                    float slope;
                    const Two v = ctl_value(ctl_elem<kXBf16>(xrow, c0 + j), w, a.c, o, r, c0 + j, &slope);
                    const float p = ex2(__fadd_rn(__fsub_rn(__fmaf_rn(v.h, f, -lh), ll), __fmul_rn(v.l, f)));
                    d = __fmul_rn(__fmul_rn(gs, slope), __fsub_rn(c0 + j == id ? 1.f : 0.f, p));
                }
                sh.table[j] = __float_as_uint(d);
            }
            const f2_t f2f = f2(f, f), l2f = f2(-lh, -lh), g2f = f2(gl, gl);
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                const int gi = t + g * kCtlThreads;
                const int64_t j = c0 + 8 * static_cast<int64_t>(gi);
                if (j >= a.vocab) continue;
                float v[8];
                ctl_unpack8<kXBf16>(raw[g], v);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f2_t d = mul2(g2f, ex2_2(fma2(f2(v[2 * q], v[2 * q + 1]), f2f, l2f)));
                    v[2 * q] = f2_lo(d);
                    v[2 * q + 1] = f2_hi(d);
                }
                Group8<kOBf16> w;
                ctl_pack8<kOBf16>(v, w);
                const uint32_t skip = group_bits(sh.allow_t, gi) ^ 0xffu;
                if (skip) ctl_fill8<kOBf16, 0u>(w, sh.lanes[skip]);
                ctl_store8<kOBf16, kVec>(orow, j, a.vocab, w);
            }
            if (n) {
                __syncthreads();  // the stream's stores come first
                for (int i = t; i < n; i += kCtlThreads) {
                    const int j = sh.list[i];
                    ctl_store1<kOBf16>(orow, c0 + j, __uint_as_float(sh.table[j]));
                    sh.table[j] = 0;
                }
            }
        }
    }
}

// ---- scoring: sums of both sides ---------------------------------------------------
// Two sides that nearly agree (the same scale, |z_t - z_r| small) take one
// exponential a column: e_t = e_r (1 + q), q = expm1(u) of the small exponent
// difference u by its Taylor series.  The difference of the two sums, e_r q
// added up, is then accurate relative to itself, where e_t - e_r of two rounded
// exponentials carries 2^-22 of the term (1e-5 of a logprob difference of
// 2e-3), and the special-function unit, which bounds the kernel beside HBM, has
// half the work.
constexpr float kNear2 = 0.0625f;   // sum of u^2 over a thread's sixteen columns: |u| <= 1/4
// A masked column of the stream holds about -1e30 (bf16 0xf149) on both sides:
// its term is 0 and its u finite.  Rows whose allowed logits are all below
// kFloorZ leave this path.
constexpr uint32_t kFillBits = 0xf149u;
constexpr float kFloorZ = -1e29f;

// expm1(u) / u up to u^5 / 720: the next term is u^6 / 5040 = 5e-8 at 1/4
__device__ __forceinline__ f2_t expm1_ratio2(f2_t u) {
    f2_t p = fma2(u, f2(1.f / 720.f, 1.f / 720.f), f2(1.f / 120.f, 1.f / 120.f));
    p = fma2(u, p, f2(1.f / 24.f, 1.f / 24.f));
    p = fma2(u, p, f2(1.f / 6.f, 1.f / 6.f));
    p = fma2(u, p, f2(0.5f, 0.5f));
    return fma2(u, p, f2(1.f, 1.f));
}

// References (mt, mr) moved up to (nmt, nmr).
__device__ __forceinline__ void raise_refs(Acc2 &a, float nmt, float nmr, float lt, float lr) {
    const float at = __fmul_rn(__fsub_rn(a.mt, nmt), lt), ar = __fmul_rn(__fsub_rn(a.mr, nmr), lr);
    const float ft = ex2(at), fr = ex2(ar);
    const float corr = scale_diff(ft, fr, at, ar);
    a.dd = add2(mul2(a.dd, f2(ft, ft)), mul2(a.sr, f2(corr, corr)));
    a.st = mul2(a.st, f2(ft, ft));
    a.sr = mul2(a.sr, f2(fr, fr));
    a.mt = nmt;
    a.mr = nmr;
}

// Sixteen columns of two sides that nearly agree; false where they do not (the
// state is valid either way).  A NaN fails the comparison of the sum of squares.
__device__ __forceinline__ bool accumulate_near(const f2_t *vt, const f2_t *vr, Acc2 &a, float l, float s) {
    const float cm = max16(vr);
    if (!(cm > kFloorZ)) return false;
    if (cm > a.mr) raise_refs(a, fmaxf(a.mt, cm), cm, l, l);
    const float dm = __fmul_rn(__fsub_rn(a.mr, a.mt), s);
    const f2_t s2 = f2(s, s), dm2 = f2(dm, dm), l2 = f2(l, l), m2 = f2(a.mr, a.mr);
    f2_t u[8], q2 = f2(0.f, 0.f);
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        u[p] = fma2(sub2(vt[p], vr[p]), s2, dm2);
        q2 = fma2(u[p], u[p], q2);
    }
    if (!(__fadd_rn(f2_lo(q2), f2_hi(q2)) <= kNear2)) return false;
    f2_t se = f2(0.f, 0.f), sd = f2(0.f, 0.f);
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const f2_t e = ex2_2(mul2(sub2(vr[p], m2), l2));
        se = add2(se, e);
        sd = fma2(mul2(e, u[p]), expm1_ratio2(u[p]), sd);
    }
    a.sr = add2(a.sr, se);
    a.dd = add2(a.dd, sd);
    a.st = add2(a.st, add2(se, sd));
    return true;
}

// Sixteen columns of any two sides, each with an exponential of its own; -inf
// adds nothing (the floor of the references keeps x - m defined).
__device__ __forceinline__ void accumulate_far(const f2_t *vt, const f2_t *vr, Acc2 &a, float lt, float lr) {
    const float ct = max16(vt), cr = max16(vr);
    if (ct > a.mt || cr > a.mr) raise_refs(a, fmaxf(a.mt, ct), fmaxf(a.mr, cr), lt, lr);
    const f2_t mt2 = f2(a.mt, a.mt), mr2 = f2(a.mr, a.mr), lt2 = f2(lt, lt), lr2 = f2(lr, lr);
    f2_t st = f2(0.f, 0.f), sr = st, sd = st;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const f2_t et = ex2_2(mul2(sub2(vt[p], mt2), lt2)), er = ex2_2(mul2(sub2(vr[p], mr2), lr2));
        st = add2(st, et);
        sr = add2(sr, er);
        sd = add2(sd, sub2(et, er));
    }
    a.st = add2(a.st, st);
    a.sr = add2(a.sr, sr);
    a.dd = add2(a.dd, sd);
}

// One pair of controlled logits (h + l of each side) into the state; an -inf
// adds nothing.
__device__ __forceinline__ void accumulate_pair(Two xt, Two xr, Acc2 &a, float lt, float lr, float s, bool same_scale) {
    if (xt.h > a.mt || xr.h > a.mr) raise_refs(a, fmaxf(a.mt, xt.h), fmaxf(a.mr, xr.h), lt, lr);
    const float er = ex2(__fmaf_rn(xr.l, lr, __fmul_rn(__fsub_rn(xr.h, a.mr), lr)));
    const float u = __fmul_rn(
        __fadd_rn(__fsub_rn(__fsub_rn(xt.h, xr.h), __fsub_rn(a.mt, a.mr)), __fsub_rn(xt.l, xr.l)), s);
    float d;
    if (same_scale && fabsf(u) <= 0.25f) {
        d = __fmul_rn(__fmul_rn(er, u), f2_lo(expm1_ratio2(f2(u, u))));
    } else {
        const float et = ex2(__fmaf_rn(xt.l, lt, __fmul_rn(__fsub_rn(xt.h, a.mt), lt)));
        d = __fsub_rn(et, er);
    }
    a.sr = add2(a.sr, f2(er, 0.f));
    a.st = add2(a.st, f2(__fadd_rn(er, d), 0.f));
    a.dd = add2(a.dd, f2(d, 0.f));
}

// A unit is kSegChunks chunks of a row, its state carried over them; the number
// is fixed, so a row's arithmetic depends on its columns alone.
constexpr int kSegChunks = 4;

// kTables: 1 when both sides count in the same history (or one side counts in
// none), else one table a side.
template <bool kTBf16, bool kRBf16, bool kVec, int kTables>
__global__ void __launch_bounds__(kCtlThreads, kTables == 1 ? 3 : 2)
    score_kernel(const __grid_constant__ CtlScoreArgs a) {
    extern __shared__ __align__(16) char smem[];
    __shared__ int warp_sum[kCtlWarps];
    __shared__ float states[5][kCtlWarps];
    __shared__ CtlRow ot, orr;
    const Shared<kChunk> sh(smem, kTables);
    uint32_t *const table_t = sh.table, *const table_r = sh.table + (kTables - 1) * kChunk;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const bool marks_t = a.t.counts || a.t.n_bias > 0, marks_r = a.r.counts || a.r.n_bias > 0;
    const bool marks = marks_t || marks_r;
    sh.init(marks ? kTables * kChunk : 0);
    sh.touched[t] = 0;
    const int n_chunks = static_cast<int>((a.vocab + kChunk - 1) / kChunk);
    const int64_t units = a.hdr->n_active * a.n_chunks;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        int64_t i;
        int k;
        unit_of(u, a.n_chunks, i, k);
        const int2 rid = a.rowid[i];
        const int64_t r = rid.x, id = rid.y;
        const char *trow = a.xt + r * a.t_stride, *rrow = a.xr + r * a.r_stride;
        const int64_t end = min(static_cast<int64_t>(k + 1) * kSegChunks * kChunk, a.vocab);
        // 16 columns of each side a thread and step: groups t and t + 256 of
        // the step's 4096 columns; each step's loads go out before the step
        // in front of it is worked on, a chunk's first ones before its scan
        Group8<kTBf16> gt[2];
        Group8<kRBf16> gr[2];
        auto load = [&](int64_t c) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int64_t j = c + 8 * (t + g * kCtlThreads);
                if (j < end) {
                    ctl_load8<kTBf16, kVec>(trow, j, a.vocab, gt[g]);
                    ctl_load8<kRBf16, kVec>(rrow, j, a.vocab, gr[g]);
                }
            }
        };
        const int ch0 = k * kSegChunks, ch1 = min(n_chunks, ch0 + kSegChunks);
        load(static_cast<int64_t>(ch0) * kChunk);
        if (t == 0) ot = ctl_row(a.t, r);
        if (t == 32) orr = ctl_row(a.r, r);
        __syncthreads();
        const float s_r = orr.scale;
        const float lt = __fmul_rn(ot.scale, kLog2e), lr = __fmul_rn(s_r, kLog2e);
        const bool same_scale = ot.scale == s_r;
        Acc2 acc = acc2_init();
#pragma unroll 1
        for (int ch = ch0; ch < ch1; ++ch) {
            const int64_t c0 = static_cast<int64_t>(ch) * kChunk;
            __syncthreads();  // the table and the bitmaps are free again
            if (marks) {
                const uint32_t len = static_cast<uint32_t>(min(static_cast<int64_t>(kChunk), a.vocab - c0));
                if (marks_t) ctl_mark(a.t, ot, r, c0, len, table_t, sh.touched, -1, nullptr);
                if (marks_r && !a.same) ctl_mark(a.r, orr, r, c0, len, table_r, sh.touched, -1, nullptr);
                __syncthreads();
            }
            const uint32_t bits = sh.touched[t];
            sh.touched[t] = 0;
            const uint32_t at = ctl_allowed(ot, c0, t, a.vocab), ar = ctl_allowed(orr, c0, t, a.vocab);
            sh.allow_t[t] = at;
            sh.allow_r[t] = ar;
            sh.skip_t[t] = bits | ~at;
            sh.skip_r[t] = bits | ~ar;
            if ((id - c0) >> 5 == t && id < a.vocab && !(bits >> (id & 31) & 1u))  // an untouched selected token
                a.pick[i] = make_double2(at >> (id & 31) & 1u ? static_cast<double>(ctl_elem<kTBf16>(trow, id)) : -CUDART_INF,
                                         ar >> (id & 31) & 1u ? static_cast<double>(ctl_elem<kRBf16>(rrow, id)) : -CUDART_INF);
            const int n = marks ? ctl_list(bits, sh.list, warp_sum) : 0;
            __syncthreads();
            for (int q = t; q < n; q += kCtlThreads) {
                const int j = sh.list[q];
                const uint32_t bit = 1u << (j & 31);
                const uint32_t wt = marks_t ? table_t[j] : 0u;
                const uint32_t wr = a.same ? wt : marks_r ? table_r[j] : 0u;
                Two vt{-INFINITY, 0.f}, vr{-INFINITY, 0.f};
                if (sh.allow_t[j >> 5] & bit)
                    vt = ctl_value(ctl_elem<kTBf16>(trow, c0 + j), wt, a.t, ot, r, c0 + j, nullptr);
                if (sh.allow_r[j >> 5] & bit)
                    vr = ctl_value(ctl_elem<kRBf16>(rrow, c0 + j), wr, a.r, orr, r, c0 + j, nullptr);
                table_t[j] = 0;
                if (kTables > 1) table_r[j] = 0;
                accumulate_pair(vt, vr, acc, lt, lr, s_r, same_scale);
                if (c0 + j == id)
                    a.pick[i] = make_double2(static_cast<double>(vt.h) + static_cast<double>(vt.l),
                                             static_cast<double>(vr.h) + static_cast<double>(vr.l));
            }
#pragma unroll 1
            for (int step = 0; step < kChunk / 16 / kCtlThreads; ++step) {
                uint32_t st[2], sr[2];
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const int gi = t + (2 * step + g) * kCtlThreads;
                    st[g] = group_bits(sh.skip_t, gi);
                    sr[g] = group_bits(sh.skip_r, gi);
                    if (st[g]) ctl_fill8<kTBf16, kFillBits>(gt[g], sh.lanes[st[g]]);
                    if (sr[g]) ctl_fill8<kRBf16, kFillBits>(gr[g], sh.lanes[sr[g]]);
                }
                float vt[16], vr[16];
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    ctl_unpack8<kTBf16>(gt[g], vt + 8 * g);
                    ctl_unpack8<kRBf16>(gr[g], vr + 8 * g);
                }
                load(c0 + (step + 1) * 16 * kCtlThreads);  // the next chunk's first step behind the last one
                if ((st[0] & st[1] & sr[0] & sr[1]) == 0xffu) continue;  // nothing allowed
                f2_t pt[8], pr[8];
#pragma unroll
                for (int p = 0; p < 8; ++p) {
                    pt[p] = f2(vt[2 * p], vt[2 * p + 1]);
                    pr[p] = f2(vr[2 * p], vr[2 * p + 1]);
                }
                if (same_scale && accumulate_near(pt, pr, acc, lr, s_r)) continue;
#pragma unroll
                for (int p = 0; p < 8; ++p) {
                    const uint32_t bt = st[p >> 2] >> (2 * (p & 3)), br = sr[p >> 2] >> (2 * (p & 3));
                    pt[p] = f2(bt & 1u ? -INFINITY : f2_lo(pt[p]), bt & 2u ? -INFINITY : f2_hi(pt[p]));
                    pr[p] = f2(br & 1u ? -INFINITY : f2_lo(pr[p]), br & 2u ? -INFINITY : f2_hi(pr[p]));
                }
                accumulate_far(pt, pr, acc, lt, lr);
            }
        }
        // the block's state: each warp's in a butterfly, then the eight warps' in another
        const Acc w = warp_reduce_acc<false>(acc2_fold(acc), lt, lr);
        if (lane == 0) {
            states[0][warp] = w.mt;
            states[1][warp] = w.st;
            states[2][warp] = w.dd;
            states[3][warp] = w.mr;
            states[4][warp] = w.sr;
        }
        __syncthreads();
        if (warp == 0) {
            const int s = lane & (kCtlWarps - 1);
            Acc b{states[0][s], states[1][s], states[2][s], states[3][s], states[4][s], 0.f, 0.f};
#pragma unroll
            for (int off = kCtlWarps / 2; off > 0; off >>= 1) {
                Acc y;
                y.mt = __shfl_xor_sync(0xffffffffu, b.mt, off);
                y.st = __shfl_xor_sync(0xffffffffu, b.st, off);
                y.dd = __shfl_xor_sync(0xffffffffu, b.dd, off);
                y.mr = __shfl_xor_sync(0xffffffffu, b.mr, off);
                y.sr = __shfl_xor_sync(0xffffffffu, b.sr, off);
                y.ht = y.hr = 0.f;
                merge_acc<false>(b, y, lt, lr);
            }
            if (lane == 0) {
                a.part_a[i * a.n_chunks + k] = make_float4(b.mt, b.st, b.dd, b.mr);
                a.part_b[i * a.n_chunks + k] = b.sr;
            }
        }
    }
}

// One warp per active row: lane l folds units l, l + 32, ... in order, the
// warp merges in a fixed butterfly, lane 0 does the row's arithmetic in double
// (the formulas of the plain scorer, with each side's scale).
__global__ void __launch_bounds__(256) score_finalize_kernel(const __grid_constant__ CtlScoreArgs a, float *out_lt,
                                                            float *out_lr, float *out_d, double *dval,
                                                            uint32_t *keys, uint32_t *status) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (i >= a.hdr->n_active) return;
    const int2 rid = a.rowid[i];
    const int64_t r = rid.x, id = rid.y;
    float s_t = a.t.scale ? a.t.scale[r] : 1.f, s_r = a.r.scale ? a.r.scale[r] : 1.f;
    if (!(s_t > 0.f && s_t <= FLT_MAX)) s_t = CUDART_NAN_F;
    if (!(s_r > 0.f && s_r <= FLT_MAX)) s_r = CUDART_NAN_F;
    const float lt = __fmul_rn(s_t, kLog2e), lr = __fmul_rn(s_r, kLog2e);
    Acc acc = acc_init();
    for (int k = lane; k < a.n_chunks; k += 32) {
        const float4 p = a.part_a[i * a.n_chunks + k];
        const Acc o{p.x, p.y, p.z, p.w, a.part_b[i * a.n_chunks + k], 0.f, 0.f};
        merge_acc<false>(acc, o, lt, lr);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        Acc o;
        o.mt = __shfl_xor_sync(0xffffffffu, acc.mt, off);
        o.st = __shfl_xor_sync(0xffffffffu, acc.st, off);
        o.dd = __shfl_xor_sync(0xffffffffu, acc.dd, off);
        o.mr = __shfl_xor_sync(0xffffffffu, acc.mr, off);
        o.sr = __shfl_xor_sync(0xffffffffu, acc.sr, off);
        o.ht = o.hr = 0.f;
        merge_acc<false>(acc, o, lt, lr);
    }
    if (lane != 0) return;
    uint32_t bad = 0;
    double d = CUDART_NAN, pt = CUDART_NAN, pr = CUDART_NAN;
    if (id < 0 || id >= a.vocab) {
        bad = LPD_STATUS_TOKEN_OOB;
    } else {
        const double2 x = a.pick[i];
        const double mt = static_cast<double>(s_t) * acc.mt, mr = static_cast<double>(s_r) * acc.mr;
        const double xt = s_t * x.x, xr = s_r * x.y;
        const double st = acc.st, sr = acc.sr, dd = acc.dd;
        const double lse_t = mt + log(st), lse_r = mr + log(sr);
        const double ratio = fabs(dd) < 0.5 * st ? log1p(-dd / st) : log(sr / st);
        d = ((xt - xr) - (mt - mr)) + ratio;
        pt = xt - lse_t;
        pr = xr - lse_r;
        if (!(isfinite(lse_t) && isfinite(lse_r) && isfinite(xt) && isfinite(xr))) bad = LPD_STATUS_NONFINITE;
    }
    if (out_lt) out_lt[r] = static_cast<float>(pt);
    if (out_lr) out_lr[r] = static_cast<float>(pr);
    if (out_d) out_d[r] = static_cast<float>(d);
    dval[i] = d;
    keys[i] = __float_as_uint(fabsf(static_cast<float>(d)));
    if (bad) atomicOr(status, bad);
}

int64_t chunks_of(int64_t vocab, int cols) { return (vocab + cols - 1) / cols; }

template <class Args, class Kernel>
cudaError_t launch_units(Kernel *kern, const Args &a, int64_t units, int per_sm, size_t smem,
                         std::atomic<uint64_t> &configured, cudaStream_t stream) {
    const cudaError_t e = set_smem_once(kern, smem, configured);
    if (e != cudaSuccess) return e;
    const int64_t most = static_cast<int64_t>(device_sm_count()) * per_sm;
    kern<<<static_cast<unsigned>(units < most ? units : most), kCtlThreads, smem, stream>>>(a);
    return cudaGetLastError();
}

// Chunks of 2048 columns where 8192 would leave multiprocessors without a unit
// (elementwise forms only: a column's value does not depend on the chunk).
bool few_units(int64_t n_rows, int64_t vocab) {
    return n_rows * chunks_of(vocab, kChunk) < 2 * static_cast<int64_t>(device_sm_count());
}

template <bool kXB, bool kOB, bool kVec, int kCols>
cudaError_t apply_typed(ApplyArgs &a, cudaStream_t stream) {
    static std::atomic<uint64_t> configured{0};
    a.n_chunks = static_cast<int>(chunks_of(a.vocab, kCols));
    a.per_unit = 1;
    return launch_units(apply_kernel<kXB, kOB, kVec, kCols>, a, a.n_rows * a.n_chunks, 4, Shared<kCols>::bytes(1),
                        configured, stream);
}

template <bool kXB, bool kOB, bool kVec, int kCols>
cudaError_t gradient_typed(GradArgs &a, cudaStream_t stream) {
    static std::atomic<uint64_t> configured{0};
    a.n_chunks = static_cast<int>(chunks_of(a.vocab, kCols));
    a.per_unit = 1;
    return launch_units(gradient_kernel<kXB, kOB, kVec, kCols>, a, a.n_rows * a.n_chunks, 4, Shared<kCols>::bytes(1),
                        configured, stream);
}

template <bool kXB, bool kOB>
cudaError_t apply_path(ApplyArgs &a, bool vec, cudaStream_t s) {
    if (few_units(a.n_rows, a.vocab))
        return vec ? apply_typed<kXB, kOB, true, kSmallChunk>(a, s) : apply_typed<kXB, kOB, false, kSmallChunk>(a, s);
    return vec ? apply_typed<kXB, kOB, true, kChunk>(a, s) : apply_typed<kXB, kOB, false, kChunk>(a, s);
}

template <bool kXB, bool kOB>
cudaError_t gradient_path(GradArgs &a, bool vec, cudaStream_t s) {
    if (few_units(a.n_rows, a.vocab))
        return vec ? gradient_typed<kXB, kOB, true, kSmallChunk>(a, s)
                   : gradient_typed<kXB, kOB, false, kSmallChunk>(a, s);
    return vec ? gradient_typed<kXB, kOB, true, kChunk>(a, s) : gradient_typed<kXB, kOB, false, kChunk>(a, s);
}

bool aligned_rows(const void *p, int64_t stride_bytes) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride_bytes % 16 == 0;
}

template <bool kTB, bool kRB, int kTables>
cudaError_t score_typed(const CtlScoreArgs &a, bool vec, int64_t n_rows, cudaStream_t s) {
    static std::atomic<uint64_t> configured[2];
    const int64_t units = n_rows * a.n_chunks;
    const int per_sm = kTables == 1 ? 3 : 2;
    const size_t smem = Shared<kChunk>::bytes(kTables);
    return vec ? launch_units(score_kernel<kTB, kRB, true, kTables>, a, units, per_sm, smem, configured[0], s)
               : launch_units(score_kernel<kTB, kRB, false, kTables>, a, units, per_sm, smem, configured[1], s);
}

}  // namespace

int controls_chunks(int64_t vocab) { return static_cast<int>(chunks_of(vocab, kChunk * kSegChunks)); }

cudaError_t launch_controls_apply(const CtlSide &c, const void *x, int x_dtype, int64_t x_stride_elems, void *out,
                                  int out_dtype, int64_t out_stride_elems, int64_t n_rows, int64_t vocab,
                                  cudaStream_t stream) {
    if (n_rows == 0) return cudaSuccess;
    const bool xb = x_dtype == LPD_BF16, ob = out_dtype == LPD_BF16;
    ApplyArgs a{};
    a.c = c;
    a.x = static_cast<const char *>(x);
    a.out = static_cast<char *>(out);
    a.x_stride = x_stride_elems * (xb ? 2 : 4);
    a.out_stride = out_stride_elems * (ob ? 2 : 4);
    a.n_rows = n_rows;
    a.vocab = vocab;
    const bool vec = aligned_rows(x, a.x_stride) && aligned_rows(out, a.out_stride);
    if (xb) return ob ? apply_path<true, true>(a, vec, stream) : apply_path<true, false>(a, vec, stream);
    return ob ? apply_path<false, true>(a, vec, stream) : apply_path<false, false>(a, vec, stream);
}

cudaError_t launch_controls_gradient(const CtlSide &c, const void *x, int x_dtype, int64_t x_stride_elems, void *out,
                                     int out_dtype, int64_t out_stride_elems, int64_t n_rows, int64_t vocab,
                                     const int32_t *ids, const uint8_t *mask, const float *logp, const float *grad,
                                     cudaStream_t stream) {
    if (n_rows == 0) return cudaSuccess;
    const bool xb = x_dtype == LPD_BF16, ob = out_dtype == LPD_BF16;
    GradArgs a{};
    a.c = c;
    a.x = static_cast<const char *>(x);
    a.out = static_cast<char *>(out);
    a.x_stride = x_stride_elems * (xb ? 2 : 4);
    a.out_stride = out_stride_elems * (ob ? 2 : 4);
    a.n_rows = n_rows;
    a.vocab = vocab;
    a.ids = ids;
    a.mask = mask;
    a.logp = logp;
    a.grad = grad;
    const bool vec = aligned_rows(x, a.x_stride) && aligned_rows(out, a.out_stride);
    if (xb) return ob ? gradient_path<true, true>(a, vec, stream) : gradient_path<true, false>(a, vec, stream);
    return ob ? gradient_path<false, true>(a, vec, stream) : gradient_path<false, false>(a, vec, stream);
}

cudaError_t launch_controls_score(const CtlScoreArgs &args, int dtype_t, int dtype_r, int64_t n_rows, float *out_lt,
                                  float *out_lr, float *out_d, double *dval, uint32_t *keys, uint32_t *status,
                                  cudaStream_t stream) {
    if (n_rows == 0) return cudaSuccess;
    CtlScoreArgs a = args;
    a.n_chunks = controls_chunks(a.vocab);
    const bool vec = aligned_rows(a.xt, a.t_stride) && aligned_rows(a.xr, a.r_stride);
    const bool tb = dtype_t == LPD_BF16, rb = dtype_r == LPD_BF16;
    const bool mt = a.t.counts || a.t.n_bias > 0, mr = a.r.counts || a.r.n_bias > 0;
    // one table serves two sides that mark the same tokens, or one side that marks any
    a.same = mt && mr && a.t.counts == a.r.counts && a.t.history == a.r.history && a.t.hist_begin == a.r.hist_begin &&
             a.t.hist_split == a.r.hist_split && a.t.hist_end == a.r.hist_end && a.t.n_history == a.r.n_history &&
             a.t.bias_ids == a.r.bias_ids && a.t.n_bias == a.r.n_bias;
    const bool one = a.same || !(mt && mr);
    cudaError_t e;
    if (one) {
        if (tb) e = rb ? score_typed<true, true, 1>(a, vec, n_rows, stream) : score_typed<true, false, 1>(a, vec, n_rows, stream);
        else e = rb ? score_typed<false, true, 1>(a, vec, n_rows, stream) : score_typed<false, false, 1>(a, vec, n_rows, stream);
    } else {
        if (tb) e = rb ? score_typed<true, true, 2>(a, vec, n_rows, stream) : score_typed<true, false, 2>(a, vec, n_rows, stream);
        else e = rb ? score_typed<false, true, 2>(a, vec, n_rows, stream) : score_typed<false, false, 2>(a, vec, n_rows, stream);
    }
    if (e != cudaSuccess) return e;
    score_finalize_kernel<<<static_cast<unsigned>((n_rows + 7) / 8), 256, 0, stream>>>(a, out_lt, out_lr, out_d, dval,
                                                                                      keys, status);
    return cudaGetLastError();
}

}  // namespace lpd
