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

template <int kCols>
struct Shared {
    uint32_t *table;
    uint16_t *list;
    uint32_t *touched, *allow_t, *allow_r;
    static constexpr size_t bytes(int tables, int sides) {
        return static_cast<size_t>(kCols) * (4 * tables + 2) + (kCols / 32) * 4 * (1 + sides);
    }
    __device__ Shared(char *p, int tables, int sides) {
        table = reinterpret_cast<uint32_t *>(p);
        p += static_cast<size_t>(kCols) * 4 * tables;
        list = reinterpret_cast<uint16_t *>(p);
        p += kCols * 2;
        touched = reinterpret_cast<uint32_t *>(p);
        allow_t = touched + kCols / 32;
        allow_r = sides > 1 ? allow_t + kCols / 32 : allow_t;
    }
};

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
    int n_chunks;
};

template <bool kXBf16, bool kOBf16, bool kVec, int kCols>
__global__ void __launch_bounds__(kCtlThreads, 4) apply_kernel(const __grid_constant__ ApplyArgs a) {
    extern __shared__ __align__(16) char smem[];
    __shared__ int warp_sum[kCtlWarps];
    const Shared<kCols> sh(smem, 1, 1);
    constexpr int kGroups = kCols / 8 / kCtlThreads;
    const int t = threadIdx.x;
    const bool marks = a.c.counts || a.c.n_bias > 0;
    if (marks)
        for (int j = t; j < kCols; j += kCtlThreads) sh.table[j] = 0;
    const int64_t units = a.n_rows * a.n_chunks;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t r = u / a.n_chunks;
        const int64_t c0 = (u - r * a.n_chunks) * kCols;
        const char *xrow = a.x + r * a.x_stride;
        char *orow = a.out + r * a.out_stride;
        Group8<kXBf16> raw[kGroups];
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            const int64_t j = c0 + 8 * (t + g * kCtlThreads);
            if (j < a.vocab) ctl_load8<kXBf16, kVec>(xrow, j, a.vocab, raw[g]);
        }
        const CtlRow o = ctl_row(a.c, r);
        if (t < kCols / 32) {
            sh.touched[t] = 0;
            sh.allow_t[t] = ctl_allowed(o, c0, t, a.vocab);
        }
        __syncthreads();
        if (marks) {
            const uint32_t len = static_cast<uint32_t>(min(static_cast<int64_t>(kCols), a.vocab - c0));
            ctl_mark(a.c, o, r, c0, len, sh.table, sh.touched, -1, nullptr);
            __syncthreads();
            const int n = ctl_list(sh.touched, kCols / 32, sh.list, warp_sum);
            __syncthreads();
            // the touched tokens' logits replace their table words
            for (int i = t; i < n; i += kCtlThreads) {
                const int j = sh.list[i];
                const uint32_t w = sh.table[j];
                float z = 0.f;
                if (sh.allow_t[j >> 5] >> (j & 31) & 1u) {
                    const Two v = ctl_value(ctl_elem<kXBf16>(xrow, c0 + j), w, a.c, o, r, c0 + j, nullptr);
                    z = __fmaf_rn(v.h, o.scale, __fmul_rn(v.l, o.scale));
                }
                sh.table[j] = __float_as_uint(z);
            }
            __syncthreads();
        }
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            const int gi = t + g * kCtlThreads;
            const int64_t j = c0 + 8 * static_cast<int64_t>(gi);
            if (j >= a.vocab) continue;
            float v[8];
            ctl_unpack8<kXBf16>(raw[g], v);
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = __fmul_rn(v[q], o.scale);
            const uint32_t allow = group_bits(sh.allow_t, gi), touched = group_bits(sh.touched, gi);
            if (touched) {
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (touched >> q & 1u) {
                        v[q] = __uint_as_float(sh.table[8 * gi + q]);
                        sh.table[8 * gi + q] = 0;
                    }
            }
            if (allow != 0xffu) {
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (!(allow >> q & 1u)) v[q] = -INFINITY;
            }
            ctl_store8<kOBf16, kVec>(orow, j, a.vocab, v);
        }
        __syncthreads();
    }
}

struct GradArgs {
    CtlSide c;
    const char *x;
    char *out;
    int64_t x_stride, out_stride;  // bytes
    int64_t n_rows, vocab;
    int n_chunks;
    const int32_t *ids;
    const uint8_t *mask;
    const float *logp, *grad;
};

// d(g logp)/dx_j = g scale (1[j = id] - p_j) dx3/dx, p_j = 2^(z_j log2 e - lse
// log2 e) with lse = z[id] - logp from the forward's own output (as the plain
// gradient does), its base-2 form kept as two floats.
template <bool kXBf16, bool kOBf16, bool kVec, int kCols>
__global__ void __launch_bounds__(kCtlThreads, 4) gradient_kernel(const __grid_constant__ GradArgs a) {
    extern __shared__ __align__(16) char smem[];
    __shared__ int warp_sum[kCtlWarps];
    __shared__ uint32_t id_word;
    __shared__ float lse2[2];
    const Shared<kCols> sh(smem, 1, 1);
    constexpr int kGroups = kCols / 8 / kCtlThreads;
    const int t = threadIdx.x;
    const bool marks = a.c.counts || a.c.n_bias > 0;
    if (marks)
        for (int j = t; j < kCols; j += kCtlThreads) sh.table[j] = 0;
    const int64_t units = a.n_rows * a.n_chunks;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t r = u / a.n_chunks;
        const int64_t c0 = (u - r * a.n_chunks) * kCols;
        const char *xrow = a.x + r * a.x_stride;
        char *orow = a.out + r * a.out_stride;
        const bool active = a.mask[r] != 0;
        const int64_t id = active ? a.ids[r] : 0;
        if (!(active && id >= 0 && id < a.vocab)) {
            // inactive rows: 0; an active row with an out-of-range id: NaN
            float v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = active ? CUDART_NAN_F : 0.f;
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                const int64_t j = c0 + 8 * static_cast<int64_t>(t + g * kCtlThreads);
                if (j < a.vocab) ctl_store8<kOBf16, kVec>(orow, j, a.vocab, v);
            }
            continue;
        }
        Group8<kXBf16> raw[kGroups];
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            const int64_t j = c0 + 8 * (t + g * kCtlThreads);
            if (j < a.vocab) ctl_load8<kXBf16, kVec>(xrow, j, a.vocab, raw[g]);
        }
        const CtlRow o = ctl_row(a.c, r);
        const float gs = __fmul_rn(a.grad[r], o.scale);
        if (t < kCols / 32) {
            sh.touched[t] = 0;
            sh.allow_t[t] = ctl_allowed(o, c0, t, a.vocab);
        }
        if (t == 0) id_word = 0;
        __syncthreads();
        const uint32_t len = static_cast<uint32_t>(min(static_cast<int64_t>(kCols), a.vocab - c0));
        int n = 0;
        if (marks) {
            ctl_mark(a.c, o, r, c0, len, sh.table, sh.touched, id, &id_word);
            __syncthreads();
            n = ctl_list(sh.touched, kCols / 32, sh.list, warp_sum);
        }
        if (t == 0) {
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
        const float lh = lse2[0], ll = lse2[1];
        const float f = __fmul_rn(o.scale, kLog2e);
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
        if (n) __syncthreads();
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            const int gi = t + g * kCtlThreads;
            const int64_t j = c0 + 8 * static_cast<int64_t>(gi);
            if (j >= a.vocab) continue;
            float v[8];
            ctl_unpack8<kXBf16>(raw[g], v);
            const int64_t at = id - j;  // the one-hot column, if it is in this group
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float p = ex2(__fsub_rn(__fmaf_rn(v[q], f, -lh), ll));
                v[q] = __fmul_rn(gs, at == q ? __fsub_rn(1.f, p) : -p);
            }
            const uint32_t allow = group_bits(sh.allow_t, gi), touched = group_bits(sh.touched, gi);
            if (touched) {
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (touched >> q & 1u) {
                        v[q] = __uint_as_float(sh.table[8 * gi + q]);
                        sh.table[8 * gi + q] = 0;
                    }
            }
            if (allow != 0xffu) {
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (!(allow >> q & 1u)) v[q] = 0.f;
            }
            ctl_store8<kOBf16, kVec>(orow, j, a.vocab, v);
        }
        __syncthreads();
    }
}

// One pair of controlled logits (h + l of each side) into the state; an -inf
// adds nothing.
__device__ __forceinline__ void accumulate_pair(Two xt, Two xr, Acc2 &a, float lt, float lr) {
    if (xt.h > a.mt || xr.h > a.mr) {
        const float nmt = fmaxf(a.mt, xt.h), nmr = fmaxf(a.mr, xr.h);
        const float at = __fmul_rn(__fsub_rn(a.mt, nmt), lt), ar = __fmul_rn(__fsub_rn(a.mr, nmr), lr);
        const float ft = ex2(at), fr = ex2(ar);
        const float corr = scale_diff(ft, fr, at, ar);
        a.dd = add2(mul2(a.dd, f2(ft, ft)), mul2(a.sr, f2(corr, corr)));
        a.st = mul2(a.st, f2(ft, ft));
        a.sr = mul2(a.sr, f2(fr, fr));
        a.mt = nmt;
        a.mr = nmr;
    }
    const float et = ex2(__fmaf_rn(xt.l, lt, __fmul_rn(__fsub_rn(xt.h, a.mt), lt)));
    const float er = ex2(__fmaf_rn(xr.l, lr, __fmul_rn(__fsub_rn(xr.h, a.mr), lr)));
    a.st = add2(a.st, f2(et, 0.f));
    a.sr = add2(a.sr, f2(er, 0.f));
    a.dd = add2(a.dd, f2(__fsub_rn(et, er), 0.f));
}

// kTables: 1 when both sides count in the same history (or one side counts in
// none), else one table a side.
template <bool kTBf16, bool kRBf16, bool kVec, int kTables>
__global__ void __launch_bounds__(kCtlThreads, kTables == 1 ? 3 : 2)
    score_kernel(const __grid_constant__ CtlScoreArgs a) {
    extern __shared__ __align__(16) char smem[];
    __shared__ int warp_sum[kCtlWarps];
    __shared__ float states[5][kCtlWarps];
    const Shared<kChunk> sh(smem, kTables, 2);
    uint32_t *const table_t = sh.table, *const table_r = sh.table + (kTables - 1) * kChunk;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const bool marks_t = a.t.counts || a.t.n_bias > 0, marks_r = a.r.counts || a.r.n_bias > 0;
    const bool marks = marks_t || marks_r;
    if (marks)
        for (int j = t; j < kTables * kChunk; j += kCtlThreads) sh.table[j] = 0;
    const int64_t units = a.hdr->n_active * a.n_chunks;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t i = u / a.n_chunks;
        const int k = static_cast<int>(u - i * a.n_chunks);
        const int64_t c0 = static_cast<int64_t>(k) * kChunk;
        const int2 rid = a.rowid[i];
        const int64_t r = rid.x, id = rid.y;
        const char *trow = a.xt + r * a.t_stride, *rrow = a.xr + r * a.r_stride;
        // 16 columns of each side a thread and step: groups t and t + 256 of
        // the step's 4096 columns; the first step's loads go out before the scan
        Group8<kTBf16> gt[2];
        Group8<kRBf16> gr[2];
        auto load = [&](int step) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int64_t j = c0 + 8 * (t + (2 * step + g) * kCtlThreads);
                if (j < a.vocab) {
                    ctl_load8<kTBf16, kVec>(trow, j, a.vocab, gt[g]);
                    ctl_load8<kRBf16, kVec>(rrow, j, a.vocab, gr[g]);
                }
            }
        };
        load(0);
        const CtlRow ot = ctl_row(a.t, r), orr = ctl_row(a.r, r);
        sh.touched[t] = 0;
        sh.allow_t[t] = ctl_allowed(ot, c0, t, a.vocab);
        sh.allow_r[t] = ctl_allowed(orr, c0, t, a.vocab);
        __syncthreads();
        const float lt = __fmul_rn(ot.scale, kLog2e), lr = __fmul_rn(orr.scale, kLog2e);
        Acc2 acc = acc2_init();
        if (marks) {
            const uint32_t len = static_cast<uint32_t>(min(static_cast<int64_t>(kChunk), a.vocab - c0));
            if (marks_t) ctl_mark(a.t, ot, r, c0, len, table_t, sh.touched, -1, nullptr);
            if (marks_r && !a.same) ctl_mark(a.r, orr, r, c0, len, table_r, sh.touched, -1, nullptr);
            __syncthreads();
            const int n = ctl_list(sh.touched, kChunk / 32, sh.list, warp_sum);
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
                accumulate_pair(vt, vr, acc, lt, lr);
                if (c0 + j == id)
                    a.pick[i] = make_double2(static_cast<double>(vt.h) + static_cast<double>(vt.l),
                                             static_cast<double>(vr.h) + static_cast<double>(vr.l));
            }
        }
        if (t == 0 && id >= c0 && id < c0 + kChunk && id < a.vocab) {
            const int j = static_cast<int>(id - c0);
            if (!(sh.touched[j >> 5] >> (j & 31) & 1u))
                a.pick[i] = make_double2(
                    sh.allow_t[j >> 5] >> (j & 31) & 1u ? static_cast<double>(ctl_elem<kTBf16>(trow, id)) : -CUDART_INF,
                    sh.allow_r[j >> 5] >> (j & 31) & 1u ? static_cast<double>(ctl_elem<kRBf16>(rrow, id)) : -CUDART_INF);
        }
#pragma unroll
        for (int step = 0; step < kChunk / 16 / kCtlThreads; ++step) {
            float vt[16], vr[16];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                ctl_unpack8<kTBf16>(gt[g], vt + 8 * g);
                ctl_unpack8<kRBf16>(gr[g], vr + 8 * g);
            }
            if (step + 1 < kChunk / 16 / kCtlThreads) load(step + 1);
            if (c0 + 8 * (t + 2 * step * kCtlThreads) >= a.vocab) continue;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int gi = t + (2 * step + g) * kCtlThreads;
                const uint32_t touched = group_bits(sh.touched, gi);
                const uint32_t st = touched | (group_bits(sh.allow_t, gi) ^ 0xffu);
                const uint32_t sr = touched | (group_bits(sh.allow_r, gi) ^ 0xffu);
                if (st | sr) {
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        vt[8 * g + q] = st >> q & 1u ? -INFINITY : vt[8 * g + q];
                        vr[8 * g + q] = sr >> q & 1u ? -INFINITY : vr[8 * g + q];
                    }
                }
            }
            f2_t pt[8], pr[8];
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                pt[p] = f2(vt[2 * p], vt[2 * p + 1]);
                pr[p] = f2(vr[2 * p], vr[2 * p + 1]);
            }
            accumulate16(pt, pr, acc, lt, lr);
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
        __syncthreads();
    }
}

// One warp per active row: lane l folds chunks l, l + 32, ... in order, the
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
    return launch_units(apply_kernel<kXB, kOB, kVec, kCols>, a, a.n_rows * a.n_chunks, 4, Shared<kCols>::bytes(1, 1),
                        configured, stream);
}

template <bool kXB, bool kOB, bool kVec, int kCols>
cudaError_t gradient_typed(GradArgs &a, cudaStream_t stream) {
    static std::atomic<uint64_t> configured{0};
    a.n_chunks = static_cast<int>(chunks_of(a.vocab, kCols));
    return launch_units(gradient_kernel<kXB, kOB, kVec, kCols>, a, a.n_rows * a.n_chunks, 4,
                        Shared<kCols>::bytes(1, 1), configured, stream);
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
    const size_t smem = Shared<kChunk>::bytes(kTables, 2);
    return vec ? launch_units(score_kernel<kTB, kRB, true, kTables>, a, units, per_sm, smem, configured[0], s)
               : launch_units(score_kernel<kTB, kRB, false, kTables>, a, units, per_sm, smem, configured[1], s);
}

}  // namespace

int controls_chunks(int64_t vocab) { return static_cast<int>(chunks_of(vocab, kChunk)); }

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
