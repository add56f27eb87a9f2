// Sampling controls on logits: penalties for repeated tokens, biases, grammar
// masks and the request's temperature, in three forms of one streaming kernel:
//   kApply   writes the controlled logits (what a sampler reads);
//   kScore   the log-sum-exp of both sides' controlled logits in one read of
//            each row, never written to memory;
//   kGrad    the selected-token logprob's gradient with respect to the raw
//            logits.
// The mathematics of a logit is in lpd_controls.cuh.
//
// Method: "WS2 Cross-Config Logprob Drift Contract", "Measurement Contract":
// the rollout's tokens are scored under the distribution that they were
// sampled from.
//
// Bound: HBM.  One persistent block per SM works through units: a row, or a
// range of its columns where there are few rows:
//   producer  one thread streams the unit's tiles (of both sides when scoring)
//             through a shared-memory ring with 1-D bulk copies (TMA,
//             completion on an mbarrier);
//   scouts    some warps prepare the next unit while this one streams: the
//             bitmap of its touched columns, and the touched tokens themselves.
//             When scoring they add these to sums of their own, and the stream
//             leaves them out; else they keep the values and store them once
//             the stream has passed over the unit;
//   stream    the other warps, 16 columns of each side a thread and tile.
// What bounds it now: waiting, in scoring, not one unit of the SM.  4096 x 151936
// bf16 pairs take 690 us with nothing to control and 840 us with a thousand
// touched tokens a row (331 us of HBM time).  In a capture of 1024 rows with
// nothing to control 53 % of the issue slots are used, the fma pipe 45 % and DRAM
// 44 %: sixteen warps, each with a chain of dependent steps a tile.  The rest is the
// scouts' reads of single logits, which a row's stream has to wait for.  The
// elementwise forms are nearer to HBM: the gradient of 2048 such rows, a tenth of
// them inactive, 252 us of 175.
// A first version gave every block a chunk, then scan, list and stream in turn
// with barriers between: 24 warps on an SM that mostly waited (39 % of issue
// slots), 1373 us for the same scoring.
#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "lpd_controls.cuh"

namespace lpd {
namespace {

constexpr int kApply = 0, kScore = 1, kGrad = 2;

constexpr int kStreamWarps = 16, kScoutWarps = 7;
constexpr int kTile = 16 * 32 * kStreamWarps;  // columns of a stage
constexpr int kStreamThreads = kStreamWarps * 32, kScoutThreads = kScoutWarps * 32;
constexpr int kThreads = kStreamThreads + kScoutThreads + 32;  // the producer's warp last
// Scoring keeps a state for each warp and segment of 57344 columns, whether one
// unit takes all segments of a row or each is a unit of its own, so a row's
// bits do not depend on how many rows there are.
constexpr int kSegment = 7 * 8192;
constexpr int kStates = kStreamWarps + kScoutWarps;
static_assert(kSegment % kTile == 0 && kSegment % 4096 == 0, "segments of whole tiles and bitmap lines");
constexpr int kMaxWidth = 3 * kSegment;        // columns of a unit: the bitmaps' room
constexpr int kWords = kMaxWidth / 32;
constexpr int kLines = (kWords + 127) / 128;   // lines of 128 bitmap words, one warp's scan each: four words a lane
// touched tokens at a time (more take several passes over the history)
constexpr int cap_of(int mode) { return mode == kScore ? 1536 : 4096; }
constexpr int kKept = 8;                       // history tokens that a scout keeps between its two passes
constexpr int kStagedBias = 128;               // bias entries kept in shared memory (more stay in global)
constexpr int kStagePad = 64;                  // a copy starts and ends on 16-byte boundaries around its columns
static_assert(2 * 8 * kStreamThreads == kTile, "two groups of eight columns a thread and tile");

constexpr unsigned long long kWaitLimitNs = 4000000000ull;
constexpr uint32_t kWaitLimitIters = 1u << 30;

// ---- barriers and copies (inline PTX) ----------------------------------------------
__device__ __forceinline__ uint32_t smem_u32(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ unsigned long long globaltimer_ns() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
__device__ __forceinline__ void mbar_init(uint64_t *bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive_expect_tx(uint64_t *bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ void bulk_g2s(void *dst, const void *src, uint32_t bytes, uint64_t *bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1], %2, [%3], %4;" ::"r"(smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}
// Bounded wait; when it gives up it raises the block's abort flag and, where
// there is a status word, sets LPD_STATUS_TIMEOUT.
__device__ __noinline__ bool wait_slow(uint64_t *bar, uint32_t parity, volatile int *abort_flag, uint32_t *status,
                                       bool honour_abort) {
    const unsigned long long t0 = globaltimer_ns();
    for (uint32_t n = 1; n < kWaitLimitIters; ++n) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((n & 255u) == 0) {
            if (honour_abort && *abort_flag) return false;
            if (globaltimer_ns() - t0 > kWaitLimitNs) break;
        }
    }
    *abort_flag = 1;
    if (status) atomicOr(status, LPD_STATUS_TIMEOUT);
    return false;
}
__device__ __forceinline__ bool wait_phase(uint64_t *bar, uint32_t parity, volatile int *abort_flag, uint32_t *status,
                                           bool honour_abort = true) {
    return mbar_try_wait(bar, parity) || wait_slow(bar, parity, abort_flag, status, honour_abort);
}
// All scouts reach it or none does: what one of them waits for, they all learn
// from it.  The barrier counts whole warps, so a warp's lanes meet first: one
// that left a loop early would otherwise arrive for the others.
__device__ __forceinline__ void scout_sync() {
    __syncwarp();
    asm volatile("bar.sync 1, %0;" ::"n"(kScoutThreads) : "memory");
}

// ---- arguments ---------------------------------------------------------------------
// One [rows, vocab] tensor as the stream reads it.
struct Plane {
    const char *base;
    int64_t stride;     // bytes
    const char *end;    // behind the last row's last column
};

struct StreamArgs {
    CtlSide c[2];       // the controls (kScore: train, rollout)
    Plane in[2];
    int64_t n_rows, vocab;
    int width, n_units; // columns of a unit (a multiple of 32; kScore: of kSegment), units a row
    int n_segs;         // kScore: segments a row
    int same;           // kScore: one count serves both sides
    uint32_t *status;
    int n_stages;
    // kApply, kGrad
    char *out;
    int64_t out_stride;  // bytes
    int in_place;        // kApply: the stream writes touched columns back as they are, for the scouts to read
    const int32_t *ids;
    const uint8_t *mask;
    const float *logp, *grad;
    // kScore
    const WsHeader *hdr;
    const int2 *rowid;
    float4 *part_a;
    float *part_b;
    double2 *pick;
};

// What the stream needs of a row, written by the scouts.
struct RowNumbers {
    float s, l, lt;    // scale (kScore: the rollout's), times log2 e, the train side's
    int same_scale;    // of at least kLeastNearScale
    float at, top, g;  // kGrad: a logit, log2 p there (upper part), -grad * scale * 2^(lower part)
    const uint8_t *mask[2];  // each side's mask bits, null: everything allowed
    int none[2];             // nothing allowed
};

template <int kMode>
struct Smem {
    static constexpr int kSides = kMode == kScore ? 2 : 1;
    static constexpr int kCap = cap_of(kMode);
    uint64_t full[16], empty[16], ready[2], done[2];
    CtlRow row[2];
    RowNumbers num[2];
    uint32_t id_word;
    int ok, abort_flag;
    int total;
    int line_base[kLines + 1];                  // touched columns in the lines in front
    float gs, low;                              // kGrad: grad * scale, the lower part of log2 p at num.at
    alignas(16) uint4 lanes[256];
    alignas(16) uint32_t touched[kMode == kGrad ? 1 : 2][kLines * 128];  // [unit parity] where the stream looks: it leaves these out
    alignas(8) uint16_t before[kLines * 128];   // touched columns in the words in front, of the same line
    uint32_t word[2][kCap];                     // kScore: a side's count words; else [unit parity], the values
    uint32_t list[kSides == 2 ? 1 : 2][kCap];   // their columns in the unit
    alignas(16) int32_t bias_ids[kSides][kStagedBias];  // the row's biases
    float bias[kSides][kStagedBias];
};
template <int kMode>
constexpr size_t ring_offset() {
    return (sizeof(Smem<kMode>) + 127) / 128 * 128;
}
constexpr size_t kSmemMost = 232448 - 1024;  // what a block may have, less the driver's own

// ---- where a tile's columns are ------------------------------------------------------
// Bulk copies start and end on 16-byte boundaries: the tile's bytes are widened
// to them as far as the tensor goes.  Column c of the tile's range sits at byte
// `lead` + (c - first) * size of the stage.  At the tensor's two ends up to
// seven columns may be missing there; the scouts take a row's first eight
// columns and its last eight to fifteen always (each unit's, in the elementwise
// forms), whether they are missing or not, so that a row's arithmetic does not
// depend on its place.
struct Span {
    const char *src;
    uint32_t bytes, at;  // copied bytes, and where in the stage they go
};
template <int kElt>
__device__ __forceinline__ Span span_of(const Plane &p, const char *row, int64_t first, int64_t end) {
    Span s;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(row + first * kElt), a1 = reinterpret_cast<uintptr_t>(row + end * kElt);
    const uintptr_t low = a0 & ~uintptr_t{15};
    uintptr_t b = low, e = (a1 + 15) & ~uintptr_t{15};
    if (b < reinterpret_cast<uintptr_t>(p.base)) b += 16;
    if (e > reinterpret_cast<uintptr_t>(p.end)) e -= 16;
    s.src = reinterpret_cast<const char *>(b);
    s.at = static_cast<uint32_t>(b - low);
    s.bytes = e > b ? static_cast<uint32_t>(e - b) : 0u;
    return s;
}
// The columns of a unit [c0, c1) that are the scouts' for their place: [c0,
// head) and [tail, c1).  When scoring they are the row's, whatever its units: a
// last unit of a few columns leaves the ends of the tensor's last row in the
// unit in front of it, and the split of a row between stream and scouts does
// not depend on its units.
template <int kMode>
__device__ __forceinline__ void edges(int64_t c0, int64_t c1, int64_t vocab, int64_t &head, int64_t &tail) {
    if (kMode == kScore) {
        head = max(c0, min(static_cast<int64_t>(8), c1));
        tail = min(max(vocab / 8 * 8 - 8, head), c1);
    } else {
        head = min(c0 + 8, c1);
        tail = max(c1 / 8 * 8 - 8, head);
    }
}

// Unit u: the row (kScore: its place among the active rows) and which of its
// units.  Each row starts at another of its units: a tokenizer's frequent
// tokens sit in the first columns, and a grid that is a multiple of n_units
// would give the same blocks every row's first unit.
__device__ __forceinline__ void unit_of(int64_t u, int n_units, int64_t &row, int &k) {
    if (n_units == 1) {
        row = u;
        k = 0;
        return;
    }
    row = u / n_units;
    k = static_cast<int>((u - row * n_units + row) % n_units);
}

// ---- scoring: sums of both sides ---------------------------------------------------
// Two sides that nearly agree (the same scale, u = z_t - z_r small) take one
// exponential a column, e = exp of the mean of the two exponents:
//   e_t - e_r = 2 e sinh(u / 2) = e (u + u^3 / 24 + ...)
//   e_t + e_r = 2 e cosh(u / 2) = e (2 + u^2 / 4 + ...)
// so four sums over the columns, of e, e u, e u^2 and e u^3, give both sides.
// Their difference is accurate relative to itself, where e_t - e_r of two
// rounded exponentials carries 2^-22 of the term (1e-5 of a logprob difference
// of 2e-3; this form: 1e-7), and the special-function unit has half the work.
// For |u| <= 1/8 the series' next terms are u^4 / 1920 = 1.3e-7 of the
// difference and u^4 / 192 = 1.3e-6 of the sum (the same on both sides).
constexpr float kNear2 = 0.015625f;  // sum of u^2 over a thread's sixteen columns
// A masked column of the stream holds about -1e30 (bf16 0xf149) on both sides:
// its term is 0 and its u finite.  Rows whose allowed logits are all below
// kFloorZ leave this path.
constexpr uint32_t kFillBits = 0xf149u;
constexpr float kFloorZ = -1e29f;
// Below this scale -1e30 need not be far below the others: each side of a column
// is then summed by itself, and a masked one left out.
constexpr float kLeastNearScale = 1e-20f;

// A side's factor from logits to base-2 exponents.  Scales from 2.4e38 on would
// make it infinite (and 0 times it NaN); differences that the largest number
// does not push below 2^-126 are below 4e-37.
__device__ __forceinline__ float exponent_factor(float scale) {
    const float l = __fmul_rn(scale, kLog2e);
    return l > FLT_MAX ? FLT_MAX : l;
}

constexpr float kLargestLow = 8.f;  // octaves

// expm1(u) / u up to u^5 / 720: the next term is u^6 / 5040 = 5e-8 at 1/4
__device__ __forceinline__ float expm1_ratio(float u) {
    float p = __fmaf_rn(u, 1.f / 720.f, 1.f / 120.f);
    p = __fmaf_rn(u, p, 1.f / 24.f);
    p = __fmaf_rn(u, p, 1.f / 6.f);
    p = __fmaf_rn(u, p, 0.5f);
    return __fmaf_rn(u, p, 1.f);
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

// The references raised to take in the maxima (ct, cr) of columns that are
// added next.  Two sides of one scale get one reference where neither can lose
// terms by it, as the sums of two sides that nearly agree need (see
// accumulate_near): the lower side goes up with the higher one only if its sum
// stays at 2^-8 of the reference's term or more, by what it holds or by what
// comes.  A sum's terms are flushed below 2^-126, so each side keeps all that
// counts, whatever the scale and however far the sides' peaks lie apart.
constexpr float kTied = 8.f;  // octaves
__device__ __forceinline__ void raise_to(Acc2 &a, float ct, float cr, float lt, float lr) {
    float nt = fmaxf(a.mt, ct), nr = fmaxf(a.mr, cr);
    if (nt != nr && lt == lr) {
        const bool t_low = nt < nr;
        const float top = t_low ? nr : nt, c = t_low ? ct : cr, m = t_low ? a.mt : a.mr;
        const f2_t held = t_low ? a.st : a.sr;
        const float sum = __fadd_rn(f2_lo(held), f2_hi(held));
        if (__fmul_rn(__fsub_rn(top, c), lr) <= kTied ||
            __fmul_rn(sum, ex2(__fmul_rn(__fsub_rn(m, top), lr))) >= 0.00390625f)
            nt = nr = top;
    }
    raise_refs(a, nt, nr, lt, lr);
}

// Columns 2 q and 2 q + 1 of a group, and the largest of two groups.  Both work
// on the raw words, so that no more than a pair is held widened at a time.
template <bool kBf16>
__device__ __forceinline__ f2_t group_pair(const Group8<kBf16> &g, int q) {
    if constexpr (kBf16) {
        const uint32_t w = q == 0 ? g.w[0].x : q == 1 ? g.w[0].y : q == 2 ? g.w[0].z : g.w[0].w;
        return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    } else {
        const uint4 &w = g.w[kBf16 ? 0 : q >> 1];
        return q & 1 ? f2(__uint_as_float(w.z), __uint_as_float(w.w)) : f2(__uint_as_float(w.x), __uint_as_float(w.y));
    }
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <bool kBf16>
__device__ __forceinline__ float groups_max(const Group8<kBf16> *g) {
    if constexpr (kBf16) {
        const uint32_t a = max_bf16x2(max_bf16x2(g[0].w[0].x, g[0].w[0].y), max_bf16x2(g[0].w[0].z, g[0].w[0].w));
        const uint32_t b = max_bf16x2(max_bf16x2(g[1].w[0].x, g[1].w[0].y), max_bf16x2(g[1].w[0].z, g[1].w[0].w));
        const uint32_t c = max_bf16x2(a, b);
        return fmaxf(__uint_as_float(c << 16), __uint_as_float(c & 0xffff0000u));
    } else {
        f2_t v[8];
#pragma unroll
        for (int p = 0; p < 8; ++p) v[p] = group_pair<kBf16>(g[p >> 2], p & 3);
        return max16(v);
    }
}

// Sixteen columns of two sides that nearly agree, by all lanes of a warp; false
// where they do not (the state is valid either way).  A NaN fails the comparison of the sum of
// squares.
template <bool kTBf16, bool kRBf16>
__device__ __forceinline__ bool accumulate_near(const Group8<kTBf16> *gt, const Group8<kRBf16> *gr, Acc2 &a, float l,
                                                float s) {
    const float ct = groups_max(gt), cr = groups_max(gr);
    const bool fit = fminf(ct, cr) > kFloorZ;
    if (__any_sync(0xffffffffu, fit && (ct > a.mt || cr > a.mr)))
        raise_to(a, fit ? ct : -INFINITY, fit ? cr : -INFINITY, l, l);
    const f2_t s2 = f2(s, s), m2 = f2(a.mr, a.mr), l2 = f2(l, l), h2 = f2(0.5f * kLog2e, 0.5f * kLog2e);
    f2_t q = f2(0.f, 0.f), e0 = q, e1 = q, e2 = q, e3 = q;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        // the mean exponent from the difference to the reference: its rounding
        // goes by the row's spread, not by where the row lies
        const f2_t xt = group_pair(gt[p >> 2], p & 3), xr = group_pair(gr[p >> 2], p & 3);
        const f2_t u = mul2(sub2(xt, xr), s2);
        const f2_t e = ex2_2(fma2(u, h2, mul2(sub2(xr, m2), l2)));
        const f2_t v = mul2(u, u), w = mul2(e, u);
        q = add2(q, v);
        e0 = add2(e0, e);
        e1 = add2(e1, w);
        e2 = fma2(e, v, e2);
        e3 = fma2(w, v, e3);
    }
    // (references apart: only where columns in front did not agree)
    if (!(fit && a.mt == a.mr && __fadd_rn(f2_lo(q), f2_hi(q)) <= kNear2)) return false;
    const f2_t d = fma2(e3, f2(1.f / 24.f, 1.f / 24.f), e1);       // e_t - e_r
    const f2_t m = fma2(e2, f2(0.125f, 0.125f), e0);               // their mean
    a.dd = add2(a.dd, d);
    a.st = add2(a.st, fma2(d, f2(0.5f, 0.5f), m));
    a.sr = add2(a.sr, fma2(d, f2(-0.5f, -0.5f), m));
    return true;
}

// Sixteen columns of any two sides, each with an exponential of its own; -inf
// adds nothing.  The differences to the references come first: a type's lowest
// value times the scale could overflow.
__device__ __forceinline__ void accumulate_far(const f2_t *vt, const f2_t *vr, Acc2 &a, float lt, float lr) {
    const float ct = max16(vt), cr = max16(vr);
    if (ct > a.mt || cr > a.mr) raise_to(a, ct, cr, lt, lr);
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

// A value whose lower part cannot lift its term far above one whose reference
// is the upper part: at scales or logits so large that it would, the value is
// the float.
__device__ __forceinline__ Two beside(Two v, float l) {
    return Two{v.h, fabsf(__fmul_rn(v.l, l)) <= kLargestLow ? v.l : 0.f};
}

// One pair of controlled logits (h + l of each side, see `beside`) into the
// state; an -inf adds nothing.
__device__ __forceinline__ void accumulate_pair(Two xt, Two xr, Acc2 &a, float lt, float lr, float s, bool same_scale) {
    if (xt.h > a.mt || xr.h > a.mr) raise_to(a, xt.h, xr.h, lt, lr);
    const float er = ex2(__fmaf_rn(xr.l, lr, __fmul_rn(__fsub_rn(xr.h, a.mr), lr)));
    const float u = __fmul_rn(
        __fadd_rn(__fsub_rn(__fsub_rn(xt.h, xr.h), __fsub_rn(a.mt, a.mr)), __fsub_rn(xt.l, xr.l)), s);
    float d, et;
    if (same_scale && fabsf(u) <= 0.25f) {
        d = __fmul_rn(__fmul_rn(er, u), expm1_ratio(u));
        et = __fadd_rn(er, d);
    } else {
        et = ex2(__fmaf_rn(xt.l, lt, __fmul_rn(__fsub_rn(xt.h, a.mt), lt)));
        d = __fsub_rn(et, er);
    }
    a.sr = add2(a.sr, f2(er, 0.f));
    a.st = add2(a.st, f2(et, 0.f));
    a.dd = add2(a.dd, f2(d, 0.f));
}

// ---- the scouts --------------------------------------------------------------------
// The tokens k, k + kScoutThreads, ... of a range, kKept of them in flight;
// those behind its end as -1 (no token).
__device__ __forceinline__ void fetch_tokens(const CtlSide &c, int64_t k, int64_t end, int32_t *t) {
#pragma unroll
    for (int u = 0; u < kKept; ++u) {
        const int64_t at = k + u * kScoutThreads;
        t[u] = at < end ? __ldg(c.history + at) : -1;
    }
}
// f(token, generated) over the row's range; `kept` holds the first tokens.
template <class F>
__device__ __forceinline__ void each_token(const CtlSide &c, const CtlRow &o, int st, const int32_t *kept, F f) {
    int64_t k = o.begin + st;
#pragma unroll
    for (int u = 0; u < kKept; ++u)
        if (kept[u] >= 0) f(kept[u], k + u * kScoutThreads >= o.split);
#pragma unroll 1
    for (k += kKept * kScoutThreads; k < o.end; k += kKept * kScoutThreads) {
        int32_t t[kKept];
        fetch_tokens(c, k, o.end, t);
#pragma unroll
        for (int u = 0; u < kKept; ++u)
            if (t[u] >= 0) f(t[u], k + u * kScoutThreads >= o.split);
    }
}

// The element type's name in templates.
template <bool kBf16>
constexpr int elt() { return kBf16 ? 2 : 4; }

template <int kMode, bool kXBf16, bool kYBf16, bool kAligned>
__global__ void __launch_bounds__(kThreads, 1) stream_kernel(const __grid_constant__ StreamArgs a) {
    // kYBf16: the rollout's logits (kScore) or the output
    extern __shared__ __align__(128) char smem_raw[];
    Smem<kMode> &sm = *reinterpret_cast<Smem<kMode> *>(smem_raw);
    char *const ring = smem_raw + ring_offset<kMode>();
    constexpr bool kTwo = kMode == kScore;
    constexpr int kXE = elt<kXBf16>(), kYE = elt<kYBf16>();
    constexpr int kStageX = kTile * kXE + kStagePad;
    constexpr int kStage = kStageX + (kTwo ? kTile * kYE + kStagePad : 0);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t n_rows = kTwo ? a.hdr->n_active : a.n_rows;
    const int64_t units = n_rows * a.n_units;

    if (threadIdx.x == 0) {
        sm.abort_flag = 0;
        for (int s = 0; s < a.n_stages; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], kStreamWarps);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sm.ready[b], 1);
            mbar_init(&sm.done[b], kStreamWarps);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (threadIdx.x < 256) sm.lanes[threadIdx.x] = ctl_lanes(threadIdx.x);
    __syncthreads();

    // kGrad: a row without a gradient (inactive, or an id out of range) has no
    // tiles and no scouting; every role decides it alike
    auto live = [&](int64_t r) -> bool {
        if (kMode != kGrad) return true;
        if (a.mask[r] == 0) return false;
        const int64_t id = a.ids[r];
        return id >= 0 && id < a.vocab;
    };
    // Columns between the start of a unit's first group of eight and the unit:
    // groups start on 16-byte boundaries of the output row.
    auto lead_in = [&](int64_t r, int64_t c0) -> int {
        if (kTwo || kAligned) return 0;
        const int at = static_cast<int>(reinterpret_cast<uintptr_t>(a.out + r * a.out_stride + c0 * kYE) & 15u) / kYE;
        return kYBf16 ? at : at & 3;
    };

    if (warp == kStreamWarps + kScoutWarps) {
        // ------------------------------------------------------------ producer
        if (lane != 0) return;
        uint64_t policy;
        asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
        int s = 0, issued = 0;
        uint32_t phase = 1;  // the first turn finds every stage empty
        bool ok = true;
        for (int64_t u = blockIdx.x; ok && u < units; u += gridDim.x) {
            int64_t i;
            int k;
            unit_of(u, a.n_units, i, k);
            const int64_t r = kTwo ? a.rowid[i].x : i;
            if (!live(r)) continue;
            const int64_t c0 = static_cast<int64_t>(k) * a.width, c1 = min(c0 + a.width, a.vocab);
            const char *const xrow = a.in[0].base + r * a.in[0].stride;
            const char *const yrow = kTwo ? a.in[1].base + r * a.in[1].stride : nullptr;
            for (int64_t tc = c0 - lead_in(r, c0); tc < c1; tc += kTile) {
                if (!wait_phase(&sm.empty[s], phase, &sm.abort_flag, a.status)) {
                    ok = false;
                    break;
                }
                char *st = ring + static_cast<size_t>(s) * kStage;
                if (kAligned && tc + kTile <= c1) {
                    mbar_arrive_expect_tx(&sm.full[s], kTile * (kXE + (kTwo ? kYE : 0)));
                    bulk_g2s(st, xrow + tc * kXE, kTile * kXE, &sm.full[s], policy);
                    if (kTwo) bulk_g2s(st + kStageX, yrow + tc * kYE, kTile * kYE, &sm.full[s], policy);
                } else {
                    const int64_t f = max(tc, c0), e = min(tc + kTile, c1);
                    const Span x = span_of<kXE>(a.in[0], xrow, f, e);
                    Span y{nullptr, 0, 0};
                    if (kTwo) y = span_of<kYE>(a.in[1], yrow, f, e);
                    mbar_arrive_expect_tx(&sm.full[s], x.bytes + y.bytes);
                    if (x.bytes) bulk_g2s(st + x.at, x.src, x.bytes, &sm.full[s], policy);
                    if (y.bytes) bulk_g2s(st + kStageX + y.at, y.src, y.bytes, &sm.full[s], policy);
                }
                issued = min(issued + 1, a.n_stages);
                if (++s == a.n_stages) {
                    s = 0;
                    phase ^= 1;
                }
            }
        }
        // every copy issued must land before the block's shared memory goes
        // away: the last turn's stages, each in the phase of its last use
        for (int j = 0; j < issued; ++j) {
            if (--s < 0) {
                s = a.n_stages - 1;
                phase ^= 1;
            }
            wait_phase(&sm.full[s], phase ^ 1, &sm.abort_flag, a.status, false);
        }
        return;
    }

    if (warp >= kStreamWarps) {
        // -------------------------------------------------------------- scouts
        const int st = threadIdx.x - kStreamThreads;
        constexpr int kCap = Smem<kMode>::kCap;
        constexpr int kLast = kTwo ? 1 : 0;
        const bool counts[2] = {a.c[0].counts != 0, kTwo && !a.same && a.c[1].counts != 0};
        uint32_t n_live = 0;
        // kApply, kGrad: the unit whose touched values wait for the stream to pass
        int64_t held_row = -1, held_c0 = 0;
        int held_n = 0;
        // one scout waits, all learn how it ended
        auto wait_all = [&](uint64_t *bar, uint32_t parity) -> bool {
            if (st == 0) sm.ok = wait_phase(bar, parity, &sm.abort_flag, a.status) ? 1 : 0;
            scout_sync();
            const bool ok = sm.ok != 0;
            scout_sync();
            return ok;
        };
        auto store_held = [&](uint32_t unit) -> bool {
            const uint32_t b = unit & 1;
            if (!wait_all(&sm.done[b], (unit >> 1) & 1)) return false;
            if constexpr (!kTwo) {
                char *orow = a.out + held_row * a.out_stride;
                for (int i = st; i < held_n; i += kScoutThreads)
                    ctl_store1<kYBf16>(orow, held_c0 + sm.list[b][i], __uint_as_float(sm.word[b][i]));
            }
            held_row = -1;
            scout_sync();
            return true;
        };
        for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
            int64_t i;
            int k;
            unit_of(u, a.n_units, i, k);
            const int2 rid = kTwo ? a.rowid[i] : make_int2(0, 0);
            const int64_t r = kTwo ? rid.x : i;
            if (!live(r)) continue;
            const int64_t id = kTwo ? static_cast<int64_t>(rid.y) : kMode == kGrad ? static_cast<int64_t>(a.ids[r]) : -1;
            const uint32_t b = n_live & 1;
            const int64_t c0 = static_cast<int64_t>(k) * a.width, c1 = min(c0 + a.width, a.vocab);
            const uint32_t len = static_cast<uint32_t>(c1 - c0);
            const int words = static_cast<int>((len + 31) / 32);
            const char *xrow = a.in[0].base + r * a.in[0].stride;
            const char *yrow = kTwo ? a.in[1].base + r * a.in[1].stride : nullptr;
            uint32_t *const touched = sm.touched[kMode == kGrad ? 0 : b];
            // the bitmap of this parity belongs to the unit before the last;
            // (store_held has waited for it in the elementwise forms)
            if (kTwo && n_live >= 2 && !wait_all(&sm.done[b], ((n_live >> 1) - 1) & 1)) return;
            if (st == 0) {
                sm.row[0] = ctl_row(a.c[0], r);
                sm.id_word = 0;
            }
            if (kTwo && st == 32) sm.row[1] = ctl_row(a.c[1], r);
            const int lines = (words + 127) / 128;
            for (int w = st; w < lines * 32; w += kScoutThreads) reinterpret_cast<uint4 *>(touched)[w] = make_uint4(0, 0, 0, 0);
            scout_sync();
            int32_t kept[2][kKept];
#pragma unroll
            for (int side = 0; side <= kLast; ++side) {
#pragma unroll
                for (int v = 0; v < kKept; ++v) kept[side][v] = -1;
                if (counts[side]) fetch_tokens(a.c[side], sm.row[side].begin + st, sm.row[side].end, kept[side]);
            }
            // first pass: which columns
            auto mark = [&](int32_t tok) {
                const uint64_t j = static_cast<uint64_t>(static_cast<int64_t>(tok) - c0);
                if (j < len) {
                    const uint32_t bit = 1u << (j & 31);
                    volatile uint32_t *w = &touched[j >> 5];
                    if (!(*w & bit)) atomicOr(&touched[j >> 5], bit);  // (a text's frequent tokens come often)
                }
            };
#pragma unroll
            for (int side = 0; side <= kLast; ++side) {
                if (counts[side])
                    each_token(a.c[side], sm.row[side], st, kept[side], [&](int32_t tok, bool gen) {
                        mark(tok);
                        if (kMode == kGrad && tok == id) {
                            if (gen) atomicAdd(&sm.id_word, 1u);
                            else atomicOr(&sm.id_word, kSeen);
                        }
                    });
                // staged ids are padded to a multiple of four
                if (a.c[side].n_bias + st < min((a.c[side].n_bias + 3) & ~3, kStagedBias))
                    sm.bias_ids[side][a.c[side].n_bias + st] = -1;
                for (int e = st; e < a.c[side].n_bias; e += kScoutThreads) {
                    const int32_t tok = __ldg(a.c[side].bias_ids + r * a.c[side].n_bias + e);
                    if (a.c[side].n_bias <= kStagedBias) {
                        sm.bias_ids[side][e] = tok;
                        sm.bias[side][e] = __ldg(a.c[side].bias + r * a.c[side].n_bias + e);
                    }
                    mark(tok);
                    if (kMode == kGrad && tok == id) atomicOr(&sm.id_word, kBiased);
                }
            }
            if (kMode == kGrad && st == 0 && id >= c0 && id < c1)
                atomicOr(&touched[(id - c0) >> 5], 1u << ((id - c0) & 31));
            {
                // the unit's edges; behind the vocabulary up to a group of eight, which the list leaves out
                int64_t head, tail;
                edges<kMode>(c0, c1, a.vocab, head, tail);
                const int n_head = static_cast<int>(head - c0), up = static_cast<int>((len + 7) / 8 * 8);
                const int at = st < n_head ? st : static_cast<int>(tail - c0) + st - n_head;
                if (at < up) atomicOr(&touched[at >> 5], 1u << (at & 31));
            }
            scout_sync();
            // the bias of a token on each side (one search where the sides share their ids)
            auto bias_of = [&](int32_t token, Two *v) {
                int at = -1, found = 0;
#pragma unroll
                for (int side = 0; side <= kLast; ++side) {
                    const int n = a.c[side].n_bias;
                    v[side] = Two{0.f, 0.f};
                    if (n == 0) continue;
                    const bool staged = n <= kStagedBias;
                    const int32_t *ids = staged ? sm.bias_ids[side] : a.c[side].bias_ids + r * n;
                    if (side == 0 || !a.same) {
                        at = -1;
                        found = 0;
                        if (staged) {
                            at = bias_find(reinterpret_cast<const int4 *>(ids), n, token, &found);
                        } else {
                            for (int e = 0; e < n; ++e)
                                if (ids[e] == token) {
                                    at = e;
                                    ++found;
                                }
                        }
                    }
                    v[side] = bias_sum(ids, staged ? sm.bias[side] : a.c[side].bias + r * n, n, token, at, found);
                }
            };
            // the row's numbers for the stream
            if (st == 0) {
                RowNumbers &num = sm.num[b];
                const float s = sm.row[kLast].scale;
                num.s = s;
                num.l = exponent_factor(s);
                if (kTwo) {
                    num.lt = exponent_factor(sm.row[0].scale);
                    num.same_scale = sm.row[0].scale == s && s >= kLeastNearScale ? 1 : 0;
                }
#pragma unroll
                for (int side = 0; side <= kLast; ++side) {
                    num.mask[side] = reinterpret_cast<const uint8_t *>(sm.row[side].mask);
                    num.none[side] = sm.row[side].none ? 1 : 0;
                }
                if (kMode == kGrad) {
                    const CtlRow &o = sm.row[0];
                    // p_j = 2^(log2 p + (x_j - at) scale log2 e) from a logit `at` whose
                    // probability is known, so that the exponents' rounding goes by the
                    // row's spread, not by where it lies: the selected token, or, where
                    // that lies far below, the log-sum-exp's own place.  A masked token
                    // gives NaN.
                    double at = 0.0, top = CUDART_NAN;
                    if (ctl_allows(o, id)) {
                        Two bias[kLast + 1];
                        bias_of(static_cast<int32_t>(id), bias);
                        const Two v = ctl_value(ctl_elem<kXBf16>(xrow, id), sm.id_word, o, bias[0], nullptr);
                        const double sc = o.scale, lp = a.logp[r];
                        if (lp > -32.0) {
                            at = v.h;
                            top = lp - static_cast<double>(v.l) * sc;
                        } else {
                            const double lse = (static_cast<double>(v.h) + static_cast<double>(v.l)) * sc - lp;
                            at = static_cast<float>(lse / sc);
                            top = at * sc - lse;
                        }
                    }
                    top *= 1.4426950408889634;
                    const float h = static_cast<float>(top), gs = __fmul_rn(a.grad[r], o.scale);
                    sm.low = static_cast<float>(top - static_cast<double>(h));
                    sm.gs = gs;
                    num.at = static_cast<float>(at);
                    num.top = h;
                    num.g = __fmul_rn(-gs, ex2(sm.low));
                }
                mbar_arrive(&sm.ready[b]);
            }
            // each word's rank within its line
            for (int line = kScoutWarps - 1 - (warp - kStreamWarps); line < lines; line += kScoutWarps) {
                const int w = 32 * line + lane;
                const uint4 bits = reinterpret_cast<const uint4 *>(touched)[w];
                const int n0 = __popc(bits.x), n1 = n0 + __popc(bits.y), n2 = n1 + __popc(bits.z), n = n2 + __popc(bits.w);
                int incl = n;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, incl, off);
                    if (lane >= off) incl += v;
                }
                const int at = incl - n;
                reinterpret_cast<ushort4 *>(sm.before)[w] =
                    make_ushort4(static_cast<uint16_t>(at), static_cast<uint16_t>(at + n0), static_cast<uint16_t>(at + n1),
                                 static_cast<uint16_t>(at + n2));
                if (lane == 31) sm.line_base[line] = incl;
            }
            scout_sync();
            if (warp == kStreamWarps) {
                // the lines' sums become what lies in front of them
                int sum = 0;
                for (int l0 = 0; l0 <= lines; l0 += 32) {
                    const int n = l0 + lane < lines ? sm.line_base[l0 + lane] : 0;
                    int incl = n;
#pragma unroll
                    for (int off = 1; off < 32; off <<= 1) {
                        const int v = __shfl_up_sync(0xffffffffu, incl, off);
                        if (lane >= off) incl += v;
                    }
                    if (l0 + lane <= lines) sm.line_base[l0 + lane] = sum + incl - n;
                    sum += __shfl_sync(0xffffffffu, incl, 31);
                }
                if (lane == 0) sm.total = sum - static_cast<int>((8 - len % 8) % 8);
            }
            scout_sync();
            const int total = sm.total;
            uint32_t *const w0 = kTwo ? sm.word[0] : sm.word[b];
            uint32_t *const w1 = sm.word[1];
            uint32_t *const list = kTwo ? sm.list[0] : sm.list[b];
            // The touched tokens of ranks [base, base + m): their columns, and
            // in a second pass over the history how often each occurs.
            auto count = [&](int base, int m) {
                for (int q = st; q < m; q += kScoutThreads) {
                    w0[q] = 0;
                    if (kTwo) w1[q] = 0;
                }
                scout_sync();
                // a column's rank among the window's; every mark of a column
                // writes it down there (the same value, so their order is free)
                auto enter = [&](uint32_t j) -> int {
                    const int p = sm.line_base[j >> 12] + sm.before[j >> 5] + __popc(touched[j >> 5] & ((1u << (j & 31)) - 1u)) - base;
                    if (p < 0 || p >= m) return -1;
                    list[p] = j;
                    // its logits and mask word will be wanted soon
                    prefetch_l1(xrow + (c0 + j) * kXE);
                    if (kTwo) prefetch_l1(yrow + (c0 + j) * kYE);
                    if (sm.row[0].mask) prefetch_l1(sm.row[0].mask + (c0 + j) / 32);
                    return p;
                };
                auto place = [&](int32_t tok) -> int {
                    const uint64_t j = static_cast<uint64_t>(static_cast<int64_t>(tok) - c0);
                    return j < len ? enter(static_cast<uint32_t>(j)) : -1;
                };
                {
                    int64_t head, tail;
                    edges<kMode>(c0, c1, a.vocab, head, tail);
                    const int n_head = static_cast<int>(head - c0);
                    const int at = st < n_head ? st : static_cast<int>(tail - c0) + st - n_head;
                    if (at < static_cast<int>(len)) enter(static_cast<uint32_t>(at));
                    if (kMode == kGrad && st == kScoutThreads - 1) place(static_cast<int32_t>(id));
                }
#pragma unroll
                for (int side = 0; side <= kLast; ++side) {
                    uint32_t *const word = side ? w1 : w0;
                    if (counts[side])
                        each_token(a.c[side], sm.row[side], st, kept[side], [&](int32_t tok, bool gen) {
                            const int p = place(tok);
                            if (p < 0) return;
                            if (gen) atomicAdd(&word[p], 1u);
                            else if (!(*static_cast<volatile uint32_t *>(&word[p]) & kSeen)) atomicOr(&word[p], kSeen);
                        });
                    if (side == 0 || !a.same) {
                        const int32_t *ids = a.c[side].n_bias <= kStagedBias ? sm.bias_ids[side]
                                                                             : a.c[side].bias_ids + r * a.c[side].n_bias;
                        for (int e = st; e < a.c[side].n_bias; e += kScoutThreads) {
                            const int p = place(ids[e]);
                            if (p >= 0) atomicOr(&word[p], kBiased);
                        }
                    }
                }
                scout_sync();
            };
            if constexpr (kTwo) {
                const float s_r = sm.num[b].s, lt = sm.num[b].lt, lr = sm.num[b].l;
                const bool same_scale = sm.num[b].same_scale != 0;
                // an untouched selected token (the stream leaves a touched one to the list below)
                if (st == 0 && id >= c0 && id < c1 && !(touched[(id - c0) >> 5] >> ((id - c0) & 31) & 1u))
                    a.pick[i] = make_double2(
                        ctl_allows(sm.row[0], id) ? static_cast<double>(ctl_elem<kXBf16>(xrow, id)) : -CUDART_INF,
                        ctl_allows(sm.row[1], id) ? static_cast<double>(ctl_elem<kYBf16>(yrow, id)) : -CUDART_INF);
                if (total > 0 && total <= kCap) count(0, total);
                for (int64_t f = c0; f < c1; f += kSegment) {
                    const int first = sm.line_base[(f - c0) >> 12];
                    const int end = f + kSegment < c1 ? sm.line_base[(f + kSegment - c0) >> 12] : total;
                    Acc2 acc = acc2_init();
                    for (int base = first; base < end; base += kCap) {
                        const int m = min(kCap, end - base);
                        if (total > kCap) count(base, m);
                        const int at = total > kCap ? 0 : base;  // list position of rank `base`
                        // two tokens at a time: their chains of arithmetic are independent
                        for (int q0 = st; q0 < m; q0 += 2 * kScoutThreads) {
                            Two vt[2], vr[2];
                            int64_t col[2];
#pragma unroll
                            for (int v = 0; v < 2; ++v) {
                                const int q = q0 + v * kScoutThreads;
                                vt[v] = vr[v] = Two{-INFINITY, 0.f};
                                col[v] = -1;
                                if (q >= m) continue;
                                col[v] = c0 + list[at + q];
                                const float x0 = ctl_elem<kXBf16>(xrow, col[v]), x1 = ctl_elem<kYBf16>(yrow, col[v]);
                                const uint32_t t0 = w0[at + q], t1 = a.same ? t0 : w1[at + q];
                                Two bias[2] = {Two{0.f, 0.f}, Two{0.f, 0.f}};
                                if ((t0 | t1) & kBiased) bias_of(static_cast<int32_t>(col[v]), bias);
                                const bool in0 = ctl_allows(sm.row[0], col[v]);
                                const bool in1 = sm.row[0].mask == sm.row[1].mask && sm.row[0].none == sm.row[1].none
                                                     ? in0
                                                     : ctl_allows(sm.row[1], col[v]);
                                const Two y0 = beside(ctl_value(x0, t0, sm.row[0], bias[0], nullptr), lt);
                                const Two y1 = beside(ctl_value(x1, t1, sm.row[1], bias[1], nullptr), lr);
                                if (in0) vt[v] = y0;
                                if (in1) vr[v] = y1;
                            }
#pragma unroll
                            for (int v = 0; v < 2; ++v) {
                                if (col[v] < 0) continue;
                                accumulate_pair(vt[v], vr[v], acc, lt, lr, s_r, same_scale);
                                if (col[v] == id)
                                    a.pick[i] = make_double2(static_cast<double>(vt[v].h) + static_cast<double>(vt[v].l),
                                                             static_cast<double>(vr[v].h) + static_cast<double>(vr[v].l));
                            }
                        }
                        if (total > kCap) scout_sync();
                    }
                    const Acc w = warp_reduce_acc<false>(acc2_fold(acc), lt, lr);
                    if (lane == 0) {
                        const int64_t o = (i * a.n_segs + f / kSegment) * kStates + warp;
                        a.part_a[o] = make_float4(w.mt, w.st, w.dd, w.mr);
                        a.part_b[o] = w.sr;
                    }
                }
                scout_sync();
            } else {
                const float s = sm.row[0].scale, f = sm.num[b].l;
                auto result = [&](int q) -> float {
                    const int64_t col = c0 + list[q];
                    const float x0 = ctl_elem<kXBf16>(xrow, col);
                    const bool in0 = ctl_allows(sm.row[0], col);
                    if (!in0) return kMode == kApply ? -INFINITY : 0.f;
                    float slope;
                    Two bias[kLast + 1] = {Two{0.f, 0.f}};
                    if (w0[q] & kBiased) bias_of(static_cast<int32_t>(col), bias);
                    const Two v = ctl_value(x0, w0[q], sm.row[0], bias[0], &slope);
                    if (kMode == kApply) return __fmaf_rn(v.h, s, __fmul_rn(v.l, s));
                    const float e = __fmaf_rn(__fsub_rn(v.h, sm.num[b].at), f, sm.num[b].top);
                    const float p = ex2(__fadd_rn(__fadd_rn(e, sm.low), __fmul_rn(v.l, f)));
                    return __fmul_rn(__fmul_rn(sm.gs, slope), __fsub_rn(col == id ? 1.f : 0.f, p));
                };
                const int m = min(kCap, total);
                if (total > 0) {
                    count(0, m);
                    for (int q = st; q < m; q += kScoutThreads) w0[q] = __float_as_uint(result(q));
                }
                scout_sync();
                // the last unit's values, now that the stream has this one to go on with
                if (held_row >= 0 && !store_held(n_live - 1)) return;
                held_row = r;
                held_c0 = c0;
                held_n = m;
                if (total > kCap) {
                    // more than kCap: straight to the output, behind the stream
                    // (in place it has left them as they were)
                    if (!store_held(n_live)) return;
                    for (int base = kCap; base < total; base += kCap) {
                        const int n = min(kCap, total - base);
                        count(base, n);
                        for (int q = st; q < n; q += kScoutThreads)
                            ctl_store1<kYBf16>(a.out + r * a.out_stride, c0 + list[q], result(q));
                        scout_sync();
                    }
                }
            }
            ++n_live;
        }
        if (!kTwo && held_row >= 0) store_held(n_live - 1);
        return;
    }

    // ------------------------------------------------------------------ stream
    const int t = threadIdx.x;
    int stage = 0;
    uint32_t phase = 0, n_live = 0;
    bool dead = false;  // a wait gave up: what is left of the output reads as NaN
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        int64_t i;
        int k;
        unit_of(u, a.n_units, i, k);
        const int64_t r = kTwo ? 0 : i;
        const int64_t c0 = static_cast<int64_t>(k) * a.width;
        const int len = static_cast<int>(min(static_cast<int64_t>(a.width), a.vocab - c0));
        const int lead = kTwo ? 0 : lead_in(r, c0);
        char *const orow = kTwo ? nullptr : a.out + r * a.out_stride + c0 * kYE;  // the unit's first column
        auto fill = [&](float value) {
            float v[8];
            Group8<kYBf16> w;
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = value;
            ctl_pack8<kYBf16>(v, w);
            for (int j = 8 * t - lead; j < len; j += 8 * kStreamThreads) {
                if (j >= 0 && j + 8 <= len) {
                    ctl_store8<kYBf16>(orow, j, w);
                } else {
                    for (int q = max(j, 0); q < min(j + 8, len); ++q) ctl_store1<kYBf16>(orow, q, value);
                }
            }
        };
        if (!kTwo && (dead || !live(r))) {
            // inactive rows: 0; an active row with an out-of-range id: NaN
            fill(!dead && a.mask[r] == 0 ? 0.f : CUDART_NAN_F);
            continue;
        }
        const uint32_t b = n_live & 1;
        {
            const bool ok = wait_phase(&sm.ready[b], (n_live >> 1) & 1, &sm.abort_flag, a.status);
            if (__any_sync(0xffffffffu, !ok)) {
                if (kTwo) return;
                dead = true;
                fill(CUDART_NAN_F);
                continue;
            }
        }
        const RowNumbers &num = sm.num[b];
        const bool same_scale = kTwo && num.same_scale != 0;
        const float n_s = num.s, n_l = num.l, n_lt = kTwo ? num.lt : 0.f;
        const float n_at = kMode == kGrad ? num.at : 0.f, n_top = kMode == kGrad ? num.top : 0.f, n_g = kMode == kGrad ? num.g : 0.f;
        // Masked columns, eight bits a group.  The mask's bytes come from global
        // memory, asked for a tile ahead; `last` keeps them inside the row's.
        const bool none0 = num.none[0] != 0, none1 = kTwo && num.none[kTwo ? 1 : 0] != 0;
        const uint8_t *const mask0 = num.mask[0], *const mask1 = kTwo ? num.mask[1] : nullptr;
        const bool one_mask = mask0 == mask1;
        const int64_t first_byte = (c0 - lead) >> 3;
        const int last_byte = static_cast<int>(((a.vocab - 1) >> 3) - first_byte);
        const int shift = kTwo || kAligned ? 0 : static_cast<int>(c0 - lead) & 7;
        uint32_t m0[2] = {0, 0}, m1[2] = {0, 0};
        auto ask1 = [&](const uint8_t *mask, int at) -> uint32_t {
            const uint8_t *p = mask + first_byte;
            if (kTwo || kAligned) return ~static_cast<uint32_t>(__ldg(p + min(at, last_byte)));
            const int low = first_byte < 0 ? 1 : 0;
            const uint32_t lo = __ldg(p + max(min(at, last_byte), low)), hi = __ldg(p + max(min(at + 1, last_byte), low));
            return ~((lo | hi << 8) >> shift);
        };
        auto ask = [&](int tile) {
            if (mask0) {
                m0[0] = ask1(mask0, tile * (kTile / 8) + t);
                m0[1] = ask1(mask0, tile * (kTile / 8) + t + kStreamThreads);
            }
            if (kTwo && mask1 && !one_mask) {
                m1[0] = ask1(mask1, tile * (kTile / 8) + t);
                m1[1] = ask1(mask1, tile * (kTile / 8) + t + kStreamThreads);
            }
        };
        ask(0);
        uint32_t at_x = 0, at_y = 0;  // where the first tile's groups start in a stage (the others': aligned alike)
        if (!kAligned) {
            const int64_t row = kTwo ? a.rowid[i].x : r;
            at_x = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(a.in[0].base + row * a.in[0].stride + (c0 - lead) * kXE)) & 15u;
            if (kTwo) at_y = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(a.in[1].base + row * a.in[1].stride + c0 * kYE)) & 15u;
        }
        Acc2 acc = acc2_init();
        const int tiles = (len + lead + kTile - 1) / kTile;
        int seg_left = kSegment / kTile;
        int64_t state = kTwo ? (i * a.n_segs + c0 / kSegment) * kStates + warp : 0;
#pragma unroll 1
        for (int tile = 0; tile < tiles; ++tile) {
            const bool ok = wait_phase(&sm.full[stage], phase, &sm.abort_flag, a.status);
            if (__any_sync(0xffffffffu, !ok)) {
                if (kTwo) return;
                dead = true;
                break;
            }
            const char *stg = ring + stage * kStage;
            Group8<kXBf16> gx[2];
            Group8<kYBf16> gy[2];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int j = 8 * (t + g * kStreamThreads);
                // A first tile that starts in front of its unit was copied from
                // the unit's first column on: its first group is the scouts',
                // the others lie where a copy from the tile's start had them.
                const uint32_t skew = !kAligned && !kTwo && tile == 0 && lead > 0
                                          ? (at_x + lead * kXE & ~15u)
                                          : 0u;
                ctl_shared8<kXBf16, kAligned>(stg, max(static_cast<int>(at_x + j * kXE - skew), 0), gx[g]);
                if constexpr (kTwo) ctl_shared8<kYBf16, kAligned>(stg + kStageX, at_y + j * kYE, gy[g]);
            }
            // The stage's next copy is the async proxy's: it is ordered behind
            // these reads by the proxy fence, not by the barrier alone (without
            // it one row in two hundred of a long run read a later tile).
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.empty[stage]);
            if (++stage == a.n_stages) {
                stage = 0;
                phase ^= 1;
            }
            uint32_t s0[2] = {m0[0] & 0xffu, m0[1] & 0xffu}, s1[2] = {m1[0] & 0xffu, m1[1] & 0xffu};
            if (one_mask) {
                s1[0] = s0[0];
                s1[1] = s0[1];
            }
            if (tile + 1 < tiles) ask(tile + 1);
            const int left = len + lead - tile * kTile;  // columns from the tile's start on
            if constexpr (kTwo) {
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const int group = t + g * kStreamThreads;
                    const uint32_t out = left > 8 * group
                                             ? reinterpret_cast<const uint8_t *>(sm.touched[b])[tile * (kTile / 8) + group]
                                             : 0xffu;
                    s0[g] |= none0 ? 0xffu : out;
                    s1[g] |= none1 ? 0xffu : out;
                }
                if (__any_sync(0xffffffffu, (s0[0] & s0[1] & s1[0] & s1[1]) != 0xffu)) {  // something is allowed
                    if (__any_sync(0xffffffffu, (s0[0] | s0[1] | s1[0] | s1[1]) != 0u)) {
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            ctl_fill8<kXBf16, kFillBits>(gx[g], sm.lanes[s0[g]]);
                            ctl_fill8<kYBf16, kFillBits>(gy[g], sm.lanes[s1[g]]);
                        }
                    }
                    const bool any = (s0[0] & s0[1] & s1[0] & s1[1]) != 0xffu;
                    const bool near = same_scale && accumulate_near(gx, gy, acc, n_l, n_s);
                    if (any && !near) {
                        f2_t pt[8], pr[8];
#pragma unroll
                        for (int p = 0; p < 8; ++p) {
                            const uint32_t bt = s0[p >> 2] >> (2 * (p & 3)), br = s1[p >> 2] >> (2 * (p & 3));
                            const f2_t xt = group_pair(gx[p >> 2], p & 3), xr = group_pair(gy[p >> 2], p & 3);
                            pt[p] = f2(bt & 1u ? -INFINITY : f2_lo(xt), bt & 2u ? -INFINITY : f2_hi(xt));
                            pr[p] = f2(br & 1u ? -INFINITY : f2_lo(xr), br & 2u ? -INFINITY : f2_hi(xr));
                        }
                        accumulate_far(pt, pr, acc, n_lt, n_l);
                    }
                }
                if (--seg_left == 0 || tile + 1 == tiles) {
                    const Acc w = warp_reduce_acc<false>(acc2_fold(acc), n_lt, n_l);
                    if (lane == 0) {
                        a.part_a[state] = make_float4(w.mt, w.st, w.dd, w.mr);
                        a.part_b[state] = w.sr;
                    }
                    state += kStates;
                    seg_left = kSegment / kTile;
                    acc = acc2_init();
                }
            } else {
                const f2_t f2f = f2(n_l, n_l), at2 = f2(n_at, n_at), top2 = f2(n_top, n_top), g2f = f2(n_g, n_g);
                const f2_t s2f = f2(n_s, n_s);
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const int group = t + g * kStreamThreads, j = tile * kTile + 8 * group - lead;
                    float v[8];
                    ctl_unpack8<kXBf16>(gx[g], v);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const f2_t z = f2(v[2 * q], v[2 * q + 1]);
                        const f2_t d = kMode == kApply ? mul2(z, s2f) : mul2(g2f, ex2_2(fma2(sub2(z, at2), f2f, top2)));
                        v[2 * q] = f2_lo(d);
                        v[2 * q + 1] = f2_hi(d);
                    }
                    Group8<kYBf16> w;
                    ctl_pack8<kYBf16>(v, w);
                    constexpr uint32_t kMasked = kMode == kApply ? 0xff80u : 0u;  // -inf, or no gradient
                    const uint32_t skip = none0 ? 0xffu : s0[g];
                    if (skip) ctl_fill8<kYBf16, kMasked>(w, sm.lanes[skip]);
                    if (j < 0 || left < 8 * group + 8) continue;  // the scouts'
                    if constexpr (kMode == kApply && kXBf16 == kYBf16) {
                        if (a.in_place) {
                            const uint8_t *bits = reinterpret_cast<const uint8_t *>(sm.touched[b]) + (j >> 3);
                            const uint32_t keep = kAligned ? bits[0] : (bits[0] | bits[1] << 8) >> (j & 7) & 0xffu;
                            if (keep) ctl_keep8<kYBf16>(w, gx[g], sm.lanes[keep]);
                        }
                    }
                    ctl_store8<kYBf16>(orow, j, w);
                }
            }
        }
        if (!kTwo && dead) fill(CUDART_NAN_F);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.done[b]);
        ++n_live;
    }
}

// One warp per active row: lane l folds the segments' warp states l, l + 32, ... in order, the
// warp merges in a fixed butterfly, lane 0 does the row's arithmetic in double
// (the formulas of the plain scorer, with each side's scale).
__global__ void __launch_bounds__(256) score_finalize_kernel(const __grid_constant__ StreamArgs a, float *out_lt,
                                                            float *out_lr, float *out_d, double *dval,
                                                            uint32_t *keys, uint32_t *status) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (i >= a.hdr->n_active) return;
    const int2 rid = a.rowid[i];
    const int64_t r = rid.x, id = rid.y;
    float s_t = a.c[0].scale ? a.c[0].scale[r] : 1.f, s_r = a.c[1].scale ? a.c[1].scale[r] : 1.f;
    if (!(s_t > 0.f && s_t <= FLT_MAX)) s_t = CUDART_NAN_F;
    if (!(s_r > 0.f && s_r <= FLT_MAX)) s_r = CUDART_NAN_F;
    const float lt = exponent_factor(s_t), lr = exponent_factor(s_r);
    Acc acc = acc_init();
    const int n = a.n_segs * kStates;
    for (int k = lane; k < n; k += 32) {
        const float4 p = a.part_a[i * n + k];
        const Acc o{p.x, p.y, p.z, p.w, a.part_b[i * n + k], 0.f, 0.f};
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
        // differences to the maxima before the scale: at a scale of 1e15 a
        // logarithm is lost beside the scaled maximum even in double
        const double xt = s_t * (x.x - acc.mt), xr = s_r * (x.y - acc.mr);
        const double st = acc.st, sr = acc.sr, dd = acc.dd;
        const double lse_t = log(st), lse_r = log(sr);  // above the scaled maxima
        // dd is st - sr with an error relative to itself where the sides move
        // together.  Where they do not (thousands on one side before its
        // dominant token is met, a few on the other) it may have lost more than
        // the sums, and has to fit them to their roundings: some 50 a side, 2^-17.
        const bool near = fabs(dd) < 0.5 * st && fabs(dd - (st - sr)) <= 7.6e-6 * st;
        const double ratio = near ? log1p(-dd / st) : log(sr / st);
        d = (xt - xr) + ratio;
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

int score_segments(int64_t vocab) { return static_cast<int>((vocab + kSegment - 1) / kSegment); }

template <int kMode, bool kXB, bool kYB, bool kAligned>
cudaError_t launch_typed(StreamArgs &a, int64_t rows, cudaStream_t stream) {
    auto kern = stream_kernel<kMode, kXB, kYB, kAligned>;
    constexpr size_t stage = (kTile * elt<kXB>() + kStagePad) + (kMode == kScore ? kTile * elt<kYB>() + kStagePad : 0);
    constexpr size_t room = kSmemMost - ring_offset<kMode>();
    constexpr int stages = static_cast<int>(room / stage < 16 ? room / stage : 16);
    static_assert(stages >= 2, "a ring of at least two stages");
    static std::atomic<uint64_t> configured{0};
    const size_t smem = ring_offset<kMode>() + stages * stage;
    const cudaError_t e = set_smem_once(kern, smem, configured);
    if (e != cudaSuccess) return e;
    a.n_stages = stages;
    const int64_t units = rows * a.n_units, sms = device_sm_count();
    kern<<<static_cast<unsigned>(units < sms ? units : sms), kThreads, smem, stream>>>(a);
    return cudaGetLastError();
}

template <int kMode, bool kAligned>
cudaError_t launch_kinds(StreamArgs &a, bool xb, bool yb, int64_t rows, cudaStream_t s) {
    if (xb) return yb ? launch_typed<kMode, true, true, kAligned>(a, rows, s) : launch_typed<kMode, true, false, kAligned>(a, rows, s);
    return yb ? launch_typed<kMode, false, true, kAligned>(a, rows, s) : launch_typed<kMode, false, false, kAligned>(a, rows, s);
}

bool aligned_rows(const void *p, int64_t stride_bytes) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride_bytes % 16 == 0;
}

Plane plane(const void *base, int64_t stride_bytes, int elt_bytes, int64_t rows, int64_t vocab) {
    const char *b = static_cast<const char *>(base);
    return Plane{b, stride_bytes, b + (rows - 1) * stride_bytes + vocab * elt_bytes};
}

// Units of the elementwise forms: as few as the bitmaps allow, and with fewer
// rows than blocks as many as keep every block to one unit, down to 2048 columns
// (a decode step's one row is cut in 63 units of a 128256-column vocabulary).
// Every unit of a row looks through its whole history, so more units a block
// cost more than the idle blocks that they avoid: 256 rows of 151936 with 8192
// tokens of history in 107 us as whole rows, 146 us as three units each; 100
// rows in 62 us, 83 us as two units each.  Rows that are not 16-byte aligned
// start up to seven columns early, which a full last tile could not take.
void set_units(StreamArgs &a, bool aligned) {
    const int64_t most = kMaxWidth - (aligned ? 0 : 32);
    int64_t n = (a.vocab + most - 1) / most;
    n = std::max(n, std::min(device_sm_count() / a.n_rows, (a.vocab + 2047) / 2048));
    a.width = static_cast<int>(((a.vocab + n - 1) / n + 31) / 32 * 32);
    a.n_units = static_cast<int>((a.vocab + a.width - 1) / a.width);
}

}  // namespace

int controls_states(int64_t vocab) { return score_segments(vocab) * kStates; }

cudaError_t launch_controls_apply(const CtlSide &c, const void *x, int x_dtype, int64_t x_stride_elems, void *out,
                                  int out_dtype, int64_t out_stride_elems, int64_t n_rows, int64_t vocab,
                                  cudaStream_t stream) {
    if (n_rows == 0) return cudaSuccess;
    const bool xb = x_dtype == LPD_BF16, ob = out_dtype == LPD_BF16;
    StreamArgs a{};
    a.c[0] = c;
    a.in[0] = plane(x, x_stride_elems * (xb ? 2 : 4), xb ? 2 : 4, n_rows, vocab);
    a.out = static_cast<char *>(out);
    a.out_stride = out_stride_elems * (ob ? 2 : 4);
    a.n_rows = n_rows;
    a.vocab = vocab;
    a.in_place = x == out ? 1 : 0;
    const bool aligned = aligned_rows(x, a.in[0].stride) && aligned_rows(out, a.out_stride);
    set_units(a, aligned);
    return aligned ? launch_kinds<kApply, true>(a, xb, ob, n_rows, stream) : launch_kinds<kApply, false>(a, xb, ob, n_rows, stream);
}

cudaError_t launch_controls_gradient(const CtlSide &c, const void *x, int x_dtype, int64_t x_stride_elems, void *out,
                                     int out_dtype, int64_t out_stride_elems, int64_t n_rows, int64_t vocab,
                                     const int32_t *ids, const uint8_t *mask, const float *logp, const float *grad,
                                     cudaStream_t stream) {
    if (n_rows == 0) return cudaSuccess;
    const bool xb = x_dtype == LPD_BF16, ob = out_dtype == LPD_BF16;
    StreamArgs a{};
    a.c[0] = c;
    a.in[0] = plane(x, x_stride_elems * (xb ? 2 : 4), xb ? 2 : 4, n_rows, vocab);
    a.out = static_cast<char *>(out);
    a.out_stride = out_stride_elems * (ob ? 2 : 4);
    a.n_rows = n_rows;
    a.vocab = vocab;
    a.ids = ids;
    a.mask = mask;
    a.logp = logp;
    a.grad = grad;
    const bool aligned = aligned_rows(x, a.in[0].stride) && aligned_rows(out, a.out_stride);
    set_units(a, aligned);
    return aligned ? launch_kinds<kGrad, true>(a, xb, ob, n_rows, stream) : launch_kinds<kGrad, false>(a, xb, ob, n_rows, stream);
}

cudaError_t launch_controls_score(const CtlScoreCall &call, cudaStream_t stream) {
    if (call.n_rows == 0) return cudaSuccess;
    const bool tb = call.dtype_t == LPD_BF16, rb = call.dtype_r == LPD_BF16;
    StreamArgs a{};
    a.c[0] = call.t;
    a.c[1] = call.r;
    a.in[0] = plane(call.xt, call.t_stride, tb ? 2 : 4, call.n_rows, call.vocab);
    a.in[1] = plane(call.xr, call.r_stride, rb ? 2 : 4, call.n_rows, call.vocab);
    a.n_rows = call.n_rows;
    a.vocab = call.vocab;
    // rows enough for two a block: whole rows (as far as the bitmaps reach); else a unit a segment
    a.n_segs = score_segments(call.vocab);
    a.width = call.n_rows >= 2 * static_cast<int64_t>(device_sm_count()) ? std::min(a.n_segs * kSegment, kMaxWidth) : kSegment;
    a.n_units = static_cast<int>((call.vocab + a.width - 1) / a.width);
    a.status = call.status;
    a.hdr = call.hdr;
    a.rowid = call.rowid;
    a.part_a = call.part_a;
    a.part_b = call.part_b;
    a.pick = call.pick;
    // one count serves two sides that mark the same tokens
    const CtlSide &t = call.t, &r = call.r;
    a.same = t.counts == r.counts && t.n_bias == r.n_bias && (t.counts || t.n_bias) &&
             (!t.counts || (t.history == r.history && t.n_history == r.n_history && t.hist_begin == r.hist_begin &&
                            t.hist_split == r.hist_split && t.hist_end == r.hist_end)) &&
             (!t.n_bias || t.bias_ids == r.bias_ids);
    const bool aligned = aligned_rows(call.xt, call.t_stride) && aligned_rows(call.xr, call.r_stride);
    const cudaError_t e = aligned ? launch_kinds<kScore, true>(a, tb, rb, call.n_rows, stream)
                                  : launch_kinds<kScore, false>(a, tb, rb, call.n_rows, stream);
    if (e != cudaSuccess) return e;
    score_finalize_kernel<<<static_cast<unsigned>((call.n_rows + 7) / 8), 256, 0, stream>>>(
        a, call.out_lt, call.out_lr, call.out_d, call.dval, call.keys, call.status);
    return cudaGetLastError();
}

}  // namespace lpd
