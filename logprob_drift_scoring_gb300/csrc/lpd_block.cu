// Block-scaled 8-bit floating point: quantisation and the matrix product.
//
// A value of an operand is q * s with q in e4m3 or e5m2 and one fp32 scale s
// for each 1 x 128 or 128 x 128 block along k ("[WS2] Framework for ablation
// experiment", LogProb knobs table, rows 9-10: the head GEMM of the rollout
// engine, whose rounding is a drift source).  The product is
//   C[m, n] = sum_kb sa[m, kb] sb[n, kb] sum_{k in block kb} A[m, k] B[n, k]:
// the inner sum of 128 terms runs on the tensor cores (tcgen05.mma
// kind::f8f6f4, fp32 accumulation in tensor memory), the outer one in fp32
// registers with one multiply-add per output and block, in ascending kb.
#include <algorithm>
#include <cfloat>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <math_constants.h>

#include "lpd_acc.cuh"
#include "lpd_internal.cuh"
#include "lpd_operators.cuh"

namespace lpd {
namespace {

constexpr int kBlk = 128;  // values along k that share one scale

// =============================================================== quantisation
// A block takes a tile of 128 x 128 input values: 16 lanes a row with 8 values
// each, two rows a warp and pass, 16 rows a pass, eight passes, all held in
// registers, so the input is read once and each maximum is known before the
// first value is rounded.  For transposed output a thread takes 8 neighbouring
// rows instead: it then has 8 bytes of each of its 8 output rows, which turn
// through shared memory in 8-byte chunks.  Chunk g of output row c lies at
// g ^ (c / 8 % 16), so that the 16 columns a half-warp stores at once meet all
// banks, and so do the 128 bytes of a row when they are read (bytes stored one
// at a time kept the shared memory 96 % busy: 1085 us for 151936 x 4096).
// Bound: HBM (input bytes + one byte a value): 151936 x 4096 bf16 in 276 us
// transposed and 272 us as it lies with 128 x 128 blocks (6.8 TB/s, the measured
// copy rate), 297 and 285 us with 1 x 128 blocks; 75968 x 4096 f32 in 238 us (6.6
// TB/s).  Rows off 16-byte boundaries are read an element at a time: 263 us for
// 75968 x 4096 bf16 instead of 145.  1024 x 4096 takes 4 us replayed from a graph,
// 11 us called from Python, most of it the host's.
constexpr int kQThreads = 256;
constexpr float kFloor = 5.421010862427522e-20f;  // 2^-64: the smallest magnitude a scale is made for

struct QuantArgs {
    const char *x;
    int64_t x_stride;  // bytes
    int64_t rows, cols;
    uint8_t *out;
    int64_t out_stride;
    float *scales;
    int64_t scale_stride;
    int n_tiles_c;
    int vec_in, vec_out;  // 16-byte aligned input rows, 8-byte (plain) or 16-byte (transposed) aligned output rows
    int pow2;
};

template <bool kE5>
__device__ __forceinline__ uint32_t pack2(float lo, float hi, float inv) {
    return __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(lo, inv), __fmul_rn(hi, inv)), __NV_SATFINITE,
                                    kE5 ? __NV_E5M2 : __NV_E4M3);
}

// scale and the factor onto the 8-bit range from the block's largest magnitude
// (as bits: NaN above infinity above numbers, so neither is lost)
template <bool kE5>
__device__ __forceinline__ void scale_of(uint32_t top_bits, int pow2, float *scale, float *inv) {
    constexpr float kMost = kE5 ? 57344.f : 448.f;
    const float raw = __uint_as_float(top_bits);
    if (!(raw <= FLT_MAX)) {  // a non-finite value: the whole block reads as NaN
        *scale = raw;
        *inv = CUDART_NAN_F;
        return;
    }
    const float top = fmaxf(raw, kFloor);
    const float s = __fdiv_rn(top, kMost);
    if (pow2) {
        const uint32_t b = __float_as_uint(s);
        *scale = __uint_as_float((b + 0x7fffffu) & 0x7f800000u);  // up to the next power of two
        *inv = __fdiv_rn(1.f, *scale);
    } else {
        *scale = s;
        *inv = __fdiv_rn(kMost, top);
    }
}

template <bool kBf16, bool kE5, bool kBlock, bool kTranspose>
__global__ void __launch_bounds__(kQThreads, kBf16 ? 4 : 2) quantize_kernel(const __grid_constant__ QuantArgs a) {
    __shared__ __align__(16) uint32_t tops[kTranspose && !kBlock ? 9 * kBlk : 8];  // (the ninth part: the columns' factors)
    __shared__ __align__(16) uint8_t turned[kTranspose ? kBlk * kBlk : 16];
    constexpr int kElt = kBf16 ? 2 : 4;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int64_t tile_r = blockIdx.x / a.n_tiles_c, tile_c = blockIdx.x % a.n_tiles_c;
    const int64_t r0 = tile_r * kBlk, c0 = tile_c * kBlk;
    const int col = (lane & 15) * 8;
    const int row_group = warp * 2 + (lane >> 4);
    const auto row_of = [&](int p) { return kTranspose ? row_group * 8 + p : p * 16 + row_group; };
    // raw words of the thread's 8 passes: 8 values each, outside the tensor 0
    uint4 raw[8][kBf16 ? 1 : 2];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int64_t r = r0 + row_of(p), c = c0 + col;
        const char *src = a.x + r * a.x_stride + c * kElt;
#pragma unroll
        for (int h = 0; h < (kBf16 ? 1 : 2); ++h) raw[p][h] = make_uint4(0, 0, 0, 0);
        if (r < a.rows && c < a.cols) {
            if (a.vec_in && c + 8 <= a.cols) {
#pragma unroll
                for (int h = 0; h < (kBf16 ? 1 : 2); ++h) raw[p][h] = __ldcs(reinterpret_cast<const uint4 *>(src) + h);
            } else {
                uint32_t w[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const bool in = c + q < a.cols;
                    if constexpr (kBf16) {
                        const uint32_t b = in ? reinterpret_cast<const unsigned short *>(src)[q] : 0u;
                        if (q & 1) w[q >> 1] |= b << 16;
                        else w[q >> 1] = b;
                    } else {
                        w[q] = in ? reinterpret_cast<const uint32_t *>(src)[q] : 0u;
                    }
                }
                raw[p][0] = make_uint4(w[0], w[1], w[2], w[3]);
                if constexpr (!kBf16) raw[p][1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
        }
    }
    auto values = [&](int p, float *v) {
        if constexpr (kBf16) {
            const uint32_t ws[4] = {raw[p][0].x, raw[p][0].y, raw[p][0].z, raw[p][0].w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                v[2 * q] = __uint_as_float(ws[q] << 16);
                v[2 * q + 1] = __uint_as_float(ws[q] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int h = 0; h < (kBf16 ? 1 : 2); ++h) {
                v[4 * h] = __uint_as_float(raw[p][h].x);
                v[4 * h + 1] = __uint_as_float(raw[p][h].y);
                v[4 * h + 2] = __uint_as_float(raw[p][h].z);
                v[4 * h + 3] = __uint_as_float(raw[p][h].w);
            }
        }
    };
    auto bits = [](float x) { return __float_as_uint(x) & 0x7fffffffu; };
    float inv_col[kTranspose && !kBlock ? 8 : 1], inv_all = 0.f;
    if constexpr (kBlock) {
        uint32_t m = 0;
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            float v[8];
            values(p, v);
#pragma unroll
            for (int q = 0; q < 8; ++q) m = max(m, bits(v[q]));
        }
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0) tops[warp] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 8; ++w) m = max(m, tops[w]);
        float s;
        scale_of<kE5>(m, a.pow2, &s, &inv_all);
        if (t == 0) a.scales[kTranspose ? tile_c * a.scale_stride + tile_r : tile_r * a.scale_stride + tile_c] = s;
    } else if constexpr (kTranspose) {
        uint32_t m[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) m[q] = 0;
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            float v[8];
            values(p, v);
#pragma unroll
            for (int q = 0; q < 8; ++q) m[q] = max(m[q], bits(v[q]));
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            m[q] = max(m[q], __shfl_xor_sync(0xffffffffu, m[q], 16));
            if (lane < 16) tops[warp * kBlk + col + q] = m[q];
        }
        __syncthreads();
        if (t < kBlk) {  // a column a thread: two divisions each
            uint32_t top = 0;
#pragma unroll
            for (int w = 0; w < 8; ++w) top = max(top, tops[w * kBlk + t]);
            float s, inv;
            scale_of<kE5>(top, a.pow2, &s, &inv);
            if (c0 + t < a.cols) a.scales[(c0 + t) * a.scale_stride + tile_r] = s;
            tops[8 * kBlk + t] = __float_as_uint(inv);
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < 8; ++q) inv_col[q] = __uint_as_float(tops[8 * kBlk + col + q]);
    } else {
        // The 8 rows' maxima over 16 lanes, halving the rows a lane keeps at
        // each step, so that a lane ends with one row (and its neighbour with
        // the same): 8 exchanges instead of 32, two divisions instead of 16.
        uint32_t m[8];
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            float v[8];
            values(p, v);
            m[p] = 0;
#pragma unroll
            for (int q = 0; q < 8; ++q) m[p] = max(m[p], bits(v[q]));
        }
#pragma unroll
        for (int off = 8, half = 4; off > 1; off >>= 1, half >>= 1) {
            const bool upper = lane & off;
#pragma unroll
            for (int p = 0; p < half; ++p) {
                const uint32_t give = upper ? m[p] : m[p + half], keep = upper ? m[p + half] : m[p];
                m[p] = max(keep, __shfl_xor_sync(0xffffffffu, give, off));
            }
        }
        const uint32_t top = max(m[0], __shfl_xor_sync(0xffffffffu, m[0], 1));
        float s;
        scale_of<kE5>(top, a.pow2, &s, &inv_all);
        const int64_t r = r0 + row_of((lane >> 1) & 7);
        if ((lane & 1) == 0 && r < a.rows) a.scales[r * a.scale_stride + tile_c] = s;
    }
    if constexpr (kTranspose) {
        uint32_t words[2][8];  // rows 0..3 and 4..7 of each column
#pragma unroll
        for (int p = 0; p < 8; p += 2) {
            float v[2][8];
            values(p, v[0]);
            values(p + 1, v[1]);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const uint32_t two = pack2<kE5>(v[0][q], v[1][q], kBlock ? inv_all : inv_col[kBlock ? 0 : q]);
                if (p & 2) words[p >> 2][q] |= two << 16;
                else words[p >> 2][q] = two;
            }
        }
#pragma unroll
        for (int q = 0; q < 8; ++q)
            *reinterpret_cast<uint2 *>(&turned[(col + q) * kBlk + ((row_group ^ (col >> 3)) << 3)]) = make_uint2(words[0][q], words[1][q]);
        __syncthreads();
        // 128 output rows (input columns) of 128 bytes: 8 lanes a row with 16 bytes each
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const int row = p * 32 + (t >> 3), at = t & 7, key = row >> 3;
            const int64_t orow = c0 + row, oc = r0 + at * 16;
            if (orow >= a.cols || oc >= a.rows) continue;
            uint4 w = *reinterpret_cast<const uint4 *>(&turned[row * kBlk + ((at ^ (key >> 1)) << 4)]);
            if (key & 1) w = make_uint4(w.z, w.w, w.x, w.y);
            uint8_t *dst = a.out + orow * a.out_stride + oc;
            if (a.vec_out && oc + 16 <= a.rows) {
                __stcs(reinterpret_cast<uint4 *>(dst), w);
            } else {
                const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
                for (int q = 0; q < 16 && oc + q < a.rows; ++q)
                    dst[q] = static_cast<uint8_t>(ws[q >> 2] >> (8 * (q & 3)));
            }
        }
    } else {
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            const int64_t r = r0 + row_of(p), c = c0 + col;
            float v[8];
            values(p, v);
            const float inv = kBlock ? inv_all : __shfl_sync(0xffffffffu, inv_all, (lane & 16) | 2 * p);
            if (r >= a.rows || c >= a.cols) continue;
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) w[q] = pack2<kE5>(v[2 * q], v[2 * q + 1], inv);
            uint8_t *dst = a.out + r * a.out_stride + c;
            if (a.vec_out && c + 8 <= a.cols) {
                __stcs(reinterpret_cast<uint2 *>(dst), make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16));
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (c + q < a.cols) dst[q] = static_cast<uint8_t>(w[q >> 1] >> (8 * (q & 1)));
            }
        }
    }
}

// ==================================================================== product
// One persistent CTA per SM.  Warpgroup 0: warp 0 streams 128-wide k blocks of A
// (128 rows) and B (256 rows) through a three-stage ring (TMA, 128-byte
// swizzle), warp 1 issues four M=128 N=256 K=32 MMAs a block into one of two
// accumulators in tensor memory, and warps 2 and 3 copy the scales of four
// blocks at a time into shared memory, one group ahead.  Warpgroups 1 and 2, the
// read-back, take each accumulator, scale it and add it to 128 fp32 registers a
// thread, a warp 32 rows and half of the 256 columns; two accumulators let the
// MMAs of block kb + 1 run under the read-back of block kb.  It reads 16 rows at
// a time, a lane four rows and every fourth pair of columns, so that a lane
// needs 4 + 32 scales a block (one row a lane needs 1 + 128: with 1 x 128 scales
// on both sides, 1024 cycles of shared-memory returns a block, and a weight
// gradient took 651 us instead of 473).
//
// Bound: tensor cores by the operations, 512 cycles a block; the read-back by
// measurement.  4096 x 128256 x 4096 takes 2.1 ms (2.0 PFLOP/s; 2.5 us a tile and
// 0.55 us a block); with the multiply-adds left out 1.53 ms, with the copies left
// out as well 1.30 ms.  128 multiply-adds a lane and block take 256 cycles of a
// sub-partition's 512, and each piece's read of tensor memory stands before them
// (tcgen05.wait::ld waits for all reads, so only one piece can be on its way).
// Tried and slower: sixteen warps of 64 registers (2.2 to 2.4 ms), pieces of half
// the size (2.2 ms), the next block's first piece under this one's last
// (4.2 ms: its registers spill), packed multiply-adds (a move each after a read
// of tensor memory), calling B into L2 ahead (no change; few rows 5 to 30 %
// slower).  A product of few rows (16 x 151936 x 4096: 136 us, 4.6 TB/s) waits
// for its 128-byte pieces of B's rows from HBM.  Output rows off 16-byte boundaries
// leave by stores of single elements: 4096 x 50257 x 4096 in 956 us dense, 822 us
// with a row stride of 50264.  A data gradient of split k (64 x 4096 x 151936: 115
// us, 93 of them HBM; 512 x 4096 x 151936: 348 us) is joined by a second kernel.
constexpr int kTM = 128, kTN = 256;
constexpr int kStages = 3;
constexpr int kABytes = kTM * kBlk, kBBytes = kTN * kBlk;
constexpr int kStageBytes = kABytes + kBBytes;  // 48 KB
constexpr int kEpiWarps = 8;
constexpr int kEpiCols = kTN / (kEpiWarps / 4);  // columns a warp
constexpr int kMmThreads = (4 + kEpiWarps) * 32;  // a warpgroup for the copies and the MMAs, two for the read-back
// registers a thread after the split (three warps a sub-partition, launched at
// 168 each: 40 + 2 * 232 = 3 * 168)
constexpr int kRegsFront = 40, kRegsEpi = 232;
// Output staging, a warp's: two boxes of 32 rows x 128 bytes.  They leave by TMA
// stores, which run under the next tile (stores by the warps themselves took
// 4200 cycles a tile); output rows that are not
// 16-byte aligned go through rows of kOutPitch bytes instead.
constexpr int kBoxBytes = 32 * 128;
constexpr int kOutPitch = 80;                   // 64 bytes a row and 16 against bank conflicts
constexpr int kOutWarp = 2 * kBoxBytes;
constexpr int kOutBytes = kEpiWarps * kOutWarp;
static_assert(32 * kOutPitch <= kOutWarp, "staging of either kind");
constexpr int kScaleGroup = 4;                  // k blocks whose scales are fetched together
constexpr int kScaleThreads = 64;
constexpr int kScaleFloats = kScaleGroup * (kTN + kTM);  // of a group: the columns', then the rows'
constexpr int kScaleBytes = 2 * kScaleFloats * 4;
constexpr size_t kMmSmem = 1024 + static_cast<size_t>(kStages) * kStageBytes + kOutBytes + kScaleBytes;
constexpr uint32_t kTmemCols = 512;
constexpr int kRaster = 16;                     // row tiles that share a B tile in L2
constexpr unsigned long long kWaitLimitNs = 4000000000ull;
constexpr uint32_t kWaitLimitIters = 1u << 30;

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
// Bounded wait of a whole warp, the same answer in every lane (so that no lane
// goes its own way); when it gives up it raises the CTA's abort flag and sets
// LPD_STATUS_TIMEOUT in the workspace's first word.  The clock is read only
// once a wait has been polled for long: a read costs more than a block's MMAs.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, volatile int *abort_flag, uint32_t *status,
                                          bool honour_abort = true) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    unsigned long long t0 = 0;
#pragma unroll 1
    for (uint32_t n = 1; n < kWaitLimitIters; ++n) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        if ((n & 255u) == 0) {
            const unsigned long long now = globaltimer_ns();
            if (t0 == 0) t0 = now;
            if (__any_sync(0xffffffffu, (honour_abort && *abort_flag) || now - t0 > kWaitLimitNs)) break;
        }
    }
    if ((threadIdx.x & 31) == 0) {
        *abort_flag = 1;
        atomicOr(status, LPD_STATUS_TIMEOUT);
    }
    return false;
}
__device__ __forceinline__ void copy_async_4(float *dst, const float *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void tma_load_2d(void *dst, const CUtensorMap *map, int x, int y, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}
// Descriptor of a K-major tile of 128-byte rows under the 128-byte swizzle
// (8-row groups of 1024 bytes): the lower word is the address / 16 (and the
// unused leading offset), the upper word is the same for every tile.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(const void *tile) { return ((smem_u32(tile) & 0x3FFFFu) >> 4) | (1u << 16); }
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint32_t a_low, uint32_t b_low, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, %5};\n\t"
        "mov.b64 db, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_low), "r"(b_low), "r"(idesc), "r"(accumulate), "r"(kDescHigh)
        : "memory");
}
// One lane of a warp, the same each time.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void umma_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// 16 lanes x 32 columns: registers 4 i + j hold row lane / 4 + 8 (j / 2), column 8 i + 2 (lane % 4) + j % 2.
__device__ __forceinline__ void tmem_ld_issue(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_issue(uint32_t taddr, uint32_t (&r)[32]) {  // the same, 64 columns
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, const void *src, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x),
                 "r"(y), "r"(z), "r"(smem_u32(src))
                 : "memory");
}
__device__ __forceinline__ void tma_store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// Until the stores so far have read their shared memory.
__device__ __forceinline__ void tma_store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
struct MmMaps {
    CUtensorMap a, b;
    CUtensorMap out;  // (column, row, split); only where vec_out
};

struct MmArgs {
    const float *sa, *sb;
    int64_t sa_stride, sb_stride;
    int sa_shift, sb_shift;    // 0: a scale a row, 7: a scale for 128 rows
    int64_t m, n;
    int kb_total, kb_per_split, n_splits;
    int n_tm, n_tn;
    uint32_t idesc;
    char *out;
    int64_t out_stride;        // bytes
    int64_t split_stride;      // bytes between the partial results of two splits
    int vec_out;               // 16-byte aligned output rows
    int whole_out;             // ... of whole 16-byte pieces
    uint32_t *status;
};

// Work items in raster order: groups of kRaster row tiles over all column
// tiles, row tiles innermost, then the splits.
__device__ __forceinline__ void item_coords(int64_t w, const MmArgs &a, int &tm, int &tn, int &split) {
    const int64_t tiles = static_cast<int64_t>(a.n_tm) * a.n_tn;
    split = static_cast<int>(w / tiles);
    const int64_t i = w - split * tiles;
    const int64_t per_group = static_cast<int64_t>(kRaster) * a.n_tn;
    const int g = static_cast<int>(i / per_group);
    const int64_t local = i - g * per_group;
    const int gm = min(kRaster, a.n_tm - g * kRaster);
    tn = static_cast<int>(local / gm);
    tm = g * kRaster + static_cast<int>(local - static_cast<int64_t>(tn) * gm);
}

// kVecB: B's scales are one a row (1 x 128 blocks), so they differ from column
// to column of the accumulator; else one for 128 columns.
template <bool kOutF32, bool kVecB>
__global__ void __launch_bounds__(kMmThreads, 1)
    product_kernel(const __grid_constant__ MmMaps maps, const __grid_constant__ MmArgs a) {
    extern __shared__ __align__(1024) char smem_raw[];
    __shared__ uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], scales_full[2], scales_empty[2], done;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    char *const smem = smem_raw + (-smem_u32(smem_raw) & 1023u);  // (an offset keeps the loads shared ones)
    char *const staged = smem + static_cast<size_t>(kStages) * kStageBytes;
    float *const scales = reinterpret_cast<float *>(staged + kOutBytes);  // [2][kScaleFloats]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t items = static_cast<int64_t>(a.n_tm) * a.n_tn * a.n_splits;

    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], kEpiWarps);
            mbar_init(&scales_full[b], kScaleThreads);
            mbar_init(&scales_empty[b], kEpiWarps);
        }
        mbar_init(&done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFront));
        // Both loops are run by whole warps, so that the compiler sees uniform
        // values (a lone thread's loop spent 855 cycles a block on issuing four
        // MMAs, most of them on moves to uniform registers); one lane issues.
        const bool leader = elect_one();
        if (warp == 0) {
            // ------------------------------------------------------------ producer
            uint32_t s = 0, phase = 1, issued = 0;  // the first turn finds every stage empty
            bool ok = true;
            for (int64_t w = blockIdx.x; ok && w < items; w += gridDim.x) {
                int tm, tn, split;
                item_coords(w, a, tm, tn, split);
                const int kb1 = min(a.kb_total, (split + 1) * a.kb_per_split);
#pragma unroll 1
                for (int kb = split * a.kb_per_split; kb < kb1; ++kb) {
                    ok = wait_warp(&empty[s], phase, &abort_flag, a.status);
                    if (!ok) break;
                    if (leader) {
                        char *st = smem + s * kStageBytes;
                        mbar_arrive_expect_tx(&full[s], kStageBytes);
                        tma_load_2d(st, &maps.a, kb * kBlk, tm * kTM, &full[s]);
                        tma_load_2d(st + kABytes, &maps.b, kb * kBlk, tn * kTN, &full[s]);
                    }
                    issued = issued < kStages ? issued + 1 : kStages;
                    if (++s == kStages) {
                        s = 0;
                        phase ^= 1;
                    }
                }
            }
            // every copy issued must land before the CTA exits: the last turn's
            // stages, each in the phase of its last use
            for (uint32_t j = 0; j < issued; ++j) {
                if (s == 0) {
                    s = kStages;
                    phase ^= 1;
                }
                --s;
                wait_warp(&full[s], phase ^ 1, &abort_flag, a.status, false);
            }
        } else if (warp == 1) {
            // ----------------------------------------------------------------- MMA
            uint32_t s = 0, phase = 0, b = 0, turn = 1;  // `turn`: the parity that an emptied accumulator shows
            bool ok = true, issued = false;
            const uint32_t base = desc_low(smem);
            for (int64_t w = blockIdx.x; ok && w < items; w += gridDim.x) {
                int tm, tn, split;
                item_coords(w, a, tm, tn, split);
                const int kbs = min(a.kb_total, (split + 1) * a.kb_per_split) - split * a.kb_per_split;
#pragma unroll 1
                for (int kb = 0; kb < kbs; ++kb) {
                    ok = wait_warp(&acc_empty[b], turn, &abort_flag, a.status) && wait_warp(&full[s], phase, &abort_flag, a.status);
                    if (!ok) break;
                    tc_fence_after();
                    if (leader) {
                        const uint32_t da = base + s * (kStageBytes >> 4), db = da + (kABytes >> 4);
#pragma unroll
                        for (int k = 0; k < kBlk / 32; ++k)  // K = 32 bytes inside the swizzle row
                            umma_f8(tmem + b * kTN, da + 2 * k, db + 2 * k, a.idesc, k > 0 ? 1u : 0u);
                        umma_commit(&empty[s]);
                        umma_commit(&acc_full[b]);
                    }
                    issued = true;
                    if (++s == kStages) {
                        s = 0;
                        phase ^= 1;
                    }
                    b ^= 1;
                    turn ^= b ^ 1;
                }
            }
            if (issued) {
                if (leader) umma_commit(&done);
                wait_warp(&done, 0, &abort_flag, a.status, false);
            }
            __syncwarp();
        } else {
            // -------------------------------------------------------------- scales
            // of four blocks at a time, the 256 columns' and the 128 rows', one
            // group ahead of the read-back (a scale for 128 of them is copied
            // 128 times: the read-back then knows one layout)
            const int u = threadIdx.x - 64;
            uint32_t group = 0;
            bool ok = true;
            for (int64_t w = blockIdx.x; ok && w < items; w += gridDim.x) {
                int tm, tn, split;
                item_coords(w, a, tm, tn, split);
                const int kb0 = split * a.kb_per_split, kb1 = min(a.kb_total, kb0 + a.kb_per_split);
#pragma unroll 1
                for (int kg = kb0; kg < kb1; kg += kScaleGroup, ++group) {
                    ok = wait_warp(&scales_empty[group & 1], ((group >> 1) & 1) ^ 1, &abort_flag, a.status);
                    if (!ok) break;
                    float *const dst = scales + (group & 1) * kScaleFloats;
#pragma unroll 1
                    for (int i = u; i < kTN; i += kScaleThreads) {
                        const float *src = a.sb + (min(static_cast<int64_t>(tn) * kTN + i, a.n - 1) >> a.sb_shift) * a.sb_stride;
#pragma unroll
                        for (int q = 0; q < kScaleGroup; ++q) copy_async_4(dst + q * kTN + i, src + min(kg + q, kb1 - 1));
                    }
#pragma unroll 1
                    for (int i = u; i < kTM; i += kScaleThreads) {
                        const float *src = a.sa + (min(static_cast<int64_t>(tm) * kTM + i, a.m - 1) >> a.sa_shift) * a.sa_stride;
#pragma unroll
                        for (int q = 0; q < kScaleGroup; ++q) copy_async_4(dst + kScaleGroup * kTN + q * kTM + i, src + min(kg + q, kb1 - 1));
                    }
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&scales_full[group & 1])) : "memory");
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpi));
        // ------------------------------------------------------------ epilogue
        const int quad = warp & 3, part = (warp - 4) >> 2;
        const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + part * kEpiCols;
        char *const mine = staged + (warp - 4) * kOutWarp;
        uint32_t it = 0, group = 0;  // k blocks and scale groups so far
        bool ok = true;
        for (int64_t w = blockIdx.x; w < items; w += gridDim.x) {
            int tm, tn, split;
            item_coords(w, a, tm, tn, split);
            const int kb0 = split * a.kb_per_split, kb1 = min(a.kb_total, kb0 + a.kb_per_split);
            const int64_t col0 = static_cast<int64_t>(tn) * kTN + part * kEpiCols;
            // A block's accumulator comes in pieces of 16 rows, each read under
            // the arithmetic of the one before it: their registers, number and
            // 8-column groups (columns of one scale each leave the registers
            // for half as many)
            constexpr int kPiece = kVecB ? 16 : 32, kPieces = kEpiCols / kPiece, kGroups = kPiece / 4;
            // the pair of columns that a lane has of 8-column group g8 and row 16 h + 8 half + lane / 4
            const auto pair_of = [](int g8, int h, int half) { return (((g8 / kGroups) * 2 + h) * kGroups + g8 % kGroups) * 4 + half * 2; };
            float acc[kEpiCols];
#pragma unroll
            for (int j = 0; j < kEpiCols; ++j) acc[j] = 0.f;
#pragma unroll 1
            for (int kg = kb0; ok && kg < kb1; kg += kScaleGroup, ++group) {
                const float *const group_scales = scales + (group & 1) * kScaleFloats;
                ok = wait_warp(&scales_full[group & 1], (group >> 1) & 1, &abort_flag, a.status);
                if (!ok) break;
                const float *const of_row = group_scales + kScaleGroup * kTN + quad * 32 + (lane >> 2);
                const float *const of_col = group_scales + part * kEpiCols + (kVecB ? (lane & 3) * 2 : 0);
#pragma unroll
                for (int g = 0; g < kScaleGroup; ++g) {
                    if (kg + g >= kb1) break;
                    const uint32_t b = it & 1;
                    ok = wait_warp(&acc_full[b], (it >> 1) & 1, &abort_flag, a.status);
                    if (!ok) break;
                    ++it;
                    tc_fence_after();
                    uint32_t r[2][kPiece];
                    const auto issue = [&](int c) {
                        tmem_ld_issue(lane_addr + b * kTN + (c >> 1) * (8 * kGroups) + ((c & 1) << 20), r[c & 1]);
                    };
                    issue(0);
                    float by_row[4];  // times the columns', where those share one
                    float2 by_col[kGroups];
#pragma unroll
                    for (int i = 0; i < 4; ++i) by_row[i] = kVecB ? of_row[g * kTM + i * 8] : __fmul_rn(of_row[g * kTM + i * 8], of_col[g * kTN]);
#pragma unroll
                    for (int c = 0; c < kPieces; ++c) {
                        if (kVecB && (c & 1) == 0) {
#pragma unroll
                            for (int i = 0; i < kGroups; ++i)
                                by_col[i] = *reinterpret_cast<const float2 *>(&of_col[g * kTN + (c / 2 * kGroups + i) * 8]);
                        }
                        tmem_wait_ld();
                        if (c + 1 < kPieces) {
                            issue(c + 1);
                        } else {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&acc_empty[b]);
                        }
#pragma unroll
                        for (int j = 0; j < kPiece; ++j) {
                            float by = by_row[(c & 1) * 2 + ((j >> 1) & 1)];
                            if (kVecB) by = __fmul_rn(by, (j & 1) ? by_col[j >> 2].y : by_col[j >> 2].x);
                            float &x = acc[c * kPiece + j];
                            x = __fmaf_rn(__uint_as_float(r[c & 1][j]), by, x);
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&scales_empty[group & 1]);
            }
            if (!ok) {  // a wait gave up: this tile reads as NaN
#pragma unroll
                for (int j = 0; j < kEpiCols; ++j) acc[j] = CUDART_NAN_F;
            }
            char *const out = a.out + split * a.split_stride;
            const int64_t row0 = static_cast<int64_t>(tm) * kTM + quad * 32;
            // (a TMA store writes whole 16-byte pieces: columns behind an n
            // between two of them are not the product's to write)
            if (a.vec_out && (a.whole_out || col0 + kEpiCols <= a.n)) {
                // boxes of 32 rows x 128 bytes under the 128-byte swizzle: chunk
                // q of row l lies at q ^ (l % 8), so a warp's stores hit all banks
                constexpr int kBoxCols = kOutF32 ? 32 : 64;
#pragma unroll
                for (int box = 0; box < kEpiCols / kBoxCols; ++box) {
                    if (box % 2 == 0) {  // both boxes' last stores have read them
                        if (lane == 0) tma_store_wait_read();
                        __syncwarp();
                    }
                    char *const dst = mine + (box & 1) * kBoxBytes;
#pragma unroll
                    for (int q = 0; q < kBoxCols / 8; ++q)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            char *to = dst + (e * 8 + (lane >> 2)) * 128;
                            const float *v = &acc[pair_of(box * (kBoxCols / 8) + q, e >> 1, e & 1)];
                            if (kOutF32) *reinterpret_cast<float2 *>(to + (((q * 2 + ((lane >> 1) & 1)) ^ (lane >> 2)) << 4) + (lane & 1) * 8) = make_float2(v[0], v[1]);
                            else *reinterpret_cast<__nv_bfloat162 *>(to + ((q ^ (lane >> 2)) << 4) + (lane & 3) * 4) = __floats2bfloat162_rn(v[0], v[1]);
                        }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    const int64_t c = col0 + box * kBoxCols;
                    if (lane == 0) {
                        if (c < a.n && row0 < a.m)
                            tma_store_3d(&maps.out, dst, static_cast<int>(c), static_cast<int>(row0), split);
                        tma_store_commit();
                    }
                }
                continue;
            }
            // 64-byte pieces of 32 rows through shared memory
            if (lane == 0) tma_store_wait_read();  // the last tile's boxes lay there
            constexpr int kCols = kOutF32 ? 16 : 32;  // columns of a piece
#pragma unroll
            for (int p = 0; p < kEpiCols / kCols; ++p) {
                __syncwarp();
#pragma unroll
                for (int q = 0; q < kCols / 8; ++q)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        char *to = mine + (e * 8 + (lane >> 2)) * kOutPitch;
                        const float *v = &acc[pair_of(p * (kCols / 8) + q, e >> 1, e & 1)];
                        if (kOutF32) *reinterpret_cast<float2 *>(to + q * 32 + (lane & 3) * 8) = make_float2(v[0], v[1]);
                        else *reinterpret_cast<__nv_bfloat162 *>(to + q * 16 + (lane & 3) * 4) = __floats2bfloat162_rn(v[0], v[1]);
                    }
                __syncwarp();
                const int64_t c = col0 + p * kCols;
                if (c >= a.n) break;
                {
                    constexpr int kRowsAtOnce = 32 / kCols;
                    for (int q = 0; q < 32 / kRowsAtOnce; ++q) {
                        const int rr = q * kRowsAtOnce + lane / kCols, cc = lane % kCols;
                        if (row0 + rr < a.m && c + cc < a.n) {
                            char *dst = out + (row0 + rr) * a.out_stride + (c + cc) * (kOutF32 ? 4 : 2);
                            if (kOutF32) *reinterpret_cast<uint32_t *>(dst) = *reinterpret_cast<const uint32_t *>(mine + rr * kOutPitch + 4 * cc);
                            else *reinterpret_cast<unsigned short *>(dst) = *reinterpret_cast<const unsigned short *>(mine + rr * kOutPitch + 2 * cc);
                        }
                    }
                }
            }
        }
    }

    if (warp >= 4 && lane == 0) tma_store_wait_read();  // shared memory outlives the last stores' reads
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

// C = the partial results added in split order, rounded once.
template <bool kOutF32>
__global__ void __launch_bounds__(256) join_kernel(const float *part, int64_t part_stride, int64_t split_stride,
                                                   int n_splits, int64_t m, int64_t n, char *out, int64_t out_stride) {
    const int64_t cells = m * n;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < cells; i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t r = i / n, c = i - r * n;
        const float *p = part + r * part_stride + c;
        float s = p[0];
        for (int k = 1; k < n_splits; ++k) s = __fadd_rn(s, p[k * split_stride]);
        if (kOutF32) *reinterpret_cast<float *>(out + r * out_stride + 4 * c) = s;
        else *reinterpret_cast<__nv_bfloat16 *>(out + r * out_stride + 2 * c) = __float2bfloat16_rn(s);
    }
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static std::atomic<EncodeTiledFn> cached{nullptr};
    EncodeTiledFn fn = cached.load(std::memory_order_acquire);
    if (!fn) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        fn = reinterpret_cast<EncodeTiledFn>(p);
        cached.store(fn, std::memory_order_release);
    }
    return fn;
}

// [rows, k] bytes, boxes of 128 x box_rows, 128-byte swizzle; what lies
// outside [rows, k] reads as 0.
bool make_map(CUtensorMap *map, const void *ptr, int64_t rows, int64_t k, int64_t stride, int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(rows)};
    // (a single row's stride may be any: it is not used)
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(rows > 1 ? stride : (k + 15) / 16 * 16)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(kBlk), static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t elem[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(ptr), dims, strides, box, elem,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The output (or its partial results) [splits, m, n] in boxes of 32 rows x 128
// bytes, 128-byte swizzle.
bool make_out_map(CUtensorMap *map, void *ptr, int64_t m, int64_t n, int64_t splits, int64_t row_bytes,
                  int64_t split_bytes, bool f32) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(n), static_cast<cuuint64_t>(m), static_cast<cuuint64_t>(splits)};
    if (m == 1) row_bytes = (n * (f32 ? 4 : 2) + 15) / 16 * 16;  // neither stride is used where there is one row, one split
    if (splits == 1) split_bytes = row_bytes;
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(split_bytes)};
    const cuuint32_t box[3] = {f32 ? 32u : 64u, 32u, 1u};
    const cuuint32_t elem[3] = {1, 1, 1};
    return fn(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, ptr, dims, strides, box,
              elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kBf16, bool kE5>
cudaError_t quantize_typed(const QuantArgs &a, bool block, bool transpose, unsigned grid, cudaStream_t s) {
    if (block) {
        if (transpose) quantize_kernel<kBf16, kE5, true, true><<<grid, kQThreads, 0, s>>>(a);
        else quantize_kernel<kBf16, kE5, true, false><<<grid, kQThreads, 0, s>>>(a);
    } else {
        if (transpose) quantize_kernel<kBf16, kE5, false, true><<<grid, kQThreads, 0, s>>>(a);
        else quantize_kernel<kBf16, kE5, false, false><<<grid, kQThreads, 0, s>>>(a);
    }
    return cudaGetLastError();
}

template <bool kOutF32, bool kVecB>
cudaError_t product_typed(const MmMaps &maps, const MmArgs &a, cudaStream_t stream) {
    static std::atomic<uint64_t> configured{0};
    const cudaError_t e = set_smem_once(product_kernel<kOutF32, kVecB>, kMmSmem, configured);
    if (e != cudaSuccess) return e;
    const int64_t items = static_cast<int64_t>(a.n_tm) * a.n_tn * a.n_splits, sms = device_sm_count();
    product_kernel<kOutF32, kVecB><<<static_cast<unsigned>(items < sms ? items : sms), kMmThreads, kMmSmem, stream>>>(maps, a);
    return cudaGetLastError();
}

}  // namespace

// The k axis is split where the output's tiles would leave half of the
// multiprocessors idle (a data gradient of few tokens: 16 tiles and a thousand
// k blocks), into parts of at least eight blocks.
BlockPlan block_plan(int64_t m, int64_t n, int64_t k) {
    BlockPlan p{};
    p.n_tm = (m + kTM - 1) / kTM;
    p.n_tn = (n + kTN - 1) / kTN;
    p.kb_total = (k + kBlk - 1) / kBlk;
    const int64_t tiles = p.n_tm * p.n_tn;
    const int64_t sms = device_sm_count();
    int64_t want = tiles > 0 ? sms / tiles : 1;
    want = std::min(want, p.kb_total / 8);
    p.n_splits = std::max<int64_t>(want, 1);
    p.kb_per_split = p.n_splits > 1 ? (p.kb_total + p.n_splits - 1) / p.n_splits : p.kb_total;
    if (p.n_splits > 1) p.n_splits = (p.kb_total + p.kb_per_split - 1) / p.kb_per_split;
    p.part_stride = (n + 3) / 4 * 4;
    p.bytes = 256;
    if (p.n_splits > 1) p.bytes += align256(static_cast<size_t>(p.n_splits) * m * p.part_stride * 4);
    return p;
}

cudaError_t launch_block_quantize(const void *x, int x_dtype, int64_t x_stride_elems, int64_t rows, int64_t cols,
                                  bool block, bool transpose, bool pow2, bool e5m2, void *out, int64_t out_stride,
                                  float *scales, int64_t scale_stride, cudaStream_t stream) {
    if (rows == 0 || cols == 0) return cudaSuccess;
    QuantArgs a{};
    const bool bf16 = x_dtype == LPD_BF16;
    a.x = static_cast<const char *>(x);
    a.x_stride = x_stride_elems * (bf16 ? 2 : 4);
    a.rows = rows;
    a.cols = cols;
    a.out = static_cast<uint8_t *>(out);
    a.out_stride = out_stride;
    a.scales = scales;
    a.scale_stride = scale_stride;
    a.n_tiles_c = static_cast<int>((cols + kBlk - 1) / kBlk);
    const uintptr_t unit = transpose ? 16 : 8;
    a.vec_in = reinterpret_cast<uintptr_t>(x) % 16 == 0 && a.x_stride % 16 == 0;
    a.vec_out = reinterpret_cast<uintptr_t>(out) % unit == 0 && static_cast<uintptr_t>(out_stride) % unit == 0;
    a.pow2 = pow2 ? 1 : 0;
    const unsigned grid = static_cast<unsigned>((rows + kBlk - 1) / kBlk * a.n_tiles_c);
    if (bf16) return e5m2 ? quantize_typed<true, true>(a, block, transpose, grid, stream)
                          : quantize_typed<true, false>(a, block, transpose, grid, stream);
    return e5m2 ? quantize_typed<false, true>(a, block, transpose, grid, stream)
                : quantize_typed<false, false>(a, block, transpose, grid, stream);
}

cudaError_t launch_block_matmul(const BlockOperand &x, const BlockOperand &y, int64_t m, int64_t n, int64_t k,
                                void *out, int out_dtype, int64_t out_stride_elems, void *workspace,
                                cudaStream_t stream) {
    const bool f32 = out_dtype == LPD_F32;
    const int64_t out_stride = out_stride_elems * (f32 ? 4 : 2);
    if (m == 0 || n == 0) return cudaSuccess;
    if (k == 0) return cudaMemset2DAsync(out, out_stride, 0, n * (f32 ? 4 : 2), m, stream);
    const BlockPlan p = block_plan(m, n, k);
    MmMaps maps;
    if (!make_map(&maps.a, x.ptr, m, k, x.row_stride, kTM) || !make_map(&maps.b, y.ptr, n, k, y.row_stride, kTN))
        return cudaErrorInvalidValue;
    MmArgs a{};
    a.sa = x.scales;
    a.sb = y.scales;
    a.sa_stride = x.scale_stride;
    a.sb_stride = y.scale_stride;
    a.sa_shift = x.block ? 7 : 0;
    a.sb_shift = y.block ? 7 : 0;
    a.m = m;
    a.n = n;
    a.kb_total = static_cast<int>(p.kb_total);
    a.kb_per_split = static_cast<int>(p.kb_per_split);
    a.n_splits = static_cast<int>(p.n_splits);
    a.n_tm = static_cast<int>(p.n_tm);
    a.n_tn = static_cast<int>(p.n_tn);
    // kind::f8f6f4: fp32 accumulator (bit 4), A's and B's format (bits 7 and 10: 0 e4m3, 1 e5m2), both K-major
    a.idesc = (1u << 4) | (static_cast<uint32_t>(x.e5m2) << 7) | (static_cast<uint32_t>(y.e5m2) << 10) |
              (static_cast<uint32_t>(kTN >> 3) << 17) | (static_cast<uint32_t>(kTM >> 4) << 24);
    a.status = static_cast<uint32_t *>(workspace);
    float *part = reinterpret_cast<float *>(static_cast<char *>(workspace) + 256);
    const bool split = p.n_splits > 1;
    a.out = split ? reinterpret_cast<char *>(part) : static_cast<char *>(out);
    a.out_stride = split ? p.part_stride * 4 : out_stride;
    a.split_stride = split ? m * p.part_stride * 4 : 0;
    a.vec_out = reinterpret_cast<uintptr_t>(a.out) % 16 == 0 && a.out_stride % 16 == 0;
    const bool to_f32 = split || f32;
    // (partial results have room up to their row stride)
    const int64_t n_written = split ? p.part_stride : n;
    a.whole_out = n_written % (to_f32 ? 4 : 8) == 0;
    if (a.vec_out && !make_out_map(&maps.out, a.out, m, n_written, p.n_splits, a.out_stride, a.split_stride, to_f32))
        return cudaErrorInvalidValue;
    cudaError_t e;
    if (to_f32) e = y.block ? product_typed<true, false>(maps, a, stream) : product_typed<true, true>(maps, a, stream);
    else e = y.block ? product_typed<false, false>(maps, a, stream) : product_typed<false, true>(maps, a, stream);
    if (e != cudaSuccess || !split) return e;
    const int64_t blocks = std::min<int64_t>((m * n + 255) / 256, static_cast<int64_t>(device_sm_count()) * 16);
    if (f32)
        join_kernel<true><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(part, p.part_stride, m * p.part_stride, a.n_splits, m, n,
                                                                          static_cast<char *>(out), out_stride);
    else
        join_kernel<false><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(part, p.part_stride, m * p.part_stride, a.n_splits, m, n,
                                                                           static_cast<char *>(out), out_stride);
    return cudaGetLastError();
}

}  // namespace lpd
