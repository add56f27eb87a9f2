// Microscaled 4-bit floating point: quantisation and the matrix product.
//
// A value of an operand is q * s * t with q in e2m1 (0, 1/2, 1, 3/2, 2, 3, 4, 6 and
// their negatives), one scale s for 16 (e4m3) or 32 (a power of two) values along k
// and one float t for the operand: a rollout engine's 4-bit head ("[WS2] Framework
// for ablation experiment", LogProb knobs table, rows 9-10: the head GEMM and its
// rounding as a drift source).  The tensor cores take the block scales themselves
// (tcgen05.mma kind::mxf4nvf4 and kind::mxf4, block_scale), so a product is a plain
// chain of MMAs over k into one accumulator; the two t enter once at the end.
#include <algorithm>
#include <cfloat>
#include <type_traits>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>
#include <math_constants.h>

#include "lpd_internal.cuh"
#include "lpd_operators.cuh"
#include "lpd_tc.cuh"

namespace lpd {
namespace {

constexpr int kAtom = 512;  // bytes of scales of 128 rows x 4 blocks: (row % 32) * 16 + (row / 32 % 4) * 4 + block % 4

// =============================================================== quantisation
// A block takes a tile of 128 x 128 input values: 16 lanes a row with 8 values
// each, two rows a warp and pass, eight passes, all held in registers, so the
// input is read once.  A scale's values lie in two (16) or four (32) neighbouring
// lanes.  For transposed output a thread takes 8 neighbouring rows: it then has
// four bytes of codes of each of its 8 output rows, which turn through shared
// memory (word g of output row c lies at g ^ (c / 8 % 16)).  The tile's scales are
// gathered in shared memory in their final order and leave as one piece.
//
// Bound: 151936 x 4096 bf16 with the values that the codes stand for take 501 us as they
// lie (0.84 of the copy rate; 68 % of the issue slots and 62 % of HBM's cycles in use) and
// 547 transposed, whose words turn through shared memory; float32, 75968 x 4096, 408 us
// (0.96).  A tile kept in registers and not in shared memory spares a write and a read of
// it; rows off 16-byte boundaries pass through shared memory all the same, since a warp
// then reads and writes 32 neighbours at once (12661 x 2051 float32: 63 us, 8 values a
// lane 71).
constexpr int kQTile = 128;
constexpr int kQThreads = 256;
constexpr float kFloor = 5.421010862427522e-20f;  // 2^-64: the smallest magnitude a power-of-two scale is made for

struct QuantArgs {
    const char *x;
    int64_t x_stride;  // bytes
    int64_t rows, cols;
    uint8_t *out;
    int64_t out_stride;
    uint8_t *scales;
    int64_t atoms;     // of scales along the output's k
    const float *tensor_scale;
    char *values;      // null: not wanted
    int64_t values_stride;
    int values_f32;
    int n_tiles_c;
    int vec_out;
};

// What a scale byte means under t: the factor onto the codes' range, and what a code's
// unit is worth before t.
template <bool kB16>
__device__ __forceinline__ float2 meaning_of(uint32_t byte, float t) {
    const float unit = kB16 ? __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte), __NV_E4M3)))
                            : __uint_as_float(byte << 23);
    const float back = __fdiv_rn(1.f, __fmul_rn(unit, t));
    return make_float2(back <= FLT_MAX ? back : 0.f, unit);
}
// Correctly rounded x / d, from the correctly rounded r = 1 / d: one step of Markstein's
// division, whose residual is exact while nothing leaves the normal range.
__device__ __forceinline__ float over(float x, float d, float r) {
    const float q = __fmul_rn(x, r);
    return __fmaf_rn(__fmaf_rn(-q, d, x), r, q);
}
struct TensorScale {
    float t, d, r;   // t; what a block's top is divided by first (6 t or t), and its reciprocal
    bool valid, plain;
};
template <bool kB16>
__device__ __forceinline__ TensorScale tensor_scale_of(const float *p) {
    TensorScale s;
    s.t = p ? *p : 1.f;
    s.d = kB16 ? __fmul_rn(6.f, s.t) : s.t;
    s.r = __fdiv_rn(1.f, s.d);
    s.valid = s.t > 0.f && s.t <= FLT_MAX;
    s.plain = s.t >= 0x1p-60f && s.t <= 0x1p60f;
    return s;
}
// The scale byte of a block.  `top`: the largest magnitude's bits (NaN above infinity
// above numbers); a non-finite value, or a tensor scale that is none, makes it NaN.
// (The divisions' general form took half of the kernel's operations.)
template <bool kB16>
__device__ __forceinline__ uint32_t scale_of(uint32_t top_bits, const TensorScale &s) {
    const float top = __uint_as_float(top_bits);
    if (!s.valid || !(top <= FLT_MAX)) return kB16 ? 0x7f : 0xff;
    const bool plain = s.plain && (top == 0.f || (top >= 0x1p-60f && top <= 0x1p60f));
    float q = plain ? over(top, s.d, s.r) : __fdiv_rn(top, s.d);
    if constexpr (kB16) return __nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
    q = fminf(fmaxf(q, kFloor), FLT_MAX);
    q = plain ? over(q, 6.f, 0x1.555556p-3f) : __fdiv_rn(q, 6.f);
    return (__float_as_uint(q) + 0x7fffffu) >> 23;  // up to the next power of two
}

__device__ __forceinline__ uint32_t codes_of(float a, float b, float inv) {
    return __nv_cvt_float2_to_fp4x2(make_float2(__fmul_rn(a, inv), __fmul_rn(b, inv)), __NV_E2M1, cudaRoundNearest);
}
// Eight codes in a word to the values that they stand for.  (A code times an e4m3 scale
// has six bits and lies between 2^-10 and 2688: exact in half precision.)
template <bool kB16>
__device__ __forceinline__ void values_of(uint32_t word, float unit, float t, float *v) {
    const __half2 u = __float2half2_rn(unit);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        __half2 h = __half2(__nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(word >> (8 * q)), __NV_E2M1));
        if constexpr (kB16) h = __hmul2(h, u);
        const float2 f = __half22float2(h);
        v[2 * q] = __fmul_rn(kB16 ? f.x : __fmul_rn(f.x, unit), t);
        v[2 * q + 1] = __fmul_rn(kB16 ? f.y : __fmul_rn(f.y, unit), t);
    }
}
// Eight neighbouring values, `n` of them inside the row.
__device__ __forceinline__ void store_values(const QuantArgs &a, int64_t r, int64_t c, int64_t n, const float *v) {
    char *dst = a.values + r * a.values_stride + c * (a.values_f32 ? 4 : 2);
    if (n >= 8) {
        if (a.values_f32) {
            __stcs(reinterpret_cast<float4 *>(dst), make_float4(v[0], v[1], v[2], v[3]));
            __stcs(reinterpret_cast<float4 *>(dst) + 1, make_float4(v[4], v[5], v[6], v[7]));
        } else {
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * q], v[2 * q + 1]);
                w[q] = *reinterpret_cast<const uint32_t *>(&h);
            }
            __stcs(reinterpret_cast<uint4 *>(dst), make_uint4(w[0], w[1], w[2], w[3]));
        }
        return;
    }
#pragma unroll
    for (int q = 0; q < 8; ++q)
        if (q < n) {
            if (a.values_f32) reinterpret_cast<float *>(dst)[q] = v[q];
            else reinterpret_cast<__nv_bfloat16 *>(dst)[q] = __float2bfloat16_rn(v[q]);
        }
}

// Two rows of 128 values that lie in shared memory, a warp's work: rows r and r + step,
// columns c to c + 127, of those that exist.
__device__ __forceinline__ void store_rows(const QuantArgs &a, int64_t r, int step, int64_t c, int64_t rows, int64_t cols, const float *v, int pitch) {
    const int lane = threadIdx.x & 31;
    const int n = static_cast<int>(min(cols - c, static_cast<int64_t>(128))) - lane;  // values from the lane's first on
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (r + h * step >= rows) break;
        char *dst = a.values + (r + h * step) * a.values_stride + (c + lane) * (a.values_f32 ? 4 : 2);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (q * 32 < n) {
                const float x = v[h * pitch + q * 32 + lane];
                if (a.values_f32) __stcs(reinterpret_cast<float *>(dst) + q * 32, x);
                else reinterpret_cast<__nv_bfloat16 *>(dst)[q * 32] = __float2bfloat16_rn(x);
            }
    }
}

// kVec: rows of x and of the values on 16-byte boundaries.
template <bool kBf16, bool kB16, bool kTranspose, bool kVec>
__global__ void __launch_bounds__(kQThreads, kBf16 && kVec ? 3 : 2) quantize_kernel(const __grid_constant__ QuantArgs a) {
    __shared__ __align__(16) uint8_t atoms[kB16 ? 2 * kAtom : kAtom];
    __shared__ __align__(16) uint32_t tops[kTranspose && !kB16 ? 8 * kQTile : 4];
    __shared__ __align__(16) uint32_t turned[kTranspose ? kQTile * 16 : 4];
    // rows that pass through shared memory, so that a warp touches neighbouring bytes: a
    // warp's two rows where rows lie off 16-byte boundaries, or 16 columns of transposed values
    constexpr int kPitch = kQTile + 4;
    __shared__ __align__(16) float staged[kVec ? 4 : 16 * kPitch];
    constexpr int kElt = kBf16 ? 2 : 4, kBlk = kB16 ? 16 : 32, kBlocks = kQTile / kBlk;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int64_t tile_r = blockIdx.x / a.n_tiles_c, tile_c = blockIdx.x % a.n_tiles_c;
    const int64_t r0 = tile_r * kQTile, c0 = tile_c * kQTile;
    const int col = (lane & 15) * 8;
    const int row_group = warp * 2 + (lane >> 4);
    const auto row_of = [&](int p) { return kTranspose ? row_group * 8 + p : p * 16 + row_group; };
    __shared__ float2 meanings[256];
    const TensorScale tensor = tensor_scale_of<kB16>(a.tensor_scale);
    const float ts = tensor.t;
    {
        const float2 m = meaning_of<kB16>(t, ts);
        const bool nan = t == (kB16 ? 0x7f : 0xff);
        meanings[t] = make_float2(m.x, nan ? CUDART_NAN_F : m.y);
    }
    __syncthreads();
    // raw words of the thread's 8 passes: 8 values each, outside the tensor 0
    uint4 raw[8][kBf16 ? 1 : 2];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int64_t r = r0 + row_of(p), c = c0 + col;
        const char *src = a.x + r * a.x_stride + c * kElt;
#pragma unroll
        for (int h = 0; h < (kBf16 ? 1 : 2); ++h) raw[p][h] = make_uint4(0, 0, 0, 0);
        if constexpr (kVec) {
            if (r < a.rows && c + 8 <= a.cols) {
#pragma unroll
                for (int h = 0; h < (kBf16 ? 1 : 2); ++h) raw[p][h] = __ldcs(reinterpret_cast<const uint4 *>(src) + h);
            } else if (r < a.rows && c < a.cols) {
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
        } else {
            // the warp's two rows side by side: values lane, lane + 32, ... of each
            uint32_t w[8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t rr = r0 + (kTranspose ? (warp * 2 + h) * 8 + p : p * 16 + warp * 2 + h);
                const char *from = a.x + rr * a.x_stride + (c0 + lane) * kElt;
                const int n = rr < a.rows ? static_cast<int>(min(a.cols - c0, static_cast<int64_t>(kQTile))) - lane : 0;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    // (without branches two bytes a load are twice as fast: 68 us instead of 136 for 12661 x
                    // 2051; four bytes a load are not: 88 instead of 63)
                    if constexpr (kBf16) {
                        const uint32_t v = __ldg(reinterpret_cast<const unsigned short *>(q * 32 < n ? from + q * 64 : a.x));
                        w[h * 4 + q] = q * 32 < n ? v << 16 : 0;
                    } else {
                        w[h * 4 + q] = 0;
                        if (q * 32 < n) w[h * 4 + q] = __ldcs(reinterpret_cast<const uint32_t *>(from) + q * 32);
                    }
                }
            }
            raw[p][0] = make_uint4(w[0], w[1], w[2], w[3]);
            if constexpr (kBf16) {
                raw[p][0].x |= w[4] >> 16;
                raw[p][0].y |= w[5] >> 16;
                raw[p][0].z |= w[6] >> 16;
                raw[p][0].w |= w[7] >> 16;
            } else {
                raw[p][1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
        }
    }
    if constexpr (!kVec) {  // each lane gets eight neighbours
        float *const mine = &staged[warp * 2 * kPitch];
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            const uint32_t w[4] = {raw[p][0].x, raw[p][0].y, raw[p][0].z, raw[p][0].w};
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if constexpr (kBf16) {
                    mine[q * 32 + lane] = __uint_as_float(w[q] & 0xffff0000u);
                    mine[kPitch + q * 32 + lane] = __uint_as_float(w[q] << 16);
                } else {
                    const uint32_t w1[4] = {raw[p][1].x, raw[p][1].y, raw[p][1].z, raw[p][1].w};
                    mine[q * 32 + lane] = __uint_as_float(w[q]);
                    mine[kPitch + q * 32 + lane] = __uint_as_float(w1[q]);
                }
            }
            __syncwarp();
            const uint4 lo = *reinterpret_cast<const uint4 *>(&mine[(lane >> 4) * kPitch + col]), hi = *reinterpret_cast<const uint4 *>(&mine[(lane >> 4) * kPitch + col + 4]);
            if constexpr (kBf16) {
                raw[p][0] = make_uint4(lo.x >> 16 | lo.y, lo.z >> 16 | lo.w, hi.x >> 16 | hi.y, hi.z >> 16 | hi.w);
            } else {
                raw[p][0] = lo;
                raw[p][1] = hi;
            }
        }
        __syncwarp();
    }
    const auto values = [&](int p, float *v) {
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
    const auto bits = [](float x) { return __float_as_uint(x) & 0x7fffffffu; };
    // the tile's scale byte of output row r, block b of the tile
    const auto put = [&](int r, int b, uint32_t byte) {
        atoms[(b >> 2) * kAtom + (r & 31) * 16 + (r >> 5) * 4 + (b & 3)] = static_cast<uint8_t>(byte);
    };
    if constexpr (!kTranspose) {
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            float v[8];
            values(p, v);
            uint32_t m = 0;
            if constexpr (kBf16) {  // two magnitudes at a time
                const uint32_t two = __vmaxu2(__vmaxu2(raw[p][0].x & 0x7fff7fffu, raw[p][0].y & 0x7fff7fffu),
                                              __vmaxu2(raw[p][0].z & 0x7fff7fffu, raw[p][0].w & 0x7fff7fffu));
                m = max(two << 16, two & 0xffff0000u);
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q) m = max(m, bits(v[q]));
            }
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            if constexpr (!kB16) m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const uint32_t byte = scale_of<kB16>(m, tensor);
            const float inv = meanings[byte].x, unit = meanings[byte].y;
            const int64_t r = r0 + row_of(p), c = c0 + col;
            const bool in = r < a.rows && c < a.cols;
            // (a block that starts behind the last value has no scale: 0)
            if ((lane & (kB16 ? 1 : 3)) == 0) put(row_of(p), col / kBlk, in ? byte : 0u);
            uint32_t word = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q) word |= codes_of(v[2 * q], v[2 * q + 1], inv) << (8 * q);
            uint8_t *dst = a.out + r * a.out_stride + c / 2;
            const int64_t n = in ? a.cols - c : 0;
            if (a.vec_out && n >= 8) {
                __stcs(reinterpret_cast<uint32_t *>(dst), word);
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (2 * q < n) dst[q] = static_cast<uint8_t>(word >> (8 * q));
            }
            if (a.values) {
                values_of<kB16>(word, unit, ts, v);
                if constexpr (kVec) {
                    store_values(a, r, c, n, v);
                } else {
                    float *const mine = &staged[warp * 2 * kPitch];
                    __syncwarp();
                    *reinterpret_cast<float4 *>(&mine[(lane >> 4) * kPitch + col]) = make_float4(v[0], v[1], v[2], v[3]);
                    *reinterpret_cast<float4 *>(&mine[(lane >> 4) * kPitch + col + 4]) = make_float4(v[4], v[5], v[6], v[7]);
                    __syncwarp();
                    store_rows(a, r0 + p * 16 + warp * 2, 1, c0, a.rows, a.cols, mine, kPitch);
                }
            }
        }
    } else {
        uint32_t m[8];
        if constexpr (kBf16) {  // two magnitudes at a time
            uint32_t two[4] = {0, 0, 0, 0};
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                const uint32_t ws[4] = {raw[p][0].x, raw[p][0].y, raw[p][0].z, raw[p][0].w};
#pragma unroll
                for (int q = 0; q < 4; ++q) two[q] = __vmaxu2(two[q], ws[q] & 0x7fff7fffu);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                m[2 * q] = two[q] << 16;
                m[2 * q + 1] = two[q] & 0xffff0000u;
            }
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q) m[q] = 0;
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                float v[8];
                values(p, v);
#pragma unroll
                for (int q = 0; q < 8; ++q) m[q] = max(m[q], bits(v[q]));
            }
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) m[q] = max(m[q], __shfl_xor_sync(0xffffffffu, m[q], 16));
        if constexpr (!kB16) {  // a block of 32 rows is two warps'
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (lane < 16) tops[warp * kQTile + col + q] = m[q];
            __syncthreads();
#pragma unroll
            for (int q = 0; q < 8; ++q) m[q] = max(m[q], tops[(warp ^ 1) * kQTile + col + q]);
        }
        const int b = warp / (kB16 ? 1 : 2);  // the tile's block
        const bool block_in = r0 + b * kBlk < a.rows;
        // the two halves of a warp have the same columns: four divisions' work each
        float inv[8], unit[8];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const bool upper = lane >= 16;
            const uint32_t byte = scale_of<kB16>(upper ? m[q + 4] : m[q], tensor);
            const float iv = meanings[byte].x, un = meanings[byte].y;
            const int c = col + q + (upper ? 4 : 0);
            if (kB16 || (warp & 1) == 0) put(c, b, block_in && c0 + c < a.cols ? byte : 0u);
            const float oi = __shfl_xor_sync(0xffffffffu, iv, 16), ou = __shfl_xor_sync(0xffffffffu, un, 16);
            inv[q] = upper ? oi : iv;
            inv[q + 4] = upper ? iv : oi;
            unit[q] = upper ? ou : un;
            unit[q + 4] = upper ? un : ou;
        }
        uint32_t words[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) words[q] = 0;
#pragma unroll
        for (int p = 0; p < 8; p += 2) {
            float v[2][8];
            values(p, v[0]);
            values(p + 1, v[1]);
#pragma unroll
            for (int q = 0; q < 8; ++q) words[q] |= codes_of(v[0][q], v[1][q], inv[q]) << (4 * p);
        }
        const int64_t oc = r0 + row_group * 8;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            turned[(col + q) * 16 + (row_group ^ (col >> 3))] = words[q];
            if (a.values) {
                float v[8];
                values_of<kB16>(words[q], unit[q], ts, v);
                if constexpr (kVec) {
                    if (c0 + col + q < a.cols && oc < a.rows) store_values(a, c0 + col + q, oc, a.rows - oc, v);
                } else {  // 16 output rows at a time
                    __syncthreads();
                    float *const to = &staged[(lane & 15) * kPitch + row_group * 8];
                    *reinterpret_cast<float4 *>(to) = make_float4(v[0], v[1], v[2], v[3]);
                    *reinterpret_cast<float4 *>(to + 4) = make_float4(v[4], v[5], v[6], v[7]);
                    __syncthreads();
                    store_rows(a, c0 + warp * 16 + q, 8, r0, a.cols, a.rows, &staged[warp * 2 * kPitch], kPitch);
                }
            }
        }
        __syncthreads();
        // 128 output rows (input columns) of 64 bytes: 4 lanes a row with 16 bytes each
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const int row = p * 64 + (t >> 2), at = t & 3, key = row >> 3;
            const int64_t orow = c0 + row, ov = r0 + at * 32;  // (the first of 32 values)
            if (orow >= a.cols || ov >= a.rows) continue;
            const uint4 w = *reinterpret_cast<const uint4 *>(&turned[row * 16 + ((at ^ (key >> 2)) << 2)]);
            const uint32_t in[4] = {w.x, w.y, w.z, w.w};
            uint32_t ws[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // word j lies at j ^ key % 4
                const uint32_t lo = (key & 1) ? in[j ^ 1] : in[j], hi = (key & 1) ? in[j ^ 3] : in[j ^ 2];
                ws[j] = (key & 2) ? hi : lo;
            }
            uint8_t *dst = a.out + orow * a.out_stride + ov / 2;
            const int64_t n = a.rows - ov;
            if (a.vec_out && n >= 32) {
                __stcs(reinterpret_cast<uint4 *>(dst), make_uint4(ws[0], ws[1], ws[2], ws[3]));
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (2 * j < n) dst[j] = static_cast<uint8_t>(ws[j >> 2] >> (8 * (j & 3)));
            }
        }
    }
    __syncthreads();
    // the tile's scales: the atoms of one group of 128 output rows, neighbours along k
    const int64_t group = kTranspose ? tile_c : tile_r, atom0 = (kTranspose ? tile_r : tile_c) * (kBlocks / 4);
    if (t < (kBlocks / 4) * (kAtom / 4) && atom0 + t / (kAtom / 4) < a.atoms)
        reinterpret_cast<uint32_t *>(a.scales + (group * a.atoms + atom0) * kAtom)[t] = reinterpret_cast<const uint32_t *>(atoms)[t];
}

// ==================================================================== product
// One persistent CTA per SM, two of them a pair where the output has more than one
// row tile.  A tile is 128 rows a CTA x 256 columns; a pair's CTAs take row tiles
// next to each other, each loads its rows of A and half of B's 256, and the leader's
// MMAs (cta_group::2, M=256 N=256 K=64) work on both CTAs' shared and tensor memory.
// Warp 0 streams 256 values of k a stage and their scales through a ring (TMA,
// 128-byte swizzle for the values).  Warp 1 copies a stage's scales into tensor memory
// (tcgen05.cp, each to all four lane quadrants) and issues its four MMAs into the one
// accumulator.  A stage's scales have columns of their own, so they are written only
// after the MMAs that read the last ones have freed the stage.  Two warpgroups read the
// accumulator into registers, 128 columns a thread, and free it at once; rounding and
// stores (TMA) run under the next tile.
//
// 4096 x 128256 x 4096: 632 us, 6.8 PFLOP/s; with a k of 16384 (38912 columns) 7.9.  A
// stage takes 0.30 us, 560 to 600 cycles, its four MMAs 512 of them; the rest is their
// issue, which is why a whole stage's runs without a test in between (0.34 us with them).
// A tile's end costs 1.2 us: its last MMAs, the read of the accumulator, the hand-over to
// the next tile's first.  Tensor memory has no room for a second accumulator of this width;
// three of half of it, used in turn, hide the hand-over, but an MMA on 128 columns takes as
// long as one on 256 (1410 us).  Without pairs (54 KB a stage, three in flight: the bytes
// from L2 bound it) the product took 896 us, with half of B brought to both CTAs by
// multicast 847.  Float32 output is bound by its boxes, one in flight a warp (37984 x 4096 x
// 2051: 190 us, 3.4 TB/s); a second one costs a stage of the ring (5 % slower), stores from
// registers in 32-byte sectors hold up the loads (246 us).
constexpr int kTM = 128, kTN = 256, kTK = 256;
template <bool kPair>
struct Ring {
    static constexpr int kStages = kPair ? 5 : 3;
    static constexpr int kBRows = kPair ? kTN / 2 : kTN;  // of B that a CTA holds
    static constexpr int kA = kTM * kTK / 2, kB = kBRows * kTK / 2;
    static constexpr int kSa = 4 * kAtom, kSb = 8 * kAtom;  // scales, all 256 columns' (blocks of 32 need half)
    static constexpr int kStage = kA + kB + kSa + kSb;      // 38 or 54 KB
    static constexpr size_t kSmem = 1024 + static_cast<size_t>(kStages) * kStage + 8 * 32 * 128;
    static_assert(kStage % 1024 == 0, "the swizzle's 1024-byte groups");
};
constexpr int kEpiWarps = 8;
constexpr int kEpiCols = kTN / (kEpiWarps / 4);  // columns a warp
constexpr int kMmThreads = (4 + kEpiWarps) * 32;
// registers a thread after the split (three warps a sub-partition, launched at
// 168 each: 40 + 2 * 232 = 3 * 168)
constexpr int kRegsFront = 40, kRegsEpi = 232;
constexpr int kOutWarp = 32 * 128;               // staging of a warp: a box of 32 rows x 128 bytes
constexpr int kOutPitch = 80;                    // or rows of 64 bytes and 16 against bank conflicts
static_assert(kEpiWarps * kOutWarp == 8 * 32 * 128, "the ring's room for staging");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kScaleCol = kTN;              // a stage's scales: 16 columns of A's, 32 of B's
constexpr uint32_t kScaleCols = 48;
static_assert(kScaleCol + 5 * kScaleCols <= kTmemCols, "tensor memory");
constexpr int kRaster = 16;                      // row tiles (or pairs) that share a B tile in L2

__device__ __forceinline__ uint32_t of_leader(const void *p) {  // the address of a pair's first CTA's own
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
    return r;
}
// A box into this CTA's memory; its bytes count at the barrier `bar` (a cluster address).
template <bool kPair>
__device__ __forceinline__ void load_box(void *dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    if constexpr (kPair)
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
            "l"(map), "r"(x), "r"(y), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
            "l"(map), "r"(x), "r"(y), "r"(bar)
            : "memory");
}
// Arrive on `bar`, of both CTAs of a pair, once every MMA issued so far completes.
template <bool kPair>
__device__ __forceinline__ void commit(uint64_t *bar) {
    if constexpr (kPair)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
            "h"(static_cast<uint16_t>(3))
            : "memory");
    else
        umma_commit(bar);
}
// The accumulator's hand-over, from an epilogue warp to the leader's MMAs.  It orders reads of
// tensor memory and nothing else, for which PTX asks no more of a barrier than to be observed:
// tcgen05.ld, wait::ld, fence::before_thread_sync and a relaxed arrival on this side, the wait
// and fence::after_thread_sync before the MMA on the other.  (A release would also wait for the
// stores under way, half a microsecond a tile: 684 us instead of 632.)
__device__ __forceinline__ void arrive_at(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// A pair's waits are at the cluster's scope: what they wait for may be the other CTA's.
struct ClusterScope {
    static __device__ __forceinline__ bool try_wait(uint64_t *bar, uint32_t parity) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        return ok != 0;
    }
};
__device__ __forceinline__ void pair_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 32 rows x 16 bytes of scales (an atom) to four columns of all lane quadrants.
constexpr uint32_t kAtomDescHigh = (128u >> 4) | (1u << 14);  // 8-row groups of 128 bytes, no swizzle
template <bool kPair>
__device__ __forceinline__ void scales_to_tmem(uint32_t col, uint32_t low) {
    if constexpr (kPair)
        asm volatile(
            "{\n\t.reg .b64 d;\n\t"
            "mov.b64 d, {%1, %2};\n\t"
            "tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], d;\n\t}" ::"r"(col),
            "r"(low), "r"(kAtomDescHigh)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .b64 d;\n\t"
            "mov.b64 d, {%1, %2};\n\t"
            "tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], d;\n\t}" ::"r"(col),
            "r"(low), "r"(kAtomDescHigh)
            : "memory");
}
template <bool kB16, bool kPair>
__device__ __forceinline__ void umma_f4(uint32_t d_tmem, uint32_t a_low, uint32_t b_low, uint32_t idesc, uint32_t sa,
                                        uint32_t sb, uint32_t accumulate) {
    if constexpr (kB16 && kPair)
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
            "mov.b64 da, {%1, %7};\n\t"
            "mov.b64 db, {%2, %7};\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], da, db, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
            "r"(a_low), "r"(b_low), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate), "r"(kDescHigh)
            : "memory");
    else if constexpr (kB16)
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
            "mov.b64 da, {%1, %7};\n\t"
            "mov.b64 db, {%2, %7};\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], da, db, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
            "r"(a_low), "r"(b_low), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate), "r"(kDescHigh)
            : "memory");
    else if constexpr (kPair)
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
            "mov.b64 da, {%1, %7};\n\t"
            "mov.b64 db, {%2, %7};\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], da, db, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
            "r"(a_low), "r"(b_low), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate), "r"(kDescHigh)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
            "mov.b64 da, {%1, %7};\n\t"
            "mov.b64 db, {%2, %7};\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], da, db, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
            "r"(a_low), "r"(b_low), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate), "r"(kDescHigh)
            : "memory");
}
// 32 lanes x 32 columns, a row a lane.
__device__ __forceinline__ void tmem_ld_32(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

// The two tensor scales as factors of the sums: f1 alone, their product, where float32 has
// that among its normal numbers; else f1 is its significand, and f2, f2 and f3 are powers of
// two, a third of its exponent each.  (Either scale may lie anywhere in float32's range, so
// their product may leave it where the scaled sums do not.  The three go in one direction:
// a step overflows only if the result does, and loses bits only where the result is denormal.)
struct SumScale {
    float f1, f2, f3;
    bool one;
    __device__ __forceinline__ SumScale(const float *ta, const float *tb) : f2(1.f), f3(1.f), one(true) {
        const float a = ta ? *ta : 1.f, b = tb ? *tb : 1.f;
        f1 = __fmul_rn(a, b);
        if (f1 == 0.f ? a == 0.f || b == 0.f : fabsf(f1) >= FLT_MIN && fabsf(f1) <= FLT_MAX) return;
        if (!(fabsf(a) <= FLT_MAX && fabsf(b) <= FLT_MAX)) return;
        int ea, eb;
        f1 = __fmul_rn(frexpf(a, &ea), frexpf(b, &eb));  // in [1/4, 1)
        const int third = (ea + eb) / 3;
        f2 = ldexpf(1.f, third);
        f3 = ldexpf(1.f, ea + eb - 2 * third);
        one = false;
    }
    __device__ __forceinline__ float rest(float x) const { return __fmul_rn(__fmul_rn(__fmul_rn(x, f2), f2), f3); }
};

struct MmMaps {
    CUtensorMap a, b;
    CUtensorMap sa, sb;  // scales: (word of an atom, atom)
    CUtensorMap out;     // (column, row, split); only where vec_out
};

struct MmArgs {
    const float *ta, *tb;
    int64_t m, n, k;
    int atoms;                 // of scales along k
    int groups_m, groups_n;    // groups of 128 rows of A and of B
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

template <bool kOutF32, bool kB16, bool kPair>
__global__ void __launch_bounds__(kMmThreads, 1)
    product_kernel(const __grid_constant__ MmMaps maps, const __grid_constant__ MmArgs a) {
    extern __shared__ __align__(1024) char smem_raw[];
    using R = Ring<kPair>;
    constexpr int kStages = R::kStages;
    __shared__ uint64_t full[kStages], empty[kStages], acc_full, acc_empty, done;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    char *const smem = smem_raw + (-smem_u32(smem_raw) & 1023u);  // (an offset keeps the loads shared ones)
    char *const staged = smem + static_cast<size_t>(kStages) * R::kStage;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t items = static_cast<int64_t>(a.n_tm) * a.n_tn * a.n_splits;
    constexpr int kAtomsPer = kB16 ? 4 : 2;  // atoms of scales along a stage's k
    constexpr int kCtas = kPair ? 2 : 1;
    using Scope = std::conditional_t<kPair, ClusterScope, CtaScope>;
    const int rank = kPair ? blockIdx.x & 1 : 0;
    const int64_t item0 = blockIdx.x / kCtas, step = gridDim.x / kCtas;

    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(&acc_full, 1);
        mbar_init(&acc_empty, kEpiWarps * kCtas);
        mbar_init(&done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        if constexpr (kPair) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)), "r"(kTmemCols) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)), "r"(kTmemCols) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (kPair) pair_sync();  // (the other's barriers stand before anything arrives at them)
    tc_fence_after();
    const uint32_t tmem = tmem_slot;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFront));
        const bool leader = elect_one();  // (whole warps run the loops, so that their values are uniform)
        if (warp == 0) {
            // ------------------------------------------------------------ producer
            uint32_t s = 0, phase = 1, issued = 0;  // the first turn finds every stage empty
            bool ok = true;
            for (int64_t w = item0; ok && w < items; w += step) {
                int tm, tn, split;
                item_coords(w, a, tm, tn, split);
                tm = tm * kCtas + rank;
                const int kb1 = min(a.kb_total, (split + 1) * a.kb_per_split);
                // (behind the last group of 128 rows any scales do)
                const int ga = min(tm, a.groups_m - 1), gb = 2 * tn, gb1 = min(gb + 1, a.groups_n - 1);
#pragma unroll 1
                for (int kb = split * a.kb_per_split; kb < kb1; ++kb) {
                    ok = wait_warp<Scope>(&empty[s], phase, &abort_flag, a.status);
                    if (!ok) break;
                    if (leader) {
                        char *st = smem + s * R::kStage;
                        constexpr uint32_t kScaleBytes = 3 * kAtomsPer * kAtom;
                        const uint32_t bar = kPair ? of_leader(&full[s]) : smem_u32(&full[s]);
                        if (rank == 0) mbar_arrive_expect_tx(&full[s], kCtas * (R::kA + R::kB + kScaleBytes));
                        load_box<kPair>(st, &maps.a, kb * (kTK / 2), tm * kTM, bar);
                        load_box<kPair>(st + R::kA, &maps.b, kb * (kTK / 2), tn * kTN + rank * R::kBRows, bar);
                        char *sc = st + R::kA + R::kB;
                        load_box<kPair>(sc, &maps.sa, 0, ga * a.atoms + kb * kAtomsPer, bar);
                        load_box<kPair>(sc + R::kSa, &maps.sb, 0, gb * a.atoms + kb * kAtomsPer, bar);
                        load_box<kPair>(sc + R::kSa + R::kSb / 2, &maps.sb, 0, gb1 * a.atoms + kb * kAtomsPer, bar);
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
                // (a pair's barriers are the leader's; the other CTA waits for it at the end)
                if (rank == 0) wait_warp<Scope>(&full[s], phase ^ 1, &abort_flag, a.status, false);
            }
        } else if (warp == 1 && rank == 0) {
            // ----------------------------------------------------------------- MMA
            uint32_t s = 0, phase = 0, turn = 1;  // `turn`: the parity that the emptied accumulator shows
            bool ok = true, issued = false;
            const int whole = static_cast<int>(a.k / kTK), tail = (static_cast<int>(a.k % kTK) + 63) / 64;  // stages of four MMAs, the last one's
            const uint32_t base = desc_low(smem), plain = (smem_u32(smem) & 0x3FFFFu) >> 4;
            for (int64_t w = item0; ok && w < items; w += step) {
                int tm, tn, split;
                item_coords(w, a, tm, tn, split);
                tm = tm * kCtas + rank;
                const int kb0 = split * a.kb_per_split, kb1 = min(a.kb_total, kb0 + a.kb_per_split);
                ok = wait_warp<Scope>(&acc_empty, turn, &abort_flag, a.status);
                turn ^= 1;
#pragma unroll 1
                for (int kb = kb0; ok && kb < kb1; ++kb) {
                    ok = wait_warp<Scope>(&full[s], phase, &abort_flag, a.status);
                    if (!ok) break;
                    tc_fence_after();
                    if (leader) {
                        const uint32_t da = base + s * (R::kStage >> 4), db = da + (R::kA >> 4);
                        const uint32_t sa = plain + s * (R::kStage >> 4) + ((R::kA + R::kB) >> 4), sb = sa + (R::kSa >> 4);
                        const uint32_t ca = tmem + kScaleCol + s * kScaleCols, cb = ca + 16;
                        const auto issue = [&](int mmas) {
#pragma unroll
                            for (int j = 0; j < kAtomsPer; ++j) {
                                if (j * (4 / kAtomsPer) >= mmas) break;
                                scales_to_tmem<kPair>(ca + 4 * j, sa + j * (kAtom >> 4));
                                scales_to_tmem<kPair>(cb + 8 * j, sb + j * (kAtom >> 4));
                                scales_to_tmem<kPair>(cb + 8 * j + 4, sb + (4 + j) * (kAtom >> 4));
                            }
#pragma unroll
                            for (int j = 0; j < 4; ++j) {  // K = 32 bytes inside the swizzle row
                                if (j >= mmas) break;
                                // (of a word of four scales of 32 an MMA takes the first or the last two)
                                const uint32_t idesc = kB16 ? a.idesc : a.idesc | (j & 1) << 5 | (j & 1) << 30;
                                const int at = kB16 ? j : j / 2;
                                umma_f4<kB16, kPair>(tmem, da + 2 * j, db + 2 * j, idesc, ca + 4 * at, cb + 4 * (kTN / kTM) * at, kb > kb0 || j > 0 ? 1u : 0u);
                            }
                        };
                        if (kb < whole) issue(4);
                        else issue(tail);
                        commit<kPair>(&empty[s]);
                        if (kb + 1 == kb1) commit<kPair>(&acc_full);
                    }
                    issued = true;
                    if (++s == kStages) {
                        s = 0;
                        phase ^= 1;
                    }
                }
            }
            if (issued) {
                if (leader) {
                    if constexpr (kPair) asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(&done)) : "memory");
                    else umma_commit(&done);
                }
                wait_warp<Scope>(&done, 0, &abort_flag, a.status, false);
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpi));
        // ------------------------------------------------------------ epilogue
        const int quad = warp & 3, part = (warp - 4) >> 2;
        const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quad * 32) << 16) + part * kEpiCols;
        char *const mine = staged + (warp - 4) * kOutWarp;
        const SumScale scale(a.ta, a.tb);
        uint32_t turn = 0;
        bool ok = true;
        for (int64_t w = item0; w < items; w += step) {
            int tm, tn, split;
            item_coords(w, a, tm, tn, split);
            tm = tm * kCtas + rank;
            const int64_t col0 = static_cast<int64_t>(tn) * kTN + part * kEpiCols;
            float acc[kEpiCols];
            ok = ok && wait_warp<Scope>(&acc_full, turn, &abort_flag, a.status);
            turn ^= 1;
            if (ok) {
                tc_fence_after();
                uint32_t *const r = reinterpret_cast<uint32_t *>(acc);
#pragma unroll
                for (int c = 0; c < kEpiCols; c += 32) tmem_ld_32(lane_addr + c, r + c);
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (kPair) arrive_at(of_leader(&acc_empty));
                    else mbar_arrive(&acc_empty);
                }
#pragma unroll
                for (int j = 0; j < kEpiCols; ++j) acc[j] = __fmul_rn(acc[j], scale.f1);
                if (!scale.one) {
#pragma unroll
                    for (int j = 0; j < kEpiCols; ++j) acc[j] = scale.rest(acc[j]);
                }
            } else {  // a wait gave up: this tile reads as NaN
#pragma unroll
                for (int j = 0; j < kEpiCols; ++j) acc[j] = CUDART_NAN_F;
            }
            char *const out = a.out + split * a.split_stride;
            const int64_t row0 = static_cast<int64_t>(tm) * kTM + quad * 32;
            if (row0 >= a.m) continue;
            // (a TMA store writes whole 16-byte pieces: columns behind an n
            // between two of them are not the product's to write)
            if (a.vec_out && (a.whole_out || col0 + kEpiCols <= a.n)) {
                // boxes of 32 rows x 128 bytes under the 128-byte swizzle: chunk
                // q of row l lies at q ^ (l % 8)
                constexpr int kBoxCols = kOutF32 ? 32 : 64;
#pragma unroll
                for (int box = 0; box < kEpiCols / kBoxCols; ++box) {
                    if (lane == 0) tma_store_wait_read();  // the last box has been read
                    __syncwarp();
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const float *v = &acc[box * kBoxCols + q * (kBoxCols / 8)];
                        uint4 u;
                        if constexpr (kOutF32) {
                            u = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
                        } else {
                            uint32_t h[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const __nv_bfloat162 two = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
                                h[e] = *reinterpret_cast<const uint32_t *>(&two);
                            }
                            u = make_uint4(h[0], h[1], h[2], h[3]);
                        }
                        *reinterpret_cast<uint4 *>(mine + lane * 128 + ((q ^ (lane & 7)) << 4)) = u;
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    const int64_t c = col0 + box * kBoxCols;
                    if (lane == 0) {
                        if (c < a.n) tma_store_3d(&maps.out, mine, static_cast<int>(c), static_cast<int>(row0), split);
                        tma_store_commit();
                    }
                }
                continue;
            }
            // 64-byte pieces of 32 rows through shared memory
            if (lane == 0) tma_store_wait_read();  // the last tile's box lay there
            constexpr int kCols = kOutF32 ? 16 : 32;  // columns of a piece
#pragma unroll
            for (int p = 0; p < kEpiCols / kCols; ++p) {
                __syncwarp();
#pragma unroll
                for (int q = 0; q < kCols; q += 2) {
                    const float *v = &acc[p * kCols + q];
                    if (kOutF32) *reinterpret_cast<float2 *>(mine + lane * kOutPitch + 4 * q) = make_float2(v[0], v[1]);
                    else *reinterpret_cast<__nv_bfloat162 *>(mine + lane * kOutPitch + 2 * q) = __floats2bfloat162_rn(v[0], v[1]);
                }
                __syncwarp();
                const int64_t c = col0 + p * kCols;
                if (c >= a.n) break;
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
            __syncwarp();
        }
    }

    if (warp >= 4 && lane == 0) tma_store_wait_read();  // shared memory outlives the last stores' reads
    tc_fence_before();
    __syncthreads();
    if constexpr (kPair) pair_sync();  // nothing of the pair's is under way any more
    if (warp == 1) {
        tc_fence_after();
        if constexpr (kPair) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
        else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

// C = the partial results added in split order, scaled, rounded once.
template <bool kOutF32>
__global__ void __launch_bounds__(256) join_kernel(const float *part, int64_t part_stride, int64_t split_stride,
                                                   int n_splits, int64_t m, int64_t n, const float *ta, const float *tb,
                                                   char *out, int64_t out_stride) {
    const int64_t cells = m * n;
    const SumScale scale(ta, tb);
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < cells; i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t r = i / n, c = i - r * n;
        const float *p = part + r * part_stride + c;
        float s = p[0];
        for (int k = 1; k < n_splits; ++k) s = __fadd_rn(s, p[k * split_stride]);
        s = __fmul_rn(s, scale.f1);
        if (!scale.one) s = scale.rest(s);
        if (kOutF32) *reinterpret_cast<float *>(out + r * out_stride + 4 * c) = s;
        else *reinterpret_cast<__nv_bfloat16 *>(out + r * out_stride + 2 * c) = __float2bfloat16_rn(s);
    }
}

// An operand's scales as atoms of 128 words, boxes of a stage's.
bool make_scale_map(CUtensorMap *map, const void *ptr, int64_t atoms, bool b16) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {kAtom / 4, static_cast<cuuint64_t>(atoms)};
    const cuuint64_t strides[1] = {kAtom};
    const cuuint32_t box[2] = {kAtom / 4, b16 ? 4u : 2u};
    const cuuint32_t elem[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void *>(ptr), dims, strides, box, elem,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kBf16, bool kVec>
cudaError_t quantize_typed(const QuantArgs &a, bool b16, bool transpose, unsigned grid, cudaStream_t s) {
    if (b16) {
        if (transpose) quantize_kernel<kBf16, true, true, kVec><<<grid, kQThreads, 0, s>>>(a);
        else quantize_kernel<kBf16, true, false, kVec><<<grid, kQThreads, 0, s>>>(a);
    } else {
        if (transpose) quantize_kernel<kBf16, false, true, kVec><<<grid, kQThreads, 0, s>>>(a);
        else quantize_kernel<kBf16, false, false, kVec><<<grid, kQThreads, 0, s>>>(a);
    }
    return cudaGetLastError();
}

template <bool kOutF32, bool kB16, bool kPair>
cudaError_t product_of(const MmMaps &maps, const MmArgs &a, cudaStream_t stream) {
    static std::atomic<uint64_t> configured{0};
    const cudaError_t e = set_smem_once(product_kernel<kOutF32, kB16, kPair>, Ring<kPair>::kSmem, configured);
    if (e != cudaSuccess) return e;
    constexpr int kCtas = kPair ? 2 : 1;
    const int64_t items = static_cast<int64_t>(a.n_tm) * a.n_tn * a.n_splits, room = device_sm_count() / kCtas;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(std::min(items, room) * kCtas));
    cfg.blockDim = dim3(kMmThreads);
    cfg.dynamicSmemBytes = Ring<kPair>::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = kCtas;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, product_kernel<kOutF32, kB16, kPair>, maps, a);
}
template <bool kOutF32, bool kB16>
cudaError_t product_typed(const MmMaps &maps, const MmArgs &a, bool pair, cudaStream_t stream) {
    return pair ? product_of<kOutF32, kB16, true>(maps, a, stream) : product_of<kOutF32, kB16, false>(maps, a, stream);
}

}  // namespace

// The k axis is split where the output's tiles would leave half of the
// multiprocessors idle, into parts of at least four stages (1024 values).
BlockPlan micro_plan(int64_t m, int64_t n, int64_t k) {
    BlockPlan p{};
    p.n_tm = (m + kTM - 1) / kTM;
    p.n_tn = (n + kTN - 1) / kTN;
    p.kb_total = (k + kTK - 1) / kTK;
    const int64_t tiles = p.n_tm * p.n_tn;
    const int64_t sms = device_sm_count();
    int64_t want = tiles > 0 ? sms / tiles : 1;
    want = std::min(want, p.kb_total / 4);
    p.n_splits = std::max<int64_t>(want, 1);
    p.kb_per_split = p.n_splits > 1 ? (p.kb_total + p.n_splits - 1) / p.n_splits : p.kb_total;
    if (p.n_splits > 1) p.n_splits = (p.kb_total + p.kb_per_split - 1) / p.kb_per_split;
    p.part_stride = (n + 3) / 4 * 4;
    p.bytes = 256;
    if (p.n_splits > 1) p.bytes += align256(static_cast<size_t>(p.n_splits) * m * p.part_stride * 4);
    return p;
}

cudaError_t launch_micro_quantize(const void *x, int x_dtype, int64_t x_stride_elems, int64_t rows, int64_t cols,
                                  bool transpose, const MicroOperand &o, void *values, int values_dtype,
                                  int64_t values_stride_elems, cudaStream_t stream) {
    if (rows == 0 || cols == 0) return cudaSuccess;
    QuantArgs a{};
    const bool bf16 = x_dtype == LPD_BF16;
    a.x = static_cast<const char *>(x);
    a.x_stride = x_stride_elems * (bf16 ? 2 : 4);
    a.rows = rows;
    a.cols = cols;
    a.out = static_cast<uint8_t *>(const_cast<void *>(o.ptr));
    a.out_stride = o.row_stride;
    a.scales = const_cast<uint8_t *>(o.scales);
    a.atoms = o.atoms;
    a.tensor_scale = o.tensor_scale;
    a.values = static_cast<char *>(values);
    a.values_f32 = values_dtype == LPD_F32 ? 1 : 0;
    a.values_stride = values_stride_elems * (a.values_f32 ? 4 : 2);
    a.n_tiles_c = static_cast<int>((cols + kQTile - 1) / kQTile);
    const uintptr_t unit = transpose ? 16 : 4;
    a.vec_out = reinterpret_cast<uintptr_t>(o.ptr) % unit == 0 && static_cast<uintptr_t>(o.row_stride) % unit == 0;
    const bool vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && a.x_stride % 16 == 0 &&
                     (!values || (reinterpret_cast<uintptr_t>(values) % 16 == 0 && a.values_stride % 16 == 0));
    const unsigned grid = static_cast<unsigned>((rows + kQTile - 1) / kQTile * a.n_tiles_c);
    if (bf16) return vec ? quantize_typed<true, true>(a, o.b16, transpose, grid, stream) : quantize_typed<true, false>(a, o.b16, transpose, grid, stream);
    return vec ? quantize_typed<false, true>(a, o.b16, transpose, grid, stream) : quantize_typed<false, false>(a, o.b16, transpose, grid, stream);
}

cudaError_t launch_micro_matmul(const MicroOperand &x, const MicroOperand &y, int64_t m, int64_t n, int64_t k,
                                void *out, int out_dtype, int64_t out_stride_elems, void *workspace,
                                cudaStream_t stream) {
    const bool f32 = out_dtype == LPD_F32;
    const int64_t out_stride = out_stride_elems * (f32 ? 4 : 2);
    if (m == 0 || n == 0) return cudaSuccess;
    if (k == 0) return cudaMemset2DAsync(out, out_stride, 0, n * (f32 ? 4 : 2), m, stream);
    const BlockPlan p = micro_plan(m, n, k);
    MmMaps maps;
    const bool pair = p.n_tm > 1;
    if (!make_map(&maps.a, x.ptr, m, (k + 1) / 2, x.row_stride, kTM) ||
        !make_map(&maps.b, y.ptr, n, (k + 1) / 2, y.row_stride, pair ? kTN / 2 : kTN) ||
        !make_scale_map(&maps.sa, x.scales, (m + 127) / 128 * x.atoms, x.b16) ||
        !make_scale_map(&maps.sb, y.scales, (n + 127) / 128 * y.atoms, y.b16))
        return cudaErrorInvalidValue;
    MmArgs a{};
    const bool split = p.n_splits > 1;
    a.ta = split ? nullptr : x.tensor_scale;  // (partial results are scaled once they are one)
    a.tb = split ? nullptr : y.tensor_scale;
    a.m = m;
    a.n = n;
    a.k = k;
    a.atoms = static_cast<int>(x.atoms);
    a.groups_m = static_cast<int>((m + 127) / 128);
    a.groups_n = static_cast<int>((n + 127) / 128);
    a.kb_total = static_cast<int>(p.kb_total);
    a.kb_per_split = static_cast<int>(p.kb_per_split);
    a.n_splits = static_cast<int>(p.n_splits);
    a.n_tm = static_cast<int>(pair ? (p.n_tm + 1) / 2 : p.n_tm);  // (pairs of row tiles)
    a.n_tn = static_cast<int>(p.n_tn);
    // block scaling: A's and B's format e2m1 (1 at bits 7 and 10), N / 8 at bit 17, scales e4m3 or
    // powers of two (bit 23), M / 16 at bit 24 (a pair's is 256); both K-major
    a.idesc = (1u << 7) | (1u << 10) | (static_cast<uint32_t>(kTN >> 3) << 17) | (x.b16 ? 0u : 1u << 23) |
              (static_cast<uint32_t>((pair ? 2 * kTM : kTM) >> 4) << 24);
    a.status = static_cast<uint32_t *>(workspace);
    float *part = reinterpret_cast<float *>(static_cast<char *>(workspace) + 256);
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
    if (to_f32) e = x.b16 ? product_typed<true, true>(maps, a, pair, stream) : product_typed<true, false>(maps, a, pair, stream);
    else e = x.b16 ? product_typed<false, true>(maps, a, pair, stream) : product_typed<false, false>(maps, a, pair, stream);
    if (e != cudaSuccess || !split) return e;
    const int64_t blocks = std::min<int64_t>((m * n + 255) / 256, static_cast<int64_t>(device_sm_count()) * 16);
    if (f32)
        join_kernel<true><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(part, p.part_stride, m * p.part_stride, a.n_splits, m, n,
                                                                          x.tensor_scale, y.tensor_scale, static_cast<char *>(out), out_stride);
    else
        join_kernel<false><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(part, p.part_stride, m * p.part_stride, a.n_splits, m, n,
                                                                           x.tensor_scale, y.tensor_scale, static_cast<char *>(out), out_stride);
    return cudaGetLastError();
}

}  // namespace lpd
