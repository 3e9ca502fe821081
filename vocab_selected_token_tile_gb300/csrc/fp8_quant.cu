// Quantisation to E4M3 with one FP32 scale for each group of 128 (sm_103a):
// the operands of the FP8 product in fp8_gemm.cu.
//
// A group is 128 consecutive elements of a row (block_rows 1), or a block of
// 128 rows x 128 columns (block_rows 128); the last group of a row and the
// last block of rows may be shorter.  With amax the group's largest magnitude,
//   s = max(amax, 2^-100) / 448,   q = e4m3(x * (1 / s)),
// each of the three operations one FP32 rounding (448 is E4M3's largest
// value; e4m3() rounds to nearest even).  The floor gives an all-zero group a
// normal scale, so no branch and no division by zero: its values are 0 * r.
// A group that holds a NaN or an infinity gets a NaN or infinite scale and
// stands for NaN throughout.
//
// Scales are laid out group-major: scale[g * rows + r] is group g of row r
// (g * ceil(rows / 128) + r / 128 for blocks), so the 128 rows of a tile of
// the product read their scales of one K group as one contiguous run.
//
// Bound: HBM.  2 (or 4) bytes read and 1 written per element, 2 written where
// the transpose is wanted too: both come from one read.  One CTA takes a
// 128 x 128 tile, which is every group of either direction that it touches,
// whole: a thread holds an 8 x 8 block of it in registers (16 threads span a
// row's 128 columns, so a row's maximum is a butterfly over 16 lanes; the
// column maxima meet in shared memory), and no element is read twice.  The
// transposed codes pass through 16 KB of shared memory in 8-byte pieces (8
// rows of one column), XOR-swizzled by the column's block of 8 so that the 16
// lanes of a half warp hit 16 different 8-byte bank pairs.
//
// What it spends: a tile is one chain of loads, maxima, barriers, conversions
// and stores, and the other CTAs of the SM (three, of BF16) are all that covers
// it; neither issue slots nor HBM are full (66% and 36%, BF16, both
// directions).  So instructions count: the maxima of BF16 are taken two at a
// time (a BF16 maximum is exact), a row's scale is formed by one lane of its
// sixteen, a column's by one thread of the CTA, and an element is widened once
// for both directions.  8192 x 4096 of BF16: both directions 28.5 us (4.8
// TB/s), rows 17.3 (5.9 TB/s); FP32, 151936 x 4096 in blocks: 443 us (7.0 TB/s:
// HBM).  Rows off the 16-byte grid are read by the element (8000 x 3517: BF16
// 27.3 us, FP32 33.8; 8000 x 3520: 16.1 and 22.5).
#include <cuda_runtime.h>
#include <stdint.h>

#include <string>

#include "rlk_internal.h"
#include "rlk_ptx.cuh"

namespace rlk {
namespace {

constexpr int kQT = 128;        // tile edge: one group in either direction
constexpr int kQThreads = 256;  // 16 (columns of 8) x 16 (rows of 8)
constexpr float kE4m3Max = 448.f;
constexpr float kAmaxFloor = 7.888609052210118e-31f;  // 2^-100

struct QuantParams {
    const void* x;
    int64_t R, C, ldx;
    uint8_t *q, *qt;      // either may be NULL
    int64_t ldq, ldqt;
    float *scale, *scale_t;
    int32_t vec;  // x rows are 16-byte aligned
};

__device__ __forceinline__ void scale_of(float amax, float& s, float& r) {
    s = __fdiv_rn(fmax_nan(amax, kAmaxFloor), kE4m3Max);
    r = __fdiv_rn(1.f, s);
}

// Two FP32 values to two E4M3 codes, round to nearest even (lo in bits 0..7).
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
    uint16_t v;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(hi), "f"(lo));
    return v;
}

// The thread's 8 x 8 block, kept as it was read (BF16 pairs, or FP32).
template <bool F32>
struct Block {
    uint32_t w[8][F32 ? 8 : 4];
    __device__ __forceinline__ float at(int i, int j) const {
        if (F32) return __uint_as_float(w[i][j]);
        return (j & 1) ? bf16hi_to_f32(w[i][j >> 1]) : bf16lo_to_f32(w[i][j >> 1]);
    }
};

template <bool F32>
__device__ __forceinline__ void load_row(Block<F32>& b, int i, const QuantParams& p, int64_t r, int64_t c0) {
    constexpr int W = F32 ? 8 : 4;
    if (r >= p.R || c0 >= p.C) {
#pragma unroll
        for (int j = 0; j < W; ++j) b.w[i][j] = 0u;
        return;
    }
    if (p.vec && c0 + 8 <= p.C) {
        const char* src = static_cast<const char*>(p.x) + (r * p.ldx + c0) * (F32 ? 4 : 2);
        const uint4 v = __ldcs(reinterpret_cast<const uint4*>(src));
        b.w[i][0] = v.x, b.w[i][1] = v.y, b.w[i][2] = v.z, b.w[i][3] = v.w;
        if (F32) {
            const uint4 u = __ldcs(reinterpret_cast<const uint4*>(src) + 1);
            b.w[i][W - 4] = u.x, b.w[i][W - 3] = u.y, b.w[i][W - 2] = u.z, b.w[i][W - 1] = u.w;
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < W; ++j) {
        if (F32) {
            b.w[i][j] = c0 + j < p.C ? static_cast<const uint32_t*>(p.x)[r * p.ldx + c0 + j] : 0u;
        } else {
            const uint16_t* src = static_cast<const uint16_t*>(p.x) + r * p.ldx + c0 + 2 * j;
            const uint32_t lo = c0 + 2 * j < p.C ? src[0] : 0u, hi = c0 + 2 * j + 1 < p.C ? src[1] : 0u;
            b.w[i][j] = lo | (hi << 16);
        }
    }
}

// 8 codes of one output row: one 8-byte store where all are inside (the row
// stride is a multiple of 16 and the column of 8), single bytes at the edge.
__device__ __forceinline__ void store_codes(uint8_t* row, int64_t c0, int64_t C, uint2 v) {
    if (c0 + 8 <= C) {
        *reinterpret_cast<uint2*>(row + c0) = v;
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (c0 + j < C) row[c0 + j] = (uint8_t)((j < 4 ? v.x >> (8 * j) : v.y >> (8 * (j - 4))) & 0xFFu);
}

// Bits of |x| of two BF16; their elementwise maximum, and the larger of the two.
__device__ __forceinline__ uint32_t abs2(uint32_t w) { return w & 0x7FFF7FFFu; }
__device__ __forceinline__ float max_of(uint32_t w) { return fmax_nan(bf16lo_to_f32(w), bf16hi_to_f32(w)); }

template <bool F32, bool BLOCKS, bool TRANS>
struct TileShared {
    uint4 colmax[TRANS && !BLOCKS ? 16 : 1][F32 ? 32 : 16];  // [8 rows][8 columns' maxima, as read]
    float4 colr[TRANS && !BLOCKS ? kQT / 4 : 1];             // a column's 1 / s
    float warpmax[8];
    uint2 tile_t[TRANS ? kQT * 16 : 1];                      // [column][8-row piece ^ (column / 8)]
};

template <bool F32, bool BLOCKS, bool TRANS>
__device__ __forceinline__ void quantize_tile(const QuantParams& p, const Block<F32>& b, int64_t ct, int64_t rt,
                                              TileShared<F32, BLOCKS, TRANS>& sh) {
    const int t = threadIdx.x, cx = t & 15, ry = t >> 4;
    const int64_t r0 = rt * kQT + ry * 8, c0 = ct * kQT + cx * 8;
    constexpr int W = F32 ? 8 : 4;  // words of a row's 8 elements

    // the columns' maxima over this thread's 8 rows, word by word
    uint32_t cm[W];
    if (BLOCKS || TRANS) {
#pragma unroll
        for (int k = 0; k < W; ++k) {
            cm[k] = F32 ? b.w[0][k] & 0x7FFFFFFFu : abs2(b.w[0][k]);
#pragma unroll
            for (int i = 1; i < 8; ++i)
                cm[k] = F32 ? __float_as_uint(fmax_nan(__uint_as_float(cm[k]), fabsf(__uint_as_float(b.w[i][k]))))
                            : bf16x2_max_nan(cm[k], abs2(b.w[i][k]));
        }
    }
    float rr[8], cc[8];  // 1 / s of the thread's rows and columns
    if (BLOCKS) {
        float m;
        if (F32) {
            m = __uint_as_float(cm[0]);
#pragma unroll
            for (int k = 1; k < W; ++k) m = fmax_nan(m, __uint_as_float(cm[k]));
        } else {
            m = max_of(bf16x2_max_nan(bf16x2_max_nan(cm[0], cm[1]), bf16x2_max_nan(cm[2], cm[W - 1])));
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmax_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        if ((t & 31) == 0) sh.warpmax[t >> 5] = m;
        __syncthreads();
        m = sh.warpmax[0];
#pragma unroll
        for (int w = 1; w < 8; ++w) m = fmax_nan(m, sh.warpmax[w]);
        float s, r;
        scale_of(m, s, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) rr[i] = cc[i] = r;
        if (t == 0) {
            const int64_t RB = (p.R + kQT - 1) / kQT, CB = (p.C + kQT - 1) / kQT;
            if (p.q) p.scale[ct * RB + rt] = s;
            if (TRANS) p.scale_t[rt * CB + ct] = s;
        }
    } else {
        if (TRANS) {
            sh.colmax[ry][(F32 ? 2 : 1) * cx] = make_uint4(cm[0], cm[1], cm[2], cm[3]);
            if (F32) sh.colmax[ry][2 * cx + 1] = make_uint4(cm[W - 4], cm[W - 3], cm[W - 2], cm[W - 1]);
        }
        if (p.q) {
            // the rows' maxima over the 16 threads of a row: lane l of the sixteen forms the scale of row l mod 8
            float m;
            if (F32) {
                m = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float v = fabsf(__uint_as_float(b.w[i][0]));
#pragma unroll
                    for (int k = 1; k < W; ++k) v = fmax_nan(v, fabsf(__uint_as_float(b.w[i][k])));
#pragma unroll
                    for (int o = 8; o; o >>= 1) v = fmax_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
                    if ((cx & 7) == i) m = v;
                }
            } else {
                uint32_t pm = 0;
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    uint32_t v[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t* w = b.w[i + h];
                        v[h] = bf16x2_max_nan(bf16x2_max_nan(abs2(w[0]), abs2(w[1])),
                                              bf16x2_max_nan(abs2(w[2]), abs2(w[W - 1])));
                    }
                    // (row i, row i + 1): the lower halves' with the upper halves' maxima
                    uint32_t m2 = bf16x2_max_nan(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[0], v[1], 0x7632));
#pragma unroll
                    for (int o = 8; o; o >>= 1) m2 = bf16x2_max_nan(m2, __shfl_xor_sync(0xFFFFFFFFu, m2, o));
                    if ((cx & 6) == i) pm = m2;
                }
                m = (cx & 1) ? bf16hi_to_f32(pm) : bf16lo_to_f32(pm);
            }
            float s, r;
            scale_of(m, s, r);
            if (cx < 8 && r0 + cx < p.R) p.scale[ct * p.R + r0 + cx] = s;
#pragma unroll
            for (int i = 0; i < 8; ++i) rr[i] = __shfl_sync(0xFFFFFFFFu, r, i, 16);
        }
        if (TRANS) {
            __syncthreads();
            if (t < kQT) {
                const uint32_t* cw = reinterpret_cast<const uint32_t*>(sh.colmax);
                float m = 0.f, s, r;
                if (F32) {
#pragma unroll
                    for (int k = 0; k < 16; ++k) m = fmax_nan(m, __uint_as_float(cw[k * 128 + t]));
                } else {
                    uint32_t v = cw[t >> 1];
#pragma unroll
                    for (int k = 1; k < 16; ++k) v = bf16x2_max_nan(v, cw[k * 64 + (t >> 1)]);
                    m = (t & 1) ? bf16hi_to_f32(v) : bf16lo_to_f32(v);
                }
                scale_of(m, s, r);
                if (ct * kQT + t < p.C) p.scale_t[rt * p.C + ct * kQT + t] = s;
                reinterpret_cast<float*>(sh.colr)[t] = r;
            }
            __syncthreads();
            const float4 lo = sh.colr[2 * cx], hi = sh.colr[2 * cx + 1];
            cc[0] = lo.x, cc[1] = lo.y, cc[2] = lo.z, cc[3] = lo.w;
            cc[4] = hi.x, cc[5] = hi.y, cc[6] = hi.z, cc[7] = hi.w;
        }
    }
    // the codes, two rows at a time: along the rows for q, along the columns for qt
    uint32_t tc[8][2] = {};  // [column][rows 0-3, 4-7]
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        uint32_t code[2][2] = {};  // [row][columns 0-3, 4-7]
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float2 v[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                v[h] = make_float2(b.at(i + h, 2 * k), b.at(i + h, 2 * k + 1));
                if (p.q || BLOCKS) {
                    const float2 y = fmul2(v[h], make_float2(rr[i + h], rr[i + h]));
                    if (BLOCKS) v[h] = y;
                    code[h][k >> 1] |= pack_e4m3x2(y.x, y.y) << (16 * (k & 1));
                }
                if (TRANS && !BLOCKS) v[h] = fmul2(v[h], make_float2(cc[2 * k], cc[2 * k + 1]));
            }
            if (TRANS) {
                tc[2 * k][i >> 2] |= pack_e4m3x2(v[0].x, v[1].x) << (8 * (i & 2));
                tc[2 * k + 1][i >> 2] |= pack_e4m3x2(v[0].y, v[1].y) << (8 * (i & 2));
            }
        }
        if (p.q) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (r0 + i + h < p.R)
                    store_codes(p.q + (r0 + i + h) * p.ldq, c0, p.C, make_uint2(code[h][0], code[h][1]));
        }
    }
    if (TRANS) {
#pragma unroll
        for (int j = 0; j < 8; ++j) sh.tile_t[(cx * 8 + j) * 16 + (ry ^ cx)] = make_uint2(tc[j][0], tc[j][1]);
        __syncthreads();
        // 128 columns x 16 pieces of 8 rows, 16 consecutive threads to a column
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int col = k * 16 + ry, piece = cx;
            if (ct * kQT + col < p.C && rt * kQT + piece * 8 < p.R)
                store_codes(p.qt + (ct * kQT + col) * p.ldqt, rt * kQT + piece * 8, p.R,
                            sh.tile_t[col * 16 + (piece ^ (col >> 3))]);
        }
    }
}

template <bool F32, bool BLOCKS, bool TRANS>
__global__ void __launch_bounds__(kQThreads, F32 ? 3 : 4) quantize_kernel(const __grid_constant__ QuantParams p) {
    __shared__ TileShared<F32, BLOCKS, TRANS> sh;
    const int cx = threadIdx.x & 15, ry = threadIdx.x >> 4;
    const int64_t ct = blockIdx.x, rt = blockIdx.y + (int64_t)blockIdx.z * 65535;
    if (rt * kQT >= p.R) return;
    Block<F32> b;
#pragma unroll
    for (int i = 0; i < 8; ++i) load_row(b, i, p, rt * kQT + ry * 8 + i, ct * kQT + cx * 8);
    quantize_tile<F32, BLOCKS, TRANS>(p, b, ct, rt, sh);
}

rlk_status quant_cuda(const char* what) {
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? RLK_OK : fail(RLK_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

template <bool F32, bool BLOCKS, bool TRANS>
rlk_status launch_as(const QuantParams& p, cudaStream_t st) {
    const int64_t ct = (p.C + kQT - 1) / kQT, rt = (p.R + kQT - 1) / kQT;
    const dim3 grid((unsigned)ct, (unsigned)(rt < 65535 ? rt : 65535), (unsigned)((rt + 65534) / 65535));
    quantize_kernel<F32, BLOCKS, TRANS><<<grid, kQThreads, 0, st>>>(p);
    return quant_cuda("fp8 quantize launch");
}

template <bool F32>
rlk_status launch_typed(const QuantParams& p, bool blocks, cudaStream_t st) {
    const bool trans = p.qt != nullptr;
    if (blocks) return trans ? launch_as<F32, true, true>(p, st) : launch_as<F32, true, false>(p, st);
    return trans ? launch_as<F32, false, true>(p, st) : launch_as<F32, false, false>(p, st);
}

}  // namespace

rlk_status launch_fp8_quantize(int64_t rows, int64_t cols, const void* x, int32_t x_f32, int64_t ldx,
                               int32_t block_rows, uint8_t* q, int64_t ldq, float* scale, uint8_t* qt, int64_t ldqt,
                               float* scale_t, cudaStream_t stream) {
    QuantParams p{};
    p.x = x;
    p.R = rows;
    p.C = cols;
    p.ldx = ldx;
    p.q = q;
    p.qt = qt;
    p.ldq = ldq;
    p.ldqt = ldqt;
    p.scale = scale;
    p.scale_t = scale_t;
    p.vec = (reinterpret_cast<uintptr_t>(x) % 16 == 0) && (ldx * (x_f32 ? 4 : 2)) % 16 == 0;
    return x_f32 ? launch_typed<true>(p, block_rows == kQT, stream) : launch_typed<false>(p, block_rows == kQT, stream);
}

}  // namespace rlk
