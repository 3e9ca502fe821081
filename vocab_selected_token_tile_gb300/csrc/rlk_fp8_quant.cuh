// A 128 x 128 tile's quantisation to E4M3 with one FP32 scale for each group of
// 128 (fp8_quant.cu has the definition and what bounds it), for the kernels that
// load or form its values: fp8_quant.cu, fp8_act_grad.cu.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <string>
#include <type_traits>

#include "rlk_groups.cuh"
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

// What the tile's 128 rows are: one matrix's; one of several matrices' (the
// batch: pointers moved to it, else as before); rows of a group, whose 128
// columns of the transpose are the group's own.
enum Rows8 : int { kOne, kBatch, kGroups };

struct QuantExtParams : QuantParams {
    int64_t x_b, q_b, qt_b, s_b, st_b;  // kBatch: elements between matrices
    const int32_t* ends;                // kGroups
    int32_t G;
    // the epilogue's backward: dy [R, C or C / 2] and z [R, C] instead of x
    const void* dy;
    const uint16_t* z;                  // NULL: dz = dy
    int64_t lddy, ldz;
    int32_t dy_f32, dy_vec, z_vec, act, gated;
    float* part;                        // NULL, or each tile's sums over its rows [row tile, C]
};

// Where a tile's rows lie: rows [row0, end) of x and q, columns [t0, t_end) of
// qt, row rt of scale_t.
struct RowTile {
    int64_t row0, end, t0, t_end, rt;
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
__device__ __forceinline__ void load_row(Block<F32>& b, int i, const QuantParams& p, int64_t r, int64_t end,
                                         int64_t c0) {
    constexpr int W = F32 ? 8 : 4;
    if (r >= end || c0 >= p.C) {
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
__device__ __forceinline__ void quantize_tile(const QuantParams& p, const Block<F32>& b, int64_t ct,
                                              const RowTile& at, TileShared<F32, BLOCKS, TRANS>& sh) {
    const int t = threadIdx.x, cx = t & 15, ry = t >> 4;
    const int64_t r0 = at.row0 + ry * 8, c0 = ct * kQT + cx * 8, rt = at.rt;
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
            if (cx < 8 && r0 + cx < at.end) p.scale[ct * p.R + r0 + cx] = s;
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
                if (r0 + i + h < at.end)
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
            if (ct * kQT + col < p.C && at.t0 + piece * 8 < at.t_end)
                store_codes(p.qt + (ct * kQT + col) * p.ldqt, at.t0 + piece * 8, at.t_end,
                            sh.tile_t[col * 16 + (piece ^ (col >> 3))]);
        }
    }
}

// The row tile of a group that blockIdx.y counts, false behind the last.  Each
// CTA looks it up for itself (rlk_groups.cuh).
__device__ __forceinline__ bool group_tile(const QuantExtParams& p, int64_t rt, GroupTable* tab, RowTile& at) {
    groups_build<kQThreads>(tab, p.ends, p.G, (int)p.R, kQT, 1, false);
    __syncthreads();
    if (rt >= tab->first[p.G]) return false;
    const int e = group_of(tab, p.G - 1, (int)rt);
    const int64_t row0 = tab->begin[e] + (rt - tab->first[e]) * kQT;
    at = RowTile{row0, min(row0 + kQT, (int64_t)tab->begin[e + 1]), rt * kQT, rt * kQT + kQT, rt};
    return true;
}

rlk_status quant_cuda(const char* what) {
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? RLK_OK : fail(RLK_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

dim3 tile_grid(int64_t C, int64_t row_tiles) {
    return dim3((unsigned)((C + kQT - 1) / kQT), (unsigned)(row_tiles < 65535 ? row_tiles : 65535),
                (unsigned)((row_tiles + 65534) / 65535));
}

}  // namespace
}  // namespace rlk
