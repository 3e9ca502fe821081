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
#include <type_traits>

#include "rlk_act.cuh"
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

// 8 consecutive elements of a row in FP32, zero from `left` on.
__device__ __forceinline__ void load8(float (&v)[8], const void* x, int64_t at, bool f32, bool vec, int64_t left) {
    if (vec && left >= 8) {
        if (f32) {
            const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
            const float4 a = __ldcs(s), b = __ldcs(s + 1);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
            const uint4 a = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at));
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) v[2 * j] = bf16lo_to_f32(w[j]), v[2 * j + 1] = bf16hi_to_f32(w[j]);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = j >= left ? 0.f
               : f32     ? static_cast<const float*>(x)[at + j]
                         : __uint_as_float((uint32_t) static_cast<const uint16_t*>(x)[at + j] << 16);
}

// Two values of dz; `up` the gate's other half (or of no use).
template <int ACT, bool GATED>
__device__ __forceinline__ float2 dz_of(float2 dy, float2 z, float2 up, bool other) {
    if (GATED) return other ? fmul2(dy, act_pair<ACT>(z)) : fmul2(fmul2(dy, up), act_slope_pair<ACT>(z));
    return ACT == RLK_ACT_NONE ? dy : fmul2(dy, act_slope_pair<ACT>(z));
}

// Row i of the thread's block of dz, 8 columns from c0 on (of one half: C / 2 is
// a multiple of 64).  Gated: columns [0, C / 2) are the gate's.
template <int ACT, bool GATED>
__device__ __forceinline__ void load_dz_row(Block<true>& b, int i, const QuantExtParams& p, int64_t r, int64_t end,
                                            int64_t c0) {
    const int64_t N = GATED ? p.C / 2 : p.C;
    const bool other = GATED && c0 >= N;
    const int64_t c = other ? c0 - N : c0, left = c0 < p.C ? N - c : 0;
    if (r >= end || left <= 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) b.w[i][j] = 0u;
        return;
    }
    float dy[8], z[8] = {}, up[8] = {};
    load8(dy, p.dy, r * p.lddy + c, p.dy_f32, p.dy_vec, left);
    if (ACT != RLK_ACT_NONE || GATED) load8(z, p.z, r * p.ldz + c, false, p.z_vec, left);
    if (GATED && !other) load8(up, p.z, r * p.ldz + N + c, false, p.z_vec, left);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const float2 d = dz_of<ACT, GATED>(make_float2(dy[j], dy[j + 1]), make_float2(z[j], z[j + 1]),
                                           make_float2(up[j], up[j + 1]), other);
        b.w[i][j] = j < left ? __float_as_uint(d.x) : 0u;
        b.w[i][j + 1] = j + 1 < left ? __float_as_uint(d.y) : 0u;
    }
}

// The thread's 8 rows of it: BF16 on the 16-byte grid by four rows' loads at a
// time (a row at a time the tile was a chain of eight memory latencies: 4096 x
// 6144 gated 145 us, XX so).
template <int ACT, bool GATED>
__device__ __forceinline__ void load_dz(Block<true>& b, const QuantExtParams& p, int64_t r0, int64_t end, int64_t c0) {
    const int64_t N = GATED ? p.C / 2 : p.C;
    const bool other = GATED && c0 >= N;
    const int64_t c = other ? c0 - N : c0;
    if (p.dy_f32 || !p.dy_vec || (!p.z_vec && (ACT != RLK_ACT_NONE || GATED)) || c + 8 > N) {
#pragma unroll
        for (int i = 0; i < 8; ++i) load_dz_row<ACT, GATED>(b, i, p, r0 + i, end, c0);
        return;
    }
    const uint16_t *dy = static_cast<const uint16_t*>(p.dy) + r0 * p.lddy + c, *z = p.z + r0 * p.ldz + c;
    const int rows = (int)min((int64_t)8, end - r0);
#pragma unroll
    for (int h = 0; h < 8; h += 4) {
        uint4 d[4], a[4], u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            d[i] = a[i] = u[i] = make_uint4(0, 0, 0, 0);
            if (h + i < rows) {
                d[i] = __ldcs(reinterpret_cast<const uint4*>(dy + (h + i) * p.lddy));
                if (ACT != RLK_ACT_NONE || GATED) a[i] = __ldcs(reinterpret_cast<const uint4*>(z + (h + i) * p.ldz));
                if (GATED && !other) u[i] = __ldcs(reinterpret_cast<const uint4*>(z + (h + i) * p.ldz + N));
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t wd[4] = {d[i].x, d[i].y, d[i].z, d[i].w}, wa[4] = {a[i].x, a[i].y, a[i].z, a[i].w};
            const uint32_t wu[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                auto two = [](uint32_t w) { return make_float2(bf16lo_to_f32(w), bf16hi_to_f32(w)); };
                const float2 v = dz_of<ACT, GATED>(two(wd[k]), two(wa[k]), two(wu[k]), other);
                b.w[h + i][2 * k] = __float_as_uint(v.x), b.w[h + i][2 * k + 1] = __float_as_uint(v.y);
            }
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

template <bool F32, bool BLOCKS, bool TRANS>
__global__ void __launch_bounds__(kQThreads, F32 ? 3 : 4) quantize_kernel(const __grid_constant__ QuantParams p) {
    __shared__ TileShared<F32, BLOCKS, TRANS> sh;
    const int cx = threadIdx.x & 15, ry = threadIdx.x >> 4;
    const int64_t ct = blockIdx.x, rt = blockIdx.y + (int64_t)blockIdx.z * 65535;
    if (rt * kQT >= p.R) return;
    Block<F32> b;
#pragma unroll
    for (int i = 0; i < 8; ++i) load_row(b, i, p, rt * kQT + ry * 8 + i, p.R, ct * kQT + cx * 8);
    quantize_tile<F32, BLOCKS, TRANS>(p, b, ct, RowTile{rt * kQT, p.R, rt * kQT, p.R, rt}, sh);
}

// The row tile of a group that blockIdx.y counts, false behind the last.  Each
// CTA looks it up for itself (rlk_groups.cuh), 0.5 us beside its own chain of 3.
__device__ __forceinline__ bool group_tile(const QuantExtParams& p, int64_t rt, GroupTable* tab, RowTile& at) {
    groups_build<kQThreads>(tab, p.ends, p.G, (int)p.R, kQT, 1, false);
    __syncthreads();
    if (rt >= tab->first[p.G]) return false;
    const int e = group_of(tab, p.G - 1, (int)rt);
    const int64_t row0 = tab->begin[e] + (rt - tab->first[e]) * kQT;
    at = RowTile{row0, min(row0 + kQT, (int64_t)tab->begin[e + 1]), rt * kQT, rt * kQT + kQT, rt};
    return true;
}

// Rows of groups, and several matrices, from x.
template <bool F32, bool TRANS, int ROWS>
__global__ void __launch_bounds__(kQThreads, F32 ? 3 : 4)
    quantize_ext_kernel(const __grid_constant__ QuantExtParams p0) {
    constexpr bool kBlocks = ROWS == kBatch;
    __shared__ TileShared<F32, kBlocks, TRANS> sh;
    __shared__ typename std::conditional<ROWS == kGroups, GroupTable, int>::type tab;
    const int cx = threadIdx.x & 15, ry = threadIdx.x >> 4;
    const int64_t ct = blockIdx.x, rt = blockIdx.y + (int64_t)blockIdx.z * 65535;
    QuantParams p = p0;
    RowTile at;
    if constexpr (ROWS == kGroups) {
        if (!group_tile(p0, rt, &tab, at)) return;
    } else {
        const int64_t tiles = (p.R + kQT - 1) / kQT, k = rt / tiles, r = rt - k * tiles;
        if (k >= p0.G) return;
        p.x = static_cast<const char*>(p.x) + k * p0.x_b * (F32 ? 4 : 2);
        if (p.q) p.q += k * p0.q_b, p.scale += k * p0.s_b;
        if (TRANS) p.qt += k * p0.qt_b, p.scale_t += k * p0.st_b;
        at = RowTile{r * kQT, p.R, r * kQT, p.R, r};
    }
    Block<F32> b;
#pragma unroll
    for (int i = 0; i < 8; ++i) load_row(b, i, p, at.row0 + ry * 8 + i, at.end, ct * kQT + cx * 8);
    quantize_tile<F32, kBlocks, TRANS>(p, b, ct, at, sh);
}

// The epilogue's backward.
template <bool TRANS, int ROWS, int ACT, bool GATED>
__global__ void __launch_bounds__(kQThreads, 2) act_grad_kernel(const __grid_constant__ QuantExtParams p) {
    __shared__ TileShared<true, false, TRANS> sh;
    __shared__ typename std::conditional<ROWS == kGroups, GroupTable, int>::type tab;
    __shared__ float4 sums[16][kQT / 4];
    const int cx = threadIdx.x & 15, ry = threadIdx.x >> 4;
    const int64_t ct = blockIdx.x, rt = blockIdx.y + (int64_t)blockIdx.z * 65535;
    RowTile at;
    if constexpr (ROWS == kGroups) {
        if (!group_tile(p, rt, &tab, at)) return;
    } else {
        if (rt * kQT >= p.R) return;
        at = RowTile{rt * kQT, p.R, rt * kQT, p.R, rt};
    }
    Block<true> b;
    load_dz<ACT, GATED>(b, p, at.row0 + ry * 8, at.end, ct * kQT + cx * 8);
    if (p.part) {
        float s[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            s[j] = b.at(0, j);
#pragma unroll
            for (int i = 1; i < 8; ++i) s[j] = __fadd_rn(s[j], b.at(i, j));
        }
        sums[ry][2 * cx] = make_float4(s[0], s[1], s[2], s[3]);
        sums[ry][2 * cx + 1] = make_float4(s[4], s[5], s[6], s[7]);
        __syncthreads();
        if (threadIdx.x < kQT && ct * kQT + threadIdx.x < p.C) {
            float v = 0.f;
#pragma unroll
            for (int k = 0; k < 16; ++k)
                v = __fadd_rn(v, reinterpret_cast<const float*>(sums[k])[threadIdx.x]);
            p.part[rt * p.C + ct * kQT + threadIdx.x] = v;
        }
    }
    if (p.q || TRANS) quantize_tile<true, false, TRANS>(p, b, ct, at, sh);
}

// dbias from the row tiles' sums: a warp of 32 columns, eight runs of a group's
// tiles at a time, joined in order.
template <int ROWS>
__global__ void __launch_bounds__(kQThreads) bias_grad_kernel(const __grid_constant__ QuantExtParams p, void* dbias,
                                                              const int f32) {
    __shared__ typename std::conditional<ROWS == kGroups, GroupTable, int>::type tab;
    __shared__ float join[8][32];
    const int run = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    if constexpr (ROWS == kGroups) {
        groups_build<kQThreads>(&tab, p.ends, p.G, (int)p.R, kQT, 1, false);
        __syncthreads();
    }
    for (int e = blockIdx.y; e < (ROWS == kGroups ? p.G : 1); e += gridDim.y) {
        int64_t t0 = 0, t1 = (p.R + kQT - 1) / kQT;
        if constexpr (ROWS == kGroups) t0 = tab.first[e], t1 = tab.first[e + 1];
        const int64_t lo = t0 + (t1 - t0) * run / 8, hi = t0 + (t1 - t0) * (run + 1) / 8;
        float v = 0.f;
        if (c < p.C) {
#pragma unroll 4
            for (int64_t t = lo; t < hi; ++t) v = __fadd_rn(v, p.part[t * p.C + c]);
        }
        join[run][lane] = v;
        __syncthreads();
        if (run == 0 && c < p.C) {
#pragma unroll
            for (int k = 1; k < 8; ++k) v = __fadd_rn(v, join[k][lane]);
            if (f32)
                static_cast<float*>(dbias)[e * p.C + c] = v;
            else
                static_cast<uint16_t*>(dbias)[e * p.C + c] = (uint16_t)pack_bf16x2_rn(v, 0.f);
        }
        __syncthreads();
    }
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

dim3 tile_grid(int64_t C, int64_t row_tiles) {
    return dim3((unsigned)((C + kQT - 1) / kQT), (unsigned)(row_tiles < 65535 ? row_tiles : 65535),
                (unsigned)((row_tiles + 65534) / 65535));
}

template <int ROWS>
rlk_status launch_ext(const QuantExtParams& p, bool f32, int64_t row_tiles, cudaStream_t st) {
    const dim3 grid = tile_grid(p.C, row_tiles);
    if (f32)
        p.qt ? quantize_ext_kernel<true, true, ROWS><<<grid, kQThreads, 0, st>>>(p)
             : quantize_ext_kernel<true, false, ROWS><<<grid, kQThreads, 0, st>>>(p);
    else
        p.qt ? quantize_ext_kernel<false, true, ROWS><<<grid, kQThreads, 0, st>>>(p)
             : quantize_ext_kernel<false, false, ROWS><<<grid, kQThreads, 0, st>>>(p);
    return quant_cuda("fp8 quantize launch");
}

template <bool TRANS, int ROWS, bool GATED>
void launch_act(const QuantExtParams& p, dim3 grid, cudaStream_t st) {
    auto go = [&](auto kernel) { kernel<<<grid, kQThreads, 0, st>>>(p); };
    switch (p.act) {
        case RLK_ACT_RELU: return go(act_grad_kernel<TRANS, ROWS, RLK_ACT_RELU, GATED>);
        case RLK_ACT_SILU: return go(act_grad_kernel<TRANS, ROWS, RLK_ACT_SILU, GATED>);
        case RLK_ACT_GELU: return go(act_grad_kernel<TRANS, ROWS, RLK_ACT_GELU, GATED>);
        case RLK_ACT_GELU_TANH: return go(act_grad_kernel<TRANS, ROWS, RLK_ACT_GELU_TANH, GATED>);
        default: return go(act_grad_kernel<TRANS, ROWS, RLK_ACT_NONE, GATED>);
    }
}

template <int ROWS>
rlk_status launch_act_rows(const QuantExtParams& p, int64_t row_tiles, void* dbias, bool f32, cudaStream_t st) {
    const dim3 grid = tile_grid(p.C, row_tiles);
    if (p.gated)
        p.qt ? launch_act<true, ROWS, true>(p, grid, st) : launch_act<false, ROWS, true>(p, grid, st);
    else
        p.qt ? launch_act<true, ROWS, false>(p, grid, st) : launch_act<false, ROWS, false>(p, grid, st);
    rlk_status s = quant_cuda("fp8 activation gradient launch");
    if (s != RLK_OK || !dbias) return s;
    const dim3 sums((unsigned)((p.C + 31) / 32), (unsigned)(p.G < 1 ? 1 : p.G < 32 ? p.G : 32));
    bias_grad_kernel<ROWS><<<sums, kQThreads, 0, st>>>(p, dbias, f32);
    return quant_cuda("bias gradient launch");
}

}  // namespace

// Row tiles that any counts of the groups' rows can ask for.
int64_t group_row_tiles(int64_t groups, int64_t rows) { return rows / kQT + (groups < rows ? groups : rows); }

rlk_status launch_fp8_quantize_grouped(int64_t G, int64_t rows, int64_t cols, const int32_t* ends, const void* x,
                                       int32_t x_f32, int64_t ldx, uint8_t* q, int64_t ldq, float* scale, uint8_t* qt,
                                       int64_t ldqt, float* scale_t, cudaStream_t stream) {
    QuantExtParams p{};
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
    p.ends = ends;
    p.G = (int32_t)G;
    return launch_ext<kGroups>(p, x_f32, group_row_tiles(G, rows), stream);
}

rlk_status launch_fp8_quantize_batch(int64_t count, int64_t rows, int64_t cols, const void* x, int32_t x_f32,
                                     int64_t ldx, int64_t x_b, uint8_t* q, int64_t ldq, int64_t q_b, float* scale,
                                     uint8_t* qt, int64_t ldqt, int64_t qt_b, float* scale_t, cudaStream_t stream) {
    QuantExtParams p{};
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
    p.x_b = x_b;
    p.q_b = q_b;
    p.qt_b = qt_b;
    p.s_b = p.st_b = ((rows + kQT - 1) / kQT) * ((cols + kQT - 1) / kQT);
    p.vec = (reinterpret_cast<uintptr_t>(x) % 16 == 0) && (ldx * (x_f32 ? 4 : 2)) % 16 == 0 &&
            (x_b * (x_f32 ? 4 : 2)) % 16 == 0;
    p.G = (int32_t)count;
    return launch_ext<kBatch>(p, x_f32, count * ((rows + kQT - 1) / kQT), stream);
}

rlk_status launch_fp8_act_grad(int64_t G, int64_t rows, int64_t wide, const int32_t* ends, const void* dy,
                               int32_t dy_f32, int64_t lddy, const void* z, int64_t ldz, int32_t act, int32_t gated,
                               uint8_t* q, int64_t ldq, float* scale, uint8_t* qt, int64_t ldqt, float* scale_t,
                               void* dbias, int32_t dbias_f32, float* part, cudaStream_t stream) {
    QuantExtParams p{};
    p.R = rows;
    p.C = wide;
    p.q = q;
    p.qt = qt;
    p.ldq = ldq;
    p.ldqt = ldqt;
    p.scale = scale;
    p.scale_t = scale_t;
    p.ends = ends;
    p.G = (int32_t)G;
    p.dy = dy;
    p.dy_f32 = dy_f32;
    p.lddy = lddy;
    p.dy_vec = (reinterpret_cast<uintptr_t>(dy) % 16 == 0) && (lddy * (dy_f32 ? 4 : 2)) % 16 == 0;
    p.z = static_cast<const uint16_t*>(z);
    p.ldz = ldz;
    p.z_vec = (reinterpret_cast<uintptr_t>(z) % 16 == 0) && (ldz * 2) % 16 == 0;
    p.act = act;
    p.gated = gated;
    p.part = dbias ? part : nullptr;
    return G > 0 ? launch_act_rows<kGroups>(p, group_row_tiles(G, rows), dbias, dbias_f32, stream)
                 : launch_act_rows<kOne>(p, (rows + kQT - 1) / kQT, dbias, dbias_f32, stream);
}

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
