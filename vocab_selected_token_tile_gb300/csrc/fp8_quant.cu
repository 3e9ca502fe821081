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
#include <cuda_runtime.h>
#include <stdint.h>

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

__device__ __forceinline__ uint2 pack_e4m3x8(const float (&v)[8]) {
    return make_uint2(pack_e4m3x2(v[0], v[1]) | (pack_e4m3x2(v[2], v[3]) << 16),
                      pack_e4m3x2(v[4], v[5]) | (pack_e4m3x2(v[6], v[7]) << 16));
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

template <bool F32, bool BLOCKS, bool TRANS>
__global__ void __launch_bounds__(kQThreads, F32 ? 2 : 4) quantize_kernel(const __grid_constant__ QuantParams p) {
    __shared__ float colmax[TRANS && !BLOCKS ? 16 : 1][kQT];
    __shared__ float warpmax[8];
    __shared__ uint2 tile_t[TRANS ? kQT * 16 : 1];  // [column][8-row piece ^ (column / 8)]
    const int t = threadIdx.x, cx = t & 15, ry = t >> 4;
    const int64_t ct = blockIdx.x, rt = blockIdx.y + (int64_t)blockIdx.z * 65535;
    const int64_t r0 = rt * kQT + ry * 8, c0 = ct * kQT + cx * 8;
    if (rt * kQT >= p.R) return;

    Block<F32> b;
#pragma unroll
    for (int i = 0; i < 8; ++i) load_row(b, i, p, r0 + i, c0);

    float bs = 0.f, br = 0.f;  // the block's scale and reciprocal (BLOCKS)
    if (BLOCKS) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) m = fmax_nan(m, fabsf(b.at(i, j)));
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmax_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        if ((t & 31) == 0) warpmax[t >> 5] = m;
        __syncthreads();
        m = warpmax[0];
#pragma unroll
        for (int w = 1; w < 8; ++w) m = fmax_nan(m, warpmax[w]);
        scale_of(m, bs, br);
        if (t == 0) {
            const int64_t RB = (p.R + kQT - 1) / kQT, CB = (p.C + kQT - 1) / kQT;
            if (p.q) p.scale[ct * RB + rt] = bs;
            if (TRANS) p.scale_t[rt * CB + ct] = bs;
        }
    }
    if (p.q) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float r = br;
            if (!BLOCKS) {
                float m = 0.f, s;
#pragma unroll
                for (int j = 0; j < 8; ++j) m = fmax_nan(m, fabsf(b.at(i, j)));
#pragma unroll
                for (int o = 8; o; o >>= 1) m = fmax_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
                scale_of(m, s, r);
                if (cx == 0 && r0 + i < p.R) p.scale[ct * p.R + r0 + i] = s;
            }
            if (r0 + i < p.R) {
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(b.at(i, j), r);
                store_codes(p.q + (r0 + i) * p.ldq, c0, p.C, pack_e4m3x8(v));
            }
        }
    }
    if (TRANS) {
        if (!BLOCKS) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float m = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) m = fmax_nan(m, fabsf(b.at(i, j)));
                colmax[ry][cx * 8 + j] = m;
            }
            __syncthreads();
            if (t < kQT) {
                float m = colmax[0][t], s, r;
#pragma unroll
                for (int k = 1; k < 16; ++k) m = fmax_nan(m, colmax[k][t]);
                scale_of(m, s, r);
                if (ct * kQT + t < p.C) p.scale_t[rt * p.C + ct * kQT + t] = s;
                colmax[0][t] = r;  // only this thread reads column t's entries
            }
            __syncthreads();
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float r = BLOCKS ? br : colmax[0][cx * 8 + j];
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(b.at(i, j), r);
            tile_t[(cx * 8 + j) * 16 + (ry ^ cx)] = pack_e4m3x8(v);
        }
        __syncthreads();
        // 128 columns x 16 pieces of 8 rows, 16 consecutive threads to a column
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int col = k * 16 + ry, piece = cx;
            if (ct * kQT + col < p.C && rt * kQT + piece * 8 < p.R)
                store_codes(p.qt + (ct * kQT + col) * p.ldqt, rt * kQT + piece * 8, p.R,
                            tile_t[col * 16 + (piece ^ (col >> 3))]);
        }
    }
}

template <bool F32>
void launch_typed(const QuantParams& p, bool blocks, dim3 grid, cudaStream_t st) {
    const bool trans = p.qt != nullptr;
    if (blocks)
        trans ? quantize_kernel<F32, true, true><<<grid, kQThreads, 0, st>>>(p)
              : quantize_kernel<F32, true, false><<<grid, kQThreads, 0, st>>>(p);
    else
        trans ? quantize_kernel<F32, false, true><<<grid, kQThreads, 0, st>>>(p)
              : quantize_kernel<F32, false, false><<<grid, kQThreads, 0, st>>>(p);
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
    const int64_t ct = (cols + kQT - 1) / kQT, rt = (rows + kQT - 1) / kQT;
    const dim3 grid((unsigned)ct, (unsigned)(rt < 65535 ? rt : 65535), (unsigned)((rt + 65534) / 65535));
    if (x_f32)
        launch_typed<true>(p, block_rows == kQT, grid, stream);
    else
        launch_typed<false>(p, block_rows == kQT, grid, stream);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(RLK_ERR_CUDA, std::string("fp8 quantize launch: ") + cudaGetErrorString(e));
    return RLK_OK;
}

}  // namespace rlk
