// Quantisation to E4M3 with one FP32 scale for each group of 128 (sm_103a):
// the operands of the FP8 products (rlk_fp8_gemm.cuh).
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
//
// Several matrices (a batch: experts' weights) are the same tiles with the
// pointers moved: 32 of 2816 x 2048, BF16, both directions 116 us (738 MB, 6.4
// TB/s).  Rows that belong to groups: a tile is up to 128 rows of one group, so
// that the transpose's groups of 128 are the group's own; each CTA looks its tile
// up by itself, which takes 18% of its time: 16384 rows of 32 groups x 2048, both
// directions 34 us, without groups 28.6 (looking up once for two or four tiles of
// columns was no faster).
#include "rlk_fp8_quant.cuh"

namespace rlk {
namespace {

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
