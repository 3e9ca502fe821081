// FP8 products of rows that belong to groups (rlk_fp8_gemm.cuh has the
// kernels): the groups' layers, and their weight gradients.
//
// The host does not know how many rows a group has, so it launches for the most
// that the sizes allow (never more CTAs than the device runs at once) and each
// CTA finds its tiles from `ends` (rlk_groups.cuh).  A group's last tile may
// load rows of the next group; they only reach rows of the accumulator that
// are not stored.
//
// Which kernel: by the average number of rows a group, all the host knows.
// Measured for 64 groups of 4096 x 2048 (us; the weights' bytes take 79), rows
// spread around the average as a router spreads them:
//   rows a group                   4     8    12    16    24    32    48    64    96   128   160   192   256
//   weight's rows on lanes, 16    84    88    93    92   111
//                           32    84    87    89    89    94   100   125
//                           64    91    96   100   101   105   108   125   151   204   245
//   half tiles (128 rows)                          110   111   112   114   114   130   149   178   206   259
//   tiles (256 rows)                               159   162   162   164   165   165   167   177   189   230
// (16 groups of 2816 x 2048: 19.0, 20.6, 25.2 us for 4 rows; 22.0 and 21.5 for 16; 24.5, 28.9, 27.2 for 32; 36 and 41
// for 128, 44 and 42 for 192).  On the lanes a group with more rows than a block takes several blocks, which run next
// to each other, so that the weight comes from L2 after the first.  So a router that is far from its average costs
// little: 1024 rows of 128 groups of 2048 x 2048 (blocks of 16 rows) take 96 us in eights, 108 with half of them in one
// group, 39 with all of them in one.  (The average is of the call's rows, those behind the groups among them.)
#include "rlk_fp8_gemm.cuh"

namespace rlk {
namespace {

enum class Shape { kLanes16, kLanes32, kHalfTiles, kTiles };

Shape shape_of(int64_t rows, int64_t groups) {
    if (rows <= 10 * groups || rows <= 16) return Shape::kLanes16;
    if (rows <= 36 * groups) return Shape::kLanes32;
    return rows <= 152 * groups ? Shape::kHalfTiles : Shape::kTiles;
}

template <int KIND>
rlk_status launch_group_tiles(const Ext8Params& p, const CUtensorMap& a, const CUtensorMap& b, int64_t tiles, int sms,
                              cudaStream_t st) {
    const int pairs = (int)(tiles < sms / 2 ? tiles : sms / 2);
    return launch_clusters<gemm_kernel<false, KIND>>(2 * pairs, kGThreads, kGSmemOf<false, KIND>, 2, false, st, a, b, p,
                                                     0, 0, 1);
}

}  // namespace

rlk_status launch_fp8_grouped_matmul(int64_t G, int64_t M, int64_t N, int64_t K, const int32_t* ends, const void* a,
                                     int64_t lda, const float* sa, const void* b, int64_t ldb, int64_t group,
                                     const float* sb, const rlk_fp8_epilogue* e, void* c, int64_t ldc, int32_t c_f32,
                                     int32_t rest, uint32_t* status, cudaStream_t stream) {
    const int sms = device_sms();
    if (sms == 0) return RLK_ERR_CUDA;
    Ext8Params p{};
    set_epilogue(p, e, N);
    p.sa = sa;
    p.sb = sb;
    p.c = c;
    p.ldc = ldc;
    p.M = (int32_t)M;
    p.N = (int32_t)N;
    p.KB = (int32_t)((K + kGK - 1) / kGK);
    p.c_f32 = c_f32;
    p.vec = reinterpret_cast<uintptr_t>(c) % 16 == 0 && (ldc * (c_f32 ? 4 : 2)) % 16 == 0;
    p.ends = ends;
    p.G = (int32_t)G;
    p.rest = rest;
    p.sb_g = (int64_t)p.KB * p.nsb;
    p.w.status = status;
    p.w.wait_ns = kDefaultWaitNs;
    const bool gated = e && e->gated;
    const int halves = gated ? 2 : 1;
    const int64_t live = G < M ? G : M;  // groups that have rows, at most
    CUtensorMap ta, tb;
    const Shape shape = shape_of(M, G);
    if (shape == Shape::kLanes16 || shape == Shape::kLanes32) {
        const int nt = shape == Shape::kLanes16 ? 16 : 32;
        p.NB = (int32_t)((N * halves + kSRows - 1) / kSRows);
        if (!make_map8(&ta, a, K, M, lda, (uint32_t)nt) ||
            !make_map_halves(&tb, b, K, N, halves, G, ldb, group, gated ? 32 : kSRows))
            return fail(RLK_ERR_CUDA, "cuTensorMapEncodeTiled failed for an operand of the grouped fp8 product");
        const int64_t most = (live + M / nt + 1) * p.NB;
        return gated ? launch_skinny_nt<false, kRowsGated>(nt, p, ta, tb, most, sms, stream)
                     : launch_skinny_nt<false, kRows>(nt, p, ta, tb, most, sms, stream);
    }
    const int rows = shape == Shape::kHalfTiles ? kGM : 2 * kGM;  // of a tile
    p.NB = (int32_t)((N * halves + kGN - 1) / kGN);
    p.band = band_of((M + 2 * kGM - 1) / (2 * kGM), K) * (2 * kGM / rows);
    const int64_t tiles = (live + M / rows + 1) * p.NB;
    if (!make_map8(&ta, a, K, M, lda, (uint32_t)rows / 2) ||
        !make_map_halves(&tb, b, K, N, halves, G, ldb, group, kGN / 2))
        return fail(RLK_ERR_CUDA, "cuTensorMapEncodeTiled failed for an operand of the grouped fp8 product");
    if (shape == Shape::kHalfTiles)
        return gated ? launch_group_tiles<kHalvesGated>(p, ta, tb, tiles, sms, stream)
                     : launch_group_tiles<kHalves>(p, ta, tb, tiles, sms, stream);
    return gated ? launch_group_tiles<kRowsGated>(p, ta, tb, tiles, sms, stream)
                 : launch_group_tiles<kRows>(p, ta, tb, tiles, sms, stream);
}

rlk_status launch_fp8_grouped_dweight(int64_t G, int64_t rows, int64_t M, int64_t N, const int32_t* ends,
                                      const void* a, int64_t lda, const float* sa, const void* b, int64_t ldb,
                                      const float* sb, void* c, int64_t ldc, int64_t group, int32_t c_f32,
                                      int32_t accumulate, uint32_t* status, cudaStream_t stream) {
    const int sms = device_sms();
    if (sms == 0) return RLK_ERR_CUDA;
    Ext8Params p{};
    p.sa = sa;
    p.sb = sb;
    p.c = c;
    p.ldc = ldc;
    p.M = (int32_t)M;
    p.N = (int32_t)N;
    p.nsb = (int32_t)N;
    p.KB = (int32_t)(rows / kGK + (G < rows ? G : rows));
    p.c_f32 = c_f32;
    p.accumulate = accumulate;
    p.vec = reinterpret_cast<uintptr_t>(c) % 16 == 0 && (ldc * (c_f32 ? 4 : 2)) % 16 == 0 &&
            (group * (c_f32 ? 4 : 2)) % 16 == 0;
    p.ends = ends;
    p.G = (int32_t)G;
    p.deep = (int32_t)rows;
    p.c_g = group;
    p.MB = (int32_t)((M + 2 * kGM - 1) / (2 * kGM));
    p.NB = (int32_t)((N + kGN - 1) / kGN);
    // A group's operands are its few tokens', which L2 holds.  32 groups of 512 tokens, 2816 x 2048 of BF16: 219 us, the
    // floors 50 (FP8 products) and 92 (369 MB written, at the 4.0 TB/s of a fill): 4 to 5 K groups of 1,250 clocks a
    // tile, and 5,000 to store it that nothing covers.  128 groups of 16 tokens, 2048 x 4096: 689 us, 2.1 GB written (a
    // fill: 517).  Half tiles were slower (247 and 738 us).
    p.band = p.MB;
    p.w.status = status;
    p.w.wait_ns = kDefaultWaitNs;
    const int64_t deep = (int64_t)kGK * p.KB, tiles = G * p.MB * p.NB;
    CUtensorMap ta, tb;
    if (!make_map8(&ta, a, deep, M, lda, kGM) || !make_map8(&tb, b, deep, N, ldb, kGN / 2))
        return fail(RLK_ERR_CUDA, "cuTensorMapEncodeTiled failed for an operand of the grouped weight gradient");
    return launch_clusters<gemm_kernel<true, kDepth>>(2 * (int)(tiles < sms / 2 ? tiles : sms / 2), kGThreads,
                                                      kGSmemOf<true, kDepth>, 2, false, stream, ta, tb, p, 0,
                                                      (int)tiles, 1);
}

}  // namespace rlk
