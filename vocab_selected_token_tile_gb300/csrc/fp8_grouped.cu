// FP8 products of rows that belong to groups (rlk_fp8_gemm.cuh has the
// kernels): the groups' layers, and their weight gradients.
//
// The host does not know how many rows a group has, so it launches for the most
// that the sizes allow (never more CTAs than the device runs at once) and each
// CTA finds its tiles from `ends` (rlk_groups.cuh).  A group's last tile may
// load rows of the next group; they only reach rows of the accumulator that
// are not stored.
//
// Which kernel: by the average number of rows a group, all the host knows.  Few
// rows: the kernel that lays the weight's rows on the lanes, in blocks of 16,
// 32 or 64 tokens; a group with more rows takes several blocks, which run next
// to each other, so that the weight comes from L2 after the first.
#include "rlk_fp8_gemm.cuh"

namespace rlk {
namespace {

// Rows of a block of few-row units, 0: tiles of CTA pairs.
int block_rows_of(int64_t rows, int64_t groups) {
    if (rows <= 16) return 16;
    if (rows <= 6 * groups) return 16;
    if (rows <= 14 * groups) return 32;
    return rows <= 48 * groups || rows <= 64 ? 64 : 0;
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
    if (const int nt = block_rows_of(M, G)) {
        p.NB = (int32_t)((N * halves + kSRows - 1) / kSRows);
        if (!make_map8(&ta, a, K, M, lda, (uint32_t)nt) ||
            !make_map_halves(&tb, b, K, N, halves, G, ldb, group, gated ? 32 : kSRows))
            return fail(RLK_ERR_CUDA, "cuTensorMapEncodeTiled failed for an operand of the grouped fp8 product");
        const int64_t most = (live + M / nt + 1) * p.NB;
        return gated ? launch_skinny_nt<false, kRowsGated>(nt, p, ta, tb, most, sms, stream)
                     : launch_skinny_nt<false, kRows>(nt, p, ta, tb, most, sms, stream);
    }
    p.MB = 0;
    p.NB = (int32_t)((N * halves + kGN - 1) / kGN);
    const int64_t tiles = (live + M / (2 * kGM) + 1) * p.NB;
    p.band = band_of((M + 2 * kGM - 1) / (2 * kGM), K);
    if (!make_map8(&ta, a, K, M, lda, kGM) || !make_map_halves(&tb, b, K, N, halves, G, ldb, group, kGN / 2))
        return fail(RLK_ERR_CUDA, "cuTensorMapEncodeTiled failed for an operand of the grouped fp8 product");
    const int blocks = 2 * (int)(tiles < sms / 2 ? tiles : sms / 2);
    return gated ? launch_clusters<gemm_kernel<false, kRowsGated>>(blocks, kGThreads, kGSmemOf<false, kRowsGated>, 2,
                                                                   false, stream, ta, tb, p, 0, 0, 1)
                 : launch_clusters<gemm_kernel<false, kRows>>(blocks, kGThreads, kGSmemOf<false, kRows>, 2, false,
                                                              stream, ta, tb, p, 0, 0, 1);
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
    p.band = p.MB;  // a group's operands are its few tokens', which L2 holds
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
