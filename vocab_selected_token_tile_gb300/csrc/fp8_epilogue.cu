// The FP8 product with a feed-forward layer's epilogue (rlk_fp8_gemm.cuh has
// the kernels): its launches.
#include "rlk_fp8_gemm.cuh"

namespace rlk {

rlk_status launch_fp8_matmul_act(int64_t M, int64_t N, int64_t K, const void* a, int64_t lda, const float* sa,
                                 const void* b, int64_t ldb, const float* sb, const rlk_fp8_epilogue* e, void* c,
                                 int64_t ldc, int32_t c_f32, uint32_t* status, cudaStream_t stream) {
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
    p.w.status = status;
    p.w.wait_ns = kDefaultWaitNs;
    const bool gated = e && e->gated;
    const int halves = gated ? 2 : 1;
    CUtensorMap ta, tb;
    if (M <= 64) {  // as for the product by itself
        const int nt = M <= 16 ? 16 : M <= 32 ? 32 : 64;
        p.NB = (int32_t)((N * halves + kSRows - 1) / kSRows);
        if (!make_map8(&ta, a, K, M, lda, (uint32_t)nt) ||
            !make_map_halves(&tb, b, K, N, halves, 1, ldb, 0, gated ? 32 : kSRows))
            return fail(RLK_ERR_CUDA, "cuTensorMapEncodeTiled failed for an operand of the fp8 product");
        return gated ? launch_skinny_nt<false, kEpiGated>(nt, p, ta, tb, p.NB, sms, stream)
                     : launch_skinny_nt<false, kEpi>(nt, p, ta, tb, p.NB, sms, stream);
    }
    p.MB = (int32_t)((M + 2 * kGM - 1) / (2 * kGM));
    p.NB = (int32_t)((N * halves + kGN - 1) / kGN);
    p.band = band_of(p.MB, K);
    if (!make_map8(&ta, a, K, M, lda, kGM) || !make_map_halves(&tb, b, K, N, halves, 1, ldb, 0, kGN / 2))
        return fail(RLK_ERR_CUDA, "cuTensorMapEncodeTiled failed for an operand of the fp8 product");
    return gated ? launch_gemm<false, kEpiGated>(p, ta, tb, sms, stream) : launch_gemm<false, kEpi>(p, ta, tb, sms, stream);
}

}  // namespace rlk
