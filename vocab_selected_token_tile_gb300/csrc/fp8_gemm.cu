// The matrix product of E4M3 operands (rlk_fp8_gemm.cuh has the kernels): its
// launches.
#include "rlk_fp8_gemm.cuh"

namespace rlk {
rlk_status launch_fp8_matmul(int64_t M, int64_t N, int64_t K, const void* a, int64_t lda, const float* sa,
                             const void* b, int64_t ldb, const float* sb, int32_t b_block_rows, void* c, int64_t ldc,
                             int32_t c_f32, int32_t accumulate, uint32_t* status, cudaStream_t stream) {
    const int sms = device_sms();
    if (sms == 0) return RLK_ERR_CUDA;
    const bool rows = b_block_rows == 1;
    Gemm8Params p{};
    p.sa = sa;
    p.sb = sb;
    p.c = c;
    p.ldc = ldc;
    p.M = (int32_t)M;
    p.N = (int32_t)N;
    p.KB = (int32_t)((K + kGK - 1) / kGK);
    p.nsb = (int32_t)(rows ? N : (N + 127) / 128);
    p.c_f32 = c_f32;
    p.accumulate = accumulate;
    p.vec = reinterpret_cast<uintptr_t>(c) % 16 == 0 && (ldc * (c_f32 ? 4 : 2)) % 16 == 0;
    p.w.status = status;
    p.w.wait_ns = kDefaultWaitNs;
    CUtensorMap ta, tb;
    // Few rows of A: the weight's rows take the lanes.  (With 65 to 128 rows a tile of 128 x 128 has more scales to
    // read and sums to keep than its share of the weight's bytes takes: 27.5 us at 128 x 16384 x 4096, the pair 24.7.)
    if (M <= 64) {
        const int nt = M <= 16 ? 16 : M <= 32 ? 32 : 64;
        p.NB = (int32_t)((N + kSRows - 1) / kSRows);
        if (!make_map8(&ta, a, K, M, lda, (uint32_t)nt) || !make_map8(&tb, b, K, N, ldb, kSRows))
            return fail(RLK_ERR_CUDA, "cuTensorMapEncodeTiled failed for an operand of the fp8 product");
        return rows ? launch_skinny_nt<true, kPlain>(nt, p, ta, tb, p.NB, sms, stream)
                    : launch_skinny_nt<false, kPlain>(nt, p, ta, tb, p.NB, sms, stream);
    }
    p.MB = (int32_t)((M + 2 * kGM - 1) / (2 * kGM));
    p.NB = (int32_t)((N + kGN - 1) / kGN);
    p.band = band_of(p.MB, K);
    if (!make_map8(&ta, a, K, M, lda, kGM) || !make_map8(&tb, b, K, N, ldb, kGN / 2))
        return fail(RLK_ERR_CUDA, "cuTensorMapEncodeTiled failed for an operand of the fp8 product");
    return rows ? launch_gemm<true, kPlain>(p, ta, tb, sms, stream) : launch_gemm<false, kPlain>(p, ta, tb, sms, stream);
}

}  // namespace rlk
