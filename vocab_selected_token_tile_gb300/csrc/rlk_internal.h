// Internal declarations shared by the C ABI (rlk_api.cu) and the kernels'
// launch planners.  Not part of the public interface.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <string>

#include "rlk_logp.h"

namespace rlk {

// Device status word bits (written by kernels with atomicOr, read by the host).
enum : uint32_t {
    kStatusTargetRange = 1u << 0,
    kStatusNonFinite = 1u << 1,
    kStatusTimeout = 1u << 2,
    kStatusInternal = 1u << 3,  // a kernel found its own bookkeeping inconsistent and stopped
};

constexpr int kMaxTiles = 1024;
constexpr int64_t kMaxTileCols = 16384;
constexpr uint64_t kDefaultWaitNs = 2000000000ull;  // 2 s
constexpr size_t kWorkspaceBytes = 256;

// kModeFused is what callers ask for; the planner runs it as kModeFusedL2
// (second read of each row from L2) unless RLK_FUSED_SCHEDULE=resident.
enum StreamMode : int { kModeFwd = 0, kModeBwd = 1, kModeFused = 2, kModeFusedL2 = 3 };

// Arguments of one streaming launch (all device pointers).
struct StreamArgs {
    const uint16_t* logits;
    uint16_t* dlogits;
    const int64_t* targets;
    const uint8_t* mask;
    const float* grad;
    const float* lse_in;
    float* logp;
    float* lse;
    float* partials;
    float* entropy;  // optional (forward): entropy of each row's softmax
    uint32_t* status;
    // kModeBwd on one vocabulary shard: an active row's target may lie in
    // another shard (any value outside [0, V_real) of this launch); it then
    // takes no one-hot term here and is not an error.
    int32_t foreign_targets;
    // The fused GRPO step (kModeFusedL2): instead of reading g, each row's g
    // is formed on chip from its logp once the fold has it,
    //   g_r = mask_r (-A_r + beta (1 - exp(ref_r - logp_r))) / N
    // (no KL term without ref), in the same FP32 operations as the GRPO loss
    // kernel, and written to grad_out.  n_active holds N.
    int32_t grpo;
    const float* adv;
    const float* ref;
    float beta;
    const unsigned long long* n_active;
    float* grad_out;
};

// Allows a kernel its dynamic shared memory, once a kernel and device (the
// call costs about as much host time as a launch's arguments).
template <auto KERNEL>
bool allow_dynamic_smem(size_t bytes) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    if (dev < 64 && (done.load(std::memory_order_acquire) >> dev & 1)) return true;
    if (cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess)
        return false;
    if (dev < 64) done.fetch_or(1ull << dev, std::memory_order_release);
    return true;
}

// Records a failure reason for rlk_last_error_message() and returns `s`.
rlk_status fail(rlk_status s, const std::string& why);

// Host check of the planner overrides in the environment (RLK_CTAS_PER_SM,
// RLK_ROW_BUFS, RLK_FUSED_SKEW, RLK_FUSED_SCHEDULE): RLK_ERR_UNSUPPORTED for
// any value outside the ring shapes the protocol model replays.
rlk_status check_planner_env();

// Launches one streaming kernel (mode kModeFwd / kModeBwd / kModeFused) for a
// validated contract; returns RLK_OK or an error with the message set.
rlk_status launch_stream(const rlk_logp_contract& c, int mode, const StreamArgs& a, cudaStream_t stream);

// Fused lm_head (lmhead.cu): host checks, workspace bytes beyond the status
// area, and the forward launch (GEMM + epilogue partials, then the fold).
rlk_status lmhead_check(const rlk_logp_contract& c, int64_t H);
size_t lmhead_fwd_workspace(const rlk_logp_contract& c);
rlk_status launch_lmhead_fwd(const rlk_logp_contract& c, const void* hidden, int64_t H, const void* weight,
                             const int64_t* targets, const uint8_t* mask, float* logp, float* lse, void* workspace,
                             uint32_t* status, cudaStream_t stream);

size_t lmhead_bwd_workspace(const rlk_logp_contract& c);
rlk_status launch_lmhead_bwd(const rlk_logp_contract& c, const void* hidden, int64_t H, const void* weight,
                             const int64_t* targets, const uint8_t* mask, const float* grad, float* logp, float* lse,
                             void* dhidden, float* dweight_f32, void* dweight_bf16, void* workspace, uint32_t* status,
                             cudaStream_t stream);
// The forward that also writes its FP32 logits [T, V_padded] to logits_f32.
rlk_status launch_lmhead_fwd_keep(const rlk_logp_contract& c, const void* hidden, int64_t H, const void* weight,
                                  const int64_t* targets, const uint8_t* mask, float* logp, float* lse,
                                  float* logits_f32, void* workspace, uint32_t* status, cudaStream_t stream);
// The backward from kept FP32 logits and the LSE: dlogits pass, then dHidden and dW.
rlk_status launch_lmhead_bwd_kept(const rlk_logp_contract& c, const void* hidden, int64_t H, const void* weight,
                                  const int64_t* targets, const uint8_t* mask, const float* grad, const float* lse,
                                  const float* logits_f32, void* dhidden, float* dweight_f32, void* dweight_bf16,
                                  void* workspace, uint32_t* status, cudaStream_t stream);
// The backward alone, from a given LSE: recompute GEMM (dlogits), then dHidden and dW.
rlk_status launch_lmhead_bwd_given_lse(const rlk_logp_contract& c, const void* hidden, int64_t H, const void* weight,
                                       const int64_t* targets, const uint8_t* mask, const float* grad,
                                       const float* lse, void* dhidden, float* dweight_f32, void* dweight_bf16,
                                       void* workspace, uint32_t* status, cudaStream_t stream);

// Vocabulary-parallel pieces (shard.cu).  A shard call's contract describes
// the whole problem with virtual_tp = the number of shards; shard j holds
// columns [j*Vs, (j+1)*Vs) of the padded vocabulary, Vs = V_padded/virtual_tp.
rlk_status check_shard_contract(const rlk_logp_contract& c, int32_t shard);
// The contract of shard j's columns as a vocabulary of its own (V_real of it
// may be 0: a shard of padding only).
rlk_logp_contract shard_local_contract(const rlk_logp_contract& c, int32_t shard);
size_t shard_workspace(const rlk_logp_contract& c);
rlk_status launch_shard_fwd(const rlk_logp_contract& c, int32_t shard, const uint16_t* logits, const int64_t* targets,
                            const uint8_t* mask, float* partials, float* target_logit, void* workspace,
                            uint32_t* status, cudaStream_t stream);
rlk_status launch_gathered_fold(const rlk_logp_contract& c, const float* gathered_partials,
                                const float* gathered_xt, const int64_t* targets, const uint8_t* mask, float* logp,
                                float* lse, uint32_t* status, cudaStream_t stream);
rlk_status launch_shard_bwd(const rlk_logp_contract& c, int32_t shard, const uint16_t* logits, const int64_t* targets,
                            const uint8_t* mask, const float* lse_in, const float* grad, uint16_t* dlogits,
                            void* workspace, uint32_t* status, cudaStream_t stream);

// Token-mean GRPO loss and its gradient (grpo_loss.cu); one cluster, fixed
// order.  grad may be NULL (the loss alone).
rlk_status launch_grpo_loss(int64_t T, const float* logp, const float* adv, const uint8_t* mask, const float* ref,
                            float beta, float* loss, float* grad, float* count, cudaStream_t stream);

// N of the fused GRPO step into *n_active (cleared first); in ignore_index
// mode (mask NULL) each row's activity also goes to mask_out.
rlk_status launch_grpo_count(int64_t T, const int64_t* targets, const uint8_t* mask, int64_t ignore_index,
                             uint8_t* mask_out, unsigned long long* n_active, int sm_count, cudaStream_t stream);

// Cross entropy of hidden @ weight^T (linear_ce.cu), for a checked contract
// whose strides are filled in.
size_t linear_ce_workspace(const rlk_linear_ce_contract& c, bool grad);
rlk_status launch_linear_ce_fwd(const rlk_linear_ce_contract& c, const void* hidden, const void* weight,
                                const int64_t* targets, const uint8_t* mask, float* loss, float* lse, void* workspace,
                                cudaStream_t stream);
rlk_status launch_linear_ce_bwd(const rlk_linear_ce_contract& c, const void* hidden, const void* weight,
                                const int64_t* targets, const uint8_t* mask, const float* lse, const float* grad,
                                void* dhidden, void* dweight, void* workspace, cudaStream_t stream);

// Quantisation to E4M3 with a scale per group of 128 (fp8_quant.cu); q and/or
// qt (the transpose), each with its scales.
rlk_status launch_fp8_quantize(int64_t rows, int64_t cols, const void* x, int32_t x_f32, int64_t ldx,
                               int32_t block_rows, uint8_t* q, int64_t ldq, float* scale, uint8_t* qt, int64_t ldqt,
                               float* scale_t, cudaStream_t stream);

// C = A B^T of such operands (fp8_gemm.cu); *status is only ever set.
rlk_status launch_fp8_matmul(int64_t M, int64_t N, int64_t K, const void* a, int64_t lda, const float* sa,
                             const void* b, int64_t ldb, const float* sb, int32_t b_block_rows, void* c, int64_t ldc,
                             int32_t c_f32, int32_t accumulate, uint32_t* status, cudaStream_t stream);

// The product with a layer's epilogue (fp8_epilogue.cu), and products of rows
// that belong to groups (fp8_grouped.cu).
rlk_status launch_fp8_matmul_act(int64_t M, int64_t N, int64_t K, const void* a, int64_t lda, const float* sa,
                                 const void* b, int64_t ldb, const float* sb, const rlk_fp8_epilogue* e, void* c,
                                 int64_t ldc, int32_t c_f32, uint32_t* status, cudaStream_t stream);
rlk_status launch_fp8_grouped_matmul(int64_t G, int64_t M, int64_t N, int64_t K, const int32_t* ends, const void* a,
                                     int64_t lda, const float* sa, const void* b, int64_t ldb, int64_t group,
                                     const float* sb, const rlk_fp8_epilogue* e, void* c, int64_t ldc, int32_t c_f32,
                                     int32_t rest, uint32_t* status, cudaStream_t stream);
rlk_status launch_fp8_grouped_dweight(int64_t G, int64_t rows, int64_t M, int64_t N, const int32_t* ends,
                                      const void* a, int64_t lda, const float* sa, const void* b, int64_t ldb,
                                      const float* sb, void* c, int64_t ldc, int64_t group, int32_t c_f32,
                                      int32_t accumulate, uint32_t* status, cudaStream_t stream);

// Quantisation of groups of rows, of several matrices, and of the epilogue's
// backward with the bias's gradient (fp8_act_grad.cu); part: the row tiles' sums.
int64_t group_row_tiles(int64_t groups, int64_t rows);
rlk_status launch_fp8_quantize_grouped(int64_t G, int64_t rows, int64_t cols, const int32_t* ends, const void* x,
                                       int32_t x_f32, int64_t ldx, uint8_t* q, int64_t ldq, float* scale, uint8_t* qt,
                                       int64_t ldqt, float* scale_t, cudaStream_t stream);
rlk_status launch_fp8_quantize_batch(int64_t count, int64_t rows, int64_t cols, const void* x, int32_t x_f32,
                                     int64_t ldx, int64_t x_b, uint8_t* q, int64_t ldq, int64_t q_b, float* scale,
                                     uint8_t* qt, int64_t ldqt, int64_t qt_b, float* scale_t, cudaStream_t stream);
rlk_status launch_fp8_act_grad(int64_t G, int64_t rows, int64_t wide, const int32_t* ends, const void* dy,
                               int32_t dy_f32, int64_t lddy, const void* z, int64_t ldz, int32_t act, int32_t gated,
                               uint8_t* q, int64_t ldq, float* scale, uint8_t* qt, int64_t ldqt, float* scale_t,
                               void* dbias, int32_t dbias_f32, float* part, cudaStream_t stream);

// Launches the bounded-wait self-test kernel (one warp waiting on an mbarrier
// that nothing arrives at).
rlk_status launch_selftest_wait(uint64_t limit_ns, uint32_t* status, cudaStream_t stream);

}  // namespace rlk
