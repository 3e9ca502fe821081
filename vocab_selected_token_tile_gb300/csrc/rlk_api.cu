// C ABI of librlk_logp.so: contract validation, argument checks, status
// handling.  Every check that can be made on the host is made here, before
// any launch (PR #289 review excerpt of the vocab-parallel entry point:
// _tile_size and _validate_invocation precede any work; "typed contract"
// commit: incompatible requests are rejected with explicit reasons and never
// served by a silent fallback).
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <initializer_list>
#include <mutex>
#include <string>

#include "rlk_internal.h"
#include "rlk_logp.h"

#define RLK_EXPORT extern "C" __attribute__((visibility("default")))

namespace rlk {

namespace {
thread_local std::string g_last_error;
}

rlk_status fail(rlk_status s, const std::string& why) {
    g_last_error = why;
    return s;
}

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

rlk_status check_contract(const rlk_logp_contract* c) {
    if (!c) return fail(RLK_ERR_INVALID_ARG, "contract is NULL");
    if (c->T < 0) return fail(RLK_ERR_INVALID_ARG, "T must be >= 0");
    if (c->T > ((int64_t)1 << 40)) return fail(RLK_ERR_UNSUPPORTED, "T above 2^40 rows");
    if (c->V_real < 1) return fail(RLK_ERR_INVALID_ARG, "V_real must be >= 1");
    if (c->V_padded < c->V_real) return fail(RLK_ERR_INVALID_ARG, "V_padded must be >= V_real");
    if (c->V_padded > ((int64_t)1 << 31)) return fail(RLK_ERR_UNSUPPORTED, "V_padded above 2^31");
    if (c->num_tiles < 1) return fail(RLK_ERR_INVALID_ARG, "num_tiles must be >= 1");
    if (c->V_padded % c->num_tiles != 0)
        return fail(RLK_ERR_NON_TILEABLE, "vocabulary is not tileable: num_tiles must divide V_padded");
    if (c->virtual_tp != 1 && c->virtual_tp != 2 && c->virtual_tp != 4 && c->virtual_tp != 8)
        return fail(RLK_ERR_UNSUPPORTED, "virtual_tp must be 1, 2, 4 or 8");
    if (c->num_tiles % c->virtual_tp != 0)
        return fail(RLK_ERR_NON_TILEABLE, "shard bounds must be tile-aligned: virtual_tp must divide num_tiles");
    if (c->num_tiles > kMaxTiles) return fail(RLK_ERR_UNSUPPORTED, "num_tiles above 1024");
    if (c->V_padded / c->num_tiles > kMaxTileCols)
        return fail(RLK_ERR_UNSUPPORTED, "tile width V_padded/num_tiles above 16384 columns");
    const int64_t stride = c->row_stride ? c->row_stride : c->V_padded;
    if (stride < c->V_padded) return fail(RLK_ERR_INVALID_ARG, "row_stride must be >= V_padded");
    if (stride % 8 != 0) return fail(RLK_ERR_MISALIGNED, "row_stride must be a multiple of 8 elements (16-byte rows)");
    if (c->mask_mode != RLK_MASK_EXPLICIT && c->mask_mode != RLK_MASK_IGNORE_INDEX)
        return fail(RLK_ERR_INVALID_ARG, "mask_mode must be RLK_MASK_EXPLICIT or RLK_MASK_IGNORE_INDEX");
    if (c->validate != 0 && c->validate != 1) return fail(RLK_ERR_INVALID_ARG, "validate must be 0 or 1");
    if (c->wait_timeout_ns < 0) return fail(RLK_ERR_INVALID_ARG, "wait_timeout_ns must be >= 0");
    return check_planner_env();
}

rlk_status check_common(const rlk_logp_contract* c, const void* logits, const int64_t* targets,
                        const uint8_t* mask, const void* workspace) {
    if (!logits) return fail(RLK_ERR_INVALID_ARG, "logits is NULL");
    if (!aligned16(logits)) return fail(RLK_ERR_MISALIGNED, "logits must be 16-byte aligned");
    if (!targets) return fail(RLK_ERR_INVALID_ARG, "targets is NULL");
    if (c->mask_mode == RLK_MASK_EXPLICIT && !mask)
        return fail(RLK_ERR_INVALID_ARG, "explicit mask mode needs active_mask");
    if (c->mask_mode == RLK_MASK_IGNORE_INDEX && mask)
        return fail(RLK_ERR_INVALID_ARG, "ignore_index mode takes no active_mask (pass NULL)");
    if (!workspace) return fail(RLK_ERR_INVALID_ARG, "workspace is NULL");
    if (!aligned16(workspace)) return fail(RLK_ERR_MISALIGNED, "workspace must be 16-byte aligned");
    return RLK_OK;
}

// dlogits may be the logits buffer itself (in place: the kernels read every
// logit before its gradient overwrites it) or a buffer of its own; any other
// overlap would let one row's gradient land on logits not yet read.
rlk_status check_dlogits_overlap(const void* logits, const void* dlogits, int64_t T, int64_t stride) {
    if (logits == dlogits) return RLK_OK;
    const uint64_t a = reinterpret_cast<uintptr_t>(logits), b = reinterpret_cast<uintptr_t>(dlogits);
    const uint64_t rows = (uint64_t)T, st = (uint64_t)stride;
    const uint64_t span = (st != 0 && rows > (UINT64_MAX / 2) / st) ? UINT64_MAX : rows * st * 2u;
    if ((a < b ? b - a : a - b) < span)
        return fail(RLK_ERR_INVALID_ARG, "dlogits overlaps logits without being the same buffer (only an exact "
                                         "in-place call, dlogits == logits, may share memory)");
    return RLK_OK;
}

// The device that holds `ptr`, if it is device memory: the driver's own query
// for those two attributes, which costs a fraction of cudaPointerGetAttributes
// (a call of seven pointers: about 4 us less of host time).  Anything else it
// leaves to the runtime's query, which tells the kinds of memory apart.
bool quick_device(const void* ptr, int* device) {
    using Query = CUresult (*)(unsigned, CUpointer_attribute*, void**, CUdeviceptr);
    static const Query query = [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPointByVersion("cuPointerGetAttributes", &fn, 12000, cudaEnableDefault, &q) ==
                            cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<Query>(fn) : nullptr;
    }();
    if (!query) return false;
    unsigned type = 0;
    CUpointer_attribute which[2] = {CU_POINTER_ATTRIBUTE_MEMORY_TYPE, CU_POINTER_ATTRIBUTE_DEVICE_ORDINAL};
    void* out[2] = {&type, device};
    return query(2, which, out, reinterpret_cast<CUdeviceptr>(ptr)) == CUDA_SUCCESS && type == CU_MEMORYTYPE_DEVICE;
}

// Makes the device that owns `ptr` current for this library's runtime.
rlk_status select_device(const void* ptr) {
    int owner = -1, now = -1;
    if (quick_device(ptr, &owner) && cudaGetDevice(&now) == cudaSuccess && owner == now) return RLK_OK;
    cudaPointerAttributes attr{};
    cudaError_t e = cudaPointerGetAttributes(&attr, ptr);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(RLK_ERR_INVALID_ARG, std::string("the first device operand is not a CUDA pointer: ") +
                                             cudaGetErrorString(e));
    }
    if (attr.type != cudaMemoryTypeDevice && attr.type != cudaMemoryTypeManaged)
        return fail(RLK_ERR_INVALID_ARG, "device buffers must be device memory");
    e = cudaSetDevice(attr.device);
    if (e != cudaSuccess) return fail(RLK_ERR_CUDA, std::string("cudaSetDevice: ") + cudaGetErrorString(e));
    return RLK_OK;
}

struct DevPtr {
    const void* ptr;
    const char* name;
};

// Every other pointer a call receives must be device memory of the device
// select_device made current (or managed memory, which that device can
// reach).  Host memory -- pinned or not -- and another GPU's memory fail
// closed here, before any launch, instead of reaching a kernel.  NULL
// entries are optional arguments the caller left out.
rlk_status check_device_ptrs(std::initializer_list<DevPtr> ptrs) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return fail(RLK_ERR_CUDA, std::string("cudaGetDevice: ") + cudaGetErrorString(e));
    for (const DevPtr& d : ptrs) {
        if (!d.ptr) continue;
        int owner = -1;
        if (quick_device(d.ptr, &owner) && owner == dev) continue;
        cudaPointerAttributes attr{};
        e = cudaPointerGetAttributes(&attr, d.ptr);
        if (e != cudaSuccess) {
            cudaGetLastError();
            return fail(RLK_ERR_INVALID_ARG, std::string(d.name) + " is not a CUDA pointer");
        }
        if (attr.type == cudaMemoryTypeManaged) continue;
        if (attr.type != cudaMemoryTypeDevice)
            return fail(RLK_ERR_INVALID_ARG, std::string(d.name) + " must be device memory (it is host memory)");
        if (attr.device != dev)
            return fail(RLK_ERR_INVALID_ARG, std::string(d.name) + " lives on device " + std::to_string(attr.device) +
                                                 ", not on device " + std::to_string(dev) +
                                                 " that holds the first operand");
    }
    return RLK_OK;
}

rlk_status decode_status(uint32_t bits) {
    if (bits & kStatusInternal)
        return fail(RLK_ERR_CUDA, "a streaming kernel found a ring slot holding an unexpected row and stopped");
    if (bits & kStatusTimeout) return fail(RLK_ERR_TIMEOUT, "a bounded device-side wait expired");
    if (bits & kStatusTargetRange) return fail(RLK_ERR_TARGET_RANGE, "an active target lies outside [0, V_real)");
    if (bits & kStatusNonFinite)
        return fail(RLK_ERR_NONFINITE_LSE,
                    "non-finite logsumexp on an active row: its real-vocabulary logits must be finite");
    return RLK_OK;
}

rlk_status read_status(const void* workspace, cudaStream_t stream) {
    uint32_t bits = 0;
    cudaError_t e = cudaMemcpyAsync(&bits, workspace, sizeof(bits), cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return fail(RLK_ERR_CUDA, std::string("reading the status word: ") + cudaGetErrorString(e));
    return decode_status(bits);
}

rlk_status begin(void* workspace, cudaStream_t stream) {
    cudaError_t e = cudaMemsetAsync(workspace, 0, sizeof(uint32_t), stream);
    if (e != cudaSuccess) return fail(RLK_ERR_CUDA, std::string("clearing the status word: ") + cudaGetErrorString(e));
    return RLK_OK;
}

}  // namespace
}  // namespace rlk

using namespace rlk;

RLK_EXPORT rlk_status rlk_logp_check_contract(const rlk_logp_contract* contract) {
    return check_contract(contract);
}

RLK_EXPORT size_t rlk_logp_workspace_size(const rlk_logp_contract* contract) {
    return check_contract(contract) == RLK_OK ? kWorkspaceBytes : 0;
}

RLK_EXPORT rlk_status rlk_logp_fwd(const rlk_logp_contract* c, const void* logits_bf16, const int64_t* targets,
                                   const uint8_t* active_mask, float* logp, float* lse, float* partials,
                                   void* workspace, rlk_stream_t stream) {
    rlk_status s = check_contract(c);
    if (s != RLK_OK) return s;
    if (c->T == 0) return RLK_OK;
    if ((s = check_common(c, logits_bf16, targets, active_mask, workspace)) != RLK_OK) return s;
    if (!logp || !lse) return fail(RLK_ERR_INVALID_ARG, "logp and lse outputs are required");
    if ((s = select_device(logits_bf16)) != RLK_OK) return s;
    if ((s = check_device_ptrs({{targets, "targets"}, {active_mask, "active_mask"}, {logp, "logp"}, {lse, "lse"},
                                {partials, "partials"}, {workspace, "workspace"}})) != RLK_OK)
        return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if ((s = begin(workspace, st)) != RLK_OK) return s;
    StreamArgs a{};
    a.logits = static_cast<const uint16_t*>(logits_bf16);
    a.targets = targets;
    a.mask = active_mask;
    a.logp = logp;
    a.lse = lse;
    a.partials = partials;
    a.status = static_cast<uint32_t*>(workspace);
    if ((s = launch_stream(*c, kModeFwd, a, st)) != RLK_OK) return s;
    return c->validate ? read_status(workspace, st) : RLK_OK;
}

RLK_EXPORT rlk_status rlk_logp_fwd_entropy(const rlk_logp_contract* c, const void* logits_bf16,
                                           const int64_t* targets, const uint8_t* active_mask, float* logp,
                                           float* lse, float* entropy, void* workspace, rlk_stream_t stream) {
    rlk_status s = check_contract(c);
    if (s != RLK_OK) return s;
    if (c->T == 0) return RLK_OK;
    if ((s = check_common(c, logits_bf16, targets, active_mask, workspace)) != RLK_OK) return s;
    if (!logp || !lse || !entropy) return fail(RLK_ERR_INVALID_ARG, "logp, lse and entropy outputs are required");
    if ((s = select_device(logits_bf16)) != RLK_OK) return s;
    if ((s = check_device_ptrs({{targets, "targets"}, {active_mask, "active_mask"}, {logp, "logp"}, {lse, "lse"},
                                {entropy, "entropy"}, {workspace, "workspace"}})) != RLK_OK)
        return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if ((s = begin(workspace, st)) != RLK_OK) return s;
    StreamArgs a{};
    a.logits = static_cast<const uint16_t*>(logits_bf16);
    a.targets = targets;
    a.mask = active_mask;
    a.logp = logp;
    a.lse = lse;
    a.entropy = entropy;
    a.status = static_cast<uint32_t*>(workspace);
    if ((s = launch_stream(*c, kModeFwd, a, st)) != RLK_OK) return s;
    return c->validate ? read_status(workspace, st) : RLK_OK;
}

RLK_EXPORT rlk_status rlk_logp_fwd_bwd_entropy(const rlk_logp_contract* c, const void* logits_bf16,
                                               const int64_t* targets, const uint8_t* active_mask,
                                               const float* grad_logp, void* dlogits_bf16, float* logp_out,
                                               float* lse_out, float* entropy_out, void* workspace,
                                               rlk_stream_t stream) {
    rlk_status s = check_contract(c);
    if (s != RLK_OK) return s;
    if (c->T == 0) return RLK_OK;
    if ((s = check_common(c, logits_bf16, targets, active_mask, workspace)) != RLK_OK) return s;
    if (!grad_logp) return fail(RLK_ERR_INVALID_ARG, "grad_logp is NULL");
    if (!dlogits_bf16) return fail(RLK_ERR_INVALID_ARG, "dlogits is NULL");
    if (!aligned16(dlogits_bf16)) return fail(RLK_ERR_MISALIGNED, "dlogits must be 16-byte aligned");
    if ((s = check_dlogits_overlap(logits_bf16, dlogits_bf16, c->T, c->row_stride ? c->row_stride : c->V_padded)) !=
        RLK_OK)
        return s;
    if (!logp_out || !lse_out || !entropy_out)
        return fail(RLK_ERR_INVALID_ARG, "logp_out, lse_out and entropy_out are required");
    if ((s = select_device(logits_bf16)) != RLK_OK) return s;
    if ((s = check_device_ptrs({{targets, "targets"}, {active_mask, "active_mask"}, {grad_logp, "grad_logp"},
                                {dlogits_bf16, "dlogits"}, {logp_out, "logp_out"}, {lse_out, "lse_out"},
                                {entropy_out, "entropy_out"}, {workspace, "workspace"}})) != RLK_OK)
        return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if ((s = begin(workspace, st)) != RLK_OK) return s;
    StreamArgs a{};
    a.logits = static_cast<const uint16_t*>(logits_bf16);
    a.dlogits = static_cast<uint16_t*>(dlogits_bf16);
    a.targets = targets;
    a.mask = active_mask;
    a.grad = grad_logp;
    a.logp = logp_out;
    a.lse = lse_out;
    a.entropy = entropy_out;
    a.status = static_cast<uint32_t*>(workspace);
    if ((s = launch_stream(*c, kModeFused, a, st)) != RLK_OK) return s;
    return c->validate ? read_status(workspace, st) : RLK_OK;
}

RLK_EXPORT rlk_status rlk_grpo_loss(int64_t T, const float* logp, const float* advantage, const uint8_t* active_mask,
                                    const float* ref_logp, float beta, float* loss, float* grad_logp,
                                    float* active_count, rlk_stream_t stream) {
    if (T < 0) return fail(RLK_ERR_INVALID_ARG, "T must be >= 0");
    if (!loss) return fail(RLK_ERR_INVALID_ARG, "loss output is required");
    if (T > 0 && (!logp || !advantage || !active_mask || !grad_logp))
        return fail(RLK_ERR_INVALID_ARG, "logp, advantage, active_mask and grad_logp are required");
    if (!(beta >= 0.f) || !isfinite(beta)) return fail(RLK_ERR_INVALID_ARG, "beta must be finite and >= 0");
    rlk_status s = select_device(loss);
    if (s != RLK_OK) return s;
    if ((s = check_device_ptrs({{logp, "logp"}, {advantage, "advantage"}, {active_mask, "active_mask"},
                                {ref_logp, "ref_logp"}, {grad_logp, "grad_logp"}, {active_count, "active_count"}})) !=
        RLK_OK)
        return s;
    return launch_grpo_loss(T, logp, advantage, active_mask, ref_logp, beta, loss, grad_logp, active_count,
                            reinterpret_cast<cudaStream_t>(stream));
}

namespace rlk {
namespace {
// Workspace of the fused GRPO step: the status word, N (8 bytes in 256), and
// in ignore_index mode each row's activity for the loss (one byte a row).
constexpr size_t kGrpoCountBytes = 256;
size_t grpo_workspace(const rlk_logp_contract& c) {
    return kWorkspaceBytes + kGrpoCountBytes + ((size_t)c.T + 255) / 256 * 256;
}
}  // namespace
}  // namespace rlk

RLK_EXPORT size_t rlk_grpo_fused_workspace_size(const rlk_logp_contract* c) {
    return check_contract(c) == RLK_OK ? grpo_workspace(*c) : 0;
}

RLK_EXPORT rlk_status rlk_grpo_fused_step(const rlk_logp_contract* c, const void* logits_bf16,
                                          const int64_t* targets, const uint8_t* active_mask, const float* advantage,
                                          const float* ref_logp, float beta, void* dlogits_bf16, float* logp_out,
                                          float* lse_out, float* grad_out, float* entropy_out, float* loss,
                                          float* active_count, void* workspace, rlk_stream_t stream) {
    rlk_status s = check_contract(c);
    if (s != RLK_OK) return s;
    if (!loss) return fail(RLK_ERR_INVALID_ARG, "loss output is required");
    if (!(beta >= 0.f) || !isfinite(beta)) return fail(RLK_ERR_INVALID_ARG, "beta must be finite and >= 0");
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (c->T == 0) {  // no rows: loss 0 (and N = 0)
        if ((s = select_device(loss)) != RLK_OK) return s;
        if ((s = check_device_ptrs({{active_count, "active_count"}})) != RLK_OK) return s;
        return launch_grpo_loss(0, nullptr, nullptr, nullptr, nullptr, beta, loss, nullptr, active_count, st);
    }
    if ((s = check_common(c, logits_bf16, targets, active_mask, workspace)) != RLK_OK) return s;
    if (!advantage) return fail(RLK_ERR_INVALID_ARG, "advantage is NULL");
    if (!dlogits_bf16) return fail(RLK_ERR_INVALID_ARG, "dlogits is NULL");
    if (!aligned16(dlogits_bf16)) return fail(RLK_ERR_MISALIGNED, "dlogits must be 16-byte aligned");
    if ((s = check_dlogits_overlap(logits_bf16, dlogits_bf16, c->T, c->row_stride ? c->row_stride : c->V_padded)) !=
        RLK_OK)
        return s;
    if (!logp_out || !lse_out || !grad_out)
        return fail(RLK_ERR_INVALID_ARG, "logp_out, lse_out and grad_out are required");
    if ((s = select_device(logits_bf16)) != RLK_OK) return s;
    if ((s = check_device_ptrs({{targets, "targets"}, {active_mask, "active_mask"}, {advantage, "advantage"},
                                {ref_logp, "ref_logp"}, {dlogits_bf16, "dlogits"}, {logp_out, "logp_out"},
                                {lse_out, "lse_out"}, {grad_out, "grad_out"}, {entropy_out, "entropy_out"},
                                {loss, "loss"}, {active_count, "active_count"}, {workspace, "workspace"}})) != RLK_OK)
        return s;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return fail(RLK_ERR_CUDA, std::string("querying the device: ") + cudaGetErrorString(e));
    if ((s = begin(workspace, st)) != RLK_OK) return s;
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    auto* n_active = reinterpret_cast<unsigned long long*>(ws + kWorkspaceBytes);
    uint8_t* mask_ws = (c->mask_mode == RLK_MASK_IGNORE_INDEX) ? ws + kWorkspaceBytes + kGrpoCountBytes : nullptr;
    if ((s = launch_grpo_count(c->T, targets, active_mask, c->ignore_index, mask_ws, n_active, sms, st)) != RLK_OK)
        return s;
    StreamArgs a{};
    a.logits = static_cast<const uint16_t*>(logits_bf16);
    a.dlogits = static_cast<uint16_t*>(dlogits_bf16);
    a.targets = targets;
    a.mask = active_mask;
    a.logp = logp_out;
    a.lse = lse_out;
    a.entropy = entropy_out;
    a.status = static_cast<uint32_t*>(workspace);
    a.grpo = 1;
    a.adv = advantage;
    a.ref = ref_logp;
    a.beta = beta;
    a.n_active = n_active;
    a.grad_out = grad_out;
    if ((s = launch_stream(*c, kModeFused, a, st)) != RLK_OK) return s;
    // the loss from this step's logp, in the GRPO loss kernel's fixed order (g is already written)
    if ((s = launch_grpo_loss(c->T, logp_out, advantage, active_mask ? active_mask : mask_ws, ref_logp, beta, loss,
                              nullptr, active_count, st)) != RLK_OK)
        return s;
    return c->validate ? read_status(workspace, st) : RLK_OK;
}

RLK_EXPORT rlk_status rlk_logp_bwd(const rlk_logp_contract* c, const void* logits_bf16, const int64_t* targets,
                                   const uint8_t* active_mask, const float* lse_in, const float* grad_logp,
                                   void* dlogits_bf16, float* logp_out, float* lse_out, void* workspace,
                                   rlk_stream_t stream) {
    rlk_status s = check_contract(c);
    if (s != RLK_OK) return s;
    if (c->T == 0) return RLK_OK;
    if ((s = check_common(c, logits_bf16, targets, active_mask, workspace)) != RLK_OK) return s;
    if (!grad_logp) return fail(RLK_ERR_INVALID_ARG, "grad_logp is NULL");
    if (!dlogits_bf16) return fail(RLK_ERR_INVALID_ARG, "dlogits is NULL");
    if (!aligned16(dlogits_bf16)) return fail(RLK_ERR_MISALIGNED, "dlogits must be 16-byte aligned");
    if ((s = check_dlogits_overlap(logits_bf16, dlogits_bf16, c->T, c->row_stride ? c->row_stride : c->V_padded)) !=
        RLK_OK)
        return s;
    if (lse_in && (logp_out || lse_out))
        return fail(RLK_ERR_INVALID_ARG, "with lse_in the forward outputs logp_out/lse_out must be NULL");
    if (!lse_in && (!logp_out || !lse_out))
        return fail(RLK_ERR_INVALID_ARG, "the fused form (lse_in NULL) needs logp_out and lse_out");
    if ((s = select_device(logits_bf16)) != RLK_OK) return s;
    if ((s = check_device_ptrs({{targets, "targets"}, {active_mask, "active_mask"}, {lse_in, "lse_in"},
                                {grad_logp, "grad_logp"}, {dlogits_bf16, "dlogits"}, {logp_out, "logp_out"},
                                {lse_out, "lse_out"}, {workspace, "workspace"}})) != RLK_OK)
        return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if ((s = begin(workspace, st)) != RLK_OK) return s;
    StreamArgs a{};
    a.logits = static_cast<const uint16_t*>(logits_bf16);
    a.dlogits = static_cast<uint16_t*>(dlogits_bf16);
    a.targets = targets;
    a.mask = active_mask;
    a.grad = grad_logp;
    a.lse_in = lse_in;
    a.logp = logp_out;
    a.lse = lse_out;
    a.status = static_cast<uint32_t*>(workspace);
    if ((s = launch_stream(*c, lse_in ? kModeBwd : kModeFused, a, st)) != RLK_OK) return s;
    return c->validate ? read_status(workspace, st) : RLK_OK;
}

// ---------------------------------------------------------------- fused lm_head

RLK_EXPORT size_t rlk_logp_lmhead_workspace_size(const rlk_logp_contract* c, int64_t H) {
    if (check_contract(c) != RLK_OK || lmhead_check(*c, H) != RLK_OK) return 0;
    return kWorkspaceBytes + lmhead_bwd_workspace(*c);
}

RLK_EXPORT rlk_status rlk_logp_fused_lmhead(const rlk_logp_contract* c, const void* hidden_bf16, int64_t H,
                                            const void* weight_bf16, const int64_t* targets,
                                            const uint8_t* active_mask, const float* grad_logp, float* logp,
                                            float* lse, void* dhidden_bf16, float* dweight_f32, void* dweight_bf16,
                                            void* workspace, rlk_stream_t stream) {
    rlk_status s = check_contract(c);
    if (s != RLK_OK) return s;
    if ((s = lmhead_check(*c, H)) != RLK_OK) return s;
    if (c->T == 0) return RLK_OK;
    if (!hidden_bf16 || !weight_bf16) return fail(RLK_ERR_INVALID_ARG, "hidden and weight are required");
    if (!aligned16(hidden_bf16) || !aligned16(weight_bf16))
        return fail(RLK_ERR_MISALIGNED, "hidden and weight must be 16-byte aligned");
    if (!targets) return fail(RLK_ERR_INVALID_ARG, "targets is NULL");
    if (c->mask_mode == RLK_MASK_EXPLICIT && !active_mask)
        return fail(RLK_ERR_INVALID_ARG, "explicit mask mode needs active_mask");
    if (c->mask_mode == RLK_MASK_IGNORE_INDEX && active_mask)
        return fail(RLK_ERR_INVALID_ARG, "ignore_index mode takes no active_mask (pass NULL)");
    if (!logp || !lse) return fail(RLK_ERR_INVALID_ARG, "logp and lse outputs are required");
    if (!workspace || !aligned16(workspace)) return fail(RLK_ERR_INVALID_ARG, "workspace must be non-NULL and 16-byte aligned");
    const bool bwd = grad_logp != nullptr;
    if (bwd && (!dhidden_bf16 || (!dweight_f32 && !dweight_bf16)))
        return fail(RLK_ERR_INVALID_ARG, "the backward (grad_logp given) needs dhidden and at least one dweight output");
    if (!bwd && (dhidden_bf16 || dweight_f32 || dweight_bf16))
        return fail(RLK_ERR_INVALID_ARG, "dhidden/dweight are written only when grad_logp is given");
    if (bwd && (!aligned16(dhidden_bf16) || !aligned16(dweight_f32) || !aligned16(dweight_bf16)))
        return fail(RLK_ERR_MISALIGNED, "dhidden and dweight must be 16-byte aligned");
    if ((s = select_device(hidden_bf16)) != RLK_OK) return s;
    if ((s = check_device_ptrs({{weight_bf16, "weight"}, {targets, "targets"}, {active_mask, "active_mask"},
                                {grad_logp, "grad_logp"}, {logp, "logp"}, {lse, "lse"}, {dhidden_bf16, "dhidden"},
                                {dweight_f32, "dweight_f32"}, {dweight_bf16, "dweight_bf16"},
                                {workspace, "workspace"}})) != RLK_OK)
        return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if ((s = begin(workspace, st)) != RLK_OK) return s;
    uint32_t* status = static_cast<uint32_t*>(workspace);
    void* ws = static_cast<unsigned char*>(workspace) + kWorkspaceBytes;
    if (bwd)
        s = launch_lmhead_bwd(*c, hidden_bf16, H, weight_bf16, targets, active_mask, grad_logp, logp, lse,
                              dhidden_bf16, dweight_f32, dweight_bf16, ws, status, st);
    else
        s = launch_lmhead_fwd(*c, hidden_bf16, H, weight_bf16, targets, active_mask, logp, lse, ws, status, st);
    if (s != RLK_OK) return s;
    return c->validate ? read_status(workspace, st) : RLK_OK;
}

RLK_EXPORT rlk_status rlk_logp_fused_lmhead_bwd(const rlk_logp_contract* c, const void* hidden_bf16, int64_t H,
                                                const void* weight_bf16, const int64_t* targets,
                                                const uint8_t* active_mask, const float* lse_in,
                                                const float* grad_logp, void* dhidden_bf16, float* dweight_f32,
                                                void* dweight_bf16, void* workspace, rlk_stream_t stream) {
    rlk_status s = check_contract(c);
    if (s != RLK_OK) return s;
    if ((s = lmhead_check(*c, H)) != RLK_OK) return s;
    if (c->T == 0) return RLK_OK;
    if (!hidden_bf16 || !weight_bf16) return fail(RLK_ERR_INVALID_ARG, "hidden and weight are required");
    if (!aligned16(hidden_bf16) || !aligned16(weight_bf16))
        return fail(RLK_ERR_MISALIGNED, "hidden and weight must be 16-byte aligned");
    if (!targets) return fail(RLK_ERR_INVALID_ARG, "targets is NULL");
    if (c->mask_mode == RLK_MASK_EXPLICIT && !active_mask)
        return fail(RLK_ERR_INVALID_ARG, "explicit mask mode needs active_mask");
    if (c->mask_mode == RLK_MASK_IGNORE_INDEX && active_mask)
        return fail(RLK_ERR_INVALID_ARG, "ignore_index mode takes no active_mask (pass NULL)");
    if (!lse_in || !grad_logp) return fail(RLK_ERR_INVALID_ARG, "lse_in and grad_logp are required");
    if (!dhidden_bf16 || (!dweight_f32 && !dweight_bf16))
        return fail(RLK_ERR_INVALID_ARG, "dhidden and at least one dweight output are required");
    if (!aligned16(dhidden_bf16) || !aligned16(dweight_f32) || !aligned16(dweight_bf16))
        return fail(RLK_ERR_MISALIGNED, "dhidden and dweight must be 16-byte aligned");
    if (!workspace || !aligned16(workspace)) return fail(RLK_ERR_INVALID_ARG, "workspace must be non-NULL and 16-byte aligned");
    if ((s = select_device(hidden_bf16)) != RLK_OK) return s;
    if ((s = check_device_ptrs({{weight_bf16, "weight"}, {targets, "targets"}, {active_mask, "active_mask"},
                                {lse_in, "lse_in"}, {grad_logp, "grad_logp"}, {dhidden_bf16, "dhidden"},
                                {dweight_f32, "dweight_f32"}, {dweight_bf16, "dweight_bf16"},
                                {workspace, "workspace"}})) != RLK_OK)
        return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if ((s = begin(workspace, st)) != RLK_OK) return s;
    if ((s = launch_lmhead_bwd_given_lse(*c, hidden_bf16, H, weight_bf16, targets, active_mask, grad_logp, lse_in,
                                         dhidden_bf16, dweight_f32, dweight_bf16,
                                         static_cast<unsigned char*>(workspace) + kWorkspaceBytes,
                                         static_cast<uint32_t*>(workspace), st)) != RLK_OK)
        return s;
    return c->validate ? read_status(workspace, st) : RLK_OK;
}

RLK_EXPORT rlk_status rlk_logp_fused_lmhead_keep(const rlk_logp_contract* c, const void* hidden_bf16, int64_t H,
                                                 const void* weight_bf16, const int64_t* targets,
                                                 const uint8_t* active_mask, float* logp, float* lse,
                                                 float* logits_f32, void* workspace, rlk_stream_t stream) {
    rlk_status s = check_contract(c);
    if (s != RLK_OK) return s;
    if ((s = lmhead_check(*c, H)) != RLK_OK) return s;
    if (c->T == 0) return RLK_OK;
    if (!hidden_bf16 || !weight_bf16) return fail(RLK_ERR_INVALID_ARG, "hidden and weight are required");
    if (!aligned16(hidden_bf16) || !aligned16(weight_bf16))
        return fail(RLK_ERR_MISALIGNED, "hidden and weight must be 16-byte aligned");
    if (!targets) return fail(RLK_ERR_INVALID_ARG, "targets is NULL");
    if (c->mask_mode == RLK_MASK_EXPLICIT && !active_mask)
        return fail(RLK_ERR_INVALID_ARG, "explicit mask mode needs active_mask");
    if (c->mask_mode == RLK_MASK_IGNORE_INDEX && active_mask)
        return fail(RLK_ERR_INVALID_ARG, "ignore_index mode takes no active_mask (pass NULL)");
    if (!logp || !lse) return fail(RLK_ERR_INVALID_ARG, "logp and lse outputs are required");
    if (!logits_f32) return fail(RLK_ERR_INVALID_ARG, "logits_f32 is NULL");
    if (!aligned16(logits_f32)) return fail(RLK_ERR_MISALIGNED, "logits_f32 must be 16-byte aligned");
    if (!workspace || !aligned16(workspace)) return fail(RLK_ERR_INVALID_ARG, "workspace must be non-NULL and 16-byte aligned");
    if ((s = select_device(hidden_bf16)) != RLK_OK) return s;
    if ((s = check_device_ptrs({{weight_bf16, "weight"}, {targets, "targets"}, {active_mask, "active_mask"},
                                {logp, "logp"}, {lse, "lse"}, {logits_f32, "logits_f32"},
                                {workspace, "workspace"}})) != RLK_OK)
        return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if ((s = begin(workspace, st)) != RLK_OK) return s;
    if ((s = launch_lmhead_fwd_keep(*c, hidden_bf16, H, weight_bf16, targets, active_mask, logp, lse, logits_f32,
                                    static_cast<unsigned char*>(workspace) + kWorkspaceBytes,
                                    static_cast<uint32_t*>(workspace), st)) != RLK_OK)
        return s;
    return c->validate ? read_status(workspace, st) : RLK_OK;
}

RLK_EXPORT rlk_status rlk_logp_fused_lmhead_bwd_kept(const rlk_logp_contract* c, const void* hidden_bf16, int64_t H,
                                                     const void* weight_bf16, const int64_t* targets,
                                                     const uint8_t* active_mask, const float* lse_in,
                                                     const float* logits_f32, const float* grad_logp,
                                                     void* dhidden_bf16, float* dweight_f32, void* dweight_bf16,
                                                     void* workspace, rlk_stream_t stream) {
    rlk_status s = check_contract(c);
    if (s != RLK_OK) return s;
    if ((s = lmhead_check(*c, H)) != RLK_OK) return s;
    if (c->T == 0) return RLK_OK;
    if (!hidden_bf16 || !weight_bf16) return fail(RLK_ERR_INVALID_ARG, "hidden and weight are required");
    if (!aligned16(hidden_bf16) || !aligned16(weight_bf16))
        return fail(RLK_ERR_MISALIGNED, "hidden and weight must be 16-byte aligned");
    if (!targets) return fail(RLK_ERR_INVALID_ARG, "targets is NULL");
    if (c->mask_mode == RLK_MASK_EXPLICIT && !active_mask)
        return fail(RLK_ERR_INVALID_ARG, "explicit mask mode needs active_mask");
    if (c->mask_mode == RLK_MASK_IGNORE_INDEX && active_mask)
        return fail(RLK_ERR_INVALID_ARG, "ignore_index mode takes no active_mask (pass NULL)");
    if (!lse_in || !grad_logp) return fail(RLK_ERR_INVALID_ARG, "lse_in and grad_logp are required");
    if (!logits_f32) return fail(RLK_ERR_INVALID_ARG, "logits_f32 is NULL");
    if (!aligned16(logits_f32)) return fail(RLK_ERR_MISALIGNED, "logits_f32 must be 16-byte aligned");
    if (!dhidden_bf16 || (!dweight_f32 && !dweight_bf16))
        return fail(RLK_ERR_INVALID_ARG, "dhidden and at least one dweight output are required");
    if (!aligned16(dhidden_bf16) || !aligned16(dweight_f32) || !aligned16(dweight_bf16))
        return fail(RLK_ERR_MISALIGNED, "dhidden and dweight must be 16-byte aligned");
    if (!workspace || !aligned16(workspace)) return fail(RLK_ERR_INVALID_ARG, "workspace must be non-NULL and 16-byte aligned");
    if ((s = select_device(hidden_bf16)) != RLK_OK) return s;
    if ((s = check_device_ptrs({{weight_bf16, "weight"}, {targets, "targets"}, {active_mask, "active_mask"},
                                {lse_in, "lse_in"}, {logits_f32, "logits_f32"}, {grad_logp, "grad_logp"},
                                {dhidden_bf16, "dhidden"}, {dweight_f32, "dweight_f32"},
                                {dweight_bf16, "dweight_bf16"}, {workspace, "workspace"}})) != RLK_OK)
        return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if ((s = begin(workspace, st)) != RLK_OK) return s;
    if ((s = launch_lmhead_bwd_kept(*c, hidden_bf16, H, weight_bf16, targets, active_mask, grad_logp, lse_in,
                                    logits_f32, dhidden_bf16, dweight_f32, dweight_bf16,
                                    static_cast<unsigned char*>(workspace) + kWorkspaceBytes,
                                    static_cast<uint32_t*>(workspace), st)) != RLK_OK)
        return s;
    return c->validate ? read_status(workspace, st) : RLK_OK;
}

// ---------------------------------------------------------------- vocabulary-parallel shards

namespace rlk {
namespace {

// A shard call's contract is the whole problem's, with virtual_tp = the
// number of shards and row_stride that of the shard's buffer (0 -> Vs).
rlk_status check_shard(const rlk_logp_contract* c, int32_t shard) {
    if (!c) return fail(RLK_ERR_INVALID_ARG, "contract is NULL");
    rlk_logp_contract whole = *c;
    whole.row_stride = 0;
    rlk_status s = check_contract(&whole);
    if (s != RLK_OK) return s;
    if (shard < 0 || shard >= c->virtual_tp) return fail(RLK_ERR_INVALID_ARG, "shard must lie in [0, virtual_tp)");
    const int64_t Vs = c->V_padded / c->virtual_tp;
    if (Vs % 8 != 0)
        return fail(RLK_ERR_MISALIGNED, "every shard must start on a 16-byte boundary: V_padded/virtual_tp must be a "
                                        "multiple of 8");
    const int64_t stride = c->row_stride ? c->row_stride : Vs;
    if (stride < Vs) return fail(RLK_ERR_INVALID_ARG, "row_stride of a shard must be >= V_padded/virtual_tp");
    if (stride % 8 != 0) return fail(RLK_ERR_MISALIGNED, "row_stride must be a multiple of 8 elements (16-byte rows)");
    return RLK_OK;
}

}  // namespace

rlk_status check_shard_contract(const rlk_logp_contract& c, int32_t shard) { return check_shard(&c, shard); }

}  // namespace rlk

RLK_EXPORT rlk_status rlk_logp_check_shard_contract(const rlk_logp_contract* c, int32_t shard) {
    return check_shard(c, shard);
}

RLK_EXPORT size_t rlk_logp_shard_workspace_size(const rlk_logp_contract* c) {
    return check_shard(c, 0) == RLK_OK ? kWorkspaceBytes + shard_workspace(*c) : 0;
}

RLK_EXPORT rlk_status rlk_logp_shard_fwd(const rlk_logp_contract* c, int32_t shard, const void* logits_shard,
                                         const int64_t* targets, const uint8_t* active_mask, float* partials_shard,
                                         float* target_logit, void* workspace, rlk_stream_t stream) {
    rlk_status s = check_shard(c, shard);
    if (s != RLK_OK) return s;
    if (c->T == 0) return RLK_OK;
    if ((s = check_common(c, logits_shard, targets, active_mask, workspace)) != RLK_OK) return s;
    if (!partials_shard || !target_logit)
        return fail(RLK_ERR_INVALID_ARG, "partials_shard and target_logit outputs are required");
    if ((s = select_device(logits_shard)) != RLK_OK) return s;
    if ((s = check_device_ptrs({{targets, "targets"}, {active_mask, "active_mask"}, {partials_shard, "partials_shard"},
                                {target_logit, "target_logit"}, {workspace, "workspace"}})) != RLK_OK)
        return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if ((s = begin(workspace, st)) != RLK_OK) return s;
    if ((s = launch_shard_fwd(*c, shard, static_cast<const uint16_t*>(logits_shard), targets, active_mask,
                              partials_shard, target_logit, static_cast<unsigned char*>(workspace) + kWorkspaceBytes,
                              static_cast<uint32_t*>(workspace), st)) != RLK_OK)
        return s;
    return c->validate ? read_status(workspace, st) : RLK_OK;
}

RLK_EXPORT rlk_status rlk_logp_fold(const rlk_logp_contract* c, const float* gathered_partials,
                                    const float* gathered_target_logit, const int64_t* targets,
                                    const uint8_t* active_mask, float* logp, float* lse, void* workspace,
                                    rlk_stream_t stream) {
    rlk_status s = check_shard(c, 0);
    if (s != RLK_OK) return s;
    if (c->T == 0) return RLK_OK;
    if (!gathered_partials || !gathered_target_logit)
        return fail(RLK_ERR_INVALID_ARG, "gathered_partials and gathered_target_logit are required");
    if (!targets) return fail(RLK_ERR_INVALID_ARG, "targets is NULL");
    if (c->mask_mode == RLK_MASK_EXPLICIT && !active_mask)
        return fail(RLK_ERR_INVALID_ARG, "explicit mask mode needs active_mask");
    if (c->mask_mode == RLK_MASK_IGNORE_INDEX && active_mask)
        return fail(RLK_ERR_INVALID_ARG, "ignore_index mode takes no active_mask (pass NULL)");
    if (!logp || !lse) return fail(RLK_ERR_INVALID_ARG, "logp and lse outputs are required");
    if (!workspace || !aligned16(workspace)) return fail(RLK_ERR_INVALID_ARG, "workspace must be non-NULL and 16-byte aligned");
    if ((s = select_device(gathered_partials)) != RLK_OK) return s;
    if ((s = check_device_ptrs({{gathered_target_logit, "gathered_target_logit"}, {targets, "targets"},
                                {active_mask, "active_mask"}, {logp, "logp"}, {lse, "lse"},
                                {workspace, "workspace"}})) != RLK_OK)
        return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if ((s = begin(workspace, st)) != RLK_OK) return s;
    if ((s = launch_gathered_fold(*c, gathered_partials, gathered_target_logit, targets, active_mask, logp, lse,
                                  static_cast<uint32_t*>(workspace), st)) != RLK_OK)
        return s;
    return c->validate ? read_status(workspace, st) : RLK_OK;
}

RLK_EXPORT rlk_status rlk_logp_shard_bwd(const rlk_logp_contract* c, int32_t shard, const void* logits_shard,
                                         const int64_t* targets, const uint8_t* active_mask, const float* lse_in,
                                         const float* grad_logp, void* dlogits_shard, void* workspace,
                                         rlk_stream_t stream) {
    rlk_status s = check_shard(c, shard);
    if (s != RLK_OK) return s;
    if (c->T == 0) return RLK_OK;
    if ((s = check_common(c, logits_shard, targets, active_mask, workspace)) != RLK_OK) return s;
    if (!lse_in || !grad_logp) return fail(RLK_ERR_INVALID_ARG, "lse_in and grad_logp are required");
    if (!dlogits_shard) return fail(RLK_ERR_INVALID_ARG, "dlogits_shard is NULL");
    if (!aligned16(dlogits_shard)) return fail(RLK_ERR_MISALIGNED, "dlogits_shard must be 16-byte aligned");
    if ((s = check_dlogits_overlap(logits_shard, dlogits_shard, c->T,
                                   c->row_stride ? c->row_stride : c->V_padded / c->virtual_tp)) != RLK_OK)
        return s;
    if ((s = select_device(logits_shard)) != RLK_OK) return s;
    if ((s = check_device_ptrs({{targets, "targets"}, {active_mask, "active_mask"}, {lse_in, "lse_in"},
                                {grad_logp, "grad_logp"}, {dlogits_shard, "dlogits_shard"},
                                {workspace, "workspace"}})) != RLK_OK)
        return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if ((s = begin(workspace, st)) != RLK_OK) return s;
    if ((s = launch_shard_bwd(*c, shard, static_cast<const uint16_t*>(logits_shard), targets, active_mask, lse_in,
                              grad_logp, static_cast<uint16_t*>(dlogits_shard),
                              static_cast<unsigned char*>(workspace) + kWorkspaceBytes, static_cast<uint32_t*>(workspace),
                              st)) != RLK_OK)
        return s;
    return c->validate ? read_status(workspace, st) : RLK_OK;
}

// ---------------------------------------------------------------- allocation-free forward
//
// rlk_logp_fwd_noalloc serves callers that may not allocate device memory
// while they run -- an engine whose memory is reserved up front, a plugin
// that is handed a stream but no allocator, a step that must not call the
// synchronising cudaMalloc.  The forward's only scratch (the 256-byte status
// word area that rlk_logp_fwd takes as `workspace`) lives in this file-scope
// array instead; every GPU that loads the library holds it until exit.

namespace rlk {
namespace {

constexpr size_t kNoAllocScratchBytes = 256;
static __device__ __align__(256) unsigned char g_noalloc_scratch[kNoAllocScratchBytes];

using CtxGetCurrentFn = CUresult (*)(CUcontext*);
using CtxGetIdFn = CUresult (*)(CUcontext, unsigned long long*);

// Process-unique id of the calling thread's current CUDA context (the
// driver never reuses one), so that an address looked up in a context that
// has since been destroyed -- by cudaDeviceReset, say -- is never used again.
rlk_status current_context_id(unsigned long long* id) {
    static std::mutex mu;
    static CtxGetCurrentFn get_current = nullptr;
    static CtxGetIdFn get_id = nullptr;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!get_current || !get_id) {
            void* f1 = nullptr;
            void* f2 = nullptr;
            cudaDriverEntryPointQueryResult q1, q2;
            if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &f1, 12000, cudaEnableDefault, &q1) != cudaSuccess ||
                q1 != cudaDriverEntryPointSuccess ||
                cudaGetDriverEntryPointByVersion("cuCtxGetId", &f2, 12000, cudaEnableDefault, &q2) != cudaSuccess ||
                q2 != cudaDriverEntryPointSuccess)
                return fail(RLK_ERR_CUDA, "cannot resolve cuCtxGetCurrent / cuCtxGetId");
            get_current = reinterpret_cast<CtxGetCurrentFn>(f1);
            get_id = reinterpret_cast<CtxGetIdFn>(f2);
        }
    }
    CUcontext ctx = nullptr;
    if (get_current(&ctx) != CUDA_SUCCESS || !ctx || get_id(ctx, id) != CUDA_SUCCESS)
        return fail(RLK_ERR_CUDA, "no current CUDA context");
    return RLK_OK;
}

// Device address of g_noalloc_scratch, looked up (cudaGetSymbolAddress, with
// the device current) once per device and context; in host code the array's
// name is only a host-side stand-in, never a device address.
rlk_status noalloc_scratch(void** out) {
    static std::mutex mu;
    static void* addr[64] = {};
    static unsigned long long ctx_of[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return fail(RLK_ERR_CUDA, std::string("cudaGetDevice: ") + cudaGetErrorString(e));
    if (dev < 0 || dev >= 64) return fail(RLK_ERR_UNSUPPORTED, "device ordinal above 63");
    unsigned long long ctx = 0;
    rlk_status s = current_context_id(&ctx);
    if (s != RLK_OK) return s;
    std::lock_guard<std::mutex> lock(mu);
    if (!addr[dev] || ctx_of[dev] != ctx) {
        void* p = nullptr;
        e = cudaGetSymbolAddress(&p, g_noalloc_scratch);
        if (e != cudaSuccess || !p)
            return fail(RLK_ERR_CUDA, std::string("cudaGetSymbolAddress of the static scratch: ") +
                                          cudaGetErrorString(e));
        addr[dev] = p;
        ctx_of[dev] = ctx;
    }
    *out = addr[dev];
    return RLK_OK;
}

}  // namespace
}  // namespace rlk

RLK_EXPORT rlk_status rlk_logp_fwd_noalloc(const rlk_logp_contract* c, const void* logits_bf16,
                                           const int64_t* targets, const uint8_t* active_mask, float* logp,
                                           float* lse, float* partials, rlk_stream_t stream) {
    rlk_status s = check_contract(c);
    if (s != RLK_OK) return s;
    if (c->T == 0) return RLK_OK;
    if (kWorkspaceBytes > kNoAllocScratchBytes)
        return fail(RLK_ERR_UNSUPPORTED, "this contract needs more scratch than the 256-byte static array; "
                                         "use rlk_logp_fwd with a workspace");
    if (!logits_bf16) return fail(RLK_ERR_INVALID_ARG, "logits is NULL");
    if ((s = select_device(logits_bf16)) != RLK_OK) return s;
    void* scratch = nullptr;
    if ((s = noalloc_scratch(&scratch)) != RLK_OK) return s;
    if ((s = check_common(c, logits_bf16, targets, active_mask, scratch)) != RLK_OK) return s;
    if (!logp || !lse) return fail(RLK_ERR_INVALID_ARG, "logp and lse outputs are required");
    if ((s = check_device_ptrs({{targets, "targets"}, {active_mask, "active_mask"}, {logp, "logp"}, {lse, "lse"},
                                {partials, "partials"}})) != RLK_OK)
        return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if ((s = begin(scratch, st)) != RLK_OK) return s;  // the status word starts at zero on every call
    StreamArgs a{};
    a.logits = static_cast<const uint16_t*>(logits_bf16);
    a.targets = targets;
    a.mask = active_mask;
    a.logp = logp;
    a.lse = lse;
    a.partials = partials;
    a.status = static_cast<uint32_t*>(scratch);
    if ((s = launch_stream(*c, kModeFwd, a, st)) != RLK_OK) return s;
    return c->validate ? read_status(scratch, st) : RLK_OK;
}

namespace rlk {
namespace {
constexpr int64_t kMaxDim8 = ((int64_t)1 << 31) - 512;

// Bytes from the first element of a [rows, stride] buffer to the end of the
// last row's `width` elements of `size` bytes.
int64_t extent(int64_t rows, int64_t stride, int64_t width, int64_t size) {
    return rows <= 0 ? 0 : ((rows - 1) * stride + width) * size;
}

struct Span {
    const void* ptr;
    int64_t bytes;
    const char* name;
};

// The first span (an output) shares no byte with the others; NULL spans are
// optional arguments left out.
rlk_status check_disjoint(const Span& out, std::initializer_list<Span> others) {
    if (!out.ptr) return RLK_OK;
    const uint64_t a = reinterpret_cast<uintptr_t>(out.ptr);
    for (const Span& o : others) {
        const uint64_t b = reinterpret_cast<uintptr_t>(o.ptr);
        if (o.ptr && a < b + (uint64_t)o.bytes && b < a + (uint64_t)out.bytes)
            return fail(RLK_ERR_INVALID_ARG, std::string(out.name) + " overlaps " + o.name);
    }
    return RLK_OK;
}

// No output shares a byte with an input or with another output.
rlk_status check_outputs(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
    for (const Span* o = outs.begin(); o != outs.end(); ++o) {
        const rlk_status s = check_disjoint(*o, ins);
        if (s != RLK_OK) return s;
        for (const Span* p = o + 1; p != outs.end(); ++p) {
            const rlk_status t = check_disjoint(*o, {*p});
            if (t != RLK_OK) return t;
        }
    }
    return RLK_OK;
}

// An E4M3 operand's pointer and row stride (whole 16-byte pieces a row).
rlk_status check_codes(const char* name, const void* p, int64_t stride, int64_t width) {
    if (!aligned16(p)) return fail(RLK_ERR_MISALIGNED, std::string(name) + " must be 16-byte aligned");
    if (stride < width) return fail(RLK_ERR_INVALID_ARG, std::string(name) + "_stride is below its row's length");
    if (stride % 16 != 0) return fail(RLK_ERR_MISALIGNED, std::string(name) + "_stride must be a multiple of 16");
    if (stride > ((int64_t)1 << 38)) return fail(RLK_ERR_UNSUPPORTED, std::string(name) + "_stride above 2^38");
    return RLK_OK;
}

rlk_status check_natural(const char* name, const void* p, int64_t size) {
    if (p && reinterpret_cast<uintptr_t>(p) % (uintptr_t)size != 0)
        return fail(RLK_ERR_MISALIGNED, std::string(name) + " must be aligned to its elements");
    return RLK_OK;
}
}  // namespace
}  // namespace rlk

RLK_EXPORT rlk_status rlk_fp8_quantize(int64_t rows, int64_t cols, const void* x, int32_t x_type, int64_t x_stride,
                                       int32_t block_rows, void* q, int64_t q_stride, float* scale, void* qt,
                                       int64_t qt_stride, float* scale_t, rlk_stream_t stream) {
    rlk_status s;
    if (rows < 0 || cols < 0) return fail(RLK_ERR_INVALID_ARG, "rows and cols must be >= 0");
    if (x_type != RLK_BF16 && x_type != RLK_F32)
        return fail(RLK_ERR_INVALID_ARG, "x_type must be RLK_BF16 or RLK_F32");
    if (block_rows != 1 && block_rows != 128) return fail(RLK_ERR_INVALID_ARG, "block_rows must be 1 or 128");
    if (rows > kMaxDim8 || cols > kMaxDim8) return fail(RLK_ERR_UNSUPPORTED, "rows or cols above 2^31 - 512");
    if (rows == 0 || cols == 0) return RLK_OK;
    if (!x) return fail(RLK_ERR_INVALID_ARG, "x is NULL");
    if (!q && !qt) return fail(RLK_ERR_INVALID_ARG, "q or qt is required");
    if ((q != nullptr) != (scale != nullptr) || (qt != nullptr) != (scale_t != nullptr))
        return fail(RLK_ERR_INVALID_ARG, "q comes with scale and qt with scale_t");
    const int64_t size = x_type == RLK_F32 ? 4 : 2;
    if (x_stride < cols) return fail(RLK_ERR_INVALID_ARG, "x_stride must be >= cols");
    if (x_stride > ((int64_t)1 << 38)) return fail(RLK_ERR_UNSUPPORTED, "x_stride above 2^38");
    if ((s = check_natural("x", x, size)) != RLK_OK) return s;
    if (q && (s = check_codes("q", q, q_stride, cols)) != RLK_OK) return s;
    if (qt && (s = check_codes("qt", qt, qt_stride, rows)) != RLK_OK) return s;
    if ((s = check_natural("scale", scale, 4)) != RLK_OK) return s;
    if ((s = check_natural("scale_t", scale_t, 4)) != RLK_OK) return s;
    const int64_t cg = (cols + 127) / 128, rg = (rows + 127) / 128;
    const Span sx{x, extent(rows, x_stride, cols, size), "x"};
    const Span sq{q, extent(rows, q_stride, cols, 1), "q"};
    const Span sqt{qt, extent(cols, qt_stride, rows, 1), "qt"};
    const Span ss{scale, 4 * cg * (block_rows == 1 ? rows : rg), "scale"};
    const Span sst{scale_t, 4 * rg * (block_rows == 1 ? cols : cg), "scale_t"};
    if ((s = check_disjoint(sq, {sx, sqt, ss, sst})) != RLK_OK) return s;
    if ((s = check_disjoint(sqt, {sx, ss, sst})) != RLK_OK) return s;
    if ((s = check_disjoint(ss, {sx, sst})) != RLK_OK) return s;
    if ((s = check_disjoint(sst, {sx})) != RLK_OK) return s;
    if ((s = select_device(x)) != RLK_OK) return s;
    if ((s = check_device_ptrs({{q, "q"}, {scale, "scale"}, {qt, "qt"}, {scale_t, "scale_t"}})) != RLK_OK) return s;
    return launch_fp8_quantize(rows, cols, x, x_type == RLK_F32, x_stride, block_rows, static_cast<uint8_t*>(q),
                               q_stride, scale, static_cast<uint8_t*>(qt), qt_stride, scale_t,
                               reinterpret_cast<cudaStream_t>(stream));
}

RLK_EXPORT rlk_status rlk_fp8_matmul(int64_t M, int64_t N, int64_t K, const void* a, int64_t a_stride,
                                     const float* a_scale, const void* b, int64_t b_stride, const float* b_scale,
                                     int32_t b_block_rows, void* c, int32_t c_type, int64_t c_stride,
                                     int32_t accumulate, void* workspace, rlk_stream_t stream) {
    rlk_status s;
    if (M < 0 || N < 0) return fail(RLK_ERR_INVALID_ARG, "M and N must be >= 0");
    if (K < 1) return fail(RLK_ERR_INVALID_ARG, "K must be >= 1");
    if (b_block_rows != 1 && b_block_rows != 128) return fail(RLK_ERR_INVALID_ARG, "b_block_rows must be 1 or 128");
    if (c_type != RLK_BF16 && c_type != RLK_F32)
        return fail(RLK_ERR_INVALID_ARG, "c_type must be RLK_BF16 or RLK_F32");
    if (accumulate != 0 && accumulate != 1) return fail(RLK_ERR_INVALID_ARG, "accumulate must be 0 or 1");
    if (accumulate && c_type != RLK_F32) return fail(RLK_ERR_INVALID_ARG, "accumulate needs an RLK_F32 c");
    if (M > kMaxDim8 || N > kMaxDim8 || K > kMaxDim8 ||
        ((M + 127) / 128) * ((N + 127) / 128) > ((int64_t)1 << 30))
        return fail(RLK_ERR_UNSUPPORTED, "M, N or K above 2^31 - 512, or above 2^30 tiles of 128 x 128");
    if (M == 0 || N == 0) return RLK_OK;
    if (!a || !b || !a_scale || !b_scale || !c)
        return fail(RLK_ERR_INVALID_ARG, "a, a_scale, b, b_scale and c are required");
    if (!workspace) return fail(RLK_ERR_INVALID_ARG, "workspace is NULL");
    if (!aligned16(workspace)) return fail(RLK_ERR_MISALIGNED, "workspace must be 16-byte aligned");
    if ((s = check_codes("a", a, a_stride, K)) != RLK_OK) return s;
    if ((s = check_codes("b", b, b_stride, K)) != RLK_OK) return s;
    if ((s = check_natural("a_scale", a_scale, 4)) != RLK_OK) return s;
    if ((s = check_natural("b_scale", b_scale, 4)) != RLK_OK) return s;
    const int64_t size = c_type == RLK_F32 ? 4 : 2, groups = (K + 127) / 128;
    if ((s = check_natural("c", c, size)) != RLK_OK) return s;
    if (c_stride < N) return fail(RLK_ERR_INVALID_ARG, "c_stride must be >= N");
    if (c_stride > ((int64_t)1 << 38)) return fail(RLK_ERR_UNSUPPORTED, "c_stride above 2^38");
    if ((s = check_disjoint({c, extent(M, c_stride, N, size), "c"},
                            {{a, extent(M, a_stride, K, 1), "a"},
                             {b, extent(N, b_stride, K, 1), "b"},
                             {a_scale, 4 * groups * M, "a_scale"},
                             {b_scale, 4 * groups * (b_block_rows == 1 ? N : (N + 127) / 128), "b_scale"},
                             {workspace, RLK_FP8_WORKSPACE, "workspace"}})) != RLK_OK)
        return s;
    if ((s = select_device(a)) != RLK_OK) return s;
    if ((s = check_device_ptrs({{a_scale, "a_scale"}, {b, "b"}, {b_scale, "b_scale"}, {c, "c"},
                                {workspace, "workspace"}})) != RLK_OK)
        return s;
    return launch_fp8_matmul(M, N, K, a, a_stride, a_scale, b, b_stride, b_scale, b_block_rows, c, c_stride,
                             c_type == RLK_F32, accumulate, static_cast<uint32_t*>(workspace),
                             reinterpret_cast<cudaStream_t>(stream));
}

namespace rlk {
namespace {
constexpr int64_t kMaxRows8 = (int64_t)1 << 30;  // rows of groups: with their padding below 2^31

rlk_status check_type(const char* name, int32_t type) {
    if (type != RLK_BF16 && type != RLK_F32)
        return fail(RLK_ERR_INVALID_ARG, std::string(name) + " must be RLK_BF16 or RLK_F32");
    return RLK_OK;
}

rlk_status check_act(int32_t activation, int32_t gated, int64_t N) {
    if (activation < RLK_ACT_NONE || activation > RLK_ACT_GELU_TANH)
        return fail(RLK_ERR_INVALID_ARG, "activation must be one of rlk_activation");
    if (gated != 0 && gated != 1) return fail(RLK_ERR_INVALID_ARG, "gated must be 0 or 1");
    if (gated && N % 64 != 0)
        return fail(RLK_ERR_UNSUPPORTED, "a gated layer's columns must be a multiple of 64");
    return RLK_OK;
}

rlk_status check_stride(const char* name, int64_t stride, int64_t width) {
    if (stride < width) return fail(RLK_ERR_INVALID_ARG, std::string(name) + "_stride is below its row's length");
    if (stride > ((int64_t)1 << 38)) return fail(RLK_ERR_UNSUPPORTED, std::string(name) + "_stride above 2^38");
    return RLK_OK;
}

// A stride between groups' matrices of E4M3, or between their results (multiple 1).
rlk_status check_group_stride(const char* name, int64_t groups, int64_t stride, int64_t least, int64_t multiple) {
    if (groups <= 1) return RLK_OK;
    if (stride < least) return fail(RLK_ERR_INVALID_ARG, std::string(name) + " is below a matrix's length");
    if (stride % multiple != 0) return fail(RLK_ERR_MISALIGNED, std::string(name) + " must be a multiple of 16");
    if (stride > ((int64_t)1 << 38)) return fail(RLK_ERR_UNSUPPORTED, std::string(name) + " above 2^38");
    return RLK_OK;
}

rlk_status check_groups(int64_t groups, int64_t rows) {
    if (groups < 1) return fail(RLK_ERR_INVALID_ARG, "groups must be >= 1");
    if (groups > 1024) return fail(RLK_ERR_UNSUPPORTED, "more than 1024 groups");
    if (rows > kMaxRows8) return fail(RLK_ERR_UNSUPPORTED, "above 2^30 rows of groups");
    return RLK_OK;
}

int64_t type_size(int32_t type) { return type == RLK_F32 ? 4 : 2; }

// Both products with an epilogue (groups 0: one B).
rlk_status matmul_act(int64_t groups, int64_t M, int64_t N, int64_t K, const int32_t* ends, const void* a,
                      int64_t a_stride, const float* a_scale, const void* b, int64_t b_stride, int64_t b_group_stride,
                      const float* b_scale, const rlk_fp8_epilogue* e, void* c, int32_t c_type, int64_t c_stride,
                      int32_t zero_rest, void* workspace, cudaStream_t stream) {
    rlk_status s;
    if (M < 0 || N < 0) return fail(RLK_ERR_INVALID_ARG, "M and N must be >= 0");
    if (K < 1) return fail(RLK_ERR_INVALID_ARG, "K must be >= 1");
    if (groups > 0 && (s = check_groups(groups, M)) != RLK_OK) return s;
    if (zero_rest != 0 && zero_rest != 1) return fail(RLK_ERR_INVALID_ARG, "zero_rest must be 0 or 1");
    if ((s = check_type("c_type", c_type)) != RLK_OK) return s;
    const bool gated = e && e->gated;
    if (e) {
        if ((s = check_act(e->activation, e->gated, N)) != RLK_OK) return s;
        if (e->bias && (s = check_type("bias_type", e->bias_type)) != RLK_OK) return s;
        if (e->residual && (s = check_type("residual_type", e->residual_type)) != RLK_OK) return s;
        if (e->residual && groups > 0)
            return fail(RLK_ERR_UNSUPPORTED, "a residual of groups' rows is not supported");
    }
    if (M > kMaxDim8 || N > kMaxDim8 / 2 || K > kMaxDim8)
        return fail(RLK_ERR_UNSUPPORTED, "M or K above 2^31 - 512, or N above 2^30 - 256");
    const int64_t wide = gated ? 2 * N : N, count = groups > 0 ? groups : 1, kg = (K + 127) / 128;
    if ((M / 16 + count + 1) * ((wide + 127) / 128) > ((int64_t)1 << 30))
        return fail(RLK_ERR_UNSUPPORTED, "above 2^30 tiles of 16 x 128");
    if (M == 0 || N == 0) return RLK_OK;
    if (!a || !b || !a_scale || !b_scale || !c || (groups > 0 && !ends))
        return fail(RLK_ERR_INVALID_ARG, groups > 0 ? "ends, a, a_scale, b, b_scale and c are required"
                                                    : "a, a_scale, b, b_scale and c are required");
    if (!workspace) return fail(RLK_ERR_INVALID_ARG, "workspace is NULL");
    if (!aligned16(workspace)) return fail(RLK_ERR_MISALIGNED, "workspace must be 16-byte aligned");
    if ((s = check_codes("a", a, a_stride, K)) != RLK_OK) return s;
    if ((s = check_codes("b", b, b_stride, K)) != RLK_OK) return s;
    const int64_t b_bytes = extent(wide, b_stride, K, 1);
    if ((s = check_group_stride("b_group_stride", groups, b_group_stride, b_bytes, 16)) != RLK_OK) return s;
    if (gated && N * b_stride >= ((int64_t)1 << 40))
        return fail(RLK_ERR_UNSUPPORTED, "N * b_stride of a gated b above 2^40");
    if ((s = check_natural("ends", ends, 4)) != RLK_OK) return s;
    if ((s = check_natural("a_scale", a_scale, 4)) != RLK_OK) return s;
    if ((s = check_natural("b_scale", b_scale, 4)) != RLK_OK) return s;
    if ((s = check_natural("c", c, type_size(c_type))) != RLK_OK) return s;
    if ((s = check_stride("c", c_stride, N)) != RLK_OK) return s;
    Span bias{nullptr, 0, "bias"}, res{nullptr, 0, "residual"}, z{nullptr, 0, "z"};
    if (e && e->bias) {
        if ((s = check_natural("bias", e->bias, type_size(e->bias_type))) != RLK_OK) return s;
        bias = Span{e->bias, count * wide * type_size(e->bias_type), "bias"};
    }
    if (e && e->residual) {
        if ((s = check_natural("residual", e->residual, type_size(e->residual_type))) != RLK_OK) return s;
        if ((s = check_stride("residual", e->residual_stride, N)) != RLK_OK) return s;
        res = Span{e->residual, extent(M, e->residual_stride, N, type_size(e->residual_type)), "residual"};
    }
    if (e && e->z) {
        if ((s = check_natural("z", e->z, 2)) != RLK_OK) return s;
        if ((s = check_stride("z", e->z_stride, wide)) != RLK_OK) return s;
        z = Span{e->z, extent(M, e->z_stride, wide, 2), "z"};
    }
    const Span out{c, extent(M, c_stride, N, type_size(c_type)), "c"}, ws{workspace, RLK_FP8_WORKSPACE, "workspace"};
    const Span sa{a, extent(M, a_stride, K, 1), "a"}, sb{b, (count - 1) * b_group_stride + b_bytes, "b"};
    const Span sas{a_scale, 4 * kg * M, "a_scale"}, sbs{b_scale, 4 * count * kg * ((wide + 127) / 128), "b_scale"};
    const Span se{ends, 4 * groups, "ends"};
    if ((s = check_outputs({out, z, ws}, {sa, sb, sas, sbs, se, bias})) != RLK_OK) return s;
    if ((s = check_outputs({z, ws}, {res})) != RLK_OK) return s;
    // in place: each element of the residual is read by the thread block that writes its place, before it does
    const bool in_place = res.ptr == c && e && e->residual_type == c_type && e->residual_stride == c_stride;
    if (!in_place && (s = check_disjoint(out, {res})) != RLK_OK) return s;
    if ((s = select_device(a)) != RLK_OK) return s;
    if ((s = check_device_ptrs({{a_scale, "a_scale"}, {b, "b"}, {b_scale, "b_scale"}, {c, "c"}, {ends, "ends"},
                                {bias.ptr, "bias"}, {res.ptr, "residual"}, {z.ptr, "z"},
                                {workspace, "workspace"}})) != RLK_OK)
        return s;
    uint32_t* status = static_cast<uint32_t*>(workspace);
    if (groups > 0)
        return launch_fp8_grouped_matmul(groups, M, N, K, ends, a, a_stride, a_scale, b, b_stride, b_group_stride,
                                         b_scale, e, c, c_stride, c_type == RLK_F32, zero_rest, status, stream);
    return launch_fp8_matmul_act(M, N, K, a, a_stride, a_scale, b, b_stride, b_scale, e, c, c_stride,
                                 c_type == RLK_F32, status, stream);
}

// The outputs of a quantisation along rows and along groups of rows: pointers, strides and their spans.
rlk_status check_quantized(int64_t rows, int64_t cols, int64_t deep, int64_t tiles, void* q, int64_t q_stride,
                           float* scale, void* qt, int64_t qt_stride, float* scale_t, Span (&out)[4]) {
    rlk_status s;
    if ((q != nullptr) != (scale != nullptr) || (qt != nullptr) != (scale_t != nullptr))
        return fail(RLK_ERR_INVALID_ARG, "q comes with scale and qt with scale_t");
    if (q && (s = check_codes("q", q, q_stride, cols)) != RLK_OK) return s;
    if (qt && (s = check_codes("qt", qt, qt_stride, deep)) != RLK_OK) return s;
    if ((s = check_natural("scale", scale, 4)) != RLK_OK) return s;
    if ((s = check_natural("scale_t", scale_t, 4)) != RLK_OK) return s;
    out[0] = Span{q, extent(rows, q_stride, cols, 1), "q"};
    out[1] = Span{scale, 4 * ((cols + 127) / 128) * rows, "scale"};
    out[2] = Span{qt, extent(cols, qt_stride, deep, 1), "qt"};
    out[3] = Span{scale_t, 4 * tiles * cols, "scale_t"};
    return RLK_OK;
}
}  // namespace
}  // namespace rlk

RLK_EXPORT rlk_status rlk_fp8_matmul_act(int64_t M, int64_t N, int64_t K, const void* a, int64_t a_stride,
                                         const float* a_scale, const void* b, int64_t b_stride, const float* b_scale,
                                         const rlk_fp8_epilogue* epilogue, void* c, int32_t c_type, int64_t c_stride,
                                         void* workspace, rlk_stream_t stream) {
    return matmul_act(0, M, N, K, nullptr, a, a_stride, a_scale, b, b_stride, 0, b_scale, epilogue, c, c_type,
                      c_stride, 0, workspace, reinterpret_cast<cudaStream_t>(stream));
}

RLK_EXPORT rlk_status rlk_fp8_grouped_matmul(int64_t groups, int64_t M, int64_t N, int64_t K, const int32_t* ends,
                                             const void* a, int64_t a_stride, const float* a_scale, const void* b,
                                             int64_t b_stride, int64_t b_group_stride, const float* b_scale,
                                             const rlk_fp8_epilogue* epilogue, void* c, int32_t c_type,
                                             int64_t c_stride, int32_t zero_rest, void* workspace,
                                             rlk_stream_t stream) {
    if (groups < 1) return fail(RLK_ERR_INVALID_ARG, "groups must be >= 1");
    return matmul_act(groups, M, N, K, ends, a, a_stride, a_scale, b, b_stride, b_group_stride, b_scale, epilogue, c,
                      c_type, c_stride, zero_rest, workspace, reinterpret_cast<cudaStream_t>(stream));
}

RLK_EXPORT rlk_status rlk_fp8_quantize_grouped(int64_t groups, int64_t rows, int64_t cols, const int32_t* ends,
                                               const void* x, int32_t x_type, int64_t x_stride, void* q,
                                               int64_t q_stride, float* scale, void* qt, int64_t qt_stride,
                                               float* scale_t, rlk_stream_t stream) {
    rlk_status s;
    if (rows < 0 || cols < 0) return fail(RLK_ERR_INVALID_ARG, "rows and cols must be >= 0");
    if ((s = check_groups(groups, rows)) != RLK_OK) return s;
    if ((s = check_type("x_type", x_type)) != RLK_OK) return s;
    if (cols > kMaxDim8) return fail(RLK_ERR_UNSUPPORTED, "cols above 2^31 - 512");
    if (rows == 0 || cols == 0) return RLK_OK;
    if (!x || !ends) return fail(RLK_ERR_INVALID_ARG, "x and ends are required");
    if (!q && !qt) return fail(RLK_ERR_INVALID_ARG, "q or qt is required");
    if ((s = check_stride("x", x_stride, cols)) != RLK_OK) return s;
    if ((s = check_natural("x", x, type_size(x_type))) != RLK_OK) return s;
    if ((s = check_natural("ends", ends, 4)) != RLK_OK) return s;
    const int64_t tiles = group_row_tiles(groups, rows);
    Span o[4];
    if ((s = check_quantized(rows, cols, 128 * tiles, tiles, q, q_stride, scale, qt, qt_stride, scale_t, o)) != RLK_OK)
        return s;
    if ((s = check_outputs({o[0], o[1], o[2], o[3]}, {{x, extent(rows, x_stride, cols, type_size(x_type)), "x"},
                                                      {ends, 4 * groups, "ends"}})) != RLK_OK)
        return s;
    if ((s = select_device(x)) != RLK_OK) return s;
    if ((s = check_device_ptrs({{ends, "ends"}, {q, "q"}, {scale, "scale"}, {qt, "qt"}, {scale_t, "scale_t"}})) !=
        RLK_OK)
        return s;
    return launch_fp8_quantize_grouped(groups, rows, cols, ends, x, x_type == RLK_F32, x_stride,
                                       static_cast<uint8_t*>(q), q_stride, scale, static_cast<uint8_t*>(qt),
                                       qt_stride, scale_t, reinterpret_cast<cudaStream_t>(stream));
}

RLK_EXPORT rlk_status rlk_fp8_quantize_batch(int64_t count, int64_t rows, int64_t cols, const void* x, int32_t x_type,
                                             int64_t x_stride, int64_t x_batch_stride, void* q, int64_t q_stride,
                                             int64_t q_batch_stride, float* scale, void* qt, int64_t qt_stride,
                                             int64_t qt_batch_stride, float* scale_t, rlk_stream_t stream) {
    rlk_status s;
    if (count < 0 || rows < 0 || cols < 0) return fail(RLK_ERR_INVALID_ARG, "count, rows and cols must be >= 0");
    if ((s = check_type("x_type", x_type)) != RLK_OK) return s;
    const int64_t rg = (rows + 127) / 128, cg = (cols + 127) / 128;
    if (rows > kMaxDim8 || cols > kMaxDim8 || count > ((int64_t)1 << 20) || (rg > 0 && count > ((int64_t)1 << 30) / rg))
        return fail(RLK_ERR_UNSUPPORTED, "rows or cols above 2^31 - 512, or above 2^20 matrices or 2^30 blocks of rows");
    if (count == 0 || rows == 0 || cols == 0) return RLK_OK;
    if (!x) return fail(RLK_ERR_INVALID_ARG, "x is NULL");
    if (!q && !qt) return fail(RLK_ERR_INVALID_ARG, "q or qt is required");
    if ((s = check_stride("x", x_stride, cols)) != RLK_OK) return s;
    if ((s = check_natural("x", x, type_size(x_type))) != RLK_OK) return s;
    const int64_t one = extent(rows, x_stride, cols, 1), size = type_size(x_type);
    if ((s = check_group_stride("x_batch_stride", count, x_batch_stride, one, 1)) != RLK_OK) return s;
    Span o[4];
    if ((s = check_quantized(rows, cols, rows, rg, q, q_stride, scale, qt, qt_stride, scale_t, o)) != RLK_OK) return s;
    if (q && (s = check_group_stride("q_batch_stride", count, q_batch_stride, o[0].bytes, 16)) != RLK_OK) return s;
    if (qt && (s = check_group_stride("qt_batch_stride", count, qt_batch_stride, o[2].bytes, 16)) != RLK_OK) return s;
    if (count > 1) o[0].bytes += (count - 1) * q_batch_stride, o[2].bytes += (count - 1) * qt_batch_stride;
    o[1].bytes = o[3].bytes = 4 * count * rg * cg;
    const int64_t x_bytes = (one + (count > 1 ? (count - 1) * x_batch_stride : 0)) * size;
    if ((s = check_outputs({o[0], o[1], o[2], o[3]}, {{x, x_bytes, "x"}})) != RLK_OK) return s;
    if ((s = select_device(x)) != RLK_OK) return s;
    if ((s = check_device_ptrs({{q, "q"}, {scale, "scale"}, {qt, "qt"}, {scale_t, "scale_t"}})) != RLK_OK) return s;
    return launch_fp8_quantize_batch(count, rows, cols, x, x_type == RLK_F32, x_stride, x_batch_stride,
                                     static_cast<uint8_t*>(q), q_stride, q_batch_stride, scale,
                                     static_cast<uint8_t*>(qt), qt_stride, qt_batch_stride, scale_t,
                                     reinterpret_cast<cudaStream_t>(stream));
}

RLK_EXPORT rlk_status rlk_fp8_grouped_dweight(int64_t groups, int64_t rows, int64_t M, int64_t N, const int32_t* ends,
                                              const void* a, int64_t a_stride, const float* a_scale, const void* b,
                                              int64_t b_stride, const float* b_scale, void* c, int32_t c_type,
                                              int64_t c_stride, int64_t c_group_stride, int32_t accumulate,
                                              void* workspace, rlk_stream_t stream) {
    rlk_status s;
    if (rows < 1 || M < 0 || N < 0) return fail(RLK_ERR_INVALID_ARG, "rows must be >= 1, M and N >= 0");
    if ((s = check_groups(groups, rows)) != RLK_OK) return s;
    if ((s = check_type("c_type", c_type)) != RLK_OK) return s;
    if (accumulate != 0 && accumulate != 1) return fail(RLK_ERR_INVALID_ARG, "accumulate must be 0 or 1");
    if (accumulate && c_type != RLK_F32) return fail(RLK_ERR_INVALID_ARG, "accumulate needs an RLK_F32 c");
    if (M > kMaxDim8 || N > kMaxDim8 || groups * ((M + 255) / 256) * ((N + 255) / 256) > ((int64_t)1 << 30))
        return fail(RLK_ERR_UNSUPPORTED, "M or N above 2^31 - 512, or above 2^30 tiles of 256 x 256");
    if (M == 0 || N == 0) return RLK_OK;
    if (!ends || !a || !b || !a_scale || !b_scale || !c)
        return fail(RLK_ERR_INVALID_ARG, "ends, a, a_scale, b, b_scale and c are required");
    if (!workspace) return fail(RLK_ERR_INVALID_ARG, "workspace is NULL");
    if (!aligned16(workspace)) return fail(RLK_ERR_MISALIGNED, "workspace must be 16-byte aligned");
    const int64_t tiles = group_row_tiles(groups, rows), deep = 128 * tiles, size = type_size(c_type);
    if ((s = check_codes("a", a, a_stride, deep)) != RLK_OK) return s;
    if ((s = check_codes("b", b, b_stride, deep)) != RLK_OK) return s;
    if ((s = check_natural("ends", ends, 4)) != RLK_OK) return s;
    if ((s = check_natural("a_scale", a_scale, 4)) != RLK_OK) return s;
    if ((s = check_natural("b_scale", b_scale, 4)) != RLK_OK) return s;
    if ((s = check_natural("c", c, size)) != RLK_OK) return s;
    if ((s = check_stride("c", c_stride, N)) != RLK_OK) return s;
    const int64_t one = extent(M, c_stride, N, 1);
    if ((s = check_group_stride("c_group_stride", groups, c_group_stride, one, 1)) != RLK_OK) return s;
    const Span out{c, (one + (groups > 1 ? (groups - 1) * c_group_stride : 0)) * size, "c"};
    if ((s = check_outputs({out, {workspace, RLK_FP8_WORKSPACE, "workspace"}},
                           {{a, extent(M, a_stride, deep, 1), "a"},
                            {b, extent(N, b_stride, deep, 1), "b"},
                            {a_scale, 4 * tiles * M, "a_scale"},
                            {b_scale, 4 * tiles * N, "b_scale"},
                            {ends, 4 * groups, "ends"}})) != RLK_OK)
        return s;
    if ((s = select_device(a)) != RLK_OK) return s;
    if ((s = check_device_ptrs({{ends, "ends"}, {a_scale, "a_scale"}, {b, "b"}, {b_scale, "b_scale"}, {c, "c"},
                                {workspace, "workspace"}})) != RLK_OK)
        return s;
    return launch_fp8_grouped_dweight(groups, rows, M, N, ends, a, a_stride, a_scale, b, b_stride, b_scale, c,
                                      c_stride, c_group_stride, c_type == RLK_F32, accumulate,
                                      static_cast<uint32_t*>(workspace), reinterpret_cast<cudaStream_t>(stream));
}

RLK_EXPORT size_t rlk_fp8_act_grad_workspace_size(int64_t groups, int64_t rows, int64_t cols, int32_t gated) {
    if (groups < 0 || rows < 0 || cols < 0 || rows > kMaxDim8 || cols > kMaxDim8 / 2) return 0;
    const int64_t tiles = groups > 0 ? group_row_tiles(groups, rows) : (rows + 127) / 128;
    return (size_t)(4 * tiles * cols * (gated ? 2 : 1));
}

RLK_EXPORT rlk_status rlk_fp8_act_grad(int64_t groups, int64_t rows, int64_t cols, const int32_t* ends, const void* dy,
                                       int32_t dy_type, int64_t dy_stride, const void* z, int64_t z_stride,
                                       int32_t activation, int32_t gated, void* q, int64_t q_stride, float* scale,
                                       void* qt, int64_t qt_stride, float* scale_t, void* dbias, int32_t dbias_type,
                                       void* workspace, rlk_stream_t stream) {
    rlk_status s;
    if (rows < 1 || cols < 0) return fail(RLK_ERR_INVALID_ARG, "rows must be >= 1 and cols >= 0");
    if (groups < 0) return fail(RLK_ERR_INVALID_ARG, "groups must be >= 0");
    if (groups > 0 && (s = check_groups(groups, rows)) != RLK_OK) return s;
    if ((s = check_type("dy_type", dy_type)) != RLK_OK) return s;
    if ((s = check_act(activation, gated, cols)) != RLK_OK) return s;
    if (dbias && (s = check_type("dbias_type", dbias_type)) != RLK_OK) return s;
    if (rows > kMaxDim8 || cols > kMaxDim8 / 2)
        return fail(RLK_ERR_UNSUPPORTED, "rows above 2^31 - 512 or cols above 2^30 - 256");
    if (cols == 0) return RLK_OK;
    const int64_t wide = gated ? 2 * cols : cols;
    const bool need_z = activation != RLK_ACT_NONE || gated;
    if (!dy || (need_z && !z) || (groups > 0 && !ends))
        return fail(RLK_ERR_INVALID_ARG, "dy, z (with an activation or a gate) and ends (with groups) are required");
    if (!q && !qt && !dbias) return fail(RLK_ERR_INVALID_ARG, "q, qt or dbias is required");
    if (dbias && !workspace) return fail(RLK_ERR_INVALID_ARG, "dbias needs a workspace");
    if (dbias && !aligned16(workspace)) return fail(RLK_ERR_MISALIGNED, "workspace must be 16-byte aligned");
    if ((s = check_stride("dy", dy_stride, cols)) != RLK_OK) return s;
    if ((s = check_natural("dy", dy, type_size(dy_type))) != RLK_OK) return s;
    if (need_z && (s = check_stride("z", z_stride, wide)) != RLK_OK) return s;
    if (need_z && (s = check_natural("z", z, 2)) != RLK_OK) return s;
    if ((s = check_natural("ends", ends, 4)) != RLK_OK) return s;
    if (dbias && (s = check_natural("dbias", dbias, type_size(dbias_type))) != RLK_OK) return s;
    const int64_t tiles = groups > 0 ? group_row_tiles(groups, rows) : (rows + 127) / 128;
    Span o[4];
    if ((s = check_quantized(rows, wide, groups > 0 ? 128 * tiles : rows, tiles, q, q_stride, scale, qt, qt_stride,
                             scale_t, o)) != RLK_OK)
        return s;
    const Span db{dbias, (groups > 0 ? groups : 1) * wide * type_size(dbias_type), "dbias"};
    const Span ws{dbias ? workspace : nullptr, 4 * tiles * wide, "workspace"};
    if ((s = check_outputs({o[0], o[1], o[2], o[3], db, ws},
                           {{dy, extent(rows, dy_stride, cols, type_size(dy_type)), "dy"},
                            {need_z ? z : nullptr, extent(rows, z_stride, wide, 2), "z"},
                            {groups > 0 ? ends : nullptr, 4 * groups, "ends"}})) != RLK_OK)
        return s;
    if ((s = select_device(dy)) != RLK_OK) return s;
    if ((s = check_device_ptrs({{need_z ? z : nullptr, "z"}, {groups > 0 ? ends : nullptr, "ends"}, {q, "q"},
                                {scale, "scale"}, {qt, "qt"}, {scale_t, "scale_t"}, {dbias, "dbias"},
                                {ws.ptr, "workspace"}})) != RLK_OK)
        return s;
    return launch_fp8_act_grad(groups, rows, wide, ends, dy, dy_type == RLK_F32, dy_stride, z, z_stride, activation,
                               gated, static_cast<uint8_t*>(q), q_stride, scale, static_cast<uint8_t*>(qt), qt_stride,
                               scale_t, dbias, dbias_type == RLK_F32, static_cast<float*>(workspace),
                               reinterpret_cast<cudaStream_t>(stream));
}

namespace rlk {
namespace {
rlk_status check_ce(const rlk_linear_ce_contract* c) {
    if (!c) return fail(RLK_ERR_INVALID_ARG, "contract is NULL");
    if (c->T < 0) return fail(RLK_ERR_INVALID_ARG, "T must be >= 0");
    if (c->V < 1 || c->H < 1) return fail(RLK_ERR_INVALID_ARG, "V and H must be >= 1");
    if (c->T > ((int64_t)1 << 31) - 512 || c->V > ((int64_t)1 << 31) - 512)
        return fail(RLK_ERR_UNSUPPORTED, "T or V above 2^31 - 512");
    if (c->H > ((int64_t)1 << 20)) return fail(RLK_ERR_UNSUPPORTED, "hidden size H above 2^20");
    const int64_t tb = (c->T + 255) / 256, vb = (c->V + 255) / 256, hb = (c->H + 255) / 256, most = (int64_t)1 << 30;
    if (tb * vb > most || tb * hb > most || vb * hb > most)
        return fail(RLK_ERR_UNSUPPORTED, "above 2^30 tiles of 256 x 256 of the logits or of a gradient");
    const struct {
        int64_t stride;
        const char* name;
    } strides[] = {{c->hidden_stride, "hidden_stride"},
                   {c->weight_stride, "weight_stride"},
                   {c->dhidden_stride, "dhidden_stride"},
                   {c->dweight_stride, "dweight_stride"}};
    for (const auto& s : strides) {
        const int64_t v = s.stride ? s.stride : c->H;
        if (v < c->H) return fail(RLK_ERR_INVALID_ARG, std::string(s.name) + " must be >= H");
        if (v % 8 != 0)
            return fail(RLK_ERR_MISALIGNED, std::string(s.name) + " must be a multiple of 8 elements (16-byte rows)");
        if (v > ((int64_t)1 << 36)) return fail(RLK_ERR_UNSUPPORTED, std::string(s.name) + " above 2^36");
    }
    if (c->mask_mode != RLK_MASK_EXPLICIT && c->mask_mode != RLK_MASK_IGNORE_INDEX)
        return fail(RLK_ERR_INVALID_ARG, "mask_mode must be RLK_MASK_EXPLICIT or RLK_MASK_IGNORE_INDEX");
    if (c->reduction != RLK_REDUCE_NONE && c->reduction != RLK_REDUCE_SUM && c->reduction != RLK_REDUCE_MEAN)
        return fail(RLK_ERR_INVALID_ARG, "reduction must be RLK_REDUCE_NONE, _SUM or _MEAN");
    if (c->validate != 0 && c->validate != 1) return fail(RLK_ERR_INVALID_ARG, "validate must be 0 or 1");
    if (c->wait_timeout_ns < 0) return fail(RLK_ERR_INVALID_ARG, "wait_timeout_ns must be >= 0");
    if (c->piece < 0) return fail(RLK_ERR_INVALID_ARG, "piece must be >= 0");
    if (!(c->label_smoothing >= 0.f && c->label_smoothing <= 1.f))
        return fail(RLK_ERR_INVALID_ARG, "label_smoothing must be in [0, 1]");
    if (!(c->z_loss >= 0.f) || !isfinite(c->z_loss))
        return fail(RLK_ERR_INVALID_ARG, "z_loss must be finite and >= 0");
    if (!(c->softcap >= 0.f) || !isfinite(c->softcap) || (c->softcap > 0.f && c->softcap < 1e-6f))
        return fail(RLK_ERR_INVALID_ARG, "softcap must be 0 or a finite value of at least 1e-6");
    return RLK_OK;
}

rlk_linear_ce_contract with_strides(const rlk_linear_ce_contract& c) {
    rlk_linear_ce_contract f = c;
    if (!f.hidden_stride) f.hidden_stride = f.H;
    if (!f.weight_stride) f.weight_stride = f.H;
    if (!f.dhidden_stride) f.dhidden_stride = f.H;
    if (!f.dweight_stride) f.dweight_stride = f.H;
    return f;
}

rlk_status check_ce_inputs(const rlk_linear_ce_contract& c, const void* hidden, const void* weight,
                           const int64_t* targets, const uint8_t* mask, const void* workspace) {
    if (!hidden || !weight) return fail(RLK_ERR_INVALID_ARG, "hidden and weight are required");
    if (!aligned16(hidden) || !aligned16(weight))
        return fail(RLK_ERR_MISALIGNED, "hidden and weight must be 16-byte aligned");
    if (!targets) return fail(RLK_ERR_INVALID_ARG, "targets is NULL");
    if (c.mask_mode == RLK_MASK_EXPLICIT && !mask)
        return fail(RLK_ERR_INVALID_ARG, "explicit mask mode needs active_mask");
    if (c.mask_mode == RLK_MASK_IGNORE_INDEX && mask)
        return fail(RLK_ERR_INVALID_ARG, "ignore_index mode takes no active_mask (pass NULL)");
    if (!workspace) return fail(RLK_ERR_INVALID_ARG, "workspace is NULL");
    if (!aligned16(workspace)) return fail(RLK_ERR_MISALIGNED, "workspace must be 16-byte aligned");
    return RLK_OK;
}
}  // namespace
}  // namespace rlk

RLK_EXPORT rlk_status rlk_linear_ce_check(const rlk_linear_ce_contract* contract) { return check_ce(contract); }

RLK_EXPORT size_t rlk_linear_ce_workspace_size(const rlk_linear_ce_contract* contract, int32_t with_grad) {
    if (check_ce(contract) != RLK_OK) return 0;
    return contract->T == 0 ? kWorkspaceBytes : linear_ce_workspace(with_strides(*contract), with_grad != 0);
}

RLK_EXPORT rlk_status rlk_linear_ce_fwd(const rlk_linear_ce_contract* contract, const void* hidden_bf16,
                                        const void* weight_bf16, const int64_t* targets, const uint8_t* active_mask,
                                        float* loss, float* lse, void* workspace, rlk_stream_t stream) {
    rlk_status s = check_ce(contract);
    if (s != RLK_OK) return s;
    const rlk_linear_ce_contract c = with_strides(*contract);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (c.T == 0) {
        if (c.reduction == RLK_REDUCE_NONE) return RLK_OK;
        if (!loss) return fail(RLK_ERR_INVALID_ARG, "loss output is required");
        if ((s = select_device(loss)) != RLK_OK) return s;
        return cudaMemsetAsync(loss, 0, sizeof(float), st) == cudaSuccess
                   ? RLK_OK
                   : fail(RLK_ERR_CUDA, "clearing the loss of no rows");
    }
    if ((s = check_ce_inputs(c, hidden_bf16, weight_bf16, targets, active_mask, workspace)) != RLK_OK) return s;
    if (!loss || !lse) return fail(RLK_ERR_INVALID_ARG, "loss and lse outputs are required");
    if ((s = check_outputs({{loss, c.reduction == RLK_REDUCE_NONE ? 4 * c.T : 4, "loss"},
                            {lse, 4 * c.T, "lse"},
                            {workspace, (int64_t)linear_ce_workspace(c, false), "workspace"}},
                           {{hidden_bf16, extent(c.T, c.hidden_stride, c.H, 2), "hidden"},
                            {weight_bf16, extent(c.V, c.weight_stride, c.H, 2), "weight"},
                            {targets, 8 * c.T, "targets"},
                            {active_mask, c.T, "active_mask"}})) != RLK_OK)
        return s;
    if ((s = select_device(hidden_bf16)) != RLK_OK) return s;
    if ((s = check_device_ptrs({{weight_bf16, "weight"}, {targets, "targets"}, {active_mask, "active_mask"},
                                {loss, "loss"}, {lse, "lse"}, {workspace, "workspace"}})) != RLK_OK)
        return s;
    if ((s = launch_linear_ce_fwd(c, hidden_bf16, weight_bf16, targets, active_mask, loss, lse, workspace, st)) !=
        RLK_OK)
        return s;
    return c.validate ? read_status(workspace, st) : RLK_OK;
}

RLK_EXPORT rlk_status rlk_linear_ce_bwd(const rlk_linear_ce_contract* contract, const void* hidden_bf16,
                                        const void* weight_bf16, const int64_t* targets, const uint8_t* active_mask,
                                        const float* lse, const float* grad_loss, void* dhidden_bf16,
                                        void* dweight_bf16, void* workspace, rlk_stream_t stream) {
    rlk_status s = check_ce(contract);
    if (s != RLK_OK) return s;
    const rlk_linear_ce_contract c = with_strides(*contract);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    // (the dhidden of no rows has no address)
    if (!dhidden_bf16 && !dweight_bf16 && c.T > 0)
        return fail(RLK_ERR_INVALID_ARG, "dhidden or dweight is required");
    if (!aligned16(dhidden_bf16) || !aligned16(dweight_bf16))
        return fail(RLK_ERR_MISALIGNED, "dhidden and dweight must be 16-byte aligned");
    if (c.T == 0) {  // no rows: a zero dweight
        if (!dweight_bf16) return RLK_OK;
        if ((s = select_device(dweight_bf16)) != RLK_OK) return s;
        return cudaMemset2DAsync(dweight_bf16, (size_t)c.dweight_stride * 2, 0, (size_t)c.H * 2, (size_t)c.V, st) ==
                       cudaSuccess
                   ? RLK_OK
                   : fail(RLK_ERR_CUDA, "clearing the gradient of no rows");
    }
    if ((s = check_ce_inputs(c, hidden_bf16, weight_bf16, targets, active_mask, workspace)) != RLK_OK) return s;
    if (!lse || !grad_loss) return fail(RLK_ERR_INVALID_ARG, "lse and grad_loss are required");
    if ((s = check_outputs({{dhidden_bf16, extent(c.T, c.dhidden_stride, c.H, 2), "dhidden"},
                            {dweight_bf16, extent(c.V, c.dweight_stride, c.H, 2), "dweight"},
                            {workspace, (int64_t)linear_ce_workspace(c, true), "workspace"}},
                           {{hidden_bf16, extent(c.T, c.hidden_stride, c.H, 2), "hidden"},
                            {weight_bf16, extent(c.V, c.weight_stride, c.H, 2), "weight"},
                            {targets, 8 * c.T, "targets"},
                            {active_mask, c.T, "active_mask"},
                            {lse, 4 * c.T, "lse"},
                            {grad_loss, c.reduction == RLK_REDUCE_NONE ? 4 * c.T : 4, "grad_loss"}})) != RLK_OK)
        return s;
    if ((s = select_device(hidden_bf16)) != RLK_OK) return s;
    if ((s = check_device_ptrs({{weight_bf16, "weight"}, {targets, "targets"}, {active_mask, "active_mask"},
                                {lse, "lse"}, {grad_loss, "grad_loss"}, {dhidden_bf16, "dhidden"},
                                {dweight_bf16, "dweight"}, {workspace, "workspace"}})) != RLK_OK)
        return s;
    if ((s = launch_linear_ce_bwd(c, hidden_bf16, weight_bf16, targets, active_mask, lse, grad_loss, dhidden_bf16,
                                  dweight_bf16, workspace, st)) != RLK_OK)
        return s;
    return c.validate ? read_status(workspace, st) : RLK_OK;
}

RLK_EXPORT rlk_status rlk_logp_workspace_status(const void* workspace, rlk_stream_t stream) {
    if (!workspace) return fail(RLK_ERR_INVALID_ARG, "workspace is NULL");
    rlk_status s = select_device(workspace);
    if (s != RLK_OK) return s;
    return read_status(workspace, reinterpret_cast<cudaStream_t>(stream));
}

RLK_EXPORT rlk_status rlk_selftest_bounded_wait(int64_t timeout_ns, void* workspace, rlk_stream_t stream) {
    if (timeout_ns <= 0 || timeout_ns > 10000000000ll)
        return fail(RLK_ERR_INVALID_ARG, "timeout_ns must be in (0, 10 s]");
    if (!workspace) return fail(RLK_ERR_INVALID_ARG, "workspace is NULL");
    if (!aligned16(workspace)) return fail(RLK_ERR_MISALIGNED, "workspace must be 16-byte aligned");
    rlk_status s = select_device(workspace);
    if (s != RLK_OK) return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if ((s = begin(workspace, st)) != RLK_OK) return s;
    if ((s = launch_selftest_wait((uint64_t)timeout_ns, static_cast<uint32_t*>(workspace), st)) != RLK_OK) return s;
    return read_status(workspace, st);
}

RLK_EXPORT const char* rlk_status_string(rlk_status s) {
    switch (s) {
        case RLK_OK: return "RLK_OK";
        case RLK_ERR_INVALID_ARG: return "RLK_ERR_INVALID_ARG";
        case RLK_ERR_UNSUPPORTED: return "RLK_ERR_UNSUPPORTED";
        case RLK_ERR_NON_TILEABLE: return "RLK_ERR_NON_TILEABLE";
        case RLK_ERR_MISALIGNED: return "RLK_ERR_MISALIGNED";
        case RLK_ERR_TARGET_RANGE: return "RLK_ERR_TARGET_RANGE";
        case RLK_ERR_NONFINITE_LSE: return "RLK_ERR_NONFINITE_LSE";
        case RLK_ERR_TIMEOUT: return "RLK_ERR_TIMEOUT";
        case RLK_ERR_CUDA: return "RLK_ERR_CUDA";
    }
    return "RLK_ERR_UNKNOWN";
}

RLK_EXPORT const char* rlk_last_error_message(void) { return g_last_error.c_str(); }
