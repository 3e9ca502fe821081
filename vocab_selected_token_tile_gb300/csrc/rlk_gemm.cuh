// What the BF16 tensor-core kernels share (lmhead.cu, linear_ce.cu): the tile
// and ring sizes, the barriers of one CTA's roles, bounded waits, the queue
// that hands work units from the producer to the other roles, and the tensor
// maps of their operands.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "rlk_internal.h"
#include "rlk_ptx.cuh"

namespace rlk {
namespace {

// TMA tile store from shared memory (bulk group); the writing threads fence
// the async proxy first.
__device__ __forceinline__ void tma_store_2d(const void* tmap, int32_t c0, int32_t c1, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(tmap), "r"(c0),
                 "r"(c1), "r"(src)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// The source of every committed store has been read (the buffer may be rewritten).
__device__ __forceinline__ void bulk_wait_read_all() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
// Every committed store has completed.
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void fence_proxy_async_smem() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

constexpr int kBM = 128;  // token rows per unit (TMEM lanes)
constexpr int kBN = 256;  // vocabulary rows per chunk (accumulator columns)
constexpr int kBK = 64;   // K per stage: 64 BF16 = one 128-byte swizzle row
constexpr int kStages = 4;
constexpr int kUq = 4;  // depth of the unit queue from the producer to the other roles
constexpr int kThreadsLm = 192;
constexpr uint32_t kTmemCols = 512;  // two accumulators of kBN columns
constexpr uint32_t kStageA = kBM * kBK * 2;
constexpr uint32_t kStageB = kBN * kBK * 2;
constexpr uint32_t kMnBlock = 64 * kBK * 2;  // one 64-wide block of an MN-major stage: 64 K rows x 128 B
constexpr uint64_t kDrainNsLm = 1000000000ull;
struct Bars {
    uint64_t full[kStages];
    uint64_t empty[kStages];
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint64_t ufull[kUq];   // unit queue entry written (the producer's arrival)
    uint64_t uempty[kUq];  // entry read by the MMA thread and the epilogue warps
    uint64_t drain;
    int64_t unit[kUq];
    uint32_t tmem_addr;
    int abort_flag;
};

struct WaitCtl {
    uint32_t* status;
    uint64_t wait_ns;
};

// Bounded wait for a phase; false when it expired or another role gave up.
// The clock is read on every 256th poll only.
__device__ bool lm_wait(Bars* bars, uint32_t bar, uint32_t parity, const WaitCtl& w) {
    volatile int* ab = &bars->abort_flag;
    uint64_t t0 = 0;
    for (uint32_t polls = 0;; ++polls) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*ab) return false;
        if ((polls & 255u) != 255u) continue;
        const uint64_t now = globaltimer_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > w.wait_ns) {
            *ab = 1;
            atomicOr(w.status, kStatusTimeout);
            return false;
        }
    }
}

__device__ void lm_drain_wait(uint32_t bar, uint32_t parity, const WaitCtl& w) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (globaltimer_ns() - t0 > kDrainNsLm) {
            atomicOr(w.status, kStatusTimeout);
            return;
        }
    }
}

// The producer publishes the CTA's n-th unit (-1: no more units).
__device__ bool unit_put(Bars* bars, int64_t n, int64_t u, const WaitCtl& w) {
    const int s = (int)(n % kUq);
    const uint32_t par = (uint32_t)((n / kUq) & 1);
    if (!lm_wait(bars, smem_u32(&bars->uempty[s]), par ^ 1u, w)) return false;
    *reinterpret_cast<volatile int64_t*>(&bars->unit[s]) = u;
    mbar_arrive(smem_u32(&bars->ufull[s]));  // release: the entry is visible to whoever acquires the phase
    return true;
}

__device__ bool unit_get(Bars* bars, int64_t n, int64_t& u, const WaitCtl& w) {
    const int s = (int)(n % kUq);
    if (!lm_wait(bars, smem_u32(&bars->ufull[s]), (uint32_t)((n / kUq) & 1), w)) return false;
    u = *reinterpret_cast<volatile int64_t*>(&bars->unit[s]);
    return true;
}

__device__ __forceinline__ void unit_done(Bars* bars, int64_t n) { mbar_arrive(smem_u32(&bars->uempty[n % kUq])); }

__device__ void init_bars(Bars* bars, int epilogue_warps = 4) {
    for (int s = 0; s < kStages; ++s) {
        mbar_init(smem_u32(&bars->full[s]), 1);
        mbar_init(smem_u32(&bars->empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
        mbar_init(smem_u32(&bars->tfull[b]), 1);
        mbar_init(smem_u32(&bars->tempty[b]), epilogue_warps);
    }
    for (int s = 0; s < kUq; ++s) {
        mbar_init(smem_u32(&bars->ufull[s]), 1);
        mbar_init(smem_u32(&bars->uempty[s]), epilogue_warps + 1);
    }
    mbar_init(smem_u32(&bars->drain), 1);
    bars->abort_flag = 0;
    fence_mbar_init();
}

// The producer's final step: every copy it issued lands before the CTA may exit.
__device__ void drain_copies(Bars* bars, int64_t issued, const WaitCtl& w) {
    const int64_t first = issued > kStages ? issued - kStages : 0;
    for (int64_t j = first; j < issued; ++j)
        lm_drain_wait(smem_u32(&bars->full[j % kStages]), (uint32_t)((j / kStages) & 1), w);
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_fn() {
    static std::mutex mu;
    static EncodeTiled fn = nullptr;
    std::lock_guard<std::mutex> lock(mu);
    if (!fn) {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiled>(ptr);
    }
    return fn;
}

// A BF16 matrix of `rows` rows of `inner` contiguous elements, `stride`
// elements apart, read in boxes of {box_inner, box_rows} with the 128-byte
// swizzle; elements outside [0, inner) x [0, rows) read as zero.
bool make_map(CUtensorMap* m, const void* base, int64_t inner, int64_t rows, int64_t stride, uint32_t box_inner,
              uint32_t box_rows) {
    EncodeTiled enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t box[2] = {box_inner, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A BF16 matrix whose contiguous dimension `inner` (a multiple of 64) is read
// in 64-element blocks: dims {64, rows, inner/64}, the blocks 128 bytes apart,
// so one box {64, box_rows, box_blocks} lands as box_blocks consecutive
// 64 x box_rows blocks of the 128-byte swizzle -- the layout of as many 2-D
// boxes {64, box_rows}.  Blocks past inner/64 read as zero.
bool make_map_mn3(CUtensorMap* m, const void* base, int64_t inner, int64_t rows, int64_t stride, uint32_t box_rows,
                  uint32_t box_blocks) {
    EncodeTiled enc = encode_fn();
    if (!enc || inner % 64 != 0) return false;
    const cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)(inner / 64)};
    const cuuint64_t strides[2] = {(cuuint64_t)stride * 2, 128};
    const cuuint32_t box[3] = {64, box_rows, box_blocks};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace rlk
