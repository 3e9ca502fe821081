// What the tensor-core kernels share (lmhead.cu, linear_ce.cu, rlk_fp8_gemm.cuh):
// the tile sizes of the BF16 ones, the bounded waits of their pipelines, and
// the tensor maps of BF16 operands.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "rlk_internal.h"
#include "rlk_ptx.cuh"

namespace rlk {
namespace {

constexpr int kBN = 256;  // vocabulary rows per chunk (accumulator columns)
constexpr int kBK = 64;   // K per stage: 64 BF16 = one 128-byte swizzle row
constexpr uint32_t kMnBlock = 64 * kBK * 2;  // one 64-wide block of an MN-major stage: 64 K rows x 128 B
constexpr uint64_t kPipeDrainNs = 1000000000ull;

struct PipeWait {
    uint32_t* status;
    uint64_t wait_ns;
};

// Bounded wait for a phase of a barrier: false, with the time-out recorded and
// *abort_flag set, when it expired, or when another role has given up.  The
// clock and the flag are read on every 256th poll.
__device__ __forceinline__ bool pipe_wait(int* abort_flag, uint32_t bar, uint32_t parity, const PipeWait& w) {
    uint64_t t0 = 0;
    for (uint32_t polls = 0;; ++polls) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((polls & 255u) != 255u) continue;
        if (*reinterpret_cast<volatile int*>(abort_flag)) return false;
        const uint64_t now = globaltimer_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > w.wait_ns) {
            *reinterpret_cast<volatile int*>(abort_flag) = 1;
            atomicOr(w.status, kStatusTimeout);
            return false;
        }
    }
}

// The wait for a role's own last copies or MMAs, which nothing may cut short.
__device__ __forceinline__ void pipe_drain(uint32_t bar, uint32_t parity, const PipeWait& w) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (globaltimer_ns() - t0 > kPipeDrainNs) {
            atomicOr(w.status, kStatusTimeout);
            return;
        }
    }
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
