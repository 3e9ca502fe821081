// What the kernels of CTA pairs share (fp8_gemm.cu, linear_ce.cu): ring
// positions, bounded waits, and the barriers of a pair's pipeline.
//
// Two CTAs work one 256 x 256 tile: each loads its 128 rows of A and half of
// B's 256, the even CTA's warp 1 issues the MMAs of both, and each CTA reads
// its 128 rows of the accumulator from its own tensor memory.  Against a tile
// of 128 x 256 a CTA it takes a third less through TMA and shared memory,
// which is what bounds a one-CTA product (about 105 bytes a clock of shared
// memory, and one 128-byte line a clock of TMA).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "rlk_internal.h"
#include "rlk_ptx.cuh"

namespace rlk {
namespace {

constexpr uint64_t kPipeDrainNs = 1000000000ull;

// Position in a ring of n slots: the slot and the parity of its current pass.
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int n) {
        if (++slot == n) {
            slot = 0;
            phase ^= 1u;
        }
    }
    __device__ __forceinline__ void back(int n) {
        if (slot-- == 0) {
            slot = n - 1;
            phase ^= 1u;
        }
    }
};

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

template <int STAGES>
struct PairBars {
    uint64_t full[STAGES];   // the even CTA's count both CTAs' copies
    uint64_t empty[STAGES];
    uint64_t tfull[2];
    uint64_t tempty[2];      // the even CTA's count both CTAs' epilogue warps
    uint64_t drain;
    uint32_t tmem_addr;
    int abort_flag;
};

template <int STAGES>
__device__ void pair_init(PairBars<STAGES>* b, int epilogue_warps) {
    for (int s = 0; s < STAGES; ++s) {
        mbar_init(smem_u32(&b->full[s]), 1);
        mbar_init(smem_u32(&b->empty[s]), 1);
    }
    for (int i = 0; i < 2; ++i) {
        mbar_init(smem_u32(&b->tfull[i]), 1);
        mbar_init(smem_u32(&b->tempty[i]), 2 * epilogue_warps);
    }
    mbar_init(smem_u32(&b->drain), 1);
    b->abort_flag = 0;
    fence_mbar_init();
}

// Start and end of a pair's kernel, by all threads of both CTAs: all 512
// columns of tensor memory are theirs in between.
template <int STAGES>
__device__ __forceinline__ uint32_t pair_begin(PairBars<STAGES>* bars, int warp, int epilogue_warps) {
    if (threadIdx.x == 0) pair_init(bars, epilogue_warps);
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(&bars->tmem_addr), 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();         // this CTA's tensor memory address
    cluster_sync_relaxed();  // both CTAs' barriers (fence_mbar_init released them)
    tc_fence_after();
    return bars->tmem_addr;
}

__device__ __forceinline__ void pair_end(uint32_t tmem, int warp) {
    tc_fence_before();
    cluster_sync_relaxed();  // the pair's MMAs and copies are done, in both CTAs' memory
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// The producer's last copies land before the pair may exit (r: its position
// after `issued` stages, STAGES at most): the even CTA's barriers count both
// CTAs' copies, and the odd one leaves only after the even one.
template <int STAGES>
__device__ void pair_drain_copies(PairBars<STAGES>* bars, Ring r, int issued, int rank, const PipeWait& w) {
    for (int j = 0; j < issued && rank == 0; ++j) {
        r.back(STAGES);
        pipe_drain(smem_u32(&bars->full[r.slot]), r.phase, w);
    }
}

// The MMA issuer's: every MMA issued so far completes.
template <int STAGES>
__device__ __forceinline__ void pair_drain_mmas(PairBars<STAGES>* bars, bool one, const PipeWait& w,
                                                uint16_t mask = 3) {
    if (one) umma_commit_pair(smem_u32(&bars->drain), mask);
    __syncwarp();
    pipe_drain(smem_u32(&bars->drain), 0u, w);
}

}  // namespace
}  // namespace rlk
