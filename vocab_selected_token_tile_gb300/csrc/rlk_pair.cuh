// What the kernels of CTA pairs share (rlk_fp8_gemm.cuh, linear_ce.cu): ring
// positions and the barriers of a pair's pipeline from its start to its end.
//
// Two CTAs work one 256 x 256 tile: each loads its 128 rows of A and half of
// B's 256, the even CTA's warp 1 issues the MMAs of both, and each CTA reads
// its 128 rows of the accumulator from its own tensor memory.  Against a tile
// of 128 x 256 a CTA it takes a third less through TMA and shared memory,
// which is what bounds a one-CTA product (about 105 bytes a clock of shared
// memory, and one 128-byte line a clock of TMA).
//
// The end of a pair.  A CTA may leave only when nothing is on its way to its
// shared memory: not its own copies, not the pair's commits, not the other
// CTA's arrivals.  So each role ends by waiting for its last hand-overs: a
// producer until its stages are free again (its copies have landed and the
// commits on its `empty` barriers have arrived), the issuer until both
// accumulators are handed back (every epilogue warp's arrival is in).  Where a
// wait expires, in any CTA of the cluster, all of them learn of it before they
// meet and take one more round (pair_give_up): each producer arms `full` for
// its own bytes only, so that a stage which only one of the two has issued is
// completed by an arrival without bytes, and every copy can be waited for.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "rlk_gemm.cuh"
#include "rlk_internal.h"
#include "rlk_ptx.cuh"

namespace rlk {
namespace {

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

// pipe_wait by a whole warp, for all of its lanes alike: one may see the phase
// complete after another has given it up, and lanes that leave a role's loop
// alone would leave the others waiting for them.  The vote costs the FP8
// product 0.6% (8192 x 12288 x 4096: 319.5 -> 321.5 us).  Voting after the step
// instead, with each lane's own result deciding whether it issues, took the
// cross entropy's issuer 10-40% longer.
__device__ __forceinline__ bool pipe_wait_warp(int* abort_flag, uint32_t bar, uint32_t parity, const PipeWait& w) {
    return __all_sync(0xFFFFFFFFu, pipe_wait(abort_flag, bar, parity, w));
}

// ACCS: accumulators in flight.
template <int STAGES, int ACCS = 2>
struct PairBars {
    uint64_t full[STAGES];   // the even CTA's count both producers' arrivals and copies
    uint64_t empty[STAGES];
    uint64_t tfull[ACCS];
    uint64_t tempty[ACCS];   // the even CTA's count both CTAs' epilogue warps
    uint64_t drain;
    uint64_t issued;         // stages that this CTA's producer has issued
    uint32_t tmem_addr;
    int abort_flag;
    uint32_t drained;        // the issuer has committed on `drain`
};

template <int STAGES, int ACCS>
__device__ void pair_init(PairBars<STAGES, ACCS>* b, int epilogue_warps) {
    for (int s = 0; s < STAGES; ++s) {
        mbar_init(smem_u32(&b->full[s]), 2);
        mbar_init(smem_u32(&b->empty[s]), 1);
    }
    for (int i = 0; i < ACCS; ++i) {
        mbar_init(smem_u32(&b->tfull[i]), 1);
        mbar_init(smem_u32(&b->tempty[i]), 2 * epilogue_warps);
    }
    mbar_init(smem_u32(&b->drain), 1);
    b->issued = 0;
    b->abort_flag = 0;
    b->drained = 0;
    fence_mbar_init();
}

// Start and end of a pair's kernel, by all threads of all CTAs of the cluster:
// all 512 columns of tensor memory are the pair's in between.
template <int STAGES, int ACCS>
__device__ __forceinline__ uint32_t pair_begin(PairBars<STAGES, ACCS>* bars, int warp, int epilogue_warps) {
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

// A stage's copies by one of the producers: `fb` is the even CTA's barrier (a
// cluster address), `local` the same in this CTA.
__device__ __forceinline__ void pair_arm(uint32_t fb, uint32_t local, int rank, uint32_t bytes) {
    if (rank == 0)
        mbar_arrive_expect_tx(local, bytes);
    else
        mbar_arrive_expect_tx_remote(fb, bytes);
}

// The end of a producer (its whole warp; r: its position, one: the thread that
// issued `issued` stages, ok: no wait has expired).
template <int STAGES, int ACCS>
__device__ __forceinline__ void pair_end_copies(PairBars<STAGES, ACCS>* bars, Ring r, bool one, uint64_t issued,
                                                bool ok, const PipeWait& w) {
    for (int j = 0; ok && j < STAGES; ++j) {
        ok = pipe_wait_warp(&bars->abort_flag, smem_u32(&bars->empty[r.slot]), r.phase ^ 1u, w);
        r.next(STAGES);
    }
    if (one) bars->issued = issued;
}

// The end of the issuer: every MMA issued so far has completed.  acc: its
// position; one: the thread that issued them.
template <int STAGES, int ACCS>
__device__ __forceinline__ void pair_end_mmas(PairBars<STAGES, ACCS>* bars, Ring acc, bool one, bool ok, const PipeWait& w,
                                              uint16_t mask = 3) {
    for (int i = 0; ok && i < ACCS; ++i) {
        ok = pipe_wait_warp(&bars->abort_flag, smem_u32(&bars->tempty[acc.slot]), acc.phase ^ 1u, w);
        acc.next(ACCS);
    }
    if (ok) return;
    if (one) {
        bars->drained = 1;
        umma_commit_pair(smem_u32(&bars->drain), mask);
    }
    __syncwarp();
    pipe_drain(smem_u32(&bars->drain), 0u, w);
}

// All CTAs have met and a wait of one of them has expired: the copies and the
// commits still under way arrive before any CTA leaves.
template <int STAGES, int ACCS>
__device__ __noinline__ void pair_give_up(PairBars<STAGES, ACCS>* bars, uint32_t* status) {
    const PipeWait w{status, 0};
    const int warp = warp_index();
    const uint32_t place = cluster_ctarank(), rank = place & 1u, even = place & ~1u;
    cluster_sync_all();  // `issued` and `drained` of both, and every thread's arrivals
    if (warp == 0 && rank == 0 && (threadIdx.x & 31) == 0) {
        const uint64_t mine = bars->issued, other = ld_cluster_u64(mapa_shared(smem_u32(&bars->issued), even + 1));
        const uint64_t lo = mine < other ? mine : other, hi = mine < other ? other : mine;
        for (uint64_t j = lo; j < hi; ++j) mbar_arrive(smem_u32(&bars->full[j % STAGES]));
        for (uint64_t j = hi > STAGES ? hi - STAGES : 0; j < hi; ++j)
            pipe_drain(smem_u32(&bars->full[j % STAGES]), (uint32_t)((j / STAGES) & 1), w);
    }
    if (warp == 1 && rank == 1 && ld_cluster_u32(mapa_shared(smem_u32(&bars->drained), even)) != 0)
        pipe_drain(smem_u32(&bars->drain), 0u, w);
    cluster_sync_all();
}

template <int STAGES, int ACCS>
__device__ __forceinline__ void pair_end(PairBars<STAGES, ACCS>* bars, uint32_t tmem, int warp, const PipeWait& w) {
    volatile int* flag = &bars->abort_flag;
    tc_fence_before();
    if (*flag) {  // the thread that set it is among those that see it here
        for (uint32_t r = 0; r < cluster_nctarank(); ++r) st_cluster_u32(mapa_shared(smem_u32(&bars->abort_flag), r), 1);
        fence_cluster();
    }
    cluster_sync_relaxed();
    if (*flag) pair_give_up(bars, w.status);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

}  // namespace
}  // namespace rlk
