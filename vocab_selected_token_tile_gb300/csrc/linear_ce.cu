// Softmax cross entropy of logits = hidden @ weight^T over a large vocabulary,
// and its gradients, without keeping the logits (sm_103a).
//
// Per row r with target t, logits x_c = hidden_r . weight_c, c < V:
//   y_c   = cap tanh(x_c / cap), or x_c without a cap;
//   lse   = log sum_c e^y_c;
//   L     = lse - (1 - eps) y_t - (eps / V) sum_c y_c + z lse^2;
//   dL/dx_c = ((1 + 2 z lse) p_c - (1 - eps) [c = t] - eps / V) (1 - (y_c / cap)^2),
//   p_c = e^(y_c - lse).
// Label smoothing eps, z-loss z and the cap are 0 when unused.
//
// Forward: one tcgen05 GEMM over units of (256 vocabulary rows, 256 tokens)
// whose epilogue turns 128 of a row's logits into one (max, sumexp[, sum])
// partial, then a merge of each row's partials in vocabulary order.  Bound:
// the tensor core, 2 T V H operations; the epilogue of one accumulator runs
// under the MMAs of the other (4096 x 151936 x 4096: 2.37-2.54 ms, 2.0-2.15
// PFLOP/s as the clock allows, the tensor pipe 96.5% busy; 2.8 ms in a long
// loop under the power cap).  Hidden whose rows lie between 128-byte lines is
// copied onto them first, as in the backward below (1000 x 50257 x 1000: 95 ->
// 76 us).  Few tokens: the weight's bytes (16 x 151936 x 1024: 61-66 us, of
// which the GEMM is 50, 6.2 TB/s).
//
// Backward, in pieces of the vocabulary: for each piece the logits are formed
// again (the price of not keeping them: 2 T V H operations more) and leave
// the epilogue as BF16 dL/dx [T, P], and one launch then runs both
//   dHidden[T, H] += dx weight[piece]     (FP32 sums across the pieces)
//   dWeight[piece] = dx^T hidden
// (8.6-9.0 ms at 4096 x 151936 x 4096, 1.7-1.75 PFLOP/s, the tensor pipe 97% busy).
// The work space is P T 2 bytes for dx, T H 4 for the sums and T H 2 for the
// rows below, whatever V is.  Only the active rows take part: their hidden is
// first copied together (a step's prompts and padding are often half of its
// rows, and a row of rubbish under a mask must not meet a zero), into rows on
// 128-byte lines, which a TMA load takes in half the time of others (1000 x
// 50257 x 1000, rows of 2000 bytes, none masked: backward 253 -> 234 us).
// P is chosen so that dx stays within kPieceBytes: the sums are read and
// written once a piece, and with pieces that large that traffic and the ends
// of the launches are under 2% of a piece's time.
//
// What is rounded to BF16 is dx / scale, with scale = (1 - eps) times the
// upstream gradient of a summed or averaged loss (the largest row's otherwise):
// with that common factor folded in, the value of every row's largest entry,
// about -(1 - eps) g, would be rounded in the same direction, a bias of up to
// 2^-8 in both gradients (eps = 0.1 alone: -0.9 becomes -0.8984, 0.17% off in
// every row of dWeight).  The scale multiplies the FP32 sums instead.
//
// Both GEMM kernels run as CTA pairs (rlk_pair.cuh) on 256 x 256 tiles: warp 0
// issues the TMA loads, warp 1 of the even CTA the MMAs, warps 2-9 are the
// epilogue.  The tiles are dealt out from the sizes alone, so every role of both
// CTAs knows its sequence and no ticket travels between them.
// Every sum has a fixed order: no split of a K range without an ordered join,
// no atomics on data.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <string>

#include "rlk_fold.cuh"
#include "rlk_gemm.cuh"
#include "rlk_internal.h"
#include "rlk_pair.cuh"
#include "rlk_ptx.cuh"

namespace rlk {
namespace {

constexpr int64_t kPieceBytes = (int64_t)512 << 20;  // BF16 dx of one piece
constexpr int kMinPiece = 2048;                      // vocabulary rows a piece at least
constexpr int kMaxPieces = 512;
constexpr int kMaxSlices = 32;                       // K slices of dHidden within a piece
constexpr int64_t kBandBytes = (int64_t)32 << 20;    // hidden of one band of token blocks (as the lm_head's)
constexpr int kBandH = 8;                            // H blocks per band of the gradient tiles (as the lm_head's)
constexpr int kFoldRows = 8, kFoldSlices = 64;       // of one CTA of the merge

// Ten warps: TMA, MMA and eight of the epilogue, each with 32 rows and half of an accumulator's 256 columns.
constexpr int kCeThreads = 320, kCeEpilogue = 8;

constexpr int kCeStages = 6;
constexpr uint32_t kCeA = 128 * 128, kCeB = 128 * 128;  // bytes of a stage: a CTA's 128 rows of A, half of B's 256; K = 64
constexpr uint32_t kCeOut = 32 * 64;                    // per epilogue warp: 32 rows x 64 bytes on their way out
constexpr size_t kCeSmem = 1024 + (size_t)kCeStages * (kCeA + kCeB) + kCeEpilogue * kCeOut + 1024;
static_assert(sizeof(PairBars<kCeStages>) <= 1024, "barriers fit their kilobyte");

enum : int { kCeForward = 0, kCeGrad = 1 };

struct CeParams {
    const int64_t* targets;
    const uint8_t* mask;
    float2* part;        // [2 chunks, T] (max, sumexp) of 128 columns  forward
    float* part_y;       // [2 chunks, T] sum of y                      forward, with smoothing
    float* yt;           // [T] the target's y                          forward
    const float* lse;    // [T]                                         gradient
    const float* grad;   // [T], NULL for a summed or averaged loss     gradient
    const float* scale;  // the common factor left out of dx            gradient
    const int32_t* count;  // the number of active rows                 gradient
    const int32_t* index;  // [count] their places in the batch         gradient
    PipeWait w;
    int64_t T, V, ignore_index;
    float cap, icap, eps, z;
    float unit;          // 1 / (1 - eps): a row's own factor in dx under a summed or averaged loss  gradient
    int32_t KB, mask_mode;
    int32_t ch0, nch;  // the launch's chunks of 256 vocabulary rows
    int32_t MB, MBg;   // blocks of 256 tokens, and per band
    int32_t box_rows;  // rows of hidden a load brings (128, or fewer where T is below it)
};

// 32 BF16 columns of a warp's 32 rows (a lane's row in v) through shared
// memory, so that a row's 64 bytes leave in one piece; 16 bytes a lane straight
// from the registers, 32 rows an instruction, took 10,700 clocks a 128 x 256
// tile.  16-byte piece j of row r is kept at j ^ (r / 2 mod 4).  Rows of
// `rows` and columns of `cols` at most; every row starts on a 16-byte boundary;
// row r of them is index[r] of dst, if index is given.
__device__ __forceinline__ void ce_store(unsigned char* out, int lane, const float (&v)[32], uint16_t* dst, int64_t ld,
                                         int rows, int cols, const int32_t* index = nullptr) {
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint4*>(out + lane * 64 + ((j ^ ((lane >> 1) & 3)) * 16)) =
            make_uint4(pack_bf16x2_rn(v[8 * j], v[8 * j + 1]), pack_bf16x2_rn(v[8 * j + 2], v[8 * j + 3]),
                       pack_bf16x2_rn(v[8 * j + 4], v[8 * j + 5]), pack_bf16x2_rn(v[8 * j + 6], v[8 * j + 7]));
    __syncwarp();
    const int j = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + (lane >> 2);
        if (r >= rows || j * 8 >= cols) continue;
        const uint4 w = *reinterpret_cast<const uint4*>(out + r * 64 + ((j ^ ((r >> 1) & 3)) * 16));
        uint16_t* d = dst + (index ? (int64_t)index[r] : (int64_t)r) * ld + j * 8;
        if (j * 8 + 8 <= cols) {
            *reinterpret_cast<uint4*>(d) = w;
        } else {
            const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (j * 8 + e < cols) d[e] = (uint16_t)(x[e >> 1] >> (16 * (e & 1)));
        }
    }
}

__device__ __forceinline__ bool ce_active(const uint8_t* mask, int mask_mode, int64_t ignore_index, int64_t target,
                                          int64_t r) {
    return mask_mode == RLK_MASK_EXPLICIT ? mask[r] != 0 : target != ignore_index;
}

// Unit u is (chunk ch of 256 vocabulary rows, block mb of 256 tokens): bands of
// MBg token blocks, chunk-major within a band, so that the units in flight
// share a few chunks of weight and one band of hidden, which L2 holds.
__device__ __forceinline__ void ce_unit(const CeParams& p, int MB, uint32_t u, int& ch, int& mb) {
    const uint32_t band = (uint32_t)p.nch * p.MBg, full = (uint32_t)MB / p.MBg;
    const uint32_t b = min(u / band, full);
    const uint32_t r = u - b * band;
    const uint32_t w = b < full ? p.MBg : MB - full * p.MBg;
    ch = p.ch0 + (int)(r / w);
    mb = (int)(b * p.MBg + r % w);
}

// y = cap tanh(x / cap), to a few 2^-24 of y whatever the cap: from u = |x| / cap = 1/2 on as cap (1 - r) with
// r = 2 / (e^(2 u) + 1), below it (where that difference loses y's digits, 10^-7 cap of them) as |x| (1 + u^2 q(u^2)),
// q interpolating (tanh(u) / u - 1) / u^2 in u^2 at the four Chebyshev nodes of [0, 1/4]: 2^-24 off at most.  And its
// slope 1 - tanh^2 = r (2 - r), which keeps its relative precision where tanh saturates.  Two logits in packed
// arithmetic: one by one the forward's epilogue took 40% longer at H = 1024 (2048 x 65536 x 1024: 229 us for 164).
__device__ __forceinline__ float2 ce_cap(float2 x, float cap, float icap, float2& slope) {
    auto both = [](float v) { return make_float2(v, v); };
    const float2 a = make_float2(fabsf(x.x), fabsf(x.y)), u = fmul2(a, both(icap)), w = fmul2(u, u);
    const float2 g = fmul2(u, both(2.f * kLog2e));
    const float2 e = fadd2(make_float2(ex2_approx(g.x), ex2_approx(g.y)), both(1.f));
    const float2 h = make_float2(rcp_approx(e.x), rcp_approx(e.y)), r = fadd2(h, h);
    slope = fmul2(r, ffma2(r, both(-1.f), both(2.f)));
    const float2 high = ffma2(r, both(-cap), both(cap));
    float2 q = ffma2(w, both(0.017988745f), both(-0.05338711f));
    q = ffma2(ffma2(q, w, both(0.13330476f)), w, both(-0.3333331f));
    const float2 low = ffma2(fmul2(q, w), a, a);
    return make_float2(copysignf(u.x < 0.5f ? low.x : high.x, x.x), copysignf(u.y < 0.5f ? low.y : high.y, x.y));
}

// One block of up to 32 logits into the row's running (max, sumexp, sum).
template <bool SMOOTH>
__device__ __forceinline__ void ce_online(const float (&y)[32], int nv, float& m_run, float& s_run, float& y_run) {
    float bm = -INFINITY;
#pragma unroll
    for (int i = 0; i < 32; ++i)
        if (i < nv) bm = fmax_nan(bm, y[i]);
    if (bm > m_run || bm != bm) {
        s_run = __fmul_rn(s_run, ex2_approx(__fmul_rn(__fsub_rn(m_run, bm), kLog2e)));
        m_run = bm;
    }
    if (SMOOTH) {
        float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < nv) a[i & 3] = __fadd_rn(a[i & 3], y[i]);
        y_run = __fadd_rn(y_run, __fadd_rn(__fadd_rn(a[0], a[1]), __fadd_rn(a[2], a[3])));
    }
    if (m_run == -INFINITY) return;  // nothing finite yet
    const float nmL = -__fmul_rn(m_run, kLog2e);
    float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const float e = ex2_approx(__fmaf_rn(y[i], kLog2e, nmL));
        if (i < nv) a[i & 3] = __fadd_rn(a[i & 3], e);
    }
    s_run = __fadd_rn(s_run, __fadd_rn(__fadd_rn(a[0], a[1]), __fadd_rn(a[2], a[3])));
}

// The pieces of shared memory of a pair's GEMM: six stages of A and B, the
// epilogue's output stages, the barriers; at the same offsets in both CTAs.
struct CeSmem {
    unsigned char *a, *b, *out;
    PairBars<kCeStages>* bars;
};
__device__ __forceinline__ CeSmem ce_smem(unsigned char* raw) {
    CeSmem m;
    m.a = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    m.b = m.a + kCeStages * kCeA;
    m.out = m.b + kCeStages * kCeB;
    m.bars = reinterpret_cast<PairBars<kCeStages>*>(m.out + kCeEpilogue * kCeOut);
    return m;
}

template <int MODE, bool CAP, bool SMOOTH>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kCeThreads, 1)
    ce_logits_kernel(const __grid_constant__ CUtensorMap tmH, const __grid_constant__ CUtensorMap tmW,
                     uint16_t* dx, const int64_t ldx, const __grid_constant__ CeParams p) {
    extern __shared__ unsigned char smem_raw[];
    const CeSmem m = ce_smem(smem_raw);
    PairBars<kCeStages>* bars = m.bars;
    const int warp = warp_index(), lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank();
    // the rows that take part: all of them, or the active ones, copied together
    const int64_t T = MODE == kCeGrad ? (int64_t)*p.count : p.T;
    const int MB = (int)((T + 255) / 256);
    const uint32_t total = (uint32_t)p.nch * MB, first = blockIdx.x / 2, step = gridDim.x / 2;
    const uint32_t tmem = pair_begin(bars, warp, kCeEpilogue);
    int* ab = &bars->abort_flag;
    if (MODE == kCeForward) grid_launch_dependents();  // the merge

    if (warp == 0) {
        const bool one = elect_one();
        const uint32_t full0 = mapa_shared(smem_u32(&bars->full[0]), 0);
        const uint64_t keep = l2_policy_evict_last();
        Ring r;
        uint64_t issued = 0;
        bool ok = true;
        for (uint32_t u = first; ok && u < total; u += step) {
            int ch, mb;
            ce_unit(p, MB, u, ch, mb);
            // a CTA without a row of its own loads no hidden: its rows of the accumulator are not used
            const int row = (2 * mb + rank) * 128;
            const bool mine = row < T;
            const uint32_t bytes = kCeB + (mine ? (uint32_t)p.box_rows * 128 : 0);
            for (int kb = 0; kb < p.KB; ++kb) {
                if (!(ok = pipe_wait_warp(ab, smem_u32(&bars->empty[r.slot]), r.phase ^ 1u, p.w))) break;
                if (one) {
                    const uint32_t fb = full0 + r.slot * 8;
                    pair_arm(fb, smem_u32(&bars->full[r.slot]), rank, bytes);
                    if (mine) tma_load_2d_pair_hint(smem_u32(m.a + r.slot * kCeA), &tmH, kb * kBK, row, fb, keep);
                    tma_load_2d_pair(smem_u32(m.b + r.slot * kCeB), &tmW, kb * kBK, ch * kBN + rank * 128, fb);
                }
                ++issued;
                r.next(kCeStages);
            }
        }
        pair_end_copies(bars, r, one, issued, ok, p.w);
    } else if (warp == 1 && rank == 0) {
        const bool one = elect_one();
        const uint64_t da = smem_desc_sw128(smem_u32(m.a)), db = smem_desc_sw128(smem_u32(m.b));
        const uint32_t idesc = idesc_bf16_f32(256, kBN);
        Ring r, acc;
        bool ok = true;
        for (uint32_t u = first; ok && u < total; u += step) {
            if (!(ok = pipe_wait_warp(ab, smem_u32(&bars->tempty[acc.slot]), acc.phase ^ 1u, p.w))) break;
            const uint32_t d = tmem + (uint32_t)(acc.slot * kBN);
            for (int kb = 0; kb < p.KB; ++kb) {
                if (!(ok = pipe_wait_warp(ab, smem_u32(&bars->full[r.slot]), r.phase, p.w))) break;
                tc_fence_after();
                if (one) {
#pragma unroll
                    for (int kk = 0; kk < kBK / 16; ++kk)
                        umma_bf16_pair(d, da + ((r.slot * kCeA + kk * 32) >> 4), db + ((r.slot * kCeB + kk * 32) >> 4),
                                       idesc, (kb | kk) != 0);
                    if (kb == p.KB - 1) umma_commit_pair(smem_u32(&bars->tfull[acc.slot]));
                    umma_commit_pair(smem_u32(&bars->empty[r.slot]));
                }
                __syncwarp();
                r.next(kCeStages);
            }
            acc.next(2);
        }
        pair_end_mmas(bars, acc, one, ok, p.w);
    } else if (warp >= 2) {
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
        unsigned char* out = m.out + (warp - 2) * kCeOut;  // kCeGrad
        const uint32_t done = mapa_shared(smem_u32(&bars->tempty[0]), 0);
        const float scale = MODE == kCeGrad ? *p.scale : 1.f;
        Ring acc;
        for (uint32_t u = first; u < total; u += step) {
            int ch, mb;
            ce_unit(p, MB, u, ch, mb);
            const int64_t row0 = (int64_t)(2 * mb + rank) * 128 + quarter * 32, row = row0 + lane;
            const bool valid = row < T;
            int64_t target = -1;
            bool active = false;
            float qa = 0.f, qb = 0.f, qc = 0.f, nlL = 0.f;
            if (valid && MODE == kCeForward) {
                target = p.targets[row];
                active = ce_active(p.mask, p.mask_mode, p.ignore_index, target, row);
            }
            if (valid && MODE == kCeGrad) {
                // dx / scale = (qa p - qc - qb [c = t]) slope
                const int64_t at = p.index[row];
                const float l = p.lse[at];
                const float g = p.grad ? __fdiv_rn(p.grad[at], scale) : p.unit;
                target = p.targets[at];
                active = true;
                qa = g * (1.f + 2.f * p.z * l);
                qb = g * (1.f - p.eps);
                qc = g * p.eps / (float)p.V;
                nlL = -__fmul_rn(l, kLog2e);
                if (ch == 0 && half == 0) {  // the device conditions of a row, once
                    if (target < 0 || target >= p.V) atomicOr(p.w.status, kStatusTargetRange);
                    if (!isfinite(l)) atomicOr(p.w.status, kStatusNonFinite);
                }
            }
            if (!__all_sync(0xFFFFFFFFu, pipe_wait(ab, smem_u32(&bars->tfull[acc.slot]), acc.phase, p.w))) break;
            tc_fence_after();
            float m_run = -INFINITY, s_run = 0.f, y_run = 0.f;
            const int64_t cbase = (int64_t)ch * kBN + half * 128;
            const int ncols = (int)max((int64_t)0, min((int64_t)128, p.V - cbase));
            for (int sub = 0; sub * 32 < ncols; ++sub) {
                float v[32];
                tmem_ld32(tmem + lane_base + (uint32_t)(acc.slot * kBN + half * 128 + sub * 32), v);
                const int nv = min(32, ncols - sub * 32);
                const int64_t hot = target - (cbase + sub * 32);
                const bool here = active && hot >= 0 && hot < nv;
                const uint32_t hot_bit = here ? 1u << (int)hot : 0u;  // an index into v would spill it
                if constexpr (MODE == kCeForward) {
                    if (CAP) {
                        float2 slope;
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            const float2 y = ce_cap(make_float2(v[i], v[i + 1]), p.cap, p.icap, slope);
                            v[i] = y.x, v[i + 1] = y.y;
                        }
                    }
                    ce_online<SMOOTH>(v, nv, m_run, s_run, y_run);
                    if (here) {
                        float yt = 0.f;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (hot_bit & (1u << i)) yt = v[i];
                        p.yt[row] = yt;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        float2 y = make_float2(v[i], v[i + 1]), slope = make_float2(1.f, 1.f);
                        if (CAP) y = ce_cap(y, p.cap, p.icap, slope);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            float d = __fmaf_rn(ex2_approx(__fmaf_rn(j ? y.y : y.x, kLog2e, nlL)), qa, -qc);
                            if (hot_bit & (1u << (i + j))) d = __fsub_rn(d, qb);
                            if (CAP) d = __fmul_rn(d, j ? slope.y : slope.x);
                            v[i + j] = active ? d : 0.f;
                        }
                    }
                    // rows past the active ones are zero: dWeight's K range ends on a whole block of 64
                    ce_store(out, lane, v, dx + row0 * ldx + (cbase - (int64_t)p.ch0 * kBN) + sub * 32, ldx,
                             (int)min((int64_t)32, p.T - row0), nv);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(done + acc.slot * 8);
            acc.next(2);
            if (MODE == kCeForward && valid) {
                p.part[(int64_t)(2 * ch + half) * p.T + row] = make_float2(m_run, s_run);
                if (SMOOTH) p.part_y[(int64_t)(2 * ch + half) * p.T + row] = y_run;
            }
        }
    }
    pair_end(bars, tmem, warp, p.w);
}

// (m, s) with (m2, s2): the larger maximum, both sums scaled to it; a maximum
// of -inf adds nothing, a NaN stays.
__device__ __forceinline__ void ce_merge(float& m, float& s, float m2, float s2) {
    if (m2 == -INFINITY) return;
    const float M = fmax_nan(m, m2);
    s = __fadd_rn(__fmul_rn(s, m == -INFINITY ? 0.f : ex2_approx(__fmul_rn(__fsub_rn(m, M), kLog2e))),
                  __fmul_rn(s2, ex2_approx(__fmul_rn(__fsub_rn(m2, M), kLog2e))));
    m = M;
}

struct CeFold {
    const float2* part;
    const float* part_y;  // NULL without smoothing
    const float* yt;
    const int64_t* targets;
    const uint8_t* mask;
    float* loss;
    float* lse;
    uint32_t* status;
    int64_t T, V, ignore_index;
    int32_t parts, mask_mode;
    float eps, z;
};

// Each row's LSE and loss from its partials: 8 rows a CTA, 64 threads a row
// take runs of partials in vocabulary order, and the runs are merged pairwise,
// neighbours first.  The order depends on the number of partials only.
__global__ void __launch_bounds__(kFoldRows* kFoldSlices) ce_fold_kernel(CeFold p) {
    __shared__ float2 sm[kFoldSlices][kFoldRows];
    __shared__ float sy[kFoldSlices][kFoldRows];
    const int lane = threadIdx.x % kFoldRows, sl = threadIdx.x / kFoldRows;
    const int64_t row = (int64_t)blockIdx.x * kFoldRows + lane;
    grid_launch_dependents();
    grid_wait_prior();
    float m = -INFINITY, s = 0.f, y = 0.f;
    if (row < p.T) {
        const int c0 = (int)((int64_t)p.parts * sl / kFoldSlices), c1 = (int)((int64_t)p.parts * (sl + 1) / kFoldSlices);
#pragma unroll 8
        for (int c = c0; c < c1; ++c) {
            const float2 q = p.part[(int64_t)c * p.T + row];
            ce_merge(m, s, q.x, q.y);
            if (p.part_y) y = __fadd_rn(y, p.part_y[(int64_t)c * p.T + row]);
        }
    }
    sm[sl][lane] = make_float2(m, s);
    sy[sl][lane] = y;
    for (int step = 1; step < kFoldSlices; step *= 2) {
        __syncthreads();
        if (sl % (2 * step) == 0) {
            ce_merge(m, s, sm[sl + step][lane].x, sm[sl + step][lane].y);
            y = __fadd_rn(y, sy[sl + step][lane]);
            sm[sl][lane] = make_float2(m, s);
            sy[sl][lane] = y;
        }
    }
    if (sl != 0 || row >= p.T) return;
    const float l = m == -INFINITY ? -INFINITY : __fadd_rn(m, logf(s));
    const int64_t t = p.targets[row];
    p.lse[row] = l;
    float loss = 0.f;
    if (ce_active(p.mask, p.mask_mode, p.ignore_index, t, row)) {
        if (t < 0 || t >= p.V) {
            loss = __int_as_float(0x7FC00000);
            atomicOr(p.status, kStatusTargetRange);
        } else {
            loss = __fmaf_rn(-(1.f - p.eps), p.yt[row], l);
            if (p.eps != 0.f) loss = __fmaf_rn(-p.eps / (float)p.V, y, loss);
            if (p.z != 0.f) loss = __fmaf_rn(p.z * l, l, loss);
        }
        if (!isfinite(l)) atomicOr(p.status, kStatusNonFinite);
    }
    p.loss[row] = loss;
}

// Sum over a CTA of 1024 threads in a fixed order; the result is warp 0's.
template <typename F>
__device__ F block_sum(F v, F* scratch) {
    for (int o = 16; o; o >>= 1) v += __shfl_down_sync(0xFFFFFFFFu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    v = scratch[threadIdx.x & 31];
    for (int o = 16; o; o >>= 1) v += __shfl_down_sync(0xFFFFFFFFu, v, o);
    return v;
}

// The sum, or the mean over the active rows (0 without any), of the rows'
// losses: one CTA, FP64, a fixed order.
__global__ void __launch_bounds__(1024) ce_reduce_kernel(const float* loss, const int64_t* targets,
                                                         const uint8_t* mask, int mask_mode, int64_t ignore_index,
                                                         int64_t T, int mean, float* out) {
    __shared__ double sums[32];
    __shared__ long long counts[32];
    grid_wait_prior();
    double s = 0.;
    long long n = 0;
    for (int64_t r = threadIdx.x; r < T; r += 1024) {
        s += (double)loss[r];
        n += ce_active(mask, mask_mode, ignore_index, mask_mode == RLK_MASK_EXPLICIT ? 0 : targets[r], r);
    }
    s = block_sum(s, sums);
    n = block_sum(n, counts);
    if (threadIdx.x == 0) *out = (float)(mean ? (n > 0 ? s / (double)n : 0.) : s);
}

struct CeRows {
    const float* grad;
    const int64_t* targets;
    const uint8_t* mask;
    float* scale;
    int32_t* count;
    int32_t* index;  // [T] the active rows, in order
    int32_t* place;  // [T] a row's place among them, -1 for an inactive one
    uint32_t* status;
    int64_t T, ignore_index;
    int32_t mask_mode, reduction;
    float keep;  // 1 - eps, the target's share of the loss
};

// The active rows in order, and the factor that is left out of every row's dx:
// the gradient of a summed loss, that of an averaged one over the active rows,
// or the largest finite magnitude of the rows' gradients (a non-finite one
// stays its own row's), each times 1 - eps.  One CTA.
__global__ void __launch_bounds__(1024) ce_rows_kernel(const CeRows p) {
    constexpr int kRuns = 4;  // 1024 rows each, loaded together
    __shared__ int counts[kRuns][32];
    __shared__ float tops[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) *p.status = 0;  // of this call; what sets it runs later
    int n = 0;
    float top = 0.f;
    for (int64_t r0 = 0; r0 < p.T; r0 += kRuns * 1024) {
        uint32_t on[kRuns];  // of the warp's 32 rows
#pragma unroll
        for (int j = 0; j < kRuns; ++j) {
            const int64_t r = r0 + j * 1024 + threadIdx.x;
            on[j] = __ballot_sync(0xFFFFFFFFu, r < p.T && ce_active(p.mask, p.mask_mode, p.ignore_index,
                                                                    p.mask_mode == RLK_MASK_EXPLICIT ? 0 : p.targets[r],
                                                                    r));
            if (lane == 0) counts[j][warp] = __popc(on[j]);
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kRuns; ++j) {
            const int64_t r = r0 + j * 1024 + threadIdx.x;
            const int c = counts[j][lane];
            const int before = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? c : 0);
            const bool mine = on[j] >> lane & 1u;
            const int at = n + before + __popc(on[j] & ((1u << lane) - 1u));
            if (r < p.T) p.place[r] = mine ? at : -1;
            if (mine) {
                p.index[at] = (int32_t)r;
                if (p.reduction == RLK_REDUCE_NONE) {
                    const float g = fabsf(p.grad[r]);
                    if (g < INFINITY) top = fmaxf(top, g);
                }
            }
            n += __reduce_add_sync(0xFFFFFFFFu, c);
        }
        __syncthreads();
    }
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if (lane == 0) tops[warp] = top;
    __syncthreads();
    if (threadIdx.x != 0) return;
    *p.count = n;
    if (p.reduction == RLK_REDUCE_NONE) {
        for (int w = 1; w < 32; ++w) top = fmaxf(top, tops[w]);
        const float s = __fmul_rn(top, p.keep);  // 0 where the product underflows
        *p.scale = s != 0.f ? s : top != 0.f ? top : 1.f;
    } else {
        const float g = p.reduction == RLK_REDUCE_SUM ? p.grad[0] : n > 0 ? (float)((double)p.grad[0] / (double)n) : 0.f;
        *p.scale = __fmul_rn(g, p.keep);
    }
}

// The active rows' hidden together, [.., Hs] with zeros past H and in the rows
// up to the next whole tile; and zeros into the inactive rows of dHidden.  Or,
// without a count, every row's.  A warp a row.
__global__ void __launch_bounds__(256) ce_gather_kernel(const uint16_t* hidden, int64_t ld, int H, int64_t T,
                                                        const int32_t* count, const int32_t* place, uint16_t* rows,
                                                        int64_t Hs, uint16_t* dhidden, int64_t ldh) {
    const int lane = threadIdx.x & 31;
    const int64_t n = count ? *count : T, whole = count ? (n + 255) / 256 * 256 : T;
    for (int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); r < T + (whole - n); r += (int64_t)gridDim.x * 8) {
        const int64_t to = r >= T ? n + (r - T) : count ? place[r] : r;
        if (to < 0) {
            if (dhidden)
                for (int c = lane * 8; c < H; c += 256) {
                    uint16_t* d = dhidden + r * ldh + c;
                    if (c + 8 <= H)
                        *reinterpret_cast<uint4*>(d) = make_uint4(0u, 0u, 0u, 0u);
                    else
                        for (int j = 0; c + j < H; ++j) d[j] = 0;
                }
            continue;
        }
#pragma unroll 2
        for (int c = lane * 8; c < Hs; c += 256) {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (r < T && c < H) {
                const uint16_t* x = hidden + r * ld + c;
                if (c + 8 <= H) {
                    v = *reinterpret_cast<const uint4*>(x);
                } else {
                    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (c + j < H) w[j >> 1] |= (uint32_t)x[j] << (16 * (j & 1));
                    v = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            *reinterpret_cast<uint4*>(rows + to * Hs + c) = v;
        }
    }
}

// ----------------------------------------------------------------- the gradients' products

struct CeGrads {
    uint16_t* dhidden;  // [T, ldh] BF16, or NULL
    uint16_t* dweight;  // the piece's rows, [cols, ldw] BF16, or NULL
    float* sums;        // [S, T, Hs] FP32 sums of dHidden across the pieces
    const float* scale;
    PipeWait w;
    const int32_t *count, *index;  // the active rows
    int64_t T, ldh, ldw, Hs;
    int32_t cols;         // vocabulary rows of the piece
    int32_t H, NB, NBg, MB1, S, KB0;
    int32_t first, last;  // the first and the last piece
};

// What follows from the number of active rows.
struct CeDeal {
    int n;        // active rows
    int MB0, KB1;
    int n0, n1;   // tiles of dHidden (S slices of MB0 x NB) and of dWeight (MB1 x NB)
    int head;     // the tiles with the longer K range: 0 dHidden's, 1 dWeight's
    int deal;     // of the others, how many make up for a long tile less (ce_walk)
};
__device__ __forceinline__ CeDeal ce_deal(const CeGrads& p, int pairs) {
    CeDeal d;
    d.n = *p.count;
    d.MB0 = (d.n + 255) / 256;
    d.KB1 = (d.n + kBK - 1) / kBK;
    d.n0 = p.dhidden ? p.S * d.MB0 * p.NB : 0;
    d.n1 = p.dweight ? p.MB1 * p.NB : 0;
    const int k0 = (p.KB0 + p.S - 1) / p.S, k1 = max(d.KB1, 1);
    d.head = k0 >= k1 ? 0 : 1;
    const int nl = d.head ? d.n1 : d.n0, ns = d.head ? d.n0 : d.n1, left = nl % pairs;
    const int64_t make_up = left ? (int64_t)(pairs - left) * ((d.head ? k1 : k0) / (d.head ? k0 : k1)) : 0;
    d.deal = (int)min(make_up, (int64_t)ns);
    return d;
}

// A pair's i-th tile: 0 .. n0 - 1 dHidden's, then dWeight's; -1 past its last.
// The longer tiles are dealt round; the pairs that the last round leaves out
// get the first `deal` of the shorter ones among themselves, and the rest are
// dealt round again.  A deal that both CTAs' roles know from the start.
__device__ __forceinline__ int ce_walk(const CeDeal& p, int i, int pair, int pairs) {
    const int nl = p.head ? p.n1 : p.n0, ns = p.head ? p.n0 : p.n1, left = nl % pairs;
    const int mine = nl / pairs + (pair < left);
    int v, is_long = 0;
    if (i < mine) {
        v = pair + i * pairs;
        is_long = 1;
    } else {
        i -= mine;
        const int k = pairs - left, at = pair - left;  // `deal` is 0 without a last round
        const int extra = at >= 0 && at < p.deal ? (p.deal - at + k - 1) / k : 0;
        v = i < extra ? at + i * k : p.deal + pair + (i - extra) * pairs;
        if (v >= ns) return -1;
    }
    return (is_long != 0) == (p.head == 0) ? v : p.n0 + v;
}

struct CeTile {
    int prob, mb, nb, wide, slice, k0, k1;  // wide: 64-column blocks of a CTA (2, or 1 in a narrow last tile)
};

// dHidden slice by slice; bands of NBg H blocks, M-major within a band.
__device__ __forceinline__ CeTile ce_tile(const CeGrads& p, const CeDeal& d, int u) {
    CeTile t;
    t.prob = u < d.n0 ? 0 : 1;
    uint32_t v = t.prob ? u - d.n0 : u;
    const uint32_t MB = t.prob ? p.MB1 : d.MB0;
    t.slice = 0;
    if (!t.prob) {
        t.slice = (int)(v / (MB * p.NB));
        v %= MB * p.NB;
    }
    const uint32_t band = MB * p.NBg, full = (uint32_t)p.NB / p.NBg;
    const uint32_t b = min(v / band, full);
    const uint32_t r = v - b * band;
    const uint32_t w = b < full ? p.NBg : p.NB - full * p.NBg;
    t.mb = (int)(r / w);
    t.nb = (int)(b * p.NBg + r % w);
    t.wide = p.H - t.nb * kBN > 128 ? 2 : 1;
    t.k0 = t.prob ? 0 : (int)((int64_t)p.KB0 * t.slice / p.S);
    t.k1 = t.prob ? d.KB1 : (int)((int64_t)p.KB0 * (t.slice + 1) / p.S);
    return t;
}

// tmB*: the MN-major operand's 64-wide blocks, two in one 3-D box; tmC*: the
// same matrix in 2-D boxes of one block, for a tile that holds H's ragged end
// or is narrow.
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kCeThreads, 1)
    ce_grads_kernel(const __grid_constant__ CUtensorMap tmA0, const __grid_constant__ CUtensorMap tmB0,
                    const __grid_constant__ CUtensorMap tmC0, const __grid_constant__ CUtensorMap tmA1,
                    const __grid_constant__ CUtensorMap tmB1, const __grid_constant__ CUtensorMap tmC1,
                    const __grid_constant__ CeGrads p) {
    extern __shared__ unsigned char smem_raw[];
    const CeSmem m = ce_smem(smem_raw);
    PairBars<kCeStages>* bars = m.bars;
    const int warp = warp_index(), lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank();
    const int pair = (int)blockIdx.x / 2, pairs = (int)gridDim.x / 2;
    const CeDeal deal = ce_deal(p, pairs);
    const uint32_t tmem = pair_begin(bars, warp, kCeEpilogue);
    int* ab = &bars->abort_flag;

    if (warp == 0) {
        const bool one = elect_one();
        const uint32_t full0 = mapa_shared(smem_u32(&bars->full[0]), 0);
        Ring r;
        uint64_t issued = 0;
        bool ok = true;
        for (int i = 0, u; ok && (u = ce_walk(deal, i, pair, pairs)) >= 0; ++i) {
            const CeTile t = ce_tile(p, deal, u);
            const int m0 = (2 * t.mb + rank) * 128, h0 = t.nb * kBN + rank * t.wide * 64;
            // (the active rows' hidden is padded with zeros to whole blocks)
            const bool box3 = t.wide == 2 && (t.prob == 1 || p.H % 64 == 0 || p.H - t.nb * kBN >= kBN);
            for (int kb = t.k0; kb < t.k1; ++kb) {
                if (!(ok = pipe_wait_warp(ab, smem_u32(&bars->empty[r.slot]), r.phase ^ 1u, p.w))) break;
                if (one) {
                    const uint32_t fb = full0 + r.slot * 8;
                    const uint32_t a = smem_u32(m.a + r.slot * kCeA), b = smem_u32(m.b + r.slot * kCeB);
                    pair_arm(fb, smem_u32(&bars->full[r.slot]), rank, kCeA + (uint32_t)t.wide * kMnBlock);
                    if (t.prob == 0) {
                        tma_load_2d_pair(a, &tmA0, kb * kBK, m0, fb);
                    } else {
                        tma_load_2d_pair(a, &tmA1, m0, kb * kBK, fb);
                        tma_load_2d_pair(a + kMnBlock, &tmA1, m0 + 64, kb * kBK, fb);
                    }
                    if (box3) {
                        tma_load_3d_pair(b, t.prob ? &tmB1 : &tmB0, 0, kb * kBK, h0 / 64, fb);
                    } else {
                        for (int j = 0; j < t.wide; ++j)
                            tma_load_2d_pair(b + j * kMnBlock, t.prob ? &tmC1 : &tmC0, h0 + j * 64, kb * kBK, fb);
                    }
                }
                ++issued;
                r.next(kCeStages);
            }
        }
        pair_end_copies(bars, r, one, issued, ok, p.w);
    } else if (warp == 1 && rank == 0) {
        const bool one = elect_one();
        const uint64_t dk = smem_desc_sw128(smem_u32(m.a)), dm = smem_desc_sw128_mn(smem_u32(m.a), kMnBlock, 1024);
        const uint64_t db = smem_desc_sw128_mn(smem_u32(m.b), kMnBlock, 1024);
        Ring r, acc;
        bool ok = true;
        for (int i = 0, u; ok && (u = ce_walk(deal, i, pair, pairs)) >= 0; ++i) {
            const CeTile t = ce_tile(p, deal, u);
            if (!(ok = pipe_wait_warp(ab, smem_u32(&bars->tempty[acc.slot]), acc.phase ^ 1u, p.w))) break;
            tc_fence_after();
            const uint32_t idesc = idesc_bf16_f32_major(256, (uint32_t)(128 * t.wide), t.prob == 1, true);
            const uint32_t d = tmem + (uint32_t)(acc.slot * kBN);
            // K-major A advances 16 elements (32 B) within its swizzle rows; an MN-major operand two 8-row K
            // groups (2 x 1024 B)
            const uint64_t da = t.prob == 0 ? dk : dm;
            const int astep = t.prob == 0 ? 32 : 2048;
            for (int kb = t.k0; kb < t.k1; ++kb) {
                if (!(ok = pipe_wait_warp(ab, smem_u32(&bars->full[r.slot]), r.phase, p.w))) break;
                tc_fence_after();
                if (one) {
#pragma unroll
                    for (int kk = 0; kk < kBK / 16; ++kk)
                        umma_bf16_pair(d, da + ((r.slot * kCeA + kk * astep) >> 4),
                                       db + ((r.slot * kCeB + kk * 2048) >> 4), idesc, kb != t.k0 || kk != 0);
                    umma_commit_pair(smem_u32(&bars->empty[r.slot]));
                }
                __syncwarp();
                r.next(kCeStages);
            }
            if (ok && one) umma_commit_pair(smem_u32(&bars->tfull[acc.slot]));
            __syncwarp();
            acc.next(2);
        }
        pair_end_mmas(bars, acc, one, ok, p.w);
    } else if (warp >= 2) {
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
        unsigned char* stage = m.out + (warp - 2) * kCeOut;
        const uint32_t done = mapa_shared(smem_u32(&bars->tempty[0]), 0);
        const float scale = *p.scale;
        Ring acc;
        for (int i = 0, u; (u = ce_walk(deal, i, pair, pairs)) >= 0; ++i) {
            const CeTile t = ce_tile(p, deal, u);
            if (!__all_sync(0xFFFFFFFFu, pipe_wait(ab, smem_u32(&bars->tfull[acc.slot]), acc.phase, p.w))) break;
            tc_fence_after();
            const int64_t row0 = (int64_t)(2 * t.mb + rank) * 128 + quarter * 32, row = row0 + lane;
            const int64_t nrows = t.prob == 0 ? deal.n : p.cols;
            // dHidden leaves as BF16 from the only slice of the last piece, else into the sums
            const bool out = t.prob == 1 || (p.S == 1 && p.last);
            for (int sub = half * 2 * t.wide; sub < (half + 1) * 2 * t.wide; ++sub) {
                if (t.nb * kBN + sub * 32 >= p.H) break;
                float v[32];
                tmem_ld32(tmem + lane_base + (uint32_t)(acc.slot * kBN + sub * 32), v);
                if (t.k0 == t.k1) {  // a slice without K blocks (a short last piece): no MMA wrote the accumulator
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = 0.f;
                }
                const int col0 = t.nb * kBN + sub * 32;
                if (t.prob == 0 && !(out && p.first) && row < nrows) {
                    float4* s4 = reinterpret_cast<float4*>(p.sums + ((int64_t)t.slice * p.T + row) * p.Hs + col0);
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        if (!p.first) {
                            const float4 o = s4[q];
                            v[4 * q] = __fadd_rn(o.x, v[4 * q]), v[4 * q + 1] = __fadd_rn(o.y, v[4 * q + 1]);
                            v[4 * q + 2] = __fadd_rn(o.z, v[4 * q + 2]), v[4 * q + 3] = __fadd_rn(o.w, v[4 * q + 3]);
                        }
                        if (!out) s4[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                    }
                }
                if (out) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = __fmul_rn(v[i], scale);
                    const int64_t ld = t.prob == 0 ? p.ldh : p.ldw;
                    ce_store(stage, lane, v, t.prob == 0 ? p.dhidden + col0 : p.dweight + row0 * ld + col0, ld,
                             (int)max((int64_t)0, min((int64_t)32, nrows - row0)), p.H - col0,
                             t.prob == 0 ? p.index + row0 : nullptr);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(done + acc.slot * 8);
            acc.next(2);
        }
    }
    pair_end(bars, tmem, warp, p.w);
}

// Up to 8 BF16 values of an output row; columns past H are not the row's.
__device__ __forceinline__ void store_bf16x8(uint16_t* row, int col, int H, const float* v) {
    const uint32_t w[4] = {pack_bf16x2_rn(v[0], v[1]), pack_bf16x2_rn(v[2], v[3]), pack_bf16x2_rn(v[4], v[5]),
                           pack_bf16x2_rn(v[6], v[7])};
    if (col + 8 <= H) {
        *reinterpret_cast<uint4*>(row + col) = make_uint4(w[0], w[1], w[2], w[3]);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (col + j < H) row[col + j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
}

// dHidden from the S slices' sums, added in order.
__global__ void __launch_bounds__(256) ce_join_kernel(const float* sums, const float* scale, int S, int64_t T,
                                                      int64_t Hs, int H, const int32_t* count, const int32_t* index,
                                                      uint16_t* dhidden, int64_t ldh) {
    const int groups = (H + 7) / 8;
    const int64_t n = (int64_t)*count * groups;
    const float sc = *scale;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / groups;
        const int col = (int)(i % groups) * 8;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int s = 0; s < S; ++s) {
            const float4* q = reinterpret_cast<const float4*>(sums + ((int64_t)s * T + row) * Hs + col);
            const float4 a = q[0], b = q[1];
            const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __fadd_rn(v[j], x[j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(v[j], sc);
        store_bf16x8(dhidden + index[row] * ldh, col, H, v);
    }
}

// ----------------------------------------------------------------- host

size_t up256(size_t b) { return (b + 255) / 256 * 256; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// How the backward cuts the vocabulary and dHidden's K range.
struct CePlan {
    int64_t P, pieces, S, Hs;
    int MB, NB;
};

CePlan plan_of(const rlk_linear_ce_contract& c) {
    CePlan q{};
    q.MB = (int)ceil_div(c.T, 256);
    q.NB = (int)ceil_div(c.H, kBN);
    q.Hs = ceil_div(c.H, 64) * 64;
    const int64_t whole = ceil_div(c.V, kBN) * kBN;
    int64_t P = c.piece > 0 ? ceil_div(c.piece, kBN) * kBN : kPieceBytes / (2 * c.T) / kBN * kBN;
    const int64_t least = ceil_div(ceil_div(c.V, kMaxPieces), kBN) * kBN;
    if (c.piece <= 0 && P < kMinPiece) P = kMinPiece;
    if (P < least) P = least;
    if (P > whole) P = whole;
    q.pieces = ceil_div(c.V, P);
    if (c.piece <= 0) P = ceil_div(ceil_div(c.V, q.pieces), kBN) * kBN;  // pieces of one size
    q.pieces = ceil_div(c.V, P);
    q.P = P;
    // dHidden has MB NB tiles with a K range of P: where they are fewer than two a pair of CTAs (76
    // pairs) the range is cut so that they are, in slices of at least 8 K blocks, with sums of their own.
    const int64_t tiles = (int64_t)q.MB * q.NB;
    int64_t S = ceil_div(152, tiles);
    if (S > P / (8 * kBK)) S = P / (8 * kBK);
    if (S > kMaxSlices) S = kMaxSlices;
    q.S = S < 1 ? 1 : S;
    return q;
}

struct CeLayout {
    size_t loss, yt, part, part_y, all, fwd_end;
    size_t scale, count, index, place, rows, dx, sums, bwd_end;
};

// Whether the forward first copies hidden onto 128-byte lines, as the backward does: where its rows' stride puts them
// between lines, and the product is large enough to repay the copy's launch and 4 T H bytes (50257 x 1000: 500 tokens
// take 62 us without and 55 with it, 1000 take 95 and 76, 4000 take 273 and 225; 250 have 6 us to gain and 4 to pay).
bool ce_copies(const rlk_linear_ce_contract& c) {
    return c.hidden_stride % 64 != 0 && c.T > 1 && (double)c.T * (double)c.V * (double)c.H >= 25e9;
}

CeLayout layout_of(const rlk_linear_ce_contract& c) {
    CeLayout l{};
    const size_t T = (size_t)c.T, parts = 2 * (size_t)ceil_div(c.V, kBN);
    const size_t at = kWorkspaceBytes;
    l.loss = at;
    l.yt = l.loss + up256(4 * T);
    l.part = l.yt + up256(4 * T);
    l.part_y = l.part + up256(8 * T * parts);
    l.all = l.part_y + (c.label_smoothing != 0.f ? up256(4 * T * parts) : 0);
    const CePlan q = plan_of(c);
    l.fwd_end = l.all + (ce_copies(c) ? up256(2 * T * (size_t)q.Hs) : 0);
    l.scale = at;
    l.count = l.scale + 16;
    l.index = l.scale + 256;
    l.place = l.index + up256(4 * T);
    l.rows = l.place + up256(4 * T);
    l.dx = l.rows + up256(2 * (size_t)q.MB * 256 * (size_t)q.Hs);
    l.sums = l.dx + up256(2 * T * (size_t)q.P);
    l.bwd_end = l.sums + (q.pieces > 1 || q.S > 1 ? up256(4 * (size_t)q.S * T * (size_t)q.Hs) : 0);
    return l;
}

// The target's share of the loss, which dx leaves out; all of the loss is the uniform distribution's at eps = 1.
float ce_keep(const rlk_linear_ce_contract& c) { return c.label_smoothing < 1.f ? 1.f - c.label_smoothing : 1.f; }

rlk_status ce_cuda(const char* what) {
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? RLK_OK : fail(RLK_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

rlk_status ce_sms(int* sms) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || *sms <= 0)
        return fail(RLK_ERR_CUDA, "cannot query the device's SM count");
    return RLK_OK;
}

// A launch that the kernel before it in the stream may overlap with its setting
// up (the kernel waits with grid_wait_prior).
template <typename... Args>
void launch_behind(void (*kernel)(Args...), int64_t blocks, int threads, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, kernel, args...);  // an error stays for ce_cuda
}

template <int MODE, bool CAP, bool SMOOTH>
rlk_status launch_logits(const CUtensorMap& h, const CUtensorMap& w, uint16_t* dx, int64_t ldx, const CeParams& p,
                         int sms, cudaStream_t st) {
    if (!allow_dynamic_smem<ce_logits_kernel<MODE, CAP, SMOOTH>>(kCeSmem))
        return ce_cuda("linear cross entropy: shared memory");
    const int64_t units = (int64_t)p.nch * p.MB, pairs = sms / 2;
    ce_logits_kernel<MODE, CAP, SMOOTH>
        <<<(unsigned)(2 * (units < pairs ? units : pairs)), kCeThreads, kCeSmem, st>>>(h, w, dx, ldx, p);
    return ce_cuda("linear cross entropy launch");
}

CeParams ce_params(const rlk_linear_ce_contract& c, const int64_t* targets, const uint8_t* mask, uint32_t* status) {
    CeParams p{};
    p.targets = targets;
    p.mask = mask;
    p.w.status = status;
    p.w.wait_ns = c.wait_timeout_ns > 0 ? (uint64_t)c.wait_timeout_ns : kDefaultWaitNs;
    p.T = c.T;
    p.V = c.V;
    p.ignore_index = c.ignore_index;
    p.cap = c.softcap;
    p.icap = c.softcap > 0.f ? 1.f / c.softcap : 0.f;
    p.eps = c.label_smoothing;
    p.z = c.z_loss;
    p.unit = 1.f / ce_keep(c);
    p.KB = (int32_t)ceil_div(c.H, kBK);
    p.mask_mode = c.mask_mode;
    p.MB = (int32_t)ceil_div(c.T, 256);
    p.box_rows = (int32_t)(c.T < 128 ? ceil_div(c.T, 8) * 8 : 128);
    const int64_t band = kBandBytes / ((int64_t)256 * c.H * 2);
    p.MBg = (int32_t)(band < 1 ? 1 : band < p.MB ? band : p.MB);
    return p;
}

void launch_gather(const rlk_linear_ce_contract& c, const void* hidden, const int32_t* count, const int32_t* place,
                   uint16_t* rows, int64_t Hs, void* dhidden, int sms, cudaStream_t st) {
    const int64_t blocks = ceil_div(c.T + 255, 8);
    ce_gather_kernel<<<(unsigned)(blocks < 8 * sms ? blocks : 8 * sms), 256, 0, st>>>(
        static_cast<const uint16_t*>(hidden), c.hidden_stride, (int)c.H, c.T, count, place, rows, Hs,
        static_cast<uint16_t*>(dhidden), c.dhidden_stride);
}

const char kMapFailed[] = "cuTensorMapEncodeTiled failed for an operand of the linear cross entropy";

}  // namespace

size_t linear_ce_workspace(const rlk_linear_ce_contract& c, bool grad) {
    const CeLayout l = layout_of(c);
    return grad ? (l.bwd_end > l.fwd_end ? l.bwd_end : l.fwd_end) : l.fwd_end;
}

rlk_status launch_linear_ce_fwd(const rlk_linear_ce_contract& c, const void* hidden, const void* weight,
                                const int64_t* targets, const uint8_t* mask, float* loss, float* lse, void* workspace,
                                cudaStream_t st) {
    int sms = 0;
    rlk_status s = ce_sms(&sms);
    if (s != RLK_OK) return s;
    const CeLayout l = layout_of(c);
    char* ws = static_cast<char*>(workspace);
    uint32_t* status = static_cast<uint32_t*>(workspace);
    if (cudaMemsetAsync(ws, 0, sizeof(uint32_t), st) != cudaSuccess) return ce_cuda("clearing the status word");
    CeParams p = ce_params(c, targets, mask, status);
    p.part = reinterpret_cast<float2*>(ws + l.part);
    p.part_y = reinterpret_cast<float*>(ws + l.part_y);
    p.yt = reinterpret_cast<float*>(ws + l.yt);
    p.ch0 = 0;
    p.nch = (int32_t)ceil_div(c.V, kBN);
    int64_t width = c.H, stride = c.hidden_stride;
    if (ce_copies(c)) {
        uint16_t* all = reinterpret_cast<uint16_t*>(ws + l.all);
        width = stride = plan_of(c).Hs;
        launch_gather(c, hidden, nullptr, nullptr, all, width, nullptr, sms, st);
        hidden = all;
    }
    CUtensorMap tmH, tmW;
    if (!make_map(&tmH, hidden, width, c.T, stride, kBK, (uint32_t)p.box_rows) ||
        !make_map(&tmW, weight, c.H, c.V, c.weight_stride, kBK, 128))
        return fail(RLK_ERR_CUDA, kMapFailed);
    const bool cap = c.softcap > 0.f, smooth = c.label_smoothing != 0.f;
    s = cap ? (smooth ? launch_logits<kCeForward, true, true>(tmH, tmW, nullptr, 0, p, sms, st)
                      : launch_logits<kCeForward, true, false>(tmH, tmW, nullptr, 0, p, sms, st))
            : (smooth ? launch_logits<kCeForward, false, true>(tmH, tmW, nullptr, 0, p, sms, st)
                      : launch_logits<kCeForward, false, false>(tmH, tmW, nullptr, 0, p, sms, st));
    if (s != RLK_OK) return s;
    CeFold f{};
    f.part = p.part;
    f.part_y = smooth ? p.part_y : nullptr;
    f.yt = p.yt;
    f.targets = targets;
    f.mask = mask;
    f.loss = c.reduction == RLK_REDUCE_NONE ? loss : reinterpret_cast<float*>(ws + l.loss);
    f.lse = lse;
    f.status = status;
    f.T = c.T;
    f.V = c.V;
    f.ignore_index = c.ignore_index;
    f.parts = 2 * p.nch;
    f.mask_mode = c.mask_mode;
    f.eps = c.label_smoothing;
    f.z = c.z_loss;
    launch_behind<CeFold>(ce_fold_kernel, ceil_div(c.T, kFoldRows), kFoldRows * kFoldSlices, st, f);
    if (c.reduction != RLK_REDUCE_NONE)
        launch_behind<const float*, const int64_t*, const uint8_t*, int, int64_t, int64_t, int, float*>(
            ce_reduce_kernel, 1, 1024, st, f.loss, targets, mask, c.mask_mode, c.ignore_index, c.T,
            c.reduction == RLK_REDUCE_MEAN, loss);
    return ce_cuda("linear cross entropy: merge");
}

rlk_status launch_linear_ce_bwd(const rlk_linear_ce_contract& c, const void* hidden, const void* weight,
                                const int64_t* targets, const uint8_t* mask, const float* lse, const float* grad,
                                void* dhidden, void* dweight, void* workspace, cudaStream_t st) {
    int sms = 0;
    rlk_status s = ce_sms(&sms);
    if (s != RLK_OK) return s;
    const CeLayout l = layout_of(c);
    const CePlan q = plan_of(c);
    char* ws = static_cast<char*>(workspace);
    uint32_t* status = static_cast<uint32_t*>(workspace);
    float* scale = reinterpret_cast<float*>(ws + l.scale);
    uint16_t* rows = reinterpret_cast<uint16_t*>(ws + l.rows);
    CeRows r{};
    r.grad = grad;
    r.targets = targets;
    r.mask = mask;
    r.scale = scale;
    r.count = reinterpret_cast<int32_t*>(ws + l.count);
    r.index = reinterpret_cast<int32_t*>(ws + l.index);
    r.place = reinterpret_cast<int32_t*>(ws + l.place);
    r.status = status;
    r.T = c.T;
    r.ignore_index = c.ignore_index;
    r.mask_mode = c.mask_mode;
    r.reduction = c.reduction;
    r.keep = ce_keep(c);
    ce_rows_kernel<<<1, 1024, 0, st>>>(r);
    launch_gather(c, hidden, r.count, r.place, rows, q.Hs, dhidden, sms, st);
    if ((s = ce_cuda("linear cross entropy: rows")) != RLK_OK) return s;

    if (!allow_dynamic_smem<ce_grads_kernel>(kCeSmem))
        return ce_cuda("linear cross entropy: shared memory");
    CeParams p = ce_params(c, targets, mask, status);
    p.lse = lse;
    p.grad = c.reduction == RLK_REDUCE_NONE ? grad : nullptr;
    p.scale = scale;
    p.count = r.count;
    p.index = r.index;
    CeGrads g{};
    g.dhidden = static_cast<uint16_t*>(dhidden);
    g.sums = reinterpret_cast<float*>(ws + l.sums);
    g.scale = scale;
    g.w = p.w;
    g.T = c.T;
    g.ldh = c.dhidden_stride;
    g.ldw = c.dweight_stride;
    g.Hs = q.Hs;
    g.H = (int32_t)c.H;
    g.NB = q.NB;
    g.NBg = q.NB < kBandH ? q.NB : kBandH;
    g.S = (int32_t)q.S;
    g.count = r.count;
    g.index = r.index;
    uint16_t* dx = reinterpret_cast<uint16_t*>(ws + l.dx);
    CUtensorMap tmH, tmB1, tmC1;
    const bool wide = c.H >= 64;
    const int64_t whole = (int64_t)q.MB * 256;
    if (!make_map(&tmH, rows, q.Hs, whole, q.Hs, kBK, (uint32_t)p.box_rows) ||
        !make_map(&tmC1, rows, q.Hs, whole, q.Hs, 64, kBK) || !make_map_mn3(&tmB1, rows, q.Hs, whole, q.Hs, kBK, 2))
        return fail(RLK_ERR_CUDA, kMapFailed);
    for (int64_t i = 0; i < q.pieces; ++i) {
        const int64_t c0 = i * q.P, cols = c.V - c0 < q.P ? c.V - c0 : q.P;
        const uint16_t* w0 = static_cast<const uint16_t*>(weight) + c0 * c.weight_stride;
        CUtensorMap tmW, tmA0, tmA1, tmB0, tmC0;
        if (!make_map(&tmW, weight, c.H, c.V, c.weight_stride, kBK, 128) ||
            !make_map(&tmA0, dx, cols, c.T, q.P, kBK, 128) ||
            !make_map(&tmA1, dx, cols, c.T, q.P, 64, kBK) ||
            !make_map(&tmC0, w0, c.H, cols, c.weight_stride, 64, kBK) ||
            (wide && !make_map_mn3(&tmB0, w0, c.H / 64 * 64, cols, c.weight_stride, kBK, 2)))
            return fail(RLK_ERR_CUDA, kMapFailed);
        if (!wide) tmB0 = tmC0;
        p.ch0 = (int32_t)(c0 / kBN);
        p.nch = (int32_t)ceil_div(cols, kBN);
        s = c.softcap > 0.f ? launch_logits<kCeGrad, true, false>(tmH, tmW, dx, q.P, p, sms, st)
                            : launch_logits<kCeGrad, false, false>(tmH, tmW, dx, q.P, p, sms, st);
        if (s != RLK_OK) return s;
        g.dweight = dweight ? static_cast<uint16_t*>(dweight) + c0 * c.dweight_stride : nullptr;
        g.cols = (int32_t)cols;
        g.KB0 = (int32_t)ceil_div(cols, kBK);
        g.MB1 = (int32_t)ceil_div(cols, 256);
        g.first = i == 0;
        g.last = i == q.pieces - 1;
        const int64_t tiles = (dhidden ? q.S * q.MB * q.NB : 0) + (dweight ? (int64_t)g.MB1 * q.NB : 0);
        const int pairs = (int)(tiles < sms / 2 ? tiles : sms / 2);
        ce_grads_kernel<<<2 * pairs, kCeThreads, kCeSmem, st>>>(tmA0, tmB0, tmC0, tmA1, tmB1, tmC1, g);
        if ((s = ce_cuda("linear cross entropy: gradients")) != RLK_OK) return s;
    }
    if (dhidden && q.S > 1) {
        const int64_t blocks = ceil_div(c.T * ceil_div(c.H, 8), 256);
        ce_join_kernel<<<(unsigned)(blocks < 8 * sms ? blocks : 8 * sms), 256, 0, st>>>(
            g.sums, g.scale, g.S, c.T, q.Hs, g.H, g.count, g.index, g.dhidden, g.ldh);
        return ce_cuda("linear cross entropy: join");
    }
    return RLK_OK;
}

}  // namespace rlk
