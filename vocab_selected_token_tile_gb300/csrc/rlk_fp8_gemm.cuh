// Matrix product of E4M3 operands with an FP32 scale for each group of 128
// along K (sm_103a):
//
//   C[m, n] = sum_g sa[g, m] sb[g, n] sum_{k in group g} a[m, k] b[n, k]
//
// A [M, K] has one scale per row and group; B [N, K] one per row and group or
// one per 128 x 128 block.  The scales are not powers of two, so they cannot
// ride in the tensor core: each group's partial product is formed by four
// tcgen05.mma (kind::f8f6f4, K = 32) into a fresh tensor-memory accumulator,
// and the epilogue warps read it, scale it and add it to the sum they hold in
// registers (FP32 throughout: a product of two scales, one rounding, then one
// fused multiply-add per element and group).
//
// Two kernels:
//
// gemm_kernel, 256 x 256 tiles by pairs of CTAs (rlk_pair.cuh), persistent, one
// CTA per SM.  A pair halves what a CTA's MMAs read of B from shared memory (a
// first kernel, single CTAs with 128 x 256 tiles, took 452 us at 8192 x 12288 x
// 4096; this one 320 by itself, 338 call after call).  Floor: the tensor core,
// 2 M N K operations.  A group's four MMAs take 512 clocks; from one
// accumulator's completion to the next it is 850-900 with block scales and
// 1,200-1,250 with row scales.  The epilogue of a group reads back 128 KB of accumulator a CTA (256 clocks of the
// tensor-memory port), scales and adds it (128 packed operations a scheduler,
// twice that and 32 KB of shared memory with row scales), and hands it back,
// and tensor memory holds two accumulators.  8192 x 8192 x 8192: 390 us (2.8
// PFLOP/s, tensor pipe 55% busy) and 548 us (2.0 PFLOP/s, 38%), 435 and 567 in
// a long loop of them under the power cap.  Roles: warp 0
// issues the TMA loads, warp 1 of the even CTA the pair's MMAs, warp 2 fetches
// the scales with cp.async (4 bytes each: a row of scales starts at any
// multiple of 4), warps 4-11 are the epilogue (a warp reads 32 tensor-memory
// lanes and 128 of the 256 columns: 128 sums a thread, which is why the first
// warpgroup gives registers away with setmaxnreg).  Sixteen epilogue warps of
// 64 sums each were slower (400 us at 8192 x 12288 x 4096).
//
// skinny_kernel, for few rows of A: B's rows take the 128 lanes and A's rows
// the accumulator's columns (16, 32 or 64), so a single token streams the
// weight once and wastes no more than 15 columns.  Bound: HBM, N K bytes (37 x
// 151936 x 4096: 100 us, 6.3 TB/s; 1 x 4096 x 4096: 7.2 us).  Two
// CTAs per SM keep loads in flight across each other's start and end.  Where N
// / 128 tiles are fewer than the SMs can hold, a cluster of 2, 4 or 8 CTAs (of a
// layer without groups any number up to 8) splits K, and adds its partial sums through distributed shared memory in
// rank order: no workspace, no second launch, the same bits every time.
//
// Both are also built for a feed-forward layer (kEpi and on): z = A B^T + bias,
// y = act(z) or act(gate) * up, c = y + residual, in FP32 and rounded where they
// are stored.  A gated layer's B is loaded so that a thread has a column's gate
// and its other half: 64 rows of each by turns for a tile of a pair (one 4-D box a
// CTA), 16 for few rows.  The epilogue warps have nothing to hide this work
// behind, so it adds to a tile's time: 8192 x 12288 x 4096, 320 us bare, 331
// through this path, 357 with silu, 380 with gelu, 326 gated with silu (half as
// many results), 340 with an FP32 bias alone and 348 with a BF16 one, 366 with z
// kept, 390 with a BF16 residual and 451 with an FP32 one; a pass over the result
// would take 60 (a read and a write of 201 MB) or 90.
//
// And for rows that belong to groups, each with a B of its own (kRows, kHalves),
// and operands whose K axis belongs to groups (kDepth), where a CTA finds its
// tiles from the groups' ends (rlk_groups.cuh).
//
// Registers decide a lot here: a layer's loop keeps 128 sums and 64 loaded values
// a thread of the 224.  A barrier for biases that another warp had fetched (so
// one more wait in the epilogue) took the bare path from 333 to 370 us, and
// finishing the tile in loops over shared memory, with little code, took it to
// 420; what is there now came out of such trials.
//
// Every wait is bounded; on expiry the CTA records the time-out in the status
// word, stops issuing, waits (bounded) for the copies and MMAs under way (a
// pair for those of both of its CTAs), frees its tensor memory and returns.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>
#include <string>
#include <type_traits>

#include "rlk_act.cuh"
#include "rlk_gemm.cuh"
#include "rlk_groups.cuh"
#include "rlk_internal.h"
#include "rlk_pair.cuh"
#include "rlk_ptx.cuh"

namespace rlk {
namespace {

constexpr int kGK = 128;         // K of a group, and of a ring stage: 128 E4M3 = one 128-byte swizzle row
constexpr int kScaleStages = 8;  // ring of scales, deeper than the operands': its loads are small and unaligned

// D[tmem] (+)= A[smem] B[smem]^T, E4M3 inputs (format 0 in both fields), FP32 accumulate.
__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// The same by a pair of CTAs (M = 256: 128 rows of each).
__device__ __forceinline__ void umma_e4m3_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__host__ __device__ constexpr uint32_t idesc_e4m3_f32(uint32_t M, uint32_t N) {
    return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// 16 consecutive FP32 columns of a warp's 32 tensor-memory lanes; the values
// are there only after tmem_wait16 on the same registers.
__device__ __forceinline__ void tmem_ld16_issue(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait16(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15])::"memory");
}

// 32 columns of a warp's 32 lanes, a lane's row a thread; the values are there
// only after tmem_wait32.
__device__ __forceinline__ void tmem_ld32_issue(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
// The same as fragments: with t the thread's lane, v[16 h
// + 4 j + 2 i + e] is row 16 h + 8 i + t / 4, column 8 j + 2 (t mod 4) + e.  A
// thread then needs 4 rows' scales and 8 columns' for its 32 values, where a
// row a thread would need all 32 columns' (and shared memory returns 128 bytes
// of registers a clock); the load itself is the slower one of the two.
__device__ __forceinline__ void tmem_ld_frag_issue(uint32_t taddr, uint32_t (&v)[32]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t* r = v + 16 * h;
        asm volatile(
            "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
            "%14, %15}, [%16];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
              "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(taddr + ((uint32_t)(16 * h) << 16))
            : "memory");
    }
}
__device__ __forceinline__ void tmem_wait32(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}

// A 4-byte asynchronous copy, zero where `ok` is false (nothing is read then).
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(ok ? 4 : 0) : "memory");
}
// This thread's arrival on `bar` once its earlier copies have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// A ring of scales: its barriers.
struct ScaleBars {
    uint64_t full[kScaleStages];
    uint64_t empty[kScaleStages];
};

__device__ void init_scales(ScaleBars* b, int epilogue_warps) {
    for (int s = 0; s < kScaleStages; ++s) {
        mbar_init(smem_u32(&b->full[s]), 32);
        mbar_init(smem_u32(&b->empty[s]), epilogue_warps);
    }
}

// The barriers of a CTA on its own (skinny_kernel).
template <int STAGES, int ACCS>
struct Bars8 {
    uint64_t full[STAGES];
    uint64_t empty[STAGES];
    uint64_t tfull[ACCS];
    uint64_t tempty[ACCS];
    ScaleBars sc;
    uint64_t drain;
    uint32_t tmem_addr;
    int abort_flag;
};

template <int STAGES, int ACCS>
__device__ void init_bars8(Bars8<STAGES, ACCS>* b, int epilogue_warps) {
    for (int s = 0; s < STAGES; ++s) {
        mbar_init(smem_u32(&b->full[s]), 1);
        mbar_init(smem_u32(&b->empty[s]), 1);
    }
    for (int i = 0; i < ACCS; ++i) {
        mbar_init(smem_u32(&b->tfull[i]), 1);
        mbar_init(smem_u32(&b->tempty[i]), epilogue_warps);
    }
    init_scales(&b->sc, epilogue_warps);
    mbar_init(smem_u32(&b->drain), 1);
    b->abort_flag = 0;
    fence_mbar_init();
}

struct Gemm8Params {
    const float *sa, *sb;
    void* c;
    int64_t ldc;
    int32_t M, N, KB;
    int32_t MB, NB;     // tiles along M (of pairs) and N
    int32_t band;       // M tiles per band of the tile order
    int32_t nsb;        // scales of B per K group: N (rows) or ceil(N / 128) (blocks)
    int32_t c_f32, accumulate, vec;
    PipeWait w;
};

// What a kernel is built for: the product by itself; with an epilogue (bias,
// activation, residual); of rows that belong to groups, each with a B of its
// own, and that epilogue; of operands whose K axis belongs to groups, each with
// a C of its own.
enum Kind8 : int { kPlain, kEpi, kEpiGated, kRows, kRowsGated, kHalves, kHalvesGated, kDepth };
__host__ __device__ constexpr bool gated_kind(int k) { return k == kEpiGated || k == kRowsGated || k == kHalvesGated; }
__host__ __device__ constexpr bool half_kind(int k) { return k == kHalves || k == kHalvesGated; }
__host__ __device__ constexpr bool rows_kind(int k) { return k == kRows || k == kRowsGated || half_kind(k); }
__host__ __device__ constexpr bool layer_kind(int k) { return k == kEpi || k == kEpiGated || rows_kind(k); }

struct Ext8Params : Gemm8Params {
    // kEpi, kRows: z = A B^T + bias, y = act(z) (gated: B holds N rows of the gate, then N more; y = act(gate) * up),
    // c = y + residual
    const void *bias, *res;
    uint16_t* z;          // NULL, or where z goes in BF16
    int64_t ldr, ldz;
    int32_t bias_f32, bias_vec, res_f32, res_vec, z_vec, act;
    // kRows, kDepth
    const int32_t* ends;
    int32_t G, rest;      // rest: the rows behind the groups are set to zero
    int32_t deep;         // kDepth: rows before their padding, what `ends` may reach
    int64_t sb_g, c_g;    // elements between the groups' scales of B, and between their C (kDepth)
};
template <int KIND>
struct ParamsOf {
    using type = Ext8Params;
};
template <>
struct ParamsOf<kPlain> {
    using type = Gemm8Params;
};

// Where a warp's rows of a result go.
struct Dest {
    void* c;
    int64_t ldc;
    int64_t limit;  // rows below it are written
    int32_t N, vec, accumulate;
};
__device__ __forceinline__ Dest dest_of(const Gemm8Params& p, int64_t limit) {
    return Dest{p.c, p.ldc, limit, p.N, p.vec, p.accumulate};
}

// 8 BF16 columns of a row on the 16-byte grid, of which `cols` are C's.
__device__ __forceinline__ void store_piece(uint16_t* c, uint4 w, int cols) {
    if (cols >= 8) {
        *reinterpret_cast<uint4*>(c) = w;
        return;
    }
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < cols) c[e] = (uint16_t)(x[e >> 1] >> (16 * (e & 1)));
}

// f(0) ... f(COUNT - 1), each number a type, for places in an array that the
// compiler is to check.
template <int COUNT, int AT = 0, typename F>
__device__ __forceinline__ void each(F&& f) {
    if constexpr (AT < COUNT) {
        f(std::integral_constant<int, AT>{});
        each<COUNT, AT + 1>(f);
    }
}

// A warp's 32 rows x 128 bytes of C (32 FP32 or 64 BF16 columns) through shared
// memory, so that a row's 128 bytes leave in one piece: 16 bytes a lane
// straight from the registers, 32 rows an instruction, took 10,700 clocks a 128
// x 256 tile, a third of the product's time at K = 4096.  16-byte piece j of
// row r is kept at j ^ turn(r), which spreads both directions over the banks.
// The pairs [FIRST, FIRST + PAIRS) of v: the lane's row (pairs of columns), or with FRAG, of each 32 columns, 4 rows
// (t / 4 and 8, 16, 24 after) x 4 pairs (2 (t mod 4) and 8, 16, 24 after).  PAIRS below 16 (FP32) or 32 (BF16): only
// the first columns, 16 bytes of them at least.
template <bool F32, bool FRAG, int FIRST, int PAIRS = F32 ? 16 : 32, int N>
__device__ __forceinline__ void store_chunk(const Dest& p, unsigned char* out, int lane, int64_t row0, int col0,
                                            const float2 (&v)[N]) {
    constexpr int kPer = F32 ? 4 : 8;  // elements of 16 bytes
    constexpr int kPieces = 2 * PAIRS / kPer;
    static_assert(FIRST >= 0 && FIRST + PAIRS <= N, "a chunk's pairs are the array's");
    static_assert(2 * PAIRS % kPer == 0 && kPieces <= 8 && (!FRAG || kPieces == 8), "a chunk is whole 16-byte pieces");
    auto turn = [](int r) { return F32 && FRAG ? 2 * (r & 3) : r & 7; };
    __syncwarp();
    if (FRAG) {
#pragma unroll
        for (int q = 0; q < (F32 ? 1 : 2); ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 x = v[FIRST + q * 16 + i * 4 + j];
                    const int r = i * 8 + (lane >> 2);
                    if (F32)
                        *reinterpret_cast<float2*>(out + r * 128 + (((2 * j + ((lane & 3) >> 1)) ^ turn(r)) * 16) +
                                                   (lane & 1) * 8) = x;
                    else
                        *reinterpret_cast<uint32_t*>(out + r * 128 + (((q * 4 + j) ^ turn(r)) * 16) +
                                                     (lane & 3) * 4) = pack_bf16x2_rn(x.x, x.y);
                }
    } else {
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
            uint4 w;
            const int at = FIRST + (F32 ? 2 : 4) * j;
            if constexpr (F32)
                w = make_uint4(__float_as_uint(v[at].x), __float_as_uint(v[at].y), __float_as_uint(v[at + 1].x),
                               __float_as_uint(v[at + 1].y));
            else
                w = make_uint4(pack_bf16x2_rn(v[at].x, v[at].y), pack_bf16x2_rn(v[at + 1].x, v[at + 1].y),
                               pack_bf16x2_rn(v[at + 2].x, v[at + 2].y), pack_bf16x2_rn(v[at + 3].x, v[at + 3].y));
            *reinterpret_cast<uint4*>(out + lane * 128 + ((j ^ turn(lane)) * 16)) = w;
        }
    }
    __syncwarp();
    const int rows = (int)min((int64_t)32, p.limit - row0), cols = min(2 * PAIRS, p.N - col0);
    if (cols <= 0) return;
    if (p.vec) {
        const int j = lane & 7, left = cols - j * kPer;
        if (left <= 0) return;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = i * 4 + (lane >> 3);
            if (r >= rows) break;
            const uint4 w = *reinterpret_cast<const uint4*>(out + r * 128 + ((j ^ turn(r)) * 16));
            const int64_t at = (row0 + r) * p.ldc + col0 + j * kPer;
            if (!F32) {
                store_piece(static_cast<uint16_t*>(p.c) + at, w, left);
                continue;
            }
            float* c = static_cast<float*>(p.c) + at;
            float x[4] = {__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w)};
            if (left >= 4) {
                float4* c4 = reinterpret_cast<float4*>(c);
                if (p.accumulate) {
                    const float4 o = *c4;
                    x[0] += o.x, x[1] += o.y, x[2] += o.z, x[3] += o.w;
                }
                *c4 = make_float4(x[0], x[1], x[2], x[3]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (e < left) c[e] = p.accumulate ? c[e] + x[e] : x[e];
            }
        }
        return;
    }
    // rows off the 16-byte grid: 4 bytes a lane, a row an instruction
    auto word = [&](int r, int l) {
        return *reinterpret_cast<const uint32_t*>(out + r * 128 + (((l >> 2) ^ turn(r)) * 16) + (l & 3) * 4);
    };
    if (F32) {
        float* c = static_cast<float*>(p.c) + row0 * p.ldc + col0 + lane;
        if (lane >= cols) return;
#pragma unroll 8
        for (int r = 0; r < rows; ++r, c += p.ldc)
            *c = p.accumulate ? *c + __uint_as_float(word(r, lane)) : __uint_as_float(word(r, lane));
        return;
    }
    uint16_t* c0 = static_cast<uint16_t*>(p.c) + row0 * p.ldc + col0;
    if (cols < 64) {
        for (int r = 0; r < rows; ++r)
            for (int e = lane; e < cols; e += 32)
                c0[r * p.ldc + e] = (uint16_t)(word(r, e >> 1) >> (16 * (e & 1)));
        return;
    }
    // The even rows, then the odd ones: all of a kind start on a word, or between words, where their words are
    // shifted by one column, and the first and the last column of all 16 rows go by themselves, a lane each (two lanes
    // a row with the row's words: 8192 x 12289 x 4096 386 us).
#pragma unroll 1
    for (int kind = 0; kind < 2; ++kind) {
        const unsigned char *at[4], *up[4];  // of rows kind + 2 k, and every eighth row after
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int r = kind + 2 * k, l = (lane + 1) & 31;
            at[k] = out + r * 128 + (((lane >> 2) ^ r) * 16) + (lane & 3) * 4;
            up[k] = out + r * 128 + (((l >> 2) ^ r) * 16) + (l & 3) * 4;
        }
        uint16_t* c = c0 + kind * p.ldc;
        if ((reinterpret_cast<uintptr_t>(c) & 2) == 0) {
            uint32_t* d = reinterpret_cast<uint32_t*>(c) + lane;
#pragma unroll
            for (int i = 0; i < 16; ++i, d += p.ldc)
                if (kind + 2 * i < rows) *d = *reinterpret_cast<const uint32_t*>(at[i & 3] + (i >> 2) * 1024);
        } else {
            uint16_t* d = c + 2 * lane + 1;
#pragma unroll
            for (int i = 0; i < 16; ++i, d += 2 * p.ldc) {
                const uint32_t w = *reinterpret_cast<const uint32_t*>(at[i & 3] + (i >> 2) * 1024);
                const uint32_t x =
                    __funnelshift_r(w, *reinterpret_cast<const uint32_t*>(up[i & 3] + (i >> 2) * 1024), 16);
                if (lane < 31 && kind + 2 * i < rows) *reinterpret_cast<uint32_t*>(d) = x;
            }
            const int r = kind + 2 * (lane >> 1), side = lane & 1;
            if (r < rows) c0[r * p.ldc + 63 * side] = (uint16_t)(word(r, 31 * side) >> (16 * side));
        }
    }
}

// ----------------------------------------------------------------- 256 x 256 tiles of a CTA pair

constexpr int kGM = 128, kGN = 256;  // a CTA's rows of a tile, and the tile's columns
constexpr int kGStages = 5;
constexpr uint32_t kGA = kGM * kGK, kGB = kGN / 2 * kGK;  // a CTA loads its rows of A and half of B's
constexpr int kGThreads = 384;
constexpr uint32_t kGOut = 32 * 128;  // an epilogue warp's output stage: 32 rows x 128 bytes
// The scales of kGroups K groups at a time, in two slots that warp 2 fills: A's 128 rows', then B's (256 rows', or
// the tile's two blocks').  By the group, their barriers' latencies were in every group's path; copied by each
// epilogue thread for itself they cost 26 us of 335.
constexpr int kGroups = 8, kGSlots = 2;
template <bool BROWS>
constexpr int kGScales = kGM + (BROWS ? kGN : 4);
template <bool BROWS>
constexpr size_t kGSmem = 1024 + (size_t)kGStages * (kGA + kGB) + 8 * kGOut +
                          (size_t)kGSlots * kGroups * kGScales<BROWS> * 4 + 1024;

// A half tile (kHalves): 128 rows of A by 256 of B, of groups of few rows.  The
// MMA takes M = 128, 64 rows of each CTA; a CTA's 128 lanes hold them twice, the
// lower 64 the tile's first 128 columns and the upper 64 the others, in 128
// columns of tensor memory.  So four accumulators are in flight, not two: from
// one's completion to the next it is the hand-overs that take the time, 530
// clocks a group against 870 for a whole tile (with two, 850).
__host__ __device__ constexpr int tile_rows(int k) { return half_kind(k) ? kGM : 2 * kGM; }  // of A, by a pair
__host__ __device__ constexpr int stages_of(int k) { return half_kind(k) ? 6 : kGStages; }
__host__ __device__ constexpr int accs_of(int k) { return half_kind(k) ? 4 : 2; }
template <bool BROWS, int KIND>
constexpr size_t kGSmemOf = kGSmem<BROWS> - (size_t)kGStages * (kGA + kGB) +
                            (size_t)stages_of(KIND) * ((half_kind(KIND) ? kGA / 2 : kGA) + kGB) +
                            (rows_kind(KIND) || KIND == kDepth ? sizeof(GroupTable) : 0);
template <int STAGES, int ACCS>
struct GemmBars {
    PairBars<STAGES, ACCS> pair;
    uint64_t sfull[kGSlots], sempty[kGSlots];
};
static_assert(sizeof(GemmBars<6, 4>) <= 1024, "barriers fit their kilobyte");
static_assert(kGSmemOf<true, kDepth> <= 232448 && kGSmemOf<false, kHalves> <= 232448, "shared memory of a CTA");

constexpr int kGSplit = 4;  // pairs that share a tile at most: a cluster of eight CTAs
constexpr int kTailSaves = 16;  // K groups that a launch of the last tiles has to save a pair
// and with an epilogue, whose code the launch fetches anew: 4096 x 4096 x 4096 66.9 us in one launch, 72.2 in two (24
// groups saved), 4096 x 6144 x 8192 176 and 167 (48)
constexpr int kLayerTailSaves = 32;
constexpr int kRedPitch = kGN + 4;
static_assert((size_t)kGM * kRedPitch * 4 <= (size_t)kGStages * (kGA + kGB), "the partial sums fit the ring");

// Tile t of the persistent order: bands of `band` M tiles, and within a band
// all M tiles of one N tile before the next, so the tiles in flight share a
// few N tiles of B and the band's rows of A, which L2 holds.
__device__ __forceinline__ void tile_of(const Gemm8Params& p, int MB, int t, int& mb, int& nb) {
    const int per = p.band * p.NB, full = MB / p.band;
    const int b = min(t / per, full);
    const int r = t - b * per;
    const int width = b < full ? p.band : MB - full * p.band;
    nb = r / width;
    mb = b * p.band + r % width;
}

struct Tile8 {
    int row0, end;  // the pair's first row of A, and the row behind the last one that is its own
    int nb, group;
    int k0, k1;     // K groups
};
template <int KIND>
__device__ __forceinline__ Tile8 tile_at(const typename ParamsOf<KIND>::type& p, const GroupTable* tab, int t, int k0,
                                         int k1) {
    Tile8 x{0, p.M, 0, 0, k0, k1};
    int mb, MB = p.MB;
    if constexpr (rows_kind(KIND)) {
        x.group = group_of(tab, p.G, t);
        t -= tab->first[x.group];
        x.row0 = tab->begin[x.group], x.end = tab->begin[x.group + 1];
        MB = (x.end - x.row0 + tile_rows(KIND) - 1) / tile_rows(KIND);
        if (x.group == p.G) x.k1 = k0;  // rows behind the groups: an empty sum
    }
    if constexpr (KIND == kDepth) {
        x.group = t / (p.MB * p.NB);
        t -= x.group * p.MB * p.NB;
        x.k0 = tab->first[x.group], x.k1 = tab->first[x.group + 1];
    }
    tile_of(p, MB, t, mb, x.nb);
    x.row0 += mb * tile_rows(KIND);
    return x;
}

// 64 columns of the residual from `col` on, added to the pairs [FIRST, FIRST + 32) of the lane's row v, through
// shared memory as store_chunk's output; eight loads under way at a time (one by
// one a tile's took 19,500 clocks), sixteen of FP32 rows off the 16-byte grid
// (1000 x 5003 x 2000: 50.6 us by eight, 44.0; thirty-two gain nothing and cost
// the loop registers).
template <bool F32, int FIRST, int N>
__device__ __forceinline__ void add_residual(const Ext8Params& p, unsigned char* out, int lane, int64_t row0,
                                             int64_t limit, int col, float2 (&v)[N]) {
    static_assert(FIRST >= 0 && FIRST + 32 <= N, "a chunk's pairs are the array's");
    constexpr int kPer = F32 ? 4 : 8, kCols = F32 ? 32 : 64;
    const int rows = (int)min((int64_t)32, limit - row0);
#pragma unroll
    for (int half = 0; half < (F32 ? 2 : 1); ++half) {
        const int at = col + half * 32, cols = min(kCols, p.N - at);
        __syncwarp();
        if (p.res_vec) {
            const int j = lane & 7, left = cols - j * kPer;
            const char* src = static_cast<const char*>(p.res) +
                              ((row0 + (lane >> 3)) * p.ldr + at + j * kPer) * (16 / kPer);
            const int64_t four = 4 * p.ldr * (16 / kPer);
            uint4 x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] = make_uint4(0, 0, 0, 0);
                if (i * 4 + (lane >> 3) < rows && left >= kPer) x[i] = __ldcs(reinterpret_cast<const uint4*>(src + i * four));
            }
            if (left > 0 && left < kPer) {  // the last columns of an N between pieces
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint32_t w[4] = {};
#pragma unroll
                    for (int e = 0; e < kPer; ++e)
                        if (i * 4 + (lane >> 3) < rows && e < left) {
                            if (F32)
                                w[e] = reinterpret_cast<const uint32_t*>(src + i * four)[e];
                            else
                                w[e >> 1] |= (uint32_t) reinterpret_cast<const uint16_t*>(src + i * four)[e] << (16 * (e & 1));
                        }
                    x[i] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = i * 4 + (lane >> 3);
                *reinterpret_cast<uint4*>(out + r * 128 + ((j ^ (r & 7)) * 16)) = x[i];
            }
        } else if (F32) {
            const uint32_t* src = static_cast<const uint32_t*>(p.res) + row0 * p.ldr + at + lane;
#pragma unroll
            for (int b = 0; b < 32; b += 16) {
                uint32_t x[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = b + i < rows && lane < cols ? __ldcs(src + (b + i) * p.ldr) : 0u;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    *reinterpret_cast<uint32_t*>(out + (b + i) * 128 + (((lane >> 2) ^ (i & 7)) * 16) + (lane & 3) * 4) = x[i];
            }
        } else {
            const uint16_t* src = static_cast<const uint16_t*>(p.res) + row0 * p.ldr + at + 2 * lane;
#pragma unroll
            for (int b = 0; b < 32; b += 8) {
                uint32_t x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[i] = 0u;
                    if (b + i < rows) {
                        if (2 * lane < cols) x[i] = src[(b + i) * p.ldr];
                        if (2 * lane + 1 < cols) x[i] |= (uint32_t)src[(b + i) * p.ldr + 1] << 16;
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<uint32_t*>(out + (b + i) * 128 + (((lane >> 2) ^ i) * 16) + (lane & 3) * 4) = x[i];
            }
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint4 x = *reinterpret_cast<const uint4*>(out + lane * 128 + ((k ^ (lane & 7)) * 16));
            if (F32) {
                const int at = FIRST + half * 16 + 2 * k;
                v[at] = fadd2(v[at], make_float2(__uint_as_float(x.x), __uint_as_float(x.y)));
                v[at + 1] = fadd2(v[at + 1], make_float2(__uint_as_float(x.z), __uint_as_float(x.w)));
            } else {
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[FIRST + 4 * k + e] =
                        fadd2(v[FIRST + 4 * k + e], make_float2(bf16lo_to_f32(w[e]), bf16hi_to_f32(w[e])));
            }
        }
    }
}

__device__ __forceinline__ float bias_at(const Ext8Params& p, int64_t i) {
    return p.bias_f32 ? static_cast<const float*>(p.bias)[i]
                      : __uint_as_float((uint32_t) static_cast<const uint16_t*>(p.bias)[i] << 16);
}
__device__ __forceinline__ float res_at(const Ext8Params& p, int64_t i) {
    return p.res_f32 ? static_cast<const float*>(p.res)[i]
                     : __uint_as_float((uint32_t) static_cast<const uint16_t*>(p.res)[i] << 16);
}

// The sums of a warp's columns start from their biases, which every lane reads
// (one address a warp), or where they lie off the 16-byte grid or end inside the
// tile through shared memory: 8192 x 12288 x 4096, 330 us without, FP32 340 read
// and 350 through shared memory, BF16 348 either way.  (Fetching them before the
// tile before was finished gained nothing, and registers of the gated product's
// loop suffered: 331 -> 348 us.)
// PAIRS: of columns a warp has, 64 or (of a half tile) 32; gated, half of them
// the gate's.  col: the first of the result's; zcol: of B's rows, so of z's.
template <int KIND, int PAIRS>
__device__ __forceinline__ void start_with_bias(const Ext8Params& p, unsigned char* out, int lane, const Tile8& t,
                                                int col, float2 (&sum)[PAIRS]) {
    constexpr bool GATED = gated_kind(KIND);
    if (rows_kind(KIND) && p.rest && t.group == p.G) return;  // rows behind the groups: zeros
    constexpr int kEach = PAIRS / 16, kOf = GATED ? 16 : 32;  // columns a lane, lanes of a half
    const int half = lane / kOf, c = col + kEach * (lane % kOf);
    const int64_t group = (int64_t)t.group * (GATED ? 2 : 1) * p.N, at = group + (half ? p.N : 0) + c;
    if (p.bias_vec && col + (GATED ? PAIRS : 2 * PAIRS) <= p.N) {
        // every lane reads all of them, one address a warp
#pragma unroll
        for (int h = 0; h < (GATED ? 2 : 1); ++h) {
            constexpr int kOwn = GATED ? PAIRS / 2 : PAIRS;
            const int64_t from = group + (h ? p.N : 0) + col;
            if (p.bias_f32) {
                const float4* b = reinterpret_cast<const float4*>(static_cast<const float*>(p.bias) + from);
#pragma unroll
                for (int i = 0; i < kOwn / 2; ++i) {
                    const float4 x = __ldg(b + i);
                    sum[kOwn * h + 2 * i] = make_float2(x.x, x.y), sum[kOwn * h + 2 * i + 1] = make_float2(x.z, x.w);
                }
            } else {
                const uint4* b = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.bias) + from);
#pragma unroll
                for (int i = 0; i < kOwn / 4; ++i) {
                    const uint4 x = __ldg(b + i);
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sum[kOwn * h + 4 * i + e] = make_float2(bf16lo_to_f32(w[e]), bf16hi_to_f32(w[e]));
                }
            }
        }
        return;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kEach; ++i)
        reinterpret_cast<float*>(out)[kEach * lane + i] = c + i < p.N ? bias_at(p, at + i) : 0.f;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < PAIRS / 2; ++i) {
        const float4 x = reinterpret_cast<const float4*>(out)[i];
        sum[2 * i] = make_float2(x.x, x.y), sum[2 * i + 1] = make_float2(x.z, x.w);
    }
    __syncwarp();
}

// The pairs [FIRST, FIRST + PAIRS) of a warp's results, which start at column `col` of c: the residual, and to memory.
template <int KIND, int FIRST, int PAIRS, int N>
__device__ __forceinline__ void finish_run(const Ext8Params& p, unsigned char* out, int lane, const Tile8& t, int col,
                                           int64_t row0, float2 (&sum)[N]) {
    const Dest d{p.c, p.ldc, t.end, p.N, p.vec, 0};
    if constexpr (!rows_kind(KIND))  // rows of groups have no residual
        if (p.res) {
            if (p.res_f32)
                add_residual<true, FIRST>(p, out, lane, row0, t.end, col, sum);
            else
                add_residual<false, FIRST>(p, out, lane, row0, t.end, col, sum);
        }
    if (p.c_f32) {
        store_chunk<true, false, FIRST>(d, out, lane, row0, col, sum);
        if constexpr (PAIRS == 32) store_chunk<true, false, FIRST + 16>(d, out, lane, row0, col + 32, sum);
    } else {
        store_chunk<false, false, FIRST, PAIRS>(d, out, lane, row0, col, sum);
    }
}

// The epilogue of a warp's 32 rows and their PAIRS pairs of columns, a row a
// lane; gated: the first half of them is the gate's and the second the other
// half's same columns, which the loads of B have laid side by side.
template <int KIND, int PAIRS>
__device__ __forceinline__ void finish_rows(const Ext8Params& p, unsigned char* out, int lane, const Tile8& t, int col0,
                                            int64_t row0, float2 (&sum)[PAIRS]) {
    constexpr bool GATED = gated_kind(KIND);
    const bool behind = rows_kind(KIND) && p.rest && t.group == p.G;  // rows behind the groups: zeros
    constexpr int kOwn = GATED ? PAIRS / 2 : PAIRS, kAt = kOwn < 32 ? kOwn : 32;  // pairs of a half, and at a time
    static_assert(PAIRS == kAt || PAIRS == 2 * kAt, "one run or two");
    if (p.z && !behind) {
        const Dest d{p.z, p.ldz, t.end, p.N, p.z_vec, 0};
        store_chunk<false, false, 0, kAt>(d, out, lane, row0, col0, sum);
        if constexpr (GATED)
            store_chunk<false, false, kAt, kAt>(Dest{p.z + p.N, p.ldz, t.end, p.N, p.z_vec, 0}, out, lane, row0, col0, sum);
        else if constexpr (PAIRS > kAt)
            store_chunk<false, false, kAt, kAt>(d, out, lane, row0, col0 + 2 * kAt, sum);
    }
    act_pairs<0, kOwn>(sum, p.act);
    if (GATED) {
#pragma unroll
        for (int i = 0; i < kOwn; ++i) sum[i] = fmul2(sum[i], sum[kOwn + i]);
    }
    finish_run<KIND, 0, kAt>(p, out, lane, t, col0, row0, sum);
    if constexpr (kOwn > kAt) finish_run<KIND, kAt, kAt>(p, out, lane, t, col0 + 2 * kAt, row0, sum);
}

// Tiles tile0 .. tiles - 1.  split: pairs of a cluster that share a tile, each
// with a part of the K groups (1: the pair's tiles are its own, one after the
// other).  A launch with tile0 > 0 runs behind the one with the tiles before,
// whose inputs are its own and whose outputs are not: it may start as that
// one's pairs end.
template <bool BROWS, int KIND>
__global__ void __launch_bounds__(kGThreads, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                const __grid_constant__ typename ParamsOf<KIND>::type p, const int tile0, const int tiles_given,
                const int split_given) {
    constexpr bool kGrouped = rows_kind(KIND) || KIND == kDepth, kLayer = layer_kind(KIND), kGated = gated_kind(KIND);
    constexpr bool kHalf = half_kind(KIND);
    constexpr int kStages = stages_of(KIND), kAccs = accs_of(KIND), kAcc = 512 / kAccs;  // columns of an accumulator
    constexpr int kOwn = tile_rows(KIND) / 2, kPairs = kHalf ? 32 : 64;  // a CTA's rows of A, a thread's pairs of sums
    constexpr uint32_t kA = kOwn * kGK;
    static_assert(!BROWS || !kLayer, "an epilogue's B has scales by the block");
    const int split = kGrouped ? 1 : split_given;
    extern __shared__ unsigned char smem_raw[];
    // The same offset in both CTAs (their dynamic shared memory starts alike): descriptors name one offset.
    unsigned char* smem =
        reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    unsigned char* sA = smem;
    unsigned char* sB = smem + kStages * kA;
    unsigned char* sOut = sB + kStages * kGB;
    float* scales = reinterpret_cast<float*>(sOut + 8 * kGOut);
    auto* all = reinterpret_cast<GemmBars<kStages, kAccs>*>(scales + kGSlots * kGroups * kGScales<BROWS>);
    PairBars<kStages, kAccs>* bars = &all->pair;
    const int warp = warp_index(), lane = threadIdx.x & 31;
    const int place = (int)cluster_ctarank(), rank = place & 1, leader = place & ~1;
    const uint16_t both = (uint16_t)(3 << leader);
    auto* tab = reinterpret_cast<GroupTable*>(reinterpret_cast<unsigned char*>(all) + 1024);
    const int first = tile0 + (int)blockIdx.x / (2 * split), step = (int)gridDim.x / (2 * split);
    const int k0 = (int)((int64_t)p.KB * (leader / 2) / split), k1 = (int)((int64_t)p.KB * (leader / 2 + 1) / split);

    if (threadIdx.x == 0) {
        for (int i = 0; i < kGSlots; ++i) {
            mbar_init(smem_u32(&all->sfull[i]), 32);
            mbar_init(smem_u32(&all->sempty[i]), 8);
        }
    }
    if constexpr (rows_kind(KIND)) groups_build<kGThreads>(tab, p.ends, p.G, p.M, tile_rows(KIND), p.NB, p.rest);
    if constexpr (KIND == kDepth) groups_build<kGThreads>(tab, p.ends, p.G, p.deep, kGK, 1, false);
    const uint32_t tmem = pair_begin(bars, warp, 8);
    int* ab = &bars->abort_flag;
    grid_launch_dependents();  // the launch of the last tiles
    int tiles = tiles_given;
    if constexpr (rows_kind(KIND)) tiles = tab->first[p.G + 1];
    auto tile = [&](int t) { return tile_at<KIND>(p, tab, t, k0, k1); };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 0) {
            // ------------------------------------------------ TMA producer: counted on the even CTA's barriers
            const bool one = elect_one();
            const uint32_t full0 = mapa_shared(smem_u32(&bars->full[0]), (uint32_t)leader);
            Ring r;
            uint64_t issued = 0;
            bool ok = true;
            for (int t = first; ok && t < tiles; t += step) {
                const Tile8 x = tile(t);
                const int a_row = x.row0 + rank * kOwn, b_row = x.nb * kGN + rank * (kGN / 2);
                // a CTA without a row of its own loads none: its rows of the accumulator are not used
                const bool mine = a_row < x.end;
                for (int kb = x.k0; kb < x.k1; ++kb) {
                    if (!(ok = pipe_wait_warp(ab, smem_u32(&bars->empty[r.slot]), r.phase ^ 1u, p.w))) break;
                    if (one) {
                        const uint32_t fb = full0 + r.slot * 8;
                        pair_arm(fb, smem_u32(&bars->full[r.slot]), rank, kGB + (mine ? kA : 0));
                        if (mine) tma_load_2d_pair(smem_u32(sA + r.slot * kA), &tmA, kb * kGK, a_row, fb);
                        if constexpr (kLayer)  // gated: half as many rows of each half
                            tma_load_4d_pair(smem_u32(sB + r.slot * kGB), &tmB, kb * kGK, kGated ? b_row / 2 : b_row,
                                             0, x.group, fb);
                        else
                            tma_load_2d_pair(smem_u32(sB + r.slot * kGB), &tmB, kb * kGK, b_row, fb);
                    }
                    ++issued;
                    r.next(kStages);
                }
            }
            pair_end_copies(bars, r, one, issued, ok, p.w);
        } else if (warp == 1 && rank == 0) {
            // ------------------------------------------------ MMA issuer of the pair
            const bool one = elect_one();
            const uint64_t da = smem_desc_sw128(smem_u32(sA)), db = smem_desc_sw128(smem_u32(sB));
            const uint32_t idesc = idesc_e4m3_f32(tile_rows(KIND), kGN);
            Ring r, acc;
            bool ok = true;
            for (int t = first; ok && t < tiles; t += step) {
                const Tile8 x = tile(t);
                for (int kb = x.k0; kb < x.k1; ++kb) {
                    // the operands first: theirs are ready early, so only the accumulator's wait is in its way
                    if (!(ok = pipe_wait_warp(ab, smem_u32(&bars->full[r.slot]), r.phase, p.w))) break;
                    if (!(ok = pipe_wait_warp(ab, smem_u32(&bars->tempty[acc.slot]), acc.phase ^ 1u, p.w))) break;
                    tc_fence_after();
                    if (one) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_e4m3_pair(tmem + (uint32_t)(acc.slot * kAcc), da + ((r.slot * kA + kk * 32) >> 4),
                                           db + ((r.slot * kGB + kk * 32) >> 4), idesc, kk != 0);
                        umma_commit_pair(smem_u32(&bars->tfull[acc.slot]), both);
                        umma_commit_pair(smem_u32(&bars->empty[r.slot]), both);
                    }
                    __syncwarp();
                    r.next(kStages);
                    acc.next(kAccs);
                }
            }
            pair_end_mmas(bars, acc, one, ok, p.w, both);
        } else if (warp == 2) {
            // ------------------------------------------------ scales
            Ring r;
            bool ok = true;
            for (int t = first; ok && t < tiles; t += step) {
                const Tile8 x = tile(t);
                const int row = x.row0 + rank * kOwn + lane, col = x.nb * kGN + lane;
                for (int kg = x.k0; kg < x.k1; kg += kGroups) {
                    ok = pipe_wait_warp(ab, smem_u32(&all->sempty[r.slot]), r.phase ^ 1u, p.w);
                    if (!ok) break;
                    if constexpr (kLayer && !rows_kind(KIND)) {
                        // the tile's residual comes into L2 meanwhile (by the tile: all tiles' at once drove the
                        // operands out)
                        if (p.res && kg == x.k0 && split == 1) {
                            const int cols = kGated ? kGN / 2 : kGN, at = x.nb * cols, size = p.res_f32 ? 4 : 2;
                            const int top = x.row0 + rank * kOwn, pieces = (min(cols, p.N - at) * size + 127) / 128;
                            const char* src = static_cast<const char*>(p.res) + ((int64_t)top * p.ldr + at) * size;
                            for (int i = lane; i < min(kOwn, x.end - top) * pieces; i += 32)
                                prefetch_l2(src + i / pieces * p.ldr * size + i % pieces * 128);
                        }
                    }
                    uint32_t dst = smem_u32(scales + r.slot * kGroups * kGScales<BROWS>) + lane * 4;
                    const float *a = p.sa + (int64_t)kg * p.M, *b = p.sb + (int64_t)kg * p.nsb;
                    if constexpr (rows_kind(KIND)) b += x.group * p.sb_g;
                    for (int kb = kg; kb < min(kg + kGroups, x.k1); ++kb) {
#pragma unroll
                        for (int i = 0; i < kOwn; i += 32)
                            cp_async4(dst + i * 4, a + (row + i < p.M ? row + i : 0), row + i < p.M);
                        if (BROWS) {
#pragma unroll
                            for (int i = 0; i < kGN; i += 32)
                                cp_async4(dst + (kGM + i) * 4, b + (col + i < p.N ? col + i : 0), col + i < p.N);
                        } else if constexpr (kGated) {
                            // of each half of the columns, of both halves of B
                            if (lane < 4) {
                                const int blk = ((lane >> 1) * p.N + x.nb * 128 + (lane & 1) * 64) >> 7;
                                cp_async4(dst + kGM * 4, b + (blk < p.nsb ? blk : 0), blk < p.nsb);
                            }
                        } else if (lane < 2) {
                            const int blk = x.nb * 2 + lane;
                            cp_async4(dst + kGM * 4, b + (blk < p.nsb ? blk : 0), blk < p.nsb);
                        }
                        dst += kGScales<BROWS> * 4;
                        a += p.M;
                        b += p.nsb;
                    }
                    cp_async_arrive(smem_u32(&all->sfull[r.slot]));
                    r.next(kGSlots);
                }
            }
            cp_async_wait_all();
        }
        __syncwarp();
    } else {
        // ------------------------------------------------ epilogue: scale and sum in registers
        asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        const int quarter = warp & 3, part = (warp - 4) >> 2;  // 32 rows, and 128 of the tile's columns
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
        // this warp's 32 of the CTA's rows, its 128 of the tile's columns, and (half) which 64 of those
        const int rows32 = kHalf ? quarter & 1 : quarter, side = kHalf ? quarter >> 1 : part;
        unsigned char* out = sOut + (warp - 4) * kGOut;
        const uint32_t done = mapa_shared(smem_u32(&bars->tempty[0]), (uint32_t)leader);
        Ring acc, sc;
        bool ok = first < tiles, ready = false;
        auto first_column = [&](const Tile8& x) {  // of the result, of this warp's
            return x.nb * (kGated ? kGN / 2 : kGN) + side * (kGated ? 64 : 128) + (kHalf ? part * (kGated ? 32 : 64) : 0);
        };
        for (int t = first; ok && t < tiles; t += step) {
            float2 sum[kPairs];
#pragma unroll
            for (int i = 0; i < kPairs; ++i) sum[i] = make_float2(0.f, 0.f);
            if constexpr (kLayer)
                if (p.bias && split == 1) start_with_bias<KIND, kPairs>(p, out, lane, tile(t), first_column(tile(t)), sum);
            const float* s = nullptr;
            const Tile8 x = tile(t);
            for (int kb = x.k0; kb < x.k1; ++kb) {
                if ((kb - x.k0) % kGroups == 0) {
                    ok = pipe_wait(ab, smem_u32(&all->sfull[sc.slot]), sc.phase, p.w);
                    s = scales + sc.slot * kGroups * kGScales<BROWS>;
                }
                // of this thread's row, times the block's; or of its fragments' four rows
                float f[4];
                if (BROWS) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) f[i] = s[quarter * 32 + i * 8 + (lane >> 2)];
                } else {
                    f[0] = __fmul_rn(s[rows32 * 32 + lane], s[kGM + side]);
                    f[1] = kGated ? __fmul_rn(s[rows32 * 32 + lane], s[kGM + 2 + side]) : f[0];
                }
                if (!ready) ok = ok && pipe_wait(ab, smem_u32(&bars->tfull[acc.slot]), acc.phase, p.w);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                tc_fence_after();
                // 32 columns at a time, the next 32 under way while these are summed
                // half: 64 of the lanes' 128 columns, or (gated) 32 of the gate's 64 and the same of the other half's
                constexpr int kChunks = kPairs / 16, kApart = kHalf && kGated ? 64 : 32;
                const uint32_t t0 = tmem + lane_base + (uint32_t)(acc.slot * kAcc + part * (kHalf ? kGated ? 32 : 64 : 128));
                uint32_t v[2][32];
                BROWS ? tmem_ld_frag_issue(t0, v[0]) : tmem_ld32_issue(t0, v[0]);
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    tmem_wait32(v[c & 1]);
                    if (c < kChunks - 1) {
                        BROWS ? tmem_ld_frag_issue(t0 + (c + 1) * kApart, v[(c + 1) & 1])
                              : tmem_ld32_issue(t0 + (c + 1) * kApart, v[(c + 1) & 1]);
                    } else {
                        // the accumulator is free again; ask for the next one before this one's last sums
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_remote(done + acc.slot * 8);
                        acc.next(kAccs);
                        ready = mbar_test_wait(smem_u32(&bars->tfull[acc.slot]), acc.phase);  // must not suspend
                    }
                    if (BROWS) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 sb =
                                *reinterpret_cast<const float2*>(s + kGM + part * 128 + c * 32 + j * 8 + 2 * (lane & 3));
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int at = (i >> 1) * 16 + j * 4 + (i & 1) * 2;
                                sum[c * 16 + i * 4 + j] = ffma2(make_float2(__uint_as_float(v[c & 1][at]),
                                                                            __uint_as_float(v[c & 1][at + 1])),
                                                                fmul2(make_float2(f[i], f[i]), sb),
                                                                sum[c * 16 + i * 4 + j]);
                            }
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            sum[c * 16 + i] = ffma2(make_float2(__uint_as_float(v[c & 1][2 * i]),
                                                                __uint_as_float(v[c & 1][2 * i + 1])),
                                                    make_float2(f[2 * c / kChunks], f[2 * c / kChunks]), sum[c * 16 + i]);
                    }
                }
                s += kGScales<BROWS>;
                if ((kb - x.k0) % kGroups == kGroups - 1 || kb == x.k1 - 1) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&all->sempty[sc.slot]));
                    sc.next(kGSlots);
                }
            }
            if (!ok) break;
            if constexpr (!kHalf) if (split > 1) {
                // every load has been consumed, so the ring's memory takes the partial sums [128][256], a row's
                // pitch 260 for the banks
                float* red = reinterpret_cast<float*>(sA) + (quarter * 32) * kRedPitch + part * 128;
                if (BROWS) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                *reinterpret_cast<float2*>(red + (i * 8 + (lane >> 2)) * kRedPitch + c * 32 + j * 8 +
                                                           2 * (lane & 3)) = sum[c * 16 + i * 4 + j];
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        *reinterpret_cast<float4*>(red + lane * kRedPitch + 4 * i) =
                            make_float4(sum[2 * i].x, sum[2 * i].y, sum[2 * i + 1].x, sum[2 * i + 1].y);
                }
                break;
            }
            const int64_t row0 = (int64_t)x.row0 + rank * kOwn + rows32 * 32;
            if constexpr (kLayer) {
                if (row0 < x.end) finish_rows<KIND, kPairs>(p, out, lane, x, first_column(x), row0, sum);
            } else {
                const int col0 = x.nb * kGN + part * 128;
                Dest d = dest_of(p, p.M);
                if constexpr (KIND == kDepth)
                    d.c = static_cast<char*>(d.c) + x.group * p.c_g * (p.c_f32 ? 4 : 2);
                if (p.c_f32)
                    each<kPairs / 16>([&](auto q) {
                        store_chunk<true, BROWS, 16 * q.value>(d, out, lane, row0, col0 + 32 * q.value, sum);
                    });
                else
                    each<kPairs / 32>([&](auto q) {
                        store_chunk<false, BROWS, 32 * q.value>(d, out, lane, row0, col0 + 64 * q.value, sum);
                    });
            }
        }
    }
    if constexpr (!kHalf) if (split > 1) {
        // This CTA adds up its share of the rows, the pairs' sums in order.
        cluster_sync_all();
        const bool failed = *reinterpret_cast<volatile int*>(ab) != 0;
        const Tile8 tl = tile(first);
        const int lo = kGM * (leader / 2) / split, hi = kGM * (leader / 2 + 1) / split;
        auto joined = [&](int r, int c, float (&x)[4]) {
            const uint32_t at = smem_u32(reinterpret_cast<float*>(sA) + r * kRedPitch + c);
            float4 v[kGSplit];  // all under way before the first is added
#pragma unroll
            for (int s = 0; s < kGSplit; ++s)
                v[s] = s < split ? ld_cluster_f32x4(mapa_shared(at, (uint32_t)(2 * s + rank)))
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
            x[0] = v[0].x, x[1] = v[0].y, x[2] = v[0].z, x[3] = v[0].w;
#pragma unroll
            for (int s = 1; s < kGSplit; ++s) {
                x[0] = __fadd_rn(x[0], v[s].x), x[1] = __fadd_rn(x[1], v[s].y);
                x[2] = __fadd_rn(x[2], v[s].z), x[3] = __fadd_rn(x[3], v[s].w);
            }
        };
        int quads = kGN / 4;  // of the result's columns, four each
        if constexpr (kGated) quads = kGN / 8;
#pragma unroll 2
        for (int e = threadIdx.x; e < (hi - lo) * quads && !failed; e += kGThreads) {
            const int r = lo + e / quads, c = e % quads * 4;
            const int64_t row = (int64_t)tl.row0 + rank * kGM + r;
            const int col = tl.nb * 4 * quads + c;
            if (row >= p.M || col >= p.N) continue;
            float x[4];
            if constexpr (kLayer) {
                float u[4] = {};
                // gated: 64 columns of the gate, then the same of the other half, for each half of the tile
                const int in = kGated ? (c & 64) * 2 + (c & 63) : c;
                joined(r, in, x);
                if (kGated) joined(r, in + 64, u);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (col + i < p.N) {
                        if (p.bias) {
                            x[i] = __fadd_rn(x[i], bias_at(p, col + i));
                            if (kGated) u[i] = __fadd_rn(u[i], bias_at(p, (int64_t)p.N + col + i));
                        }
                        if (p.z) {
                            uint16_t* z = p.z + row * p.ldz + col + i;
                            z[0] = (uint16_t)pack_bf16x2_rn(x[i], 0.f);
                            if (kGated) z[p.N] = (uint16_t)pack_bf16x2_rn(u[i], 0.f);
                        }
                        x[i] = act_one(x[i], p.act);
                        if (kGated) x[i] = __fmul_rn(x[i], u[i]);
                        if (p.res) x[i] = __fadd_rn(x[i], res_at(p, row * p.ldr + col + i));
                    }
            } else {
                joined(r, c, x);
            }
            if (p.c_f32) {
                float* d = static_cast<float*>(p.c) + row * p.ldc + col;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (col + i < p.N) d[i] = p.accumulate ? d[i] + x[i] : x[i];
            } else {
                uint16_t* d = static_cast<uint16_t*>(p.c) + row * p.ldc + col;
                const uint2 w = make_uint2(pack_bf16x2_rn(x[0], x[1]), pack_bf16x2_rn(x[2], x[3]));
                if (p.vec && col + 4 <= p.N) {
                    *reinterpret_cast<uint2*>(d) = w;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (col + i < p.N) d[i] = (uint16_t)((i < 2 ? w.x : w.y) >> (16 * (i & 1)));
                }
            }
        }
    }
    if (tile0 > 0) grid_wait_prior();  // what follows in the stream follows both launches
    pair_end(bars, tmem, warp, p.w);
}

// ----------------------------------------------------------------- few rows of A

constexpr int kSThreads = 256;
constexpr int kSRows = 128;  // rows of B a tile

template <int NT>
struct Skinny {
    static constexpr int kPerSm = 2;
    static constexpr int kStages = NT <= 16 ? 5 : 4;
    static constexpr uint32_t kW = kSRows * kGK, kX = NT * kGK;
    static constexpr uint32_t kTmem = 2 * NT < 32 ? 32 : 2 * NT;
    static constexpr int kScale = NT + kSRows;
    static constexpr size_t kRing = (size_t)kStages * (kW + kX);
    static constexpr size_t kReduce = (size_t)NT * kSRows * 4;  // partial sums of a K slice, over the drained ring
    static constexpr size_t kSmem = 1024 + kRing + kScaleStages * kScale * 4 + 1024;
    static_assert(kReduce <= kRing, "the partial sums fit the ring");
};

template <int NT, int KIND>
constexpr size_t kSSmemOf = Skinny<NT>::kSmem + (rows_kind(KIND) ? sizeof(GroupTable) : 0);
// the largest that are launched: 64 rows of one product, 32 of groups
static_assert(2 * (kSSmemOf<64, kEpi> + 1024) <= 233472 && 2 * (kSSmemOf<32, kRows> + 1024) <= 233472, "two CTAs an SM");

// A unit: 128 rows of B (gated: 64 of each half, 16 and 16 by turns, so that a
// warp's lanes l and l + 16 hold a column's gate and its other half) against
// all rows of A, or NT rows of a group.
struct Unit8 {
    int row0, rows;  // of A
    int nb, group;
    int k0, k1;
};
template <int NT, int KIND>
__device__ __forceinline__ Unit8 unit_at(const typename ParamsOf<KIND>::type& p, const GroupTable* tab, int t, int k0,
                                         int k1) {
    if constexpr (rows_kind(KIND)) {
        // the blocks of rows that share 128 rows of B come one after the other
        const int e = group_of(tab, p.G, t), begin = tab->begin[e], n = tab->begin[e + 1] - begin;
        const int blocks = (n + NT - 1) / NT, at = t - tab->first[e], j = at % blocks;
        return Unit8{begin + j * NT, min(n - j * NT, NT), at / blocks, e, k0, e == p.G ? k0 : k1};
    }
    return Unit8{0, p.M, t, 0, k0, k1};
}

// One result of K split over a cluster: z and its other half u (gated) of `row` and `col`.
template <int KIND>
__device__ __forceinline__ void finish_one(const Ext8Params& p, int64_t row, int col, float z, float u) {
    float y = act_one(z, p.act);
    if (gated_kind(KIND)) y = __fmul_rn(y, u);
    if (!rows_kind(KIND) && p.res) y = __fadd_rn(y, res_at(p, row * p.ldr + col));
    if (p.c_f32)
        static_cast<float*>(p.c)[row * p.ldc + col] = y;
    else
        static_cast<uint16_t*>(p.c)[row * p.ldc + col] = (uint16_t)pack_bf16x2_rn(y, 0.f);
}

// The epilogue of few rows: a lane has a row of B against up to NT rows of A.
// Gated: lanes l and l + 16 have a column's gate and its other half, and after
// one exchange the first finishes the even rows and the second the odd ones.
// Sixteen rows at a time, which bounds the registers.
template <int NT, int KIND>
__device__ __forceinline__ void finish_lanes(const Ext8Params& p, const Unit8& x, int quarter, int lane,
                                             const float2 (&sum)[NT / 2]) {
    constexpr bool GATED = gated_kind(KIND);
    const bool behind = rows_kind(KIND) && p.rest && x.group == p.G;  // rows behind the groups: zeros
    const int half = GATED ? lane >> 4 : 0;
    const int col = GATED ? x.nb * 64 + quarter * 16 + (lane & 15) : x.nb * 128 + quarter * 32 + lane;
    const bool in = col < p.N;
    const int64_t zc = col + (half ? (int64_t)p.N : 0);  // its row of the group's B
    float b = 0.f;
    if (p.bias && in && !behind) b = bias_at(p, (int64_t)x.group * (GATED ? 2 : 1) * p.N + zc);
    constexpr int kStep = GATED ? 2 : 1, kPairs = 8 / kStep;  // value i of a lane is row kStep i + half of the sixteen
#pragma unroll
    for (int r0 = 0; r0 < NT; r0 += 16) {
        if (r0 >= x.rows) break;
        float2 v[8], u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = fadd2(sum[r0 / 2 + i], make_float2(b, b));
        if (p.z && in && !behind) {
            uint16_t* z = p.z + (int64_t)(x.row0 + r0) * p.ldz + zc;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (r0 + i < x.rows) z[i * p.ldz] = (uint16_t)pack_bf16x2_rn(i & 1 ? v[i >> 1].y : v[i >> 1].x, 0.f);
        }
        if (GATED) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float g[2], o[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 w = v[2 * i + e];
                    const float got = __shfl_xor_sync(0xFFFFFFFFu, half ? w.x : w.y, 16);
                    g[e] = half ? got : w.x, o[e] = half ? w.y : got;
                }
                v[i] = make_float2(g[0], g[1]), u[i] = make_float2(o[0], o[1]);
            }
        }
        act_pairs<0, kPairs, true>(v, p.act);  // of different rows
        if (GATED) {
#pragma unroll
            for (int i = 0; i < kPairs; ++i) v[i] = fmul2(v[i], u[i]);
        }
        const int64_t row = (int64_t)x.row0 + r0 + half;
        const int left = in ? x.rows - r0 - half : 0;
        if constexpr (!rows_kind(KIND))  // rows of groups have no residual
            if (p.res) {
                float r[2 * kPairs];
#pragma unroll
                for (int i = 0; i < 2 * kPairs; ++i)
                    r[i] = kStep * i < left ? res_at(p, (row + kStep * i) * p.ldr + col) : 0.f;
#pragma unroll
                for (int i = 0; i < kPairs; ++i) v[i] = fadd2(v[i], make_float2(r[2 * i], r[2 * i + 1]));
            }
        if (p.c_f32) {
            float* c = static_cast<float*>(p.c) + row * p.ldc + col;
#pragma unroll
            for (int i = 0; i < 2 * kPairs; ++i)
                if (kStep * i < left) c[kStep * i * p.ldc] = i & 1 ? v[i >> 1].y : v[i >> 1].x;
        } else {
            uint16_t* c = static_cast<uint16_t*>(p.c) + row * p.ldc + col;
#pragma unroll
            for (int i = 0; i < 2 * kPairs; ++i)
                if (kStep * i < left)
                    c[kStep * i * p.ldc] = (uint16_t)pack_bf16x2_rn(i & 1 ? v[i >> 1].y : v[i >> 1].x, 0.f);
        }
    }
}

template <int NT, bool BROWS, int KIND>
__global__ void __launch_bounds__(kSThreads, Skinny<NT>::kPerSm)
    skinny_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                  const __grid_constant__ typename ParamsOf<KIND>::type p, const int split) {
    using S = Skinny<NT>;
    constexpr bool kExt = KIND != kPlain, kGated = gated_kind(KIND);
    static_assert(!BROWS || !kExt, "an epilogue's B has scales by the block");
    // A layer's accumulators are four: with fewer CTAs than the device holds, the hand-overs of two are what a CTA waits
    // for (37 x 4096 to 2 x 12288 gated: 28.4 us with two, 25.7 with four).
    constexpr int kAccs = kExt ? 4 : 2;
    constexpr uint32_t kTmem = kExt ? (uint32_t)kAccs * NT : S::kTmem;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem =
        reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    unsigned char* sW = smem;
    unsigned char* sX = smem + S::kStages * S::kW;
    float* scales = reinterpret_cast<float*>(sX + S::kStages * S::kX);
    auto* bars = reinterpret_cast<Bars8<S::kStages, kAccs>*>(scales + kScaleStages * S::kScale);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto* tab = reinterpret_cast<GroupTable*>(reinterpret_cast<unsigned char*>(bars) + 1024);
    const int rank = split > 1 ? (int)cluster_ctarank() : 0;
    const int first = (int)blockIdx.x / split, step = (int)gridDim.x / split;
    const int k0 = (int)((int64_t)p.KB * rank / split), k1 = (int)((int64_t)p.KB * (rank + 1) / split);

    if (threadIdx.x == 0) init_bars8(bars, 4);
    if constexpr (rows_kind(KIND)) groups_build<kSThreads>(tab, p.ends, p.G, p.M, NT, p.NB, p.rest);
    if (warp == 1) {
        tmem_alloc(smem_u32(&bars->tmem_addr), kTmem);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_addr;
    int* ab = &bars->abort_flag;
    const int quarter = warp & 3, row_in = quarter * 32 + lane;
    int tiles = p.NB;  // of 128 rows of B; all of A's rows are one block
    if constexpr (rows_kind(KIND)) tiles = tab->first[p.G + 1];
    auto unit = [&](int t) { return unit_at<NT, KIND>(p, tab, t, k0, k1); };
    float sum[NT];  // epilogue: this thread's row of B against the NT rows of A
    float2 pairs[kExt ? NT / 2 : 1];

    if (warp == 0) {
        if (lane == 0) {
            Ring r;
            int64_t issued = 0;
            bool ok = true;
            for (int t = first; ok && t < tiles; t += step) {
                const Unit8 x = unit(t);
                for (int kb = x.k0; kb < x.k1; ++kb) {
                    if (!(ok = pipe_wait(ab, smem_u32(&bars->empty[r.slot]), r.phase ^ 1u, p.w))) break;
                    const uint32_t fb = smem_u32(&bars->full[r.slot]);
                    mbar_arrive_expect_tx(fb, S::kW + S::kX);
                    if constexpr (kExt) {
                        if constexpr (kGated) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                tma_load_4d(smem_u32(sW + r.slot * S::kW + i * (S::kW / 4)), &tmB, kb * kGK,
                                            x.nb * (kSRows / 2) + i * 16, 0, x.group, fb);
                        } else {
                            tma_load_4d(smem_u32(sW + r.slot * S::kW), &tmB, kb * kGK, x.nb * kSRows, 0, x.group, fb);
                        }
                    } else {
                        tma_load_2d(smem_u32(sW + r.slot * S::kW), &tmB, kb * kGK, t * kSRows, fb);
                    }
                    tma_load_2d(smem_u32(sX + r.slot * S::kX), &tmA, kb * kGK, x.row0, fb);
                    ++issued;
                    r.next(S::kStages);
                }
            }
            for (int64_t j = issued > S::kStages ? issued - S::kStages : 0; j < issued; ++j)
                pipe_drain(smem_u32(&bars->full[j % S::kStages]), (uint32_t)((j / S::kStages) & 1), p.w);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            Ring r, acc;
            bool ok = true;
            const uint32_t idesc = idesc_e4m3_f32(kSRows, NT);
            for (int t = first; ok && t < tiles; t += step) {
                const Unit8 x = unit(t);
                for (int kb = x.k0; kb < x.k1; ++kb) {
                    if (!(ok = pipe_wait(ab, smem_u32(&bars->full[r.slot]), r.phase, p.w))) break;
                    if (!(ok = pipe_wait(ab, smem_u32(&bars->tempty[acc.slot]), acc.phase ^ 1u, p.w))) break;
                    tc_fence_after();
                    const uint32_t w0 = smem_u32(sW + r.slot * S::kW), x0 = smem_u32(sX + r.slot * S::kX);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_e4m3(tmem + (uint32_t)(acc.slot * NT), smem_desc_sw128(w0 + kk * 32),
                                  smem_desc_sw128(x0 + kk * 32), idesc, kk != 0);
                    umma_commit(smem_u32(&bars->empty[r.slot]));
                    umma_commit(smem_u32(&bars->tfull[acc.slot]));
                    r.next(S::kStages);
                    acc.next(kAccs);
                }
            }
            umma_commit(smem_u32(&bars->drain));
            pipe_drain(smem_u32(&bars->drain), 0u, p.w);
        }
    } else if (warp == 2) {
        Ring r;
        bool ok = true;
        for (int t = first; ok && t < tiles; t += step) {
            const Unit8 x = unit(t);
            for (int kb = x.k0; kb < x.k1; ++kb) {
                ok = __all_sync(0xFFFFFFFFu, pipe_wait(ab, smem_u32(&bars->sc.empty[r.slot]), r.phase ^ 1u, p.w));
                if (!ok) break;
                const uint32_t dst = smem_u32(scales + r.slot * S::kScale);
                const float* a = p.sa + (int64_t)kb * p.M + x.row0;
                const float* b = p.sb + (int64_t)kb * p.nsb;
                if constexpr (rows_kind(KIND)) b += x.group * p.sb_g;
                for (int i = lane; i < NT; i += 32) cp_async4(dst + i * 4, a + (i < x.rows ? i : 0), i < x.rows);
                if (BROWS) {
#pragma unroll
                    for (int i = lane; i < kSRows; i += 32) {
                        const int row = t * kSRows + i;
                        cp_async4(dst + (NT + i) * 4, b + (row < p.N ? row : 0), row < p.N);
                    }
                } else if constexpr (kExt) {
                    if (lane < (kGated ? 2 : 1)) {
                        const int blk = kGated ? (lane * p.N + x.nb * (kSRows / 2)) >> 7 : x.nb;
                        cp_async4(dst + (NT + lane) * 4, b + (blk < p.nsb ? blk : 0), blk < p.nsb);
                    }
                } else if (lane == 0) {
                    cp_async4(dst + NT * 4, b + t, true);
                }
                cp_async_arrive(smem_u32(&bars->sc.full[r.slot]));
                r.next(kScaleStages);
            }
        }
        cp_async_wait_all();
    } else if (warp >= 4) {
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
        Ring acc, sc;
        bool ok = true;
        for (int t = first; ok && t < tiles; t += step) {
#pragma unroll
            for (int i = 0; i < NT; ++i) sum[i] = 0.f;
            for (float2& x : pairs) x = make_float2(0.f, 0.f);
            const Unit8 x = unit(t);
            const int half = kGated ? lane >> 4 : 0;  // of B that this lane's row is of
            for (int kb = x.k0; kb < x.k1; ++kb) {
                ok = pipe_wait(ab, smem_u32(&bars->sc.full[sc.slot]), sc.phase, p.w);
                const float* s = scales + sc.slot * S::kScale;
                const float sb = s[NT + (BROWS ? row_in : half)];
                ok = __all_sync(0xFFFFFFFFu, ok && pipe_wait(ab, smem_u32(&bars->tfull[acc.slot]), acc.phase, p.w));
                if (!ok) break;
                tc_fence_after();
                const uint32_t t0 = tmem + lane_base + (uint32_t)(acc.slot * NT);
                uint32_t v[2][16];
                tmem_ld16_issue(t0, v[0]);
#pragma unroll
                for (int c = 0; c < NT / 16; ++c) {
                    tmem_wait16(v[c & 1]);
                    if (c < NT / 16 - 1) {
                        tmem_ld16_issue(t0 + (c + 1) * 16, v[(c + 1) & 1]);
                    } else {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_u32(&bars->tempty[acc.slot]));
                    }
                    if constexpr (kExt) {
#pragma unroll
                        for (int i = 0; i < 16; i += 4) {
                            const float4 f = *reinterpret_cast<const float4*>(s + c * 16 + i);
                            const float2 lo = fmul2(make_float2(f.x, f.y), make_float2(sb, sb));
                            const float2 hi = fmul2(make_float2(f.z, f.w), make_float2(sb, sb));
                            const uint32_t* w = &v[c & 1][i];
                            float2* d = pairs + (c * 16 + i) / 2;
                            d[0] = ffma2(make_float2(__uint_as_float(w[0]), __uint_as_float(w[1])), lo, d[0]);
                            d[1] = ffma2(make_float2(__uint_as_float(w[2]), __uint_as_float(w[3])), hi, d[1]);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            sum[c * 16 + i] = __fmaf_rn(__uint_as_float(v[c & 1][i]), __fmul_rn(s[c * 16 + i], sb),
                                                        sum[c * 16 + i]);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars->sc.empty[sc.slot]));
                acc.next(kAccs);
                sc.next(kScaleStages);
            }
            if (!ok || split > 1) break;  // a split launch has one tile a cluster, added up below
            if constexpr (kExt) {
                finish_lanes<NT, KIND>(p, x, quarter, lane, pairs);
                continue;
            }
            const int col = t * kSRows + row_in;
            if (col < p.N) {
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const int64_t at = (int64_t)i * p.ldc + col;
                    if (i >= p.M) break;
                    if (p.c_f32) {
                        float* c = static_cast<float*>(p.c) + at;
                        *c = p.accumulate ? *c + sum[i] : sum[i];
                    } else {
                        static_cast<uint16_t*>(p.c)[at] = (uint16_t)pack_bf16x2_rn(sum[i], 0.f);
                    }
                }
            }
        }
    }
    __syncwarp();
    if (split > 1) {
        // every load has been consumed, so the ring's memory takes the partial sums [NT][128]
        float* red = reinterpret_cast<float*>(smem);
        __syncthreads();
        if (warp >= 4) {
#pragma unroll
            for (int i = 0; i < NT; ++i) red[i * kSRows + row_in] = !kExt ? sum[i] : i & 1 ? pairs[i / 2].y : pairs[i / 2].x;
        }
        cluster_sync_all();
        const bool failed = *reinterpret_cast<volatile int*>(ab) != 0;
        // this CTA adds up rows [lo, hi) of A: 128 consecutive columns of C a row
        const int lo = NT * rank / split, hi = NT * (rank + 1) / split;
        auto joined = [&](int i, int at_row) {
            const uint32_t at = smem_u32(red + i * kSRows + at_row);
            float v = 0.f;
            for (int r = 0; r < split; ++r) v = __fadd_rn(v, ld_cluster_f32(mapa_shared(at, (uint32_t)r)));
            return v;
        };
        if constexpr (kExt) {
            if (first < tiles && !failed) {
                const Unit8 x = unit(first);
                const bool behind = rows_kind(KIND) && p.rest && x.group == p.G;
                const int per = kGated ? kSRows / 2 : kSRows;
                const int64_t at_b = (int64_t)x.group * (kGated ? 2 : 1) * p.N;
                for (int e = threadIdx.x; e < (hi - lo) * per; e += kSThreads) {
                    const int i = lo + e / per, c = e % per, col = x.nb * per + c;
                    if (i >= x.rows || col >= p.N) continue;
                    const int64_t row = (int64_t)x.row0 + i;
                    const int in = kGated ? (c >> 4) * 32 + (c & 15) : c;
                    float z = joined(i, in), u = kGated ? joined(i, in + 16) : 0.f;
                    if (p.bias && !behind) {
                        z = __fadd_rn(z, bias_at(p, at_b + col));
                        if (kGated) u = __fadd_rn(u, bias_at(p, at_b + p.N + col));
                    }
                    if (p.z && !behind) {
                        p.z[row * p.ldz + col] = (uint16_t)pack_bf16x2_rn(z, 0.f);
                        if (kGated) p.z[row * p.ldz + p.N + col] = (uint16_t)pack_bf16x2_rn(u, 0.f);
                    }
                    finish_one<KIND>(p, row, col, z, u);
                }
            }
        }
        for (int e = threadIdx.x; !kExt && e < (hi - lo) * kSRows && !failed; e += kSThreads) {
            const int i = lo + e / kSRows, col = first * kSRows + e % kSRows;
            if (i >= p.M || col >= p.N) continue;
            const float v = joined(i, e % kSRows);
            const int64_t o = (int64_t)i * p.ldc + col;
            if (p.c_f32) {
                float* c = static_cast<float*>(p.c) + o;
                *c = p.accumulate ? *c + v : v;
            } else {
                static_cast<uint16_t*>(p.c)[o] = (uint16_t)pack_bf16x2_rn(v, 0.f);
            }
        }
        cluster_sync_all();  // no CTA leaves while another reads its sums
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmem);
    }
}

// ----------------------------------------------------------------- host

// A byte matrix of `rows` rows of `inner` bytes, `stride` apart, in boxes of
// 128 bytes x box_rows with the 128-byte swizzle; bytes outside read as zero.
bool make_map8(CUtensorMap* m, const void* base, int64_t inner, int64_t rows, int64_t stride, uint32_t box_rows) {
    EncodeTiled enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)stride};
    const cuuint32_t box[2] = {kGK, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// B of an epilogue: G groups (`group` bytes apart) of `halves` halves of `rows` rows, in boxes of 128 bytes x box_rows /
// halves rows of each half; the rows behind a half read as zero.
bool make_map_halves(CUtensorMap* m, const void* base, int64_t inner, int64_t rows, int halves, int64_t groups,
                     int64_t stride, int64_t group, uint32_t box_rows) {
    EncodeTiled enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)inner, (cuuint64_t)rows, (cuuint64_t)halves, (cuuint64_t)groups};
    // the strides of dimensions of one element are not used, but have to pass the checks
    const cuuint64_t strides[3] = {(cuuint64_t)stride, (cuuint64_t)(halves > 1 ? rows * stride : stride),
                                   (cuuint64_t)(groups > 1 ? group : stride)};
    const cuuint32_t box[4] = {kGK, box_rows / (uint32_t)halves, (cuuint32_t)halves, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

rlk_status cuda_fail(const char* what, cudaError_t e) {
    return fail(RLK_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

template <auto KERNEL>
rlk_status allow_smem(size_t bytes) {
    return allow_dynamic_smem<KERNEL>(bytes) ? RLK_OK : cuda_fail("fp8 product: shared memory", cudaGetLastError());
}

// behind: may start while the kernel before it in the stream ends.
template <auto KERNEL, typename... Args>
rlk_status launch_clusters(int blocks, int threads, size_t smem, int cluster, bool behind, cudaStream_t st,
                           Args... args) {
    const rlk_status s = allow_smem<KERNEL>(smem);
    if (s != RLK_OK) return s;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)cluster;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = behind ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, KERNEL, args...);
    return e == cudaSuccess ? RLK_OK : cuda_fail("fp8 product launch", e);
}

// Clusters of `cluster` CTAs that the device runs at once (asked once a kernel, size and device).
template <auto KERNEL>
int clusters_at_once(int threads, size_t smem, int cluster) {
    static std::mutex mu;
    static int known[64][9] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64 || cluster < 1 || cluster > 8) return 0;
    std::lock_guard<std::mutex> lock(mu);
    int& n = known[dev][cluster];
    if (n == 0) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)cluster);
        cfg.blockDim = dim3((unsigned)threads);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = (unsigned)cluster;
        at[0].val.clusterDim.y = 1;
        at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        if (allow_smem<KERNEL>(smem) != RLK_OK || cudaOccupancyMaxActiveClusters(&n, KERNEL, &cfg) != cudaSuccess) {
            cudaGetLastError();
            n = 0;
            return 0;
        }
    }
    return n;
}

template <bool BROWS, int KIND>
rlk_status launch_gemm(const typename ParamsOf<KIND>::type& p, const CUtensorMap& a, const CUtensorMap& b, int sms,
                       cudaStream_t st) {
    // Tiles that would leave half of the pairs idle are split along K, over two or four pairs of a cluster of eight
    // CTAs at most, while each keeps four groups and all clusters run at once: the CTAs of a cluster share a GPC, and
    // a second round of clusters costs more than the split gains (16 tiles over four pairs each 30 us, over two 19).
    // The tiles of a last, partial round of the pairs are such tiles too, in a launch of their own; its start and
    // the sums' joining cost about as much as 12 K groups, so it has to save 16 (4096 x 4096 x 8192, scales by the
    // row, FP32: 172 us in one launch, 157 in two; 2560 x 4096 of BF16: 31 and 32 at K = 2048, 48.8 and 45.3 at 4096).
    constexpr auto kernel = gemm_kernel<BROWS, KIND>;
    constexpr size_t smem = kGSmemOf<BROWS, KIND>;
    const int tiles = p.MB * p.NB, pairs = sms / 2, whole = tiles / pairs * pairs, rest = tiles - whole;
    int split = rest > 0 ? kGSplit : 1;
    while (split > 1 && (p.KB < split * 4 || rest > clusters_at_once<kernel>(kGThreads, smem, 2 * split))) split /= 2;
    if (whole > 0 && p.KB * (split - 1) < (layer_kind(KIND) ? kLayerTailSaves : kTailSaves) * split) split = 1;
    if (split == 1)
        return launch_clusters<kernel>(2 * (tiles < pairs ? tiles : pairs), kGThreads, smem, 2, false, st, a, b, p, 0,
                                       tiles, 1);
    if (whole > 0) {
        const rlk_status s =
            launch_clusters<kernel>(2 * pairs, kGThreads, smem, 2, false, st, a, b, p, 0, whole, 1);
        if (s != RLK_OK) return s;
    }
    return launch_clusters<kernel>(2 * rest * split, kGThreads, smem, 2 * split, whole > 0, st, a, b, p, whole, tiles,
                                   split);
}

template <int NT, bool BROWS, int KIND>
rlk_status launch_skinny(const typename ParamsOf<KIND>::type& p, const CUtensorMap& a, const CUtensorMap& b,
                         int64_t most, int sms, cudaStream_t st) {
    const int tiles = (int)most, room = Skinny<NT>::kPerSm * sms;
    int split = 1;
    if constexpr (KIND == kEpi || KIND == kEpiGated) {
        // as many CTAs a tile as run at once, of three too (37 x 4096 to 12288, 96 tiles: 22.4 us over two, 20.1 over
        // three; 1 x 4096: 15.3 and 14.9).  A second round of clusters costs more than it saves: 16 x 4096 gated to
        // 2 x 12288, 192 tiles, 21.3 us unsplit, 27.6 over three.
        for (int s = 2; s <= 8 && s * 2 <= p.KB && (int64_t)tiles * s <= room; ++s) split = s;
    } else {
        while (split < 8 && (int64_t)tiles * split * 2 <= room && split * 4 <= p.KB) split *= 2;
    }
    return launch_clusters<skinny_kernel<NT, BROWS, KIND>>(split > 1 ? tiles * split : tiles < room ? tiles : room,
                           kSThreads, kSSmemOf<NT, KIND>, split, false, st, a, b, p, split);
}

// most: units of work, at most.
template <bool BROWS, int KIND>
rlk_status launch_skinny_nt(int nt, const typename ParamsOf<KIND>::type& p, const CUtensorMap& a,
                            const CUtensorMap& b, int64_t most, int sms, cudaStream_t st) {
    if (nt == 16) return launch_skinny<16, BROWS, KIND>(p, a, b, most, sms, st);
    if constexpr (!rows_kind(KIND))  // of groups, more rows a group take half tiles
        if (nt == 64) return launch_skinny<64, BROWS, KIND>(p, a, b, most, sms, st);
    return launch_skinny<32, BROWS, KIND>(p, a, b, most, sms, st);
}

// The device's SMs, for a launch; 0 and a reason if they cannot be had.
int device_sms() {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess && sms > 0) return sms;
    fail(RLK_ERR_CUDA, "cannot query the device's SM count");
    return 0;
}

// M tiles of a band, whose rows of A take 32 MB of L2.
int32_t band_of(int64_t MB, int64_t K) {
    const int64_t band = ((int64_t)32 << 20) / ((int64_t)2 * kGM * K);
    return (int32_t)(band < 1 ? 1 : band < MB ? band : MB);
}

// What a product with an epilogue takes from its call.
void set_epilogue(Ext8Params& p, const rlk_fp8_epilogue* e, int64_t N) {
    p.act = e ? e->activation : RLK_ACT_NONE;
    p.nsb = (int32_t)(((e && e->gated ? 2 * N : N) + 127) / 128);
    if (!e) return;
    p.bias = e->bias;
    p.bias_f32 = e->bias_type == RLK_F32;
    p.bias_vec = reinterpret_cast<uintptr_t>(p.bias) % 16 == 0 && (N * (p.bias_f32 ? 4 : 2)) % 16 == 0;
    p.res = e->residual;
    p.res_f32 = e->residual_type == RLK_F32;
    p.ldr = e->residual_stride;
    p.res_vec = reinterpret_cast<uintptr_t>(p.res) % 16 == 0 && (p.ldr * (p.res_f32 ? 4 : 2)) % 16 == 0;
    p.z = static_cast<uint16_t*>(e->z);
    p.ldz = e->z_stride;
    p.z_vec = reinterpret_cast<uintptr_t>(p.z) % 16 == 0 && (p.ldz * 2) % 16 == 0;
}

}  // namespace
}  // namespace rlk
