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
// / 128 tiles are fewer than the SMs can hold, a cluster of 2, 4 or 8 CTAs
// splits K, and adds its partial sums through distributed shared memory in
// rank order: no workspace, no second launch, the same bits every time.
//
// Every wait is bounded; on expiry the CTA records the time-out in the status
// word, stops issuing, waits (bounded) for the copies and MMAs under way (a
// pair for those of both of its CTAs), frees its tensor memory and returns.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>
#include <string>

#include "rlk_gemm.cuh"
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
template <int STAGES>
struct Bars8 {
    uint64_t full[STAGES];
    uint64_t empty[STAGES];
    uint64_t tfull[2];
    uint64_t tempty[2];
    ScaleBars sc;
    uint64_t drain;
    uint32_t tmem_addr;
    int abort_flag;
};

template <int STAGES>
__device__ void init_bars8(Bars8<STAGES>* b, int epilogue_warps) {
    for (int s = 0; s < STAGES; ++s) {
        mbar_init(smem_u32(&b->full[s]), 1);
        mbar_init(smem_u32(&b->empty[s]), 1);
    }
    for (int i = 0; i < 2; ++i) {
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

// A warp's 32 rows x 128 bytes of C (32 FP32 or 64 BF16 columns) through shared
// memory, so that a row's 128 bytes leave in one piece: 16 bytes a lane
// straight from the registers, 32 rows an instruction, took 10,700 clocks a 128
// x 256 tile, a third of the product's time at K = 4096.  16-byte piece j of
// row r is kept at j ^ turn(r), which spreads both directions over the banks.
// v: the lane's row (pairs of columns), or with FRAG, of each 32 columns, 4 rows
// (t / 4 and 8, 16, 24 after) x 4 pairs (2 (t mod 4) and 8, 16, 24 after).
template <bool F32, bool FRAG>
__device__ __forceinline__ void store_chunk(const Gemm8Params& p, unsigned char* out, int lane, int64_t row0, int col0,
                                            const float2* v) {
    constexpr int kPer = F32 ? 4 : 8;  // elements of 16 bytes
    auto turn = [](int r) { return F32 && FRAG ? 2 * (r & 3) : r & 7; };
    __syncwarp();
    if (FRAG) {
#pragma unroll
        for (int q = 0; q < (F32 ? 1 : 2); ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 x = v[q * 16 + i * 4 + j];
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
        for (int j = 0; j < 8; ++j) {
            uint4 w;
            if (F32)
                w = make_uint4(__float_as_uint(v[2 * j].x), __float_as_uint(v[2 * j].y),
                               __float_as_uint(v[2 * j + 1].x), __float_as_uint(v[2 * j + 1].y));
            else
                w = make_uint4(pack_bf16x2_rn(v[4 * j].x, v[4 * j].y), pack_bf16x2_rn(v[4 * j + 1].x, v[4 * j + 1].y),
                               pack_bf16x2_rn(v[4 * j + 2].x, v[4 * j + 2].y),
                               pack_bf16x2_rn(v[4 * j + 3].x, v[4 * j + 3].y));
            *reinterpret_cast<uint4*>(out + lane * 128 + ((j ^ turn(lane)) * 16)) = w;
        }
    }
    __syncwarp();
    const int rows = (int)min((int64_t)32, p.M - row0), cols = min(8 * kPer, p.N - col0);
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
struct GemmBars {
    PairBars<kGStages> pair;
    uint64_t sfull[kGSlots], sempty[kGSlots];
};
static_assert(sizeof(GemmBars) <= 1024, "barriers fit their kilobyte");
static_assert(kGSmem<true> <= 232448, "shared memory of a CTA");

constexpr int kGSplit = 4;  // pairs that share a tile at most: a cluster of eight CTAs
constexpr int kTailSaves = 16;  // K groups that a launch of the last tiles has to save a pair
constexpr int kRedPitch = kGN + 4;
static_assert((size_t)kGM * kRedPitch * 4 <= (size_t)kGStages * (kGA + kGB), "the partial sums fit the ring");

// Tile t of the persistent order: bands of `band` M tiles, and within a band
// all M tiles of one N tile before the next, so the tiles in flight share a
// few N tiles of B and the band's rows of A, which L2 holds.
__device__ __forceinline__ void tile_of(const Gemm8Params& p, int t, int& mb, int& nb) {
    const int per = p.band * p.NB, full = p.MB / p.band;
    const int b = min(t / per, full);
    const int r = t - b * per;
    const int width = b < full ? p.band : p.MB - full * p.band;
    nb = r / width;
    mb = b * p.band + r % width;
}

// Tiles tile0 .. tiles - 1.  split: pairs of a cluster that share a tile, each
// with a part of the K groups (1: the pair's tiles are its own, one after the
// other).  A launch with tile0 > 0 runs behind the one with the tiles before,
// whose inputs are its own and whose outputs are not: it may start as that
// one's pairs end.
template <bool BROWS>
__global__ void __launch_bounds__(kGThreads, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                const __grid_constant__ Gemm8Params p, const int tile0, const int tiles, const int split) {
    extern __shared__ unsigned char smem_raw[];
    // The same offset in both CTAs (their dynamic shared memory starts alike): descriptors name one offset.
    unsigned char* smem =
        reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    unsigned char* sA = smem;
    unsigned char* sB = smem + kGStages * kGA;
    unsigned char* sOut = sB + kGStages * kGB;
    float* scales = reinterpret_cast<float*>(sOut + 8 * kGOut);
    auto* all = reinterpret_cast<GemmBars*>(scales + kGSlots * kGroups * kGScales<BROWS>);
    PairBars<kGStages>* bars = &all->pair;
    const int warp = warp_index(), lane = threadIdx.x & 31;
    const int place = (int)cluster_ctarank(), rank = place & 1, leader = place & ~1;
    const uint16_t both = (uint16_t)(3 << leader);
    const int first = tile0 + (int)blockIdx.x / (2 * split), step = (int)gridDim.x / (2 * split);
    const int k0 = (int)((int64_t)p.KB * (leader / 2) / split), k1 = (int)((int64_t)p.KB * (leader / 2 + 1) / split);

    if (threadIdx.x == 0) {
        for (int i = 0; i < kGSlots; ++i) {
            mbar_init(smem_u32(&all->sfull[i]), 32);
            mbar_init(smem_u32(&all->sempty[i]), 8);
        }
    }
    const uint32_t tmem = pair_begin(bars, warp, 8);
    int* ab = &bars->abort_flag;
    grid_launch_dependents();  // the launch of the last tiles

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
                int mb, nb;
                tile_of(p, t, mb, nb);
                const int a_row = (2 * mb + rank) * kGM, b_row = nb * kGN + rank * (kGN / 2);
                // a CTA without a row of its own loads none: its rows of the accumulator are not used
                const bool mine = a_row < p.M;
                for (int kb = k0; kb < k1; ++kb) {
                    if (!(ok = pipe_wait_warp(ab, smem_u32(&bars->empty[r.slot]), r.phase ^ 1u, p.w))) break;
                    if (one) {
                        const uint32_t fb = full0 + r.slot * 8;
                        pair_arm(fb, smem_u32(&bars->full[r.slot]), rank, kGB + (mine ? kGA : 0));
                        if (mine) tma_load_2d_pair(smem_u32(sA + r.slot * kGA), &tmA, kb * kGK, a_row, fb);
                        tma_load_2d_pair(smem_u32(sB + r.slot * kGB), &tmB, kb * kGK, b_row, fb);
                    }
                    ++issued;
                    r.next(kGStages);
                }
            }
            pair_end_copies(bars, r, one, issued, ok, p.w);
        } else if (warp == 1 && rank == 0) {
            // ------------------------------------------------ MMA issuer of the pair
            const bool one = elect_one();
            const uint64_t da = smem_desc_sw128(smem_u32(sA)), db = smem_desc_sw128(smem_u32(sB));
            const uint32_t idesc = idesc_e4m3_f32(2 * kGM, kGN);
            Ring r, acc;
            bool ok = true;
            for (int t = first; ok && t < tiles; t += step) {
                for (int kb = k0; kb < k1; ++kb) {
                    // the operands first: theirs are ready early, so only the accumulator's wait is in its way
                    if (!(ok = pipe_wait_warp(ab, smem_u32(&bars->full[r.slot]), r.phase, p.w))) break;
                    if (!(ok = pipe_wait_warp(ab, smem_u32(&bars->tempty[acc.slot]), acc.phase ^ 1u, p.w))) break;
                    tc_fence_after();
                    if (one) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma_e4m3_pair(tmem + (uint32_t)(acc.slot * kGN), da + ((r.slot * kGA + kk * 32) >> 4),
                                           db + ((r.slot * kGB + kk * 32) >> 4), idesc, kk != 0);
                        umma_commit_pair(smem_u32(&bars->tfull[acc.slot]), both);
                        umma_commit_pair(smem_u32(&bars->empty[r.slot]), both);
                    }
                    __syncwarp();
                    r.next(kGStages);
                    acc.next(2);
                }
            }
            pair_end_mmas(bars, acc, one, ok, p.w, both);
        } else if (warp == 2) {
            // ------------------------------------------------ scales
            Ring r;
            bool ok = true;
            for (int t = first; ok && t < tiles; t += step) {
                int mb, nb;
                tile_of(p, t, mb, nb);
                const int row = (2 * mb + rank) * kGM + lane, col = nb * kGN + lane;
                for (int kg = k0; kg < k1; kg += kGroups) {
                    ok = pipe_wait_warp(ab, smem_u32(&all->sempty[r.slot]), r.phase ^ 1u, p.w);
                    if (!ok) break;
                    uint32_t dst = smem_u32(scales + r.slot * kGroups * kGScales<BROWS>) + lane * 4;
                    const float *a = p.sa + (int64_t)kg * p.M, *b = p.sb + (int64_t)kg * p.nsb;
                    for (int kb = kg; kb < min(kg + kGroups, k1); ++kb) {
#pragma unroll
                        for (int i = 0; i < kGM; i += 32)
                            cp_async4(dst + i * 4, a + (row + i < p.M ? row + i : 0), row + i < p.M);
                        if (BROWS) {
#pragma unroll
                            for (int i = 0; i < kGN; i += 32)
                                cp_async4(dst + (kGM + i) * 4, b + (col + i < p.N ? col + i : 0), col + i < p.N);
                        } else if (lane < 2) {
                            const int blk = nb * 2 + lane;
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
        unsigned char* out = sOut + (warp - 4) * kGOut;
        const uint32_t done = mapa_shared(smem_u32(&bars->tempty[0]), (uint32_t)leader);
        Ring acc, sc;
        bool ok = first < tiles, ready = false;
        for (int t = first; ok && t < tiles; t += step) {
            float2 sum[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) sum[i] = make_float2(0.f, 0.f);
            const float* s = nullptr;
            for (int kb = k0; kb < k1; ++kb) {
                if ((kb - k0) % kGroups == 0) {
                    ok = pipe_wait(ab, smem_u32(&all->sfull[sc.slot]), sc.phase, p.w);
                    s = scales + sc.slot * kGroups * kGScales<BROWS>;
                }
                // of this thread's row, times the block's; or of its fragments' four rows
                float f[4];
                if (BROWS) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) f[i] = s[quarter * 32 + i * 8 + (lane >> 2)];
                } else {
                    f[0] = __fmul_rn(s[quarter * 32 + lane], s[kGM + part]);
                }
                if (!ready) ok = ok && pipe_wait(ab, smem_u32(&bars->tfull[acc.slot]), acc.phase, p.w);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                tc_fence_after();
                // 32 columns at a time, the next 32 under way while these are summed
                const uint32_t t0 = tmem + lane_base + (uint32_t)(acc.slot * kGN + part * 128);
                uint32_t v[2][32];
                BROWS ? tmem_ld_frag_issue(t0, v[0]) : tmem_ld32_issue(t0, v[0]);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    tmem_wait32(v[c & 1]);
                    if (c < 3) {
                        BROWS ? tmem_ld_frag_issue(t0 + (c + 1) * 32, v[(c + 1) & 1])
                              : tmem_ld32_issue(t0 + (c + 1) * 32, v[(c + 1) & 1]);
                    } else {
                        // the accumulator is free again; ask for the next one before this one's last sums
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_remote(done + acc.slot * 8);
                        acc.next(2);
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
                                                    make_float2(f[0], f[0]), sum[c * 16 + i]);
                    }
                }
                s += kGScales<BROWS>;
                if ((kb - k0) % kGroups == kGroups - 1 || kb == k1 - 1) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&all->sempty[sc.slot]));
                    sc.next(kGSlots);
                }
            }
            if (!ok) break;
            if (split > 1) {
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
            int mb, nb;
            tile_of(p, t, mb, nb);
            const int64_t row0 = (int64_t)(2 * mb + rank) * kGM + quarter * 32;
            const int col0 = nb * kGN + part * 128;
            if (p.c_f32) {
#pragma unroll
                for (int q = 0; q < 4; ++q) store_chunk<true, BROWS>(p, out, lane, row0, col0 + q * 32, sum + q * 16);
            } else {
#pragma unroll
                for (int q = 0; q < 2; ++q) store_chunk<false, BROWS>(p, out, lane, row0, col0 + q * 64, sum + q * 32);
            }
        }
    }
    if (split > 1) {
        // This CTA adds up its share of the rows, the pairs' sums in order.
        cluster_sync_all();
        const bool failed = *reinterpret_cast<volatile int*>(ab) != 0;
        int mb, nb;
        tile_of(p, first, mb, nb);
        const int lo = kGM * (leader / 2) / split, hi = kGM * (leader / 2 + 1) / split;
#pragma unroll 2
        for (int e = threadIdx.x; e < (hi - lo) * (kGN / 4) && !failed; e += kGThreads) {
            const int r = lo + e / (kGN / 4), c = e % (kGN / 4) * 4;
            const int64_t row = (int64_t)(2 * mb + rank) * kGM + r;
            const int col = nb * kGN + c;
            if (row >= p.M || col >= p.N) continue;
            const uint32_t at = smem_u32(reinterpret_cast<float*>(sA) + r * kRedPitch + c);
            float4 v[kGSplit];  // all under way before the first is added
#pragma unroll
            for (int s = 0; s < kGSplit; ++s)
                v[s] = s < split ? ld_cluster_f32x4(mapa_shared(at, (uint32_t)(2 * s + rank)))
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
            float x[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
            for (int s = 1; s < kGSplit; ++s) {
                x[0] = __fadd_rn(x[0], v[s].x), x[1] = __fadd_rn(x[1], v[s].y);
                x[2] = __fadd_rn(x[2], v[s].z), x[3] = __fadd_rn(x[3], v[s].w);
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

template <int NT, bool BROWS>
__global__ void __launch_bounds__(kSThreads, Skinny<NT>::kPerSm)
    skinny_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                  const __grid_constant__ Gemm8Params p, const int split) {
    using S = Skinny<NT>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem =
        reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    unsigned char* sW = smem;
    unsigned char* sX = smem + S::kStages * S::kW;
    float* scales = reinterpret_cast<float*>(sX + S::kStages * S::kX);
    auto* bars = reinterpret_cast<Bars8<S::kStages>*>(scales + kScaleStages * S::kScale);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tiles = p.NB;  // of 128 rows of B; all of A's rows are one block
    const int rank = split > 1 ? (int)cluster_ctarank() : 0;
    const int first = (int)blockIdx.x / split, step = (int)gridDim.x / split;
    const int k0 = (int)((int64_t)p.KB * rank / split), k1 = (int)((int64_t)p.KB * (rank + 1) / split);

    if (threadIdx.x == 0) init_bars8(bars, 4);
    if (warp == 1) {
        tmem_alloc(smem_u32(&bars->tmem_addr), S::kTmem);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_addr;
    int* ab = &bars->abort_flag;
    const int quarter = warp & 3, row_in = quarter * 32 + lane;
    float sum[NT];  // epilogue: this thread's row of B against the NT rows of A

    if (warp == 0) {
        if (lane == 0) {
            Ring r;
            int64_t issued = 0;
            bool ok = true;
            for (int t = first; ok && t < tiles; t += step) {
                for (int kb = k0; kb < k1; ++kb) {
                    if (!(ok = pipe_wait(ab, smem_u32(&bars->empty[r.slot]), r.phase ^ 1u, p.w))) break;
                    const uint32_t fb = smem_u32(&bars->full[r.slot]);
                    mbar_arrive_expect_tx(fb, S::kW + S::kX);
                    tma_load_2d(smem_u32(sW + r.slot * S::kW), &tmB, kb * kGK, t * kSRows, fb);
                    tma_load_2d(smem_u32(sX + r.slot * S::kX), &tmA, kb * kGK, 0, fb);
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
                for (int kb = k0; kb < k1; ++kb) {
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
                    acc.next(2);
                }
            }
            umma_commit(smem_u32(&bars->drain));
            pipe_drain(smem_u32(&bars->drain), 0u, p.w);
        }
    } else if (warp == 2) {
        Ring r;
        bool ok = true;
        for (int t = first; ok && t < tiles; t += step) {
            for (int kb = k0; kb < k1; ++kb) {
                ok = __all_sync(0xFFFFFFFFu, pipe_wait(ab, smem_u32(&bars->sc.empty[r.slot]), r.phase ^ 1u, p.w));
                if (!ok) break;
                const uint32_t dst = smem_u32(scales + r.slot * S::kScale);
                const float* a = p.sa + (int64_t)kb * p.M;
                const float* b = p.sb + (int64_t)kb * p.nsb;
                for (int i = lane; i < NT; i += 32) cp_async4(dst + i * 4, a + (i < p.M ? i : 0), i < p.M);
                if (BROWS) {
#pragma unroll
                    for (int i = lane; i < kSRows; i += 32) {
                        const int row = t * kSRows + i;
                        cp_async4(dst + (NT + i) * 4, b + (row < p.N ? row : 0), row < p.N);
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
            for (int kb = k0; kb < k1; ++kb) {
                ok = pipe_wait(ab, smem_u32(&bars->sc.full[sc.slot]), sc.phase, p.w);
                const float* s = scales + sc.slot * S::kScale;
                const float sb = s[NT + (BROWS ? row_in : 0)];
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
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        sum[c * 16 + i] = __fmaf_rn(__uint_as_float(v[c & 1][i]), __fmul_rn(s[c * 16 + i], sb),
                                                    sum[c * 16 + i]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bars->sc.empty[sc.slot]));
                acc.next(2);
                sc.next(kScaleStages);
            }
            if (!ok || split > 1) break;  // a split launch has one tile a cluster, added up below
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
            for (int i = 0; i < NT; ++i) red[i * kSRows + row_in] = sum[i];
        }
        cluster_sync_all();
        const bool failed = *reinterpret_cast<volatile int*>(ab) != 0;
        // this CTA adds up rows [lo, hi) of A: 128 consecutive columns of C a row
        const int lo = NT * rank / split, hi = NT * (rank + 1) / split;
        for (int e = threadIdx.x; e < (hi - lo) * kSRows && !failed; e += kSThreads) {
            const int i = lo + e / kSRows, col = first * kSRows + e % kSRows;
            if (i >= p.M || col >= p.N) continue;
            const uint32_t at = smem_u32(red + i * kSRows + e % kSRows);
            float v = 0.f;
            for (int r = 0; r < split; ++r) v = __fadd_rn(v, ld_cluster_f32(mapa_shared(at, (uint32_t)r)));
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
        tmem_dealloc(tmem, S::kTmem);
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

template <bool BROWS>
rlk_status launch_gemm(const Gemm8Params& p, const CUtensorMap& a, const CUtensorMap& b, int sms, cudaStream_t st) {
    // Tiles that would leave half of the pairs idle are split along K, over two or four pairs of a cluster of eight
    // CTAs at most, while each keeps four groups and all clusters run at once: the CTAs of a cluster share a GPC, and
    // a second round of clusters costs more than the split gains (16 tiles over four pairs each 30 us, over two 19).
    // The tiles of a last, partial round of the pairs are such tiles too, in a launch of their own; its start and
    // the sums' joining cost about as much as 12 K groups, so it has to save 16 (4096 x 4096 x 8192, scales by the
    // row, FP32: 172 us in one launch, 157 in two; 2560 x 4096 of BF16: 31 and 32 at K = 2048, 48.8 and 45.3 at 4096).
    constexpr auto kernel = gemm_kernel<BROWS>;
    constexpr size_t smem = kGSmem<BROWS>;
    const int tiles = p.MB * p.NB, pairs = sms / 2, whole = tiles / pairs * pairs, rest = tiles - whole;
    int split = rest > 0 ? kGSplit : 1;
    while (split > 1 && (p.KB < split * 4 || rest > clusters_at_once<kernel>(kGThreads, smem, 2 * split))) split /= 2;
    if (whole > 0 && p.KB * (split - 1) < kTailSaves * split) split = 1;
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

template <int NT, bool BROWS>
rlk_status launch_skinny(const Gemm8Params& p, const CUtensorMap& a, const CUtensorMap& b, int sms,
                         cudaStream_t st) {
    const int tiles = p.NB, room = Skinny<NT>::kPerSm * sms;
    int split = 1;
    while (split < 8 && tiles * split * 2 <= room && split * 4 <= p.KB) split *= 2;
    return launch_clusters<skinny_kernel<NT, BROWS>>(split > 1 ? tiles * split : tiles < room ? tiles : room,
                           kSThreads, Skinny<NT>::kSmem, split, false, st, a, b, p, split);
}

template <bool BROWS>
rlk_status launch_skinny_nt(int nt, const Gemm8Params& p, const CUtensorMap& a, const CUtensorMap& b, int sms,
                            cudaStream_t st) {
    switch (nt) {
        case 16: return launch_skinny<16, BROWS>(p, a, b, sms, st);
        case 32: return launch_skinny<32, BROWS>(p, a, b, sms, st);
        default: return launch_skinny<64, BROWS>(p, a, b, sms, st);
    }
}

}  // namespace

rlk_status launch_fp8_matmul(int64_t M, int64_t N, int64_t K, const void* a, int64_t lda, const float* sa,
                             const void* b, int64_t ldb, const float* sb, int32_t b_block_rows, void* c, int64_t ldc,
                             int32_t c_f32, int32_t accumulate, uint32_t* status, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess || sms <= 0) return fail(RLK_ERR_CUDA, "cannot query the device's SM count");
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
        return rows ? launch_skinny_nt<true>(nt, p, ta, tb, sms, stream)
                    : launch_skinny_nt<false>(nt, p, ta, tb, sms, stream);
    }
    p.MB = (int32_t)((M + 2 * kGM - 1) / (2 * kGM));
    p.NB = (int32_t)((N + kGN - 1) / kGN);
    const int64_t band = ((int64_t)32 << 20) / ((int64_t)2 * kGM * K);
    p.band = (int32_t)(band < 1 ? 1 : band < p.MB ? band : p.MB);
    if (!make_map8(&ta, a, K, M, lda, kGM) || !make_map8(&tb, b, K, N, ldb, kGN / 2))
        return fail(RLK_ERR_CUDA, "cuTensorMapEncodeTiled failed for an operand of the fp8 product");
    return rows ? launch_gemm<true>(p, ta, tb, sms, stream) : launch_gemm<false>(p, ta, tb, sms, stream);
}

}  // namespace rlk
