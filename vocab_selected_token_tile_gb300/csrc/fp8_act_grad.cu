// The backward of a feed-forward layer's epilogue, quantised (sm_103a): from dy
// and the kept pre-activation z, in FP32,
//   dz = dy act'(z);   gated: dz_gate = dy z_up act'(z_gate), dz_up = dy act(z_gate),
// the E4M3 codes of dz along its rows and along its columns, and the sum of dz
// over the rows for the bias.  dz is never stored: a CTA forms a 128 x 128 tile of
// it in registers and quantises that as fp8_quant.cu does, and leaves the sums of
// its 128 columns, which a second launch adds up in order.
//
// Bound: HBM, in principle: dy and z read once (2 bytes each; a gated layer's
// gate and other half read the same dy and, between them, z one and a half times,
// the second time from L2), two codes written an element.  What it spends: as
// fp8_quant.cu's tiles, a chain of loads, maxima, barriers, conversions and
// stores, and beside that about ten packed instructions and 1.5 of the
// special-function unit a pair for the derivative; 1,950 instructions a warp run
// straight through, and 44% of the issue slots are used (instruction fetches,
// waits and memory share the rest evenly).  Two CTAs an SM with four rows' loads
// under way each; three with two rows' spilled registers.  4096 x 6144, BF16:
// gated silu 73 us (350 MB: 4.8 TB/s), of which the quantisation of as many FP32
// values takes 63; 8192 x 4096, silu without a gate 51 us (201 MB; 43).
#include "rlk_act.cuh"
#include "rlk_fp8_quant.cuh"

namespace rlk {
namespace {

// 8 consecutive elements of a row in FP32, zero from `left` on.
__device__ __forceinline__ void load8(float (&v)[8], const void* x, int64_t at, bool f32, bool vec, int64_t left) {
    if (vec && left >= 8) {
        if (f32) {
            const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
            const float4 a = __ldcs(s), b = __ldcs(s + 1);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
            const uint4 a = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at));
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) v[2 * j] = bf16lo_to_f32(w[j]), v[2 * j + 1] = bf16hi_to_f32(w[j]);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = j >= left ? 0.f
               : f32     ? static_cast<const float*>(x)[at + j]
                         : __uint_as_float((uint32_t) static_cast<const uint16_t*>(x)[at + j] << 16);
}

// The part of dz that a column is of: all of it; gated, the gate's half or the other one.
enum Part8 : int { kWhole, kGate, kOther };

// Two values of dz; `up` (kGate) the other half of z.
template <int ACT, int PART>
__device__ __forceinline__ float2 dz_of(float2 dy, float2 z, float2 up) {
    if (PART == kOther) return fmul2(dy, act_pair<ACT>(z));
    return act_back_pair<ACT>(PART == kGate ? fmul2(dy, up) : dy, z);
}

// The thread's 8 x 8 block of dz from row r0 on: 8 columns from column c of
// their part, whose width is N.
template <int ACT, int PART>
__device__ __forceinline__ void load_dz(Block<true>& b, const QuantExtParams& p, int64_t r0, int64_t end, int64_t c,
                                        int64_t N) {
    constexpr bool kZ = ACT != RLK_ACT_NONE || PART != kWhole;  // z is read
    const uint16_t* z = kZ ? p.z + r0 * p.ldz + c : nullptr;
    if (p.dy_f32 || !p.dy_vec || (kZ && !p.z_vec) || c + 8 > N) {
        const int64_t left = N - c;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float dy[8] = {}, a[8] = {}, u[8] = {};
            if (r0 + i < end && left > 0) {
                load8(dy, p.dy, (r0 + i) * p.lddy + c, p.dy_f32, p.dy_vec, left);
                if (kZ) load8(a, z, i * p.ldz, false, p.z_vec, left);
                if (PART == kGate) load8(u, z, i * p.ldz + N, false, p.z_vec, left);
            }
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float2 d = dz_of<ACT, PART>(make_float2(dy[j], dy[j + 1]), make_float2(a[j], a[j + 1]),
                                                  make_float2(u[j], u[j + 1]));
                b.w[i][j] = j < left ? __float_as_uint(d.x) : 0u;
                b.w[i][j + 1] = j + 1 < left ? __float_as_uint(d.y) : 0u;
            }
        }
        return;
    }
    // BF16 on the 16-byte grid: four rows' loads at a time (a row at a time the tile was a chain of eight memory
    // latencies: 4096 x 6144 gated 145 us, 87 so)
    const uint16_t* dy = static_cast<const uint16_t*>(p.dy) + r0 * p.lddy + c;
    const int rows = (int)min((int64_t)8, end - r0);
#pragma unroll
    for (int h = 0; h < 8; h += 4) {
        uint4 d[4], a[4], u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            d[i] = a[i] = u[i] = make_uint4(0, 0, 0, 0);
            if (h + i < rows) {
                d[i] = __ldcs(reinterpret_cast<const uint4*>(dy + (h + i) * p.lddy));
                if (kZ) a[i] = __ldcs(reinterpret_cast<const uint4*>(z + (h + i) * p.ldz));
                if (PART == kGate) u[i] = __ldcs(reinterpret_cast<const uint4*>(z + (h + i) * p.ldz + N));
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t wd[4] = {d[i].x, d[i].y, d[i].z, d[i].w}, wa[4] = {a[i].x, a[i].y, a[i].z, a[i].w};
            const uint32_t wu[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                auto two = [](uint32_t w) { return make_float2(bf16lo_to_f32(w), bf16hi_to_f32(w)); };
                const float2 v = dz_of<ACT, PART>(two(wd[k]), two(wa[k]), two(wu[k]));
                b.w[h + i][2 * k] = __float_as_uint(v.x), b.w[h + i][2 * k + 1] = __float_as_uint(v.y);
            }
        }
    }
}

// The epilogue's backward.
template <bool TRANS, int ROWS, int ACT, bool GATED>
__global__ void __launch_bounds__(kQThreads, 2) act_grad_kernel(const __grid_constant__ QuantExtParams p) {
    __shared__ TileShared<true, false, TRANS> sh;
    __shared__ typename std::conditional<ROWS == kGroups, GroupTable, int>::type tab;
    __shared__ float4 sums[16][kQT / 4];
    const int cx = threadIdx.x & 15, ry = threadIdx.x >> 4;
    const int64_t ct = blockIdx.x, rt = blockIdx.y + (int64_t)blockIdx.z * 65535;
    RowTile at;
    if constexpr (ROWS == kGroups) {
        if (!group_tile(p, rt, &tab, at)) return;
    } else {
        if (rt * kQT >= p.R) return;
        at = RowTile{rt * kQT, p.R, rt * kQT, p.R, rt};
    }
    Block<true> b;
    const int64_t r0 = at.row0 + ry * 8, c0 = ct * kQT + cx * 8;
    if constexpr (GATED) {  // 8 columns are of one half: C / 2 is a multiple of 64
        const int64_t N = p.C / 2;
        if (c0 < N)
            load_dz<ACT, kGate>(b, p, r0, at.end, c0, N);
        else
            load_dz<ACT, kOther>(b, p, r0, at.end, c0 - N, N);
    } else {
        load_dz<ACT, kWhole>(b, p, r0, at.end, c0, p.C);
    }
    if (p.part) {
        float s[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            s[j] = b.at(0, j);
#pragma unroll
            for (int i = 1; i < 8; ++i) s[j] = __fadd_rn(s[j], b.at(i, j));
        }
        sums[ry][2 * cx] = make_float4(s[0], s[1], s[2], s[3]);
        sums[ry][2 * cx + 1] = make_float4(s[4], s[5], s[6], s[7]);
        __syncthreads();
        if (threadIdx.x < kQT && ct * kQT + threadIdx.x < p.C) {
            float v = 0.f;
#pragma unroll
            for (int k = 0; k < 16; ++k)
                v = __fadd_rn(v, reinterpret_cast<const float*>(sums[k])[threadIdx.x]);
            p.part[rt * p.C + ct * kQT + threadIdx.x] = v;
        }
    }
    if (p.q || TRANS) quantize_tile<true, false, TRANS>(p, b, ct, at, sh);
}

// dbias from the row tiles' sums: a warp of 32 columns, eight runs of a group's
// tiles at a time, joined in order.
template <int ROWS>
__global__ void __launch_bounds__(kQThreads) bias_grad_kernel(const __grid_constant__ QuantExtParams p, void* dbias,
                                                              const int f32) {
    __shared__ typename std::conditional<ROWS == kGroups, GroupTable, int>::type tab;
    __shared__ float join[8][32];
    const int run = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    if constexpr (ROWS == kGroups) {
        groups_build<kQThreads>(&tab, p.ends, p.G, (int)p.R, kQT, 1, false);
        __syncthreads();
    }
    for (int e = blockIdx.y; e < (ROWS == kGroups ? p.G : 1); e += gridDim.y) {
        int64_t t0 = 0, t1 = (p.R + kQT - 1) / kQT;
        if constexpr (ROWS == kGroups) t0 = tab.first[e], t1 = tab.first[e + 1];
        const int64_t lo = t0 + (t1 - t0) * run / 8, hi = t0 + (t1 - t0) * (run + 1) / 8;
        float v = 0.f;
        if (c < p.C) {
#pragma unroll 4
            for (int64_t t = lo; t < hi; ++t) v = __fadd_rn(v, p.part[t * p.C + c]);
        }
        join[run][lane] = v;
        __syncthreads();
        if (run == 0 && c < p.C) {
#pragma unroll
            for (int k = 1; k < 8; ++k) v = __fadd_rn(v, join[k][lane]);
            if (f32)
                static_cast<float*>(dbias)[e * p.C + c] = v;
            else
                static_cast<uint16_t*>(dbias)[e * p.C + c] = (uint16_t)pack_bf16x2_rn(v, 0.f);
        }
        __syncthreads();
    }
}

template <bool TRANS, int ROWS, bool GATED>
void launch_act(const QuantExtParams& p, dim3 grid, cudaStream_t st) {
    auto go = [&](auto kernel) { kernel<<<grid, kQThreads, 0, st>>>(p); };
    switch (p.act) {
        case RLK_ACT_RELU: return go(act_grad_kernel<TRANS, ROWS, RLK_ACT_RELU, GATED>);
        case RLK_ACT_SILU: return go(act_grad_kernel<TRANS, ROWS, RLK_ACT_SILU, GATED>);
        case RLK_ACT_GELU: return go(act_grad_kernel<TRANS, ROWS, RLK_ACT_GELU, GATED>);
        case RLK_ACT_GELU_TANH: return go(act_grad_kernel<TRANS, ROWS, RLK_ACT_GELU_TANH, GATED>);
        default: return go(act_grad_kernel<TRANS, ROWS, RLK_ACT_NONE, GATED>);
    }
}

template <int ROWS>
rlk_status launch_act_rows(const QuantExtParams& p, int64_t row_tiles, void* dbias, bool f32, cudaStream_t st) {
    const dim3 grid = tile_grid(p.C, row_tiles);
    if (p.gated)
        p.qt ? launch_act<true, ROWS, true>(p, grid, st) : launch_act<false, ROWS, true>(p, grid, st);
    else
        p.qt ? launch_act<true, ROWS, false>(p, grid, st) : launch_act<false, ROWS, false>(p, grid, st);
    rlk_status s = quant_cuda("fp8 activation gradient launch");
    if (s != RLK_OK || !dbias) return s;
    const dim3 sums((unsigned)((p.C + 31) / 32), (unsigned)(p.G < 1 ? 1 : p.G < 32 ? p.G : 32));
    bias_grad_kernel<ROWS><<<sums, kQThreads, 0, st>>>(p, dbias, f32);
    return quant_cuda("bias gradient launch");
}

}  // namespace

rlk_status launch_fp8_act_grad(int64_t G, int64_t rows, int64_t wide, const int32_t* ends, const void* dy,
                               int32_t dy_f32, int64_t lddy, const void* z, int64_t ldz, int32_t act, int32_t gated,
                               uint8_t* q, int64_t ldq, float* scale, uint8_t* qt, int64_t ldqt, float* scale_t,
                               void* dbias, int32_t dbias_f32, float* part, cudaStream_t stream) {
    QuantExtParams p{};
    p.R = rows;
    p.C = wide;
    p.q = q;
    p.qt = qt;
    p.ldq = ldq;
    p.ldqt = ldqt;
    p.scale = scale;
    p.scale_t = scale_t;
    p.ends = ends;
    p.G = (int32_t)G;
    p.dy = dy;
    p.dy_f32 = dy_f32;
    p.lddy = lddy;
    p.dy_vec = (reinterpret_cast<uintptr_t>(dy) % 16 == 0) && (lddy * (dy_f32 ? 4 : 2)) % 16 == 0;
    p.z = static_cast<const uint16_t*>(z);
    p.ldz = ldz;
    p.z_vec = (reinterpret_cast<uintptr_t>(z) % 16 == 0) && (ldz * 2) % 16 == 0;
    p.act = act;
    p.gated = gated;
    p.part = dbias ? part : nullptr;
    return G > 0 ? launch_act_rows<kGroups>(p, group_row_tiles(G, rows), dbias, dbias_f32, stream)
                 : launch_act_rows<kOne>(p, (rows + kQT - 1) / kQT, dbias, dbias_f32, stream);
}

}  // namespace rlk
