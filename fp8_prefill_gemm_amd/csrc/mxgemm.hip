// MXFP4 x MXFP4 products with fp32 accumulation on the block-scaled matrix
// cores, plain and gated:
//
//     y[i][j] = sum_b 2^(ea + ew) sum_{32 values of block b} a w
//     h[i][j] = silu(g) * u,  g = a wg^T, u = a wu^T  (one pass over a)
//
// One v_mfma_scale_f32_32x32x64_f8f6f4 in its E2M1 form multiplies a 32 x 64
// activation block by a 32 x 64 weight block in 32 cycles, twice the E4M3
// rate, and applies both operands' block scales itself: lane l holds row
// l % 32 and columns 32 (l / 32) .. + 31, 16 bytes and one scale byte.  The
// tiled layout (mx_device.h) keeps exactly these operands in whole 1 KB runs
// and the scale bytes of four K steps in one dword a lane.  The activation
// is the A operand (result rows = tokens): a lane holds output column
// l % 32, and a store covers 128 bytes of two rows.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_common.h"
#include "mx_device.h"
#include "rz_internal.h"

namespace rz {
namespace {
using namespace mx;
using gemm::kNonTemporal;
using gemm::kXcds;
using gemm::v16f;
using gemm::v4i;
using gemm::v8i;

// acc += a w for one 32 x 32 block and 64 columns; Q: the byte of the scale
// dwords.
template <int Q>
__device__ __forceinline__ v16f mma(u32x4 a, u32x4 w, v16f acc, uint32_t sa, uint32_t sw) {
    const v4i a4 = __builtin_bit_cast(v4i, a), w4 = __builtin_bit_cast(v4i, w);
    const v8i a8 = __builtin_shufflevector(a4, a4, 0, 1, 2, 3, -1, -1, -1, -1);
    const v8i w8 = __builtin_shufflevector(w4, w4, 0, 1, 2, 3, -1, -1, -1, -1);
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a8, w8, acc, 4, 4, Q, (int)sa, Q, (int)sw);
}

struct Args {
    const uint8_t* a_codes;
    const uint8_t* a_scales;
    MxWeights w;
    float* y;          // fp32 output, or
    uint8_t* h_codes;  // tiled MXFP4 output
    uint8_t* h_scales;
    uint32_t m, n, k;
    uint32_t tiles_m, tiles_n, group_m;
};

enum Out { kOutF32 = 0, kOutMX = 1 };

__host__ __device__ __forceinline__ uint32_t min_u32(uint32_t a, uint32_t b) { return a < b ? a : b; }

// A row group's codes or scales as a buffer: `per` bytes for each 256-column slab.
__device__ __forceinline__ const uint8_t* group_base(const uint8_t* base, uint32_t grp, uint32_t slabs, uint32_t per) {
    return base + (uint64_t)grp * slabs * per;
}

// The 32 x 32 block v (v[e]: row 8 (e/4) + 4 (lane/32) + e%4, column lane%32)
// of row group grp and columns col0 .. + 31 to y; rows and columns outside
// [0, m) x [0, n) are dropped (rows by the buffer's range).
__device__ __forceinline__ void store_f32(const Args& P, const float (&v)[16], uint32_t grp, uint32_t col0, uint32_t lane) {
    const uint32_t row0 = grp * 32u;
    if (row0 >= P.m) return;
    const uint32_t rows = min_u32(32u, P.m - row0);
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(P.y + (uint64_t)row0 * P.n, (short)0,
                                                                        (int)(rows * P.n * 4u), 0x00020000);
    const uint32_t col = col0 + (lane & 31u);
    if (col >= P.n) return;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const uint32_t row = 8u * (e >> 2) + 4u * (lane >> 5) + (e & 3);
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[e]), rs, (row * P.n + col) * 4u, 0, kNonTemporal);
    }
}

// The same block as tiled MXFP4: through this wave's 4 KB of LDS, so that a
// quad of lanes gets a row's 32 values.  Pad rows are products of zero rows
// and quantise to zero.
__device__ __forceinline__ void store_mx(const Args& P, const float (&v)[16], uint32_t grp, uint32_t col0, uint32_t lane,
                                         float* lds) {
    if (grp * 32u >= P.m) return;
#pragma unroll
    for (int e = 0; e < 16; ++e) lds[(8 * (e >> 2) + 4 * (lane >> 5) + (e & 3)) * 32 + (lane & 31)] = v[e];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const uint32_t blk = col0 / 32u, part = lane & 3u;
    uint8_t* codes = P.h_codes + ((uint64_t)grp * (P.n / 64u) + blk / 2u) * 1024u + (blk & 1u) * 512u;
    uint8_t* scales = P.h_scales + ((uint64_t)grp * (P.n / 256u) + blk / 8u) * 256u + (blk & 1u) * 128u + (blk / 2u) % 4u;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t row = 16u * i + (lane >> 2);
        float x[8];
        *reinterpret_cast<f32x4*>(x) = *reinterpret_cast<const f32x4*>(lds + row * 32 + part * 8);
        *reinterpret_cast<f32x4*>(x + 4) = *reinterpret_cast<const f32x4*>(lds + row * 32 + part * 8 + 4);
        uint32_t byte;
        const uint32_t c = quantise8(x, byte);
        *reinterpret_cast<uint32_t*>(codes + row * 16u + part * 4u) = c;
        if (part == 0) scales[row * 4u] = (uint8_t)byte;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// ---------------------------------------------------------------------------
// Tile kernel: 128 tokens x 256 weight rows a workgroup (gated: 128 gate and
// 128 up rows), four waves along the weight rows, each 128 x 64.
//
// The four waves read the same activation blocks, so those go through LDS
// (two 16 KB stages of 256 columns, one barrier each); a weight block is
// used by one wave only and goes from the L2 straight to registers, a step
// ahead.  Two workgroups share a CU: while one stores its tile or waits, the
// other computes.
// ---------------------------------------------------------------------------
constexpr int kTM = 4;             // activation blocks of 32 rows
constexpr int kWN = 2;             // weight blocks a wave
constexpr int kStage = kTM * 4096; // one 256-column step of the activation rows

template <bool GATED, int OUT>
__global__ __launch_bounds__(256, 2) void mx_gemm_tile_kernel(Args P) {
    __shared__ __attribute__((aligned(16))) uint8_t smem[2][kStage];
    const uint32_t tid = threadIdx.x, lane = tid & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t slabs = P.k / 256u;

    // workgroup -> tile: the dispatcher sends workgroup w to XCD w % 8; each
    // XCD takes a contiguous run of tiles, m fastest in groups of group_m
    const uint32_t T = P.tiles_m * P.tiles_n, x = blockIdx.x % kXcds, j0 = blockIdx.x / kXcds;
    const uint32_t t = x * (T / kXcds) + min_u32(x, T % kXcds) + j0;
    const uint32_t per = P.group_m * P.tiles_n, gi = t / per, first = gi * P.group_m;
    const uint32_t gm = min_u32(P.group_m, P.tiles_m - first), tin = t - gi * per;
    const uint32_t tn = tin / gm, tm = first + tin % gm;

    const uint32_t a_groups = pad32(P.m) / 32u, w_groups = pad32(P.n) / 32u;
    uint32_t wg[kWN], wcol[kWN];  // each weight block's row group, first output column
    const uint8_t *wc[kWN], *ws[kWN];
#pragma unroll
    for (int i = 0; i < kWN; ++i) {
        wg[i] = GATED ? tn * 4u + wave : tn * 8u + wave * 2u + i;
        wcol[i] = wg[i] * 32u;
        const uint32_t g = min_u32(wg[i], w_groups - 1u);  // past the last group: any rows, not stored
        wc[i] = group_base(P.w.codes[GATED ? i : 0], g, slabs, 4096u) + lane * 16u;
        ws[i] = group_base(P.w.scales[GATED ? i : 0], g, slabs, 256u) + lane * 4u;
    }
    const uint8_t *ac[kTM], *as[kTM];
#pragma unroll
    for (int j = 0; j < kTM; ++j) {
        const uint32_t g = min_u32(tm * kTM + j, a_groups - 1u);
        ac[j] = group_base(P.a_codes, g, slabs, 4096u) + tid * 16u;
        as[j] = group_base(P.a_scales, g, slabs, 256u) + lane * 4u;
    }

    v16f acc[kWN][kTM] = {};
    u32x4 st[kTM];             // activation rows on their way to LDS
    u32x4 w[2][kWN][4];        // weight blocks of this step and the next
    uint32_t sa[2][kTM], sw[2][kWN];

    auto load_a = [&](uint32_t s) {
#pragma unroll
        for (int j = 0; j < kTM; ++j) st[j] = *reinterpret_cast<const u32x4*>(ac[j] + (uint64_t)s * 4096u);
    };
    auto put_a = [&](uint8_t* dst) {
#pragma unroll
        for (int j = 0; j < kTM; ++j) *reinterpret_cast<u32x4*>(dst + j * 4096 + tid * 16) = st[j];
    };
    auto load_w = [&](int b, uint32_t s) {
#pragma unroll
        for (int i = 0; i < kWN; ++i) {
            sw[b][i] = *reinterpret_cast<const uint32_t*>(ws[i] + (uint64_t)s * 256u);
#pragma unroll
            for (int q = 0; q < 4; ++q)
                w[b][i][q] = *reinterpret_cast<const u32x4*>(wc[i] + (uint64_t)s * 4096u + q * 1024);
        }
#pragma unroll
        for (int j = 0; j < kTM; ++j) sa[b][j] = *reinterpret_cast<const uint32_t*>(as[j] + (uint64_t)s * 256u);
    };
    auto step = [&](int b, uint32_t s) {
        __syncthreads();
        const uint8_t* cur = smem[b];
        load_w(b ^ 1, min_u32(s + 1u, slabs - 1u));
        auto part = [&](auto qc) {
            constexpr int q = decltype(qc)::value;
#pragma unroll
            for (int j = 0; j < kTM; ++j) {
                const u32x4 a = *reinterpret_cast<const u32x4*>(cur + j * 4096 + q * 1024 + lane * 16);
#pragma unroll
                for (int i = 0; i < kWN; ++i) acc[i][j] = mma<q>(a, w[b][i][q], acc[i][j], sa[b][j], sw[b][i]);
            }
        };
        part(std::integral_constant<int, 0>{});
        part(std::integral_constant<int, 1>{});
        put_a(smem[b ^ 1]);
        load_a(min_u32(s + 2u, slabs - 1u));
        part(std::integral_constant<int, 2>{});
        part(std::integral_constant<int, 3>{});
    };
    load_a(0);
    load_w(0, 0);
    put_a(smem[0]);
    load_a(min_u32(1u, slabs - 1u));
    for (uint32_t s = 0; s < slabs; s += 2) {
        step(0, s);
        if (s + 1 < slabs) step(1, s + 1);
    }

    if constexpr (OUT == kOutMX) __syncthreads();  // the stages become the waves' exchange space
#pragma unroll
    for (int j = 0; j < kTM; ++j) {
        float v[16];
        if constexpr (GATED) {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = silu(acc[0][j][e]) * acc[kWN - 1][j][e];
            if constexpr (OUT == kOutMX) {
                if (wcol[0] < P.n)
                    store_mx(P, v, tm * kTM + j, wcol[0], lane, reinterpret_cast<float*>(smem[0]) + wave * 1024);
            } else {
                store_f32(P, v, tm * kTM + j, wcol[0], lane);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kWN; ++i) {
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = acc[i][j][e];
                store_f32(P, v, tm * kTM + j, wcol[i], lane);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Split kernel, for few tiles: 32 TM tokens x 32 weight rows (gated: 32 gate
// and 32 up rows) a workgroup, whose eight waves share the K range (256
// columns a turn) and add their sums through LDS in a fixed order.  Every
// operand goes straight to registers; the activation rows come from the L2.
// ---------------------------------------------------------------------------
constexpr int kSplit = 8;

template <int TM, int G, int OUT>
__global__ __launch_bounds__(64 * kSplit) void mx_gemm_split_kernel(Args P) {
    __shared__ __attribute__((aligned(16))) float sums[kSplit][G * TM][16][64];
    const uint32_t tid = threadIdx.x, lane = tid & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t slabs = P.k / 256u;
    const uint32_t tn = blockIdx.x % P.tiles_n, tm = blockIdx.x / P.tiles_n;
    const uint32_t a_groups = pad32(P.m) / 32u;
    const uint8_t *wc[G], *ws[G], *ac[TM], *as[TM];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        wc[g] = group_base(P.w.codes[g], tn, slabs, 4096u) + lane * 16u;
        ws[g] = group_base(P.w.scales[g], tn, slabs, 256u) + lane * 4u;
    }
#pragma unroll
    for (int j = 0; j < TM; ++j) {
        const uint32_t g = min_u32(tm * TM + j, a_groups - 1u);
        ac[j] = group_base(P.a_codes, g, slabs, 4096u) + lane * 16u;
        as[j] = group_base(P.a_scales, g, slabs, 256u) + lane * 4u;
    }
    v16f acc[G][TM] = {};
    for (uint32_t s = wave; s < slabs; s += kSplit) {
        u32x4 a[TM][4], w[G][4];
        uint32_t sa[TM], sw[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                w[g][q] = *reinterpret_cast<const u32x4*>(wc[g] + (uint64_t)s * 4096u + q * 1024);
            sw[g] = *reinterpret_cast<const uint32_t*>(ws[g] + (uint64_t)s * 256u);
        }
#pragma unroll
        for (int j = 0; j < TM; ++j) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                a[j][q] = *reinterpret_cast<const u32x4*>(ac[j] + (uint64_t)s * 4096u + q * 1024);
            sa[j] = *reinterpret_cast<const uint32_t*>(as[j] + (uint64_t)s * 256u);
        }
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                acc[g][j] = mma<0>(a[j][0], w[g][0], acc[g][j], sa[j], sw[g]);
                acc[g][j] = mma<1>(a[j][1], w[g][1], acc[g][j], sa[j], sw[g]);
                acc[g][j] = mma<2>(a[j][2], w[g][2], acc[g][j], sa[j], sw[g]);
                acc[g][j] = mma<3>(a[j][3], w[g][3], acc[g][j], sa[j], sw[g]);
            }
    }
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int j = 0; j < TM; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) sums[wave][g * TM + j][e][lane] = acc[g][j][e];
    __syncthreads();
    // the block's 16 x TM register rows, two a wave (TM = 1) or more
    constexpr int kPer = 16 * TM / kSplit;
    float v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = (int)wave * kPer + i;
        float s[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            s[g] = 0.0f;
#pragma unroll
            for (int u = 0; u < kSplit; ++u) s[g] += sums[u][g * TM + e / 16][e % 16][lane];
        }
        if constexpr (G == 2)
            v[i] = silu(s[0]) * s[G - 1];
        else
            v[i] = s[0];
    }
    const uint32_t col = tn * 32u + (lane & 31u);
    if constexpr (OUT == kOutF32) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const uint32_t e = wave * kPer + i;
            const uint32_t row = (tm * TM + e / 16u) * 32u + 8u * ((e & 15u) >> 2) + 4u * (lane >> 5) + (e & 3u);
            if (row < P.m && col < P.n) P.y[(uint64_t)row * P.n + col] = v[i];
        }
    } else {
        __syncthreads();
        float* blk = &sums[0][0][0][0];  // TM row groups of 32 x 32, as store_mx reads them
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const uint32_t e = wave * kPer + i;
            blk[(e / 16u) * 1024u + (8u * ((e & 15u) >> 2) + 4u * (lane >> 5) + (e & 3u)) * 32u + (lane & 31u)] = v[i];
        }
        __syncthreads();
        if (wave < TM) {  // one row group a wave
            float b[16];
            const float* src = blk + wave * 1024;
#pragma unroll
            for (int e = 0; e < 16; ++e) b[e] = src[(8 * (e >> 2) + 4 * (lane >> 5) + (e & 3)) * 32 + (lane & 31)];
            store_mx(P, b, tm * TM + wave, tn * 32u, lane, blk + wave * 1024);
        }
    }
}

template <bool GATED, int OUT>
void launch_as(Args P, hipStream_t st) {
    const uint32_t a_groups = pad32(P.m) / 32u, w_groups = pad32(P.n) / 32u;
    const uint32_t wn = GATED ? 4u : 8u;  // output blocks of 32 columns a tile
    P.tiles_m = (a_groups + kTM - 1) / kTM;
    P.tiles_n = (w_groups + wn - 1) / wn;
    if ((uint64_t)P.tiles_m * P.tiles_n >= 192u) {
        P.group_m = min_u32(P.tiles_m, 8u);
        mx_gemm_tile_kernel<GATED, OUT><<<P.tiles_m * P.tiles_n, 256, 0, st>>>(P);
        return;
    }
    constexpr int G = GATED ? 2 : 1;
    const uint32_t tm = a_groups > 1 ? 2u : 1u;
    P.tiles_n = w_groups;
    P.tiles_m = (a_groups + tm - 1) / tm;
    if (tm == 1)
        mx_gemm_split_kernel<1, G, OUT><<<P.tiles_m * P.tiles_n, 64 * kSplit, 0, st>>>(P);
    else
        mx_gemm_split_kernel<2, G, OUT><<<P.tiles_m * P.tiles_n, 64 * kSplit, 0, st>>>(P);
}

}  // namespace

hipError_t launch_mx_gemm(const uint8_t* a_codes, const uint8_t* a_scales, uint32_t m, const MxWeights& W, bool gated,
                          uint32_t n, uint32_t k, float* y, uint8_t* h_codes, uint8_t* h_scales, hipStream_t st) {
    Args P = {};
    P.a_codes = a_codes;
    P.a_scales = a_scales;
    P.w = W;
    P.y = y;
    P.h_codes = h_codes;
    P.h_scales = h_scales;
    P.m = m;
    P.n = n;
    P.k = k;
    if (!gated)
        launch_as<false, kOutF32>(P, st);
    else if (h_codes)
        launch_as<true, kOutMX>(P, st);
    else
        launch_as<true, kOutF32>(P, st);
    return hipGetLastError();
}

}  // namespace rz
