// Small-batch products straight from an MXFP4 weight, fp32 in and out:
//
//     y[i][j] = sum_kk x[i][kk] * w[j][kk]                       (1 <= m <= 8)
//     h[i][j] = silu(x wg^T)[i][j] * (x wu^T)[i][j]              (gated form)
//
// the single-token companions of mxgemm.hip: x is not quantised, the weight
// is read once at 17/32 B a value, which bounds the kernel (a 4608 x 3584
// weight: 8.8 MB).  A workgroup owns one group of 32 rows; its waves share
// the 256-column slabs.  In a slab, lane 8 r + 4 h + p takes columns 32 h +
// 8 p .. + 7 of rows r, r + 8, r + 16, r + 24, so each x value it reads
// serves four rows (twice that in the gated form), and a load covers 256
// bytes.  E2M1 codes become floats two at a time (v_cvt_scalef32_pk_f32_fp4);
// the eight products of a run are summed before the block's scale is
// applied, everything in fp32.  The order of every sum is fixed.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_device.h"
#include "rz_device.h"
#include "rz_internal.h"

namespace rz {
namespace {
using namespace mx;

// 2^(byte - 127): exact for every byte (byte 0 is a subnormal, 255 NaN).
__device__ __forceinline__ float scale_value(uint32_t byte) { return times_scale(1.0f, byte); }

// Sum over the eight lanes 8i .. 8i+7; every lane gets it.
__device__ __forceinline__ float oct_sum(float v) {
    auto dpp = [](float x, auto ctrl) {
        return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(x), decltype(ctrl)::value, 0xF, 0xF, true));
    };
    v += dpp(v, std::integral_constant<int, 0xB1>{});
    v += dpp(v, std::integral_constant<int, 0x4E>{});
    v += dpp(v, std::integral_constant<int, 0x141>{});  // row_half_mirror: the other quad
    return v;
}

template <int M, int G>
__global__ __launch_bounds__(1024) void mx_gemv_kernel(MxWeights W, uint32_t n, uint32_t k, const float* __restrict__ x,
                                                       float* __restrict__ y) {
    extern __shared__ float part[];  // [waves][G][M][32]
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const uint32_t r = lane >> 3, h = (lane >> 2) & 1u, p = lane & 3u;
    const uint32_t slabs = k / 256u;
    const uint32_t coff = h * 512u + r * 16u + p * 4u, soff = h * 128u + r * 4u;
    float acc[G][4][M] = {};
    for (uint32_t s = wave; s < slabs; s += waves) {
        const uint64_t tile = (uint64_t)blockIdx.x * slabs + s;
        uint32_t w[G][4][4], sc[G][4];
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int o = 0; o < 4; ++o) {
                sc[g][o] = *reinterpret_cast<const uint32_t*>(W.scales[g] + tile * 256u + soff + 32 * o);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    w[g][o][q] = *reinterpret_cast<const uint32_t*>(W.codes[g] + tile * 4096u + q * 1024 + coff + 128 * o);
            }
        const float* xp = x + s * 256u + 32u * h + 8u * p;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            f32x4 xv[M][2];
#pragma unroll
            for (int i = 0; i < M; ++i) {
                xv[i][0] = *reinterpret_cast<const f32x4*>(xp + (uint64_t)i * k + 64 * q);
                xv[i][1] = *reinterpret_cast<const f32x4*>(xp + (uint64_t)i * k + 64 * q + 4);
            }
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int o = 0; o < 4; ++o) {
                    float v[8];
                    decode8(w[g][o][q], v);
                    const float xs = scale_value((sc[g][o] >> (8 * q)) & 0xFFu);
#pragma unroll
                    for (int i = 0; i < M; ++i) {
                        float d = v[0] * xv[i][0][0];
#pragma unroll
                        for (int e = 1; e < 8; ++e) d = __builtin_fmaf(v[e], xv[i][e >> 2][e & 3], d);
                        acc[g][o][i] = __builtin_fmaf(d, xs, acc[g][o][i]);
                    }
                }
        }
    }
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int o = 0; o < 4; ++o)
#pragma unroll
            for (int i = 0; i < M; ++i) {
                const float v = oct_sum(acc[g][o][i]);
                if ((lane & 7u) == 0) part[((wave * G + g) * M + i) * 32 + 8 * o + r] = v;
            }
    __syncthreads();
    for (uint32_t t = threadIdx.x; t < 32u * M; t += blockDim.x) {
        float v[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            v[g] = 0.0f;
            for (uint32_t u = 0; u < waves; ++u) v[g] += part[(u * G + g) * M * 32 + t];
        }
        const uint32_t row = blockIdx.x * 32u + (t & 31u);
        if (row < n) {
            if constexpr (G == 2)
                y[(uint64_t)(t >> 5) * n + row] = silu(v[0]) * v[G - 1];
            else
                y[(uint64_t)(t >> 5) * n + row] = v[0];
        }
    }
}

template <int G>
hipError_t launch(const MxWeights& W, uint32_t n, uint32_t k, const float* x, uint32_t m, float* y, hipStream_t st) {
    const uint32_t slabs = k / 256u;
    // as many waves as share the slabs evenly, at most 16
    const uint32_t waves = (slabs + (slabs + 15u) / 16u - 1u) / ((slabs + 15u) / 16u);
    const dim3 grid(pad32(n) / 32u), block(64u * waves);
    const size_t lds = (size_t)waves * G * m * 32 * sizeof(float);
    switch (m) {
#define RZ_CASE(M) case M: mx_gemv_kernel<M, G><<<grid, block, lds, st>>>(W, n, k, x, y); break;
        RZ_CASE(1) RZ_CASE(2) RZ_CASE(3) RZ_CASE(4) RZ_CASE(5) RZ_CASE(6) RZ_CASE(7) RZ_CASE(8)
#undef RZ_CASE
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_gemv(const MxWeights& W, bool gated, uint32_t n, uint32_t k, const float* x, uint32_t m, float* y,
                          hipStream_t st) {
    return gated ? launch<2>(W, n, k, x, m, y, st) : launch<1>(W, n, k, x, m, y, st);
}

}  // namespace rz
