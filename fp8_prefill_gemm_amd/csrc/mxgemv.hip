// Small-batch products straight from an MXFP4 weight, fp32 in and out:
//
//     y[i][j] = sum_kk x[i][kk] * w[j][kk]                       (1 <= m <= 8)
//     h[i][j] = silu(x wg^T)[i][j] * (x wu^T)[i][j]              (gated form)
//
// the single-token companions of mxgemm.hip: x is not quantised, the weight
// is read once at 17/32 B a value, which bounds the kernel at one token.  A
// workgroup owns 16 rows; its waves share the 256-column slabs.  Lane 32 q +
// 16 h + r holds row r's blocks of half h in the 64-column slabs q and q + 2,
// 16 bytes a load.  A wave puts its slab of x into LDS (nobody else reads it:
// no barrier), from where the rows take each value at once.  E2M1 codes
// become floats two at a time (v_cvt_scalef32_pk_f32_fp4); the 32 products of
// a block are summed before its scale is applied, everything in fp32.  The
// order of every sum is fixed.
//
// Measured, one token: 4608 x 3584 (8.8 MB) 4.5 us, mostly launch and the
// first load's latency; 18944 x 3584 8.6 us, 4.2 TB/s; gated 18944 x 3584
// (72 MB) 15.7 us, 4.6 TB/s, the rate of a large copy.  Workgroups of 32
// rows: 4.7, 9.9 and 17.4 us; lanes with 8 values of four rows, which read x
// four times less often but load 4 bytes at a time: 5.2, 13.6 and 31.  With
// more tokens the multiply-adds bound it (8 tokens, 18944 x 3584: 31 us; two
// rows a lane, half the reads of x, 33 us).
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

constexpr int kRun = 36;          // floats a 32-column run of x takes in LDS: the runs start in different banks
constexpr int kSlabX = 8 * kRun;  // floats of a slab of one token

template <int M, int G>
__global__ __launch_bounds__(1024) void mx_gemv_kernel(MxWeights W, uint32_t n, uint32_t k, const float* __restrict__ x,
                                                       float* __restrict__ y) {
    // [waves][M][kSlabX], then [waves][G][M][16] in the same place
    extern __shared__ __attribute__((aligned(16))) float lds[];
    const uint32_t lane = threadIdx.x & 63u, waves = blockDim.x >> 6;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t r = lane & 15u, h = (lane >> 4) & 1u, q0 = lane >> 5;
    const uint32_t slabs = k / 256u;
    const uint32_t grp = blockIdx.x / 2u, row = (blockIdx.x % 2u) * 16u + r;  // row of its group
    const uint32_t coff = q0 * 1024u + h * 512u + row * 16u, soff = h * 128u + row * 4u;
    float* xs = lds + wave * (M * kSlabX);
    float acc[G][M] = {};
    for (uint32_t s = wave; s < slabs; s += waves) {
        const uint64_t tile = (uint64_t)grp * slabs + s;
        u32x4 w[G][2];
        uint32_t sc[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
                w[g][t] = *reinterpret_cast<const u32x4*>(W.codes[g] + tile * 4096u + coff + t * 2048);
            sc[g] = *reinterpret_cast<const uint32_t*>(W.scales[g] + tile * 256u + soff) >> (8u * q0);
        }
#pragma unroll
        for (int i = 0; i < M; ++i)
            *reinterpret_cast<f32x4*>(xs + i * kSlabX + (lane >> 3) * kRun + (lane & 7u) * 4u) =
                *reinterpret_cast<const f32x4*>(x + (uint64_t)i * k + s * 256u + lane * 4u);
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            float d[G][M] = {};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float v[G][8];
#pragma unroll
                for (int g = 0; g < G; ++g) decode8(w[g][t][c], v[g]);
#pragma unroll
                for (int i = 0; i < M; ++i) {
                    const float* xp = xs + i * kSlabX + (2 * (q0 + 2 * t) + h) * kRun + 8 * c;
                    const f32x4 lo = *reinterpret_cast<const f32x4*>(xp), hi = *reinterpret_cast<const f32x4*>(xp + 4);
#pragma unroll
                    for (int g = 0; g < G; ++g)
#pragma unroll
                        for (int e = 0; e < 8; ++e) d[g][i] = __builtin_fmaf(v[g][e], e < 4 ? lo[e & 3] : hi[e & 3], d[g][i]);
                }
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const float f = scale_value((sc[g] >> (16 * t)) & 0xFFu);
#pragma unroll
                for (int i = 0; i < M; ++i) acc[g][i] = __builtin_fmaf(d[g][i], f, acc[g][i]);
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();  // x is no longer needed
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int i = 0; i < M; ++i) {
            float v = acc[g][i];
            v += __shfl_xor(v, 16, kWave);
            v += __shfl_xor(v, 32, kWave);
            if (lane < 16u) lds[((wave * G + g) * M + i) * 16 + lane] = v;
        }
    __syncthreads();
    for (uint32_t t = threadIdx.x; t < 16u * M; t += blockDim.x) {
        float v[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            v[g] = 0.0f;
            for (uint32_t u = 0; u < waves; ++u) v[g] += lds[(u * G + g) * M * 16 + t];
        }
        const uint32_t j = blockIdx.x * 16u + t % 16u;
        if (j < n) y[(uint64_t)(t / 16u) * n + j] = G == 2 ? silu(v[0]) * v[G - 1] : v[0];
    }
}

// Waves: as many as share the slabs evenly, up to 16 when there is at most
// one workgroup a CU, else up to 8, so that several workgroups take turns on
// one (us, up to 16 / up to 8 waves: 3584 x 18944, 224 workgroups, 8.9 /
// 10.4; 18944 x 3584, 1184 workgroups, 9.9 / 8.6, gated 19.6 / 15.7).
template <int M, int G>
hipError_t launch_m(const MxWeights& W, uint32_t n, uint32_t k, const float* x, float* y, hipStream_t st) {
    const uint32_t slabs = k / 256u, grid = pad32(n) / 16u, cap = grid <= 256u ? 16u : 8u;
    const uint32_t turns = (slabs + cap - 1u) / cap, waves = (slabs + turns - 1u) / turns;
    const size_t lds = (size_t)waves * M * kSlabX * sizeof(float);  // more than the sums take
    static_assert(kSlabX >= 2 * 16, "the sums' place");
    mx_gemv_kernel<M, G><<<grid, 64u * waves, lds, st>>>(W, n, k, x, y);
    return hipGetLastError();
}

template <int G>
hipError_t launch(const MxWeights& W, uint32_t n, uint32_t k, const float* x, uint32_t m, float* y, hipStream_t st) {
    switch (m) {
        case 1: return launch_m<1, G>(W, n, k, x, y, st);
        case 2: return launch_m<2, G>(W, n, k, x, y, st);
        case 3: return launch_m<3, G>(W, n, k, x, y, st);
        case 4: return launch_m<4, G>(W, n, k, x, y, st);
        case 5: return launch_m<5, G>(W, n, k, x, y, st);
        case 6: return launch_m<6, G>(W, n, k, x, y, st);
        case 7: return launch_m<7, G>(W, n, k, x, y, st);
        case 8: return launch_m<8, G>(W, n, k, x, y, st);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_mx_gemv(const MxWeights& W, bool gated, uint32_t n, uint32_t k, const float* x, uint32_t m, float* y,
                          hipStream_t st) {
    return gated ? launch<2>(W, n, k, x, m, y, st) : launch<1>(W, n, k, x, m, y, st);
}

}  // namespace rz
