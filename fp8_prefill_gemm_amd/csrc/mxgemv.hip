// Small-batch products straight from an MXFP4 weight, fp32 in and out:
//
//     y[i][j] = sum_kk x[i][kk] * w[j][kk]                       (1 <= m <= 8)
//     h[i][j] = silu(x wg^T)[i][j] * (x wu^T)[i][j]              (gated form)
//
// the small-batch companions of mxgemm.hip: x is not quantised, the weight is
// read once at 17/32 B a value, which bounds the kernels.  One token goes to
// the vector units, two to eight to the bf16 matrix cores; sums are fp32 and
// have a fixed order.
//
// Measured, one token: 4608 x 3584 (8.8 MB) 4.5 us, mostly launch and the
// first load's latency; 18944 x 3584 8.6 us, 4.2 TB/s; gated 18944 x 3584
// (72 MB) 15.7 us, 4.6 TB/s, the rate of a large copy.  Four tokens 4.8, 10.5
// and 18.7 us, eight 7.1, 14.6 and 21.7.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_device.h"
#include "rz_device.h"
#include "rz_internal.h"

namespace rz {
namespace {
using namespace mx;

constexpr int kRun = 36;          // floats a 32-column run of x takes in LDS: the runs start in different banks
constexpr int kSlabX = 8 * kRun;  // floats of a slab

// One token.  A workgroup owns 16 rows; its waves share the 256-column slabs.
// Lane 32 q + 16 h + r holds row r's blocks of half h in the 64-column slabs
// q and q + 2, 16 bytes a load.  A wave puts its slab of x into LDS (nobody
// else reads it: no barrier), from where the rows take each value at once.
// v_cvt_scalef32_pk_f32_fp4 makes floats of two codes and the block's scale at
// a time.  Workgroups of 32 rows: 4.7, 9.9 and 17.4 us (the shapes above); lanes with 8 values of
// four rows, which read x four times less often but load 4 bytes at a time:
// 5.2, 13.6 and 31.
template <int G>
__global__ __launch_bounds__(1024) void mx_gemv_token_kernel(MxWeights W, uint32_t n, uint32_t k, const float* __restrict__ x,
                                                             float* __restrict__ y) {
    // [waves][kSlabX], then [waves][G][16] in the same place
    extern __shared__ __attribute__((aligned(16))) float lds[];
    const uint32_t lane = threadIdx.x & 63u, waves = blockDim.x >> 6;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t r = lane & 15u, h = (lane >> 4) & 1u, q0 = lane >> 5;
    const uint32_t slabs = k / 256u;
    const uint32_t grp = blockIdx.x / 2u, row = (blockIdx.x % 2u) * 16u + r;  // row of its group
    const uint32_t coff = q0 * 1024u + h * 512u + row * 16u, soff = h * 128u + row * 4u;
    float* xs = lds + wave * kSlabX;
    float acc[G] = {};
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
        *reinterpret_cast<f32x4*>(xs + (lane >> 3) * kRun + (lane & 7u) * 4u) =
            *reinterpret_cast<const f32x4*>(x + s * 256u + lane * 4u);
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            float f[G];
#pragma unroll
            for (int g = 0; g < G; ++g) f[g] = cvt_scale((sc[g] >> (16 * t)) & 0xFFu);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float* xp = xs + (2 * (q0 + 2 * t) + h) * kRun + 8 * c;
                const f32x4 lo = *reinterpret_cast<const f32x4*>(xp), hi = *reinterpret_cast<const f32x4*>(xp + 4);
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    float v[8];
                    decode8(w[g][t][c], v, f[g]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[g] = __builtin_fmaf(v[e], e < 4 ? lo[e & 3] : hi[e & 3], acc[g]);
                }
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();  // x is no longer needed
#pragma unroll
    for (int g = 0; g < G; ++g) {
        float v = acc[g];
        v += __shfl_xor(v, 16, kWave);
        v += __shfl_xor(v, 32, kWave);
        if (lane < 16u) lds[(wave * G + g) * 16 + lane] = v;
    }
    __syncthreads();
    if (threadIdx.x < 16u) {
        float v[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            v[g] = 0.0f;
            for (uint32_t u = 0; u < waves; ++u) v[g] += lds[(u * G + g) * 16 + threadIdx.x];
        }
        const uint32_t j = blockIdx.x * 16u + threadIdx.x;
        if (j < n) y[j] = G == 2 ? silu(v[0]) * v[G - 1] : v[0];
    }
}

// Waves: as many as share the slabs evenly, up to 16 when there is at most
// one workgroup a CU, else up to 8, so that several workgroups take turns on
// one (us, up to 16 / up to 8 waves: 3584 x 18944, 224 workgroups, 8.9 /
// 10.4; 18944 x 3584, 1184 workgroups, 9.9 / 8.6, gated 19.6 / 15.7).
uint32_t even_waves(uint32_t slabs, uint32_t cap) {
    const uint32_t turns = (slabs + cap - 1u) / cap;
    return (slabs + turns - 1u) / turns;
}

template <int G>
hipError_t launch_token(const MxWeights& W, uint32_t n, uint32_t k, const float* x, float* y, hipStream_t st) {
    const uint32_t grid = pad32(n) / 16u, waves = even_waves(k / 256u, grid <= 256u ? 16u : 8u);
    static_assert(kSlabX >= 2 * 16, "the sums' place");
    mx_gemv_token_kernel<G><<<grid, 64u * waves, waves * kSlabX * sizeof(float), st>>>(W, n, k, x, y);
    return hipGetLastError();
}

// Two to eight tokens.  On the vector units the multiply-adds would bound it
// (eight tokens, 18944 x 3584: 31 us, gated 52); here the bf16 matrix cores
// do them.  Truncation cuts an fp32 value into three bf16
// ones whose sum it is exactly (8 significant bits each, all of its sign), and
// an E2M1 code times its block's scale is a bf16 value, so the products are
// exact and their sums in fp32, as above.  The 3 M parts are the columns of a
// 16x16x32 MFMA's B operand, 16 weight rows its A operand: lane group l / 16
// of both holds the same 8 columns of K.  A wave splits its slab of x once
// into LDS for the workgroup's 32 rows (64 gated).  The matrix cores take
// bf16 subnormals as they are: only what x holds below 2^-133 is lost.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4v __attribute__((ext_vector_type(4)));

constexpr int kColBytes = 528;  // a part's 256 bf16 values and 16 bytes, so that 16 columns' reads hit all banks

// The upper halves of two words: {a's, b's} bf16 values by truncation.
__device__ __forceinline__ uint32_t high_halves(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }

template <int M, int G>
__global__ __launch_bounds__(1024) void mx_gemv_batch_kernel(MxWeights W, uint32_t n, uint32_t k, const float* __restrict__ x,
                                                            float* __restrict__ y) {
    constexpr int kCols = 3 * M, kTiles = (kCols + 15) / 16;
    // [waves][kCols][kColBytes], then floats [waves][G][32][kCols] in the same place
    extern __shared__ __attribute__((aligned(16))) uint8_t xs_all[];
    const uint32_t lane = threadIdx.x & 63u, waves = blockDim.x >> 6;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t r = lane & 15u, j = lane >> 4, h = j & 1u, q0 = j >> 1;
    const uint32_t slabs = k / 256u;
    const uint32_t coff = q0 * 1024u + h * 512u + r * 16u, soff = h * 128u + r * 4u;
    uint8_t* xs = xs_all + wave * (kCols * kColBytes);
    f32x4v acc[G][2][kTiles] = {};
    for (uint32_t s = wave; s < slabs; s += waves) {
        const uint64_t tile = (uint64_t)blockIdx.x * slabs + s;
        u32x4 w[G][2][2];
        uint32_t sc[G][2];
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    w[g][u][t] = *reinterpret_cast<const u32x4*>(W.codes[g] + tile * 4096u + coff + t * 2048 + u * 256);
                sc[g][u] = *reinterpret_cast<const uint32_t*>(W.scales[g] + tile * 256u + soff + u * 64) >> (8u * q0);
            }
#pragma unroll
        for (int i = 0; i < M; ++i) {
            const f32x4 v = *reinterpret_cast<const f32x4*>(x + (uint64_t)i * k + s * 256u + lane * 4u);
            uint32_t b[3][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                b[0][e] = __float_as_uint(v[e]);
                float rest = v[e] - __uint_as_float(b[0][e] & 0xFFFF0000u);
                rest = mag_key(v[e]) == 0x7F800000u ? 0.0f : rest;  // an infinity is its first part
                b[1][e] = __float_as_uint(rest);
                b[2][e] = __float_as_uint(rest - __uint_as_float(b[1][e] & 0xFFFF0000u));
            }
#pragma unroll
            for (int p = 0; p < 3; ++p)
                *reinterpret_cast<u32x2*>(xs + (p * M + i) * kColBytes + lane * 8u) =
                    (u32x2){high_halves(b[p][0], b[p][1]), high_halves(b[p][2], b[p][3])};
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const uint8_t* xb[kTiles];
#pragma unroll
        for (int c = 0; c < kTiles; ++c) {
            const uint32_t col = c * 16u + r < (uint32_t)kCols ? c * 16u + r : kCols - 1u;  // past the last: a copy, not stored
            xb[c] = xs + col * kColBytes + j * 64u;
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            float f[G][2];
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int u = 0; u < 2; ++u) f[g][u] = cvt_scale((sc[g][u] >> (16 * t)) & 0xFFu);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                bf16x8 b[kTiles];
#pragma unroll
                for (int z = 0; z < kTiles; ++z) b[z] = *reinterpret_cast<const bf16x8*>(xb[z] + t * 256 + c * 16);
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const bf16x2 a0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[g][u][t][c], f[g][u], 0);
                        const bf16x2 a1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[g][u][t][c], f[g][u], 1);
                        const bf16x2 a2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[g][u][t][c], f[g][u], 2);
                        const bf16x2 a3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[g][u][t][c], f[g][u], 3);
                        const bf16x8 a = {a0.x, a0.y, a1.x, a1.y, a2.x, a2.y, a3.x, a3.y};
#pragma unroll
                        for (int z = 0; z < kTiles; ++z)
                            acc[g][u][z] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b[z], acc[g][u][z], 0, 0, 0);
                    }
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();  // x is no longer needed
    float* sums = reinterpret_cast<float*>(xs_all);
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int z = 0; z < kTiles; ++z)
#pragma unroll
                for (int e = 0; e < 4; ++e)  // acc[..][e]: row 4 j + e, column r
                    if (z * 16u + r < (uint32_t)kCols)
                        sums[((wave * G + g) * 32 + 16 * u + 4 * j + e) * kCols + z * 16 + r] = acc[g][u][z][e];
    __syncthreads();
    for (uint32_t o = threadIdx.x; o < 32u * M; o += blockDim.x) {
        const uint32_t row = o & 31u, i = o >> 5;
        float v[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            v[g] = 0.0f;
            for (uint32_t u = 0; u < waves; ++u) {
                const float* p = sums + ((u * G + g) * 32 + row) * kCols + i;
                v[g] += p[0] + (p[M] + p[2 * M]);
            }
        }
        const uint32_t c = blockIdx.x * 32u + row;
        if (c < n) y[(uint64_t)i * n + c] = G == 2 ? silu(v[0]) * v[G - 1] : v[0];
    }
}

// Waves as above; an LDS part of 53 KB lets three workgroups share a CU
// (eight tokens, 18944 x 3584, with up to 160 / 80 / 53 / 40 KB: 20.6 / 17.2 /
// 14.6 / 16.5 us, gated 28.7 / 24.4 / 21.7 / 23.3).
template <int M, int G>
hipError_t launch_batch(const MxWeights& W, uint32_t n, uint32_t k, const float* x, float* y, hipStream_t st) {
    constexpr uint32_t kPart = 3 * M * kColBytes;  // LDS of a wave
    constexpr uint32_t kAlone = (160u << 10) / kPart, kShared = (53u << 10) / kPart;
    static_assert(kColBytes >= 2 * 32 * 4, "the sums' place");
    const uint32_t grid = pad32(n) / 32u;
    const uint32_t waves = even_waves(k / 256u, grid <= 256u ? (kAlone < 16u ? kAlone : 16u) : (kShared < 8u ? kShared : 8u));
    mx_gemv_batch_kernel<M, G><<<grid, 64u * waves, (size_t)waves * kPart, st>>>(W, n, k, x, y);
    return hipGetLastError();
}

template <int G>
hipError_t launch(const MxWeights& W, uint32_t n, uint32_t k, const float* x, uint32_t m, float* y, hipStream_t st) {
    switch (m) {
        case 1: return launch_token<G>(W, n, k, x, y, st);
        case 2: return launch_batch<2, G>(W, n, k, x, y, st);
        case 3: return launch_batch<3, G>(W, n, k, x, y, st);
        case 4: return launch_batch<4, G>(W, n, k, x, y, st);
        case 5: return launch_batch<5, G>(W, n, k, x, y, st);
        case 6: return launch_batch<6, G>(W, n, k, x, y, st);
        case 7: return launch_batch<7, G>(W, n, k, x, y, st);
        case 8: return launch_batch<8, G>(W, n, k, x, y, st);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_mx_gemv(const MxWeights& W, bool gated, uint32_t n, uint32_t k, const float* x, uint32_t m, float* y,
                          hipStream_t st) {
    return gated ? launch<2>(W, n, k, x, m, y, st) : launch<1>(W, n, k, x, m, y, st);
}

}  // namespace rz
