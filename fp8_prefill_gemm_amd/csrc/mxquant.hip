// MXFP4 quantisation of activations and K-quant weights, and its inverse.
//
//     x -> per 32 consecutive values: scale byte, 32 E2M1 codes  (mx_device.h)
//
// Unlike the FP8 path there is no tensor-wide absmax: a block's scale depends
// on the block alone, so one pass reads the input once and writes codes and
// scales, 4 + 17/32 bytes a value (activations).  All three kernels are bound
// by memory.  A workgroup of four waves covers 32 rows x 256 columns, the
// unit of the tiled layout: each lane holds eight consecutive values of a
// block shared by its quad (two DPP maxima finish the block's absmax), reads
// are 256-byte runs of eight rows, each wave writes 128-byte runs of codes,
// and the four 64-column slabs of a lane are in flight together.
//
// Measured: quantising 2048 x 18944 31.0 us (5.7 TB/s), reading it back in
// bf16 and fp16 15.5 us (6.4 TB/s), in fp32 28.6 us; packing 18944 x 3584 from
// Q4_K 19.5 us in a trace, 18.5 back to back (4.0 TB/s; 19.9 with neighbouring
// tiles on different XCDs, whose caches then fetch the 144-byte blocks' shared
// lines twice), 3584 x 18944 from Q6_K 23.5 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_device.h"
#include "rz_device.h"
#include "rz_internal.h"

namespace rz {
namespace {
using namespace mx;

constexpr int kThreads = 256;

// Codes and scales of the 32 x 256 tile (grp, slab) from each lane's four
// runs of eight values.
__device__ __forceinline__ void store_tile(const float (&x)[4][8], const TileLane& t, uint8_t* __restrict__ codes,
                                           uint8_t* __restrict__ scales, uint64_t tile) {
    uint32_t word = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t byte;
        const uint32_t c = quantise8(x[q], byte);
        *reinterpret_cast<uint32_t*>(codes + tile * 4096u + q * 1024u + t.code()) = c;
        word |= byte << (8 * q);
    }
    if (t.part == 0) *reinterpret_cast<uint32_t*>(scales + tile * 256u + t.scale()) = word;
}

// x fp32 [m][k] -> codes, scales.  Workgroup b: row group b / slabs, 256-column
// slab b % slabs.  Rows at and past m quantise as zeros.
__global__ __launch_bounds__(kThreads) void mx_quant_kernel(const float* __restrict__ x, uint32_t m, uint32_t k,
                                                            uint32_t slabs, uint8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales) {
    const TileLane t;
    const uint64_t tile = blockIdx.x;
    const uint32_t grp = blockIdx.x / slabs, slab = blockIdx.x % slabs;
    const uint32_t row = grp * 32u + t.row;
    float v[4][8];
    if (row < m) {
        const float* p = x + (uint64_t)row * k + slab * 256u + t.half * 32u + t.part * 8u;
        f32x4 a[4][2];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            a[q][0] = *reinterpret_cast<const f32x4*>(p + 64 * q);
            a[q][1] = *reinterpret_cast<const f32x4*>(p + 64 * q + 4);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[q][i] = a[q][i >> 2][i & 3];
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[q][i] = 0.0f;
    }
    store_tile(v, t, codes, scales, tile);
}

// Eight bytes at a 2-byte-aligned address p (a field of a Q6_K block): the
// two or three dwords that hold them.  Every byte read lies in [p - 2, p + 10).
__device__ __forceinline__ u32x2 ld8_a2(const uint8_t* p) {
    const uint32_t sh = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 2u);
    const uint32_t* w = reinterpret_cast<const uint32_t*>(p - sh);
    const uint32_t a = w[0], b = w[1], c = w[sh ? 2 : 1];
    u32x2 r;
    r.x = __builtin_amdgcn_alignbyte(b, a, sh);
    r.y = __builtin_amdgcn_alignbyte(c, b, sh);
    return r;
}

// Eight bytes of w as floats.
__device__ __forceinline__ void bytes_f32(u32x2 w, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)((w[i >> 2] >> (8 * (i & 3))) & 0xFFu);
}

// A K-quant weight [n][k] -> codes, scales, without the fp32 weight in
// memory: each value is the correctly rounded fp32 that rz_dequant_f32 gives.
// A 256-column slab of a row is one super-block.  Q4_K: block (q, h) of the
// slab is sub-block 2q + h (low or high nibbles of quant bytes 32q .. 32q+31),
// so an MXFP4 block has one Q4_K scale and minimum.  Q6_K: half q/2, part
// 2(q%2) + h of the super-block.
template <int QT>
__global__ __launch_bounds__(kThreads) void mx_pack_kernel(const uint8_t* __restrict__ blocks, uint32_t n,
                                                           uint32_t slabs, uint8_t* __restrict__ codes,
                                                           uint8_t* __restrict__ scales) {
    const TileLane t;
    const uint32_t T = gridDim.x, xcd = blockIdx.x % 8u;
    const uint64_t tile = xcd * (T / 8u) + (xcd < T % 8u ? xcd : T % 8u) + blockIdx.x / 8u;
    const uint32_t grp = (uint32_t)tile / slabs, slab = (uint32_t)tile % slabs;
    const uint32_t row = grp * 32u + t.row;
    float v[4][8];
    if (row < n) {
        const uint64_t blk = (uint64_t)row * slabs + slab;
        if constexpr (QT == 12) {
            const uint8_t* b = blocks + blk * kQ4Bytes;
            const uint4 head = *reinterpret_cast<const uint4*>(b);
            u32x2 qs[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) qs[q] = *reinterpret_cast<const u32x2*>(b + 16 + 32 * q + 8 * t.part);
            const float d = half_bits_to_float(head.x & 0xFFFFu);
            const float dmin = half_bits_to_float(head.x >> 16);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t sc, mn;
                q4k_scale_min(head, 2 * q + (int)t.half, sc, mn);
                const float ds = d * (float)sc, o = dmin * (float)mn;
                const u32x2 w = (qs[q] >> (4u * t.half)) & 0x0F0F0F0Fu;
                float f[8];
                bytes_f32(w, f);
                // ds * f is exact, so the fused form rounds once (q4k_decode_unit)
#pragma unroll
                for (int i = 0; i < 8; ++i) v[q][i] = __builtin_fmaf(ds, f[i], -o);
            }
        } else {
            const uint8_t* b = blocks + blk * kQ6Bytes;
            const float d = half_bits_to_float(*reinterpret_cast<const uint16_t*>(b + 208));
            u32x2 ql[4], qh[2];
#pragma unroll
            for (int q = 0; q < 4; ++q)  // part p = 2(q%2) + h: ql run p%2 = h, nibble p/2 = q%2
                ql[q] = (q & 1) ? ql[q - 1] : ld8_a2(b + 64 * (q >> 1) + 32 * t.half + 8 * t.part);
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) qh[hh] = ld8_a2(b + 128 + 32 * hh + 8 * t.part);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t hh = q >> 1, p = 2u * (q & 1) + t.half;
                const float ds = d * (float)(int8_t)b[192 + 8 * hh + 2 * p + (t.part >> 1)];
                const u32x2 w = ((ql[q] >> (4u * (q & 1))) & 0x0F0F0F0Fu) | (((qh[hh] >> (2u * p)) & 0x03030303u) << 4u);
                float f[8];
                bytes_f32(w, f);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[q][i] = ds * (f[i] - 32.0f);
            }
        }
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[q][i] = 0.0f;
    }
    store_tile(v, t, codes, scales, tile);
}

// codes, scales -> [m][k] in fp32, fp16 or bf16.  E2M1 times a power of two
// is exact in fp32 and bf16; fp16 rounds once, to nearest even.
template <int DT>
__global__ __launch_bounds__(kThreads) void mx_dequant_kernel(const uint8_t* __restrict__ codes,
                                                              const uint8_t* __restrict__ scales, uint32_t m,
                                                              uint32_t k, uint32_t slabs, void* __restrict__ out) {
    const TileLane t;
    const uint64_t tile = blockIdx.x;
    const uint32_t grp = blockIdx.x / slabs, slab = blockIdx.x % slabs;
    const uint32_t row = grp * 32u + t.row;
    if (row >= m) return;
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) w[q] = *reinterpret_cast<const uint32_t*>(codes + tile * 4096u + q * 1024u + t.code());
    const uint32_t sc = *reinterpret_cast<const uint32_t*>(scales + tile * 256u + t.scale());
    const uint64_t at = (uint64_t)row * k + slab * 256u + t.half * 32u + t.part * 8u;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        float v[8];
        decode8(w[q], v, cvt_scale((sc >> (8 * q)) & 0xFFu));
        store8<DT>(out, at + 64u * q, v);
    }
}

}  // namespace

hipError_t launch_mx_quant(const float* x, uint32_t m, uint32_t k, uint8_t* codes, uint8_t* scales, hipStream_t st) {
    const uint32_t slabs = k / 256u;
    mx_quant_kernel<<<pad32(m) / 32u * slabs, kThreads, 0, st>>>(x, m, k, slabs, codes, scales);
    return hipGetLastError();
}

hipError_t launch_mx_pack(int qtype, const uint8_t* blocks, uint32_t n, uint32_t k, uint8_t* codes, uint8_t* scales,
                          hipStream_t st) {
    const uint32_t slabs = k / 256u, grid = pad32(n) / 32u * slabs;
    if (qtype == 12)
        mx_pack_kernel<12><<<grid, kThreads, 0, st>>>(blocks, n, slabs, codes, scales);
    else
        mx_pack_kernel<14><<<grid, kThreads, 0, st>>>(blocks, n, slabs, codes, scales);
    return hipGetLastError();
}

hipError_t launch_mx_dequant(const uint8_t* codes, const uint8_t* scales, uint32_t m, uint32_t k, int dtype, void* out,
                             hipStream_t st) {
    const uint32_t slabs = k / 256u, grid = pad32(m) / 32u * slabs;
    if (dtype == kF32)
        mx_dequant_kernel<kF32><<<grid, kThreads, 0, st>>>(codes, scales, m, k, slabs, out);
    else if (dtype == kF16)
        mx_dequant_kernel<kF16><<<grid, kThreads, 0, st>>>(codes, scales, m, k, slabs, out);
    else
        mx_dequant_kernel<kBF16><<<grid, kThreads, 0, st>>>(codes, scales, m, k, slabs, out);
    return hipGetLastError();
}

}  // namespace rz
