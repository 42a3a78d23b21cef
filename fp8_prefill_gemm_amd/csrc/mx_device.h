// MXFP4 device helpers: the block codec and the tiled layout (gfx950, wave64).
//
// MXFP4 is the OCP microscaling format with E2M1 elements: 32 consecutive
// values of a row share one power of two X = 2^(byte - 127) (E8M0), each
// value is an E2M1 code of x / X (+-{0, .5, 1, 1.5, 2, 3, 4, 6}).  With a =
// max|x| of the block, byte = max(floor(log2 a) - 2 + 127, 0), so the largest
// value lies in [4, 8) and those past 6 saturate; codes round to nearest,
// ties to the even code, and keep the sign (of a zero too).  A block that
// holds a NaN or an infinity has byte 255, which the format defines as NaN,
// and zero codes: all 32 of its values read as NaN.
//
// Layout of a tensor [rows][k], k a multiple of 256, rows padded to a
// multiple of 32 (pad rows: zero codes and zero scale bytes):
//   codes  [rows/32][k/64][2][32][16]: 64-column slab, half of 32 columns,
//          row, the 16 bytes of that row's block (element 2i in the low
//          nibble of byte i).  One slab of a row group is 1 KB: exactly the
//          operand of one 32x32x64 MFMA, lane l's 16 bytes at 16 l.
//   scales [rows/32][k/256][2][32][4]: 256-column slab, half, row, the bytes
//          of the slab's four 64-column slabs: one dword a lane holds the
//          scales of four MFMAs, whose op_sel picks the byte.
// So operands go from memory to registers in whole 1 KB and 256 B runs, and
// through LDS without a swizzle.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace rz {
namespace mx {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kNanByte = 255;

// |x| as an ordered integer: NaN above infinity above every finite value.
__device__ __forceinline__ uint32_t mag_key(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// Scale byte of a block whose largest mag_key is `key`: the exponent field
// is floor(log2 a) + 127 for a normal a; fields up to 2 (subnormals among
// them) give byte 0.
__device__ __forceinline__ uint32_t scale_byte(uint32_t key) {
    const uint32_t e = key >> 23;
    return e == 255u ? kNanByte : (e > 2u ? e - 2u : 0u);
}

// The scale operand of the v_cvt_scalef32 conversions, of which they read the
// exponent field as an E8M0 byte: 2^(byte - 127), 255 NaN.
__device__ __forceinline__ float cvt_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// E2M1 codes of eight values divided by `scale`, value i in nibble i:
// nearest, ties to even, saturating.
__device__ __forceinline__ uint32_t encode8(const float (&v)[8], float scale) {
    uint32_t w = __builtin_nondeterministic_value(0u);  // every byte is written
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], scale, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], scale, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], scale, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], scale, 3);
}

// The eight E2M1 values of a word of codes, times `scale`: exact in fp32 (its
// subnormals too), infinite past its range, NaN where scale is NaN.
__device__ __forceinline__ void decode8(uint32_t w, float (&v)[8], float scale) {
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 0);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 1);
    const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 2);
    const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 3);
    v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
    v[4] = c.x; v[5] = c.y; v[6] = d.x; v[7] = d.y;
}

// Maximum over the four lanes of a quad (lanes 4i .. 4i+3), every lane gets it.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    const uint32_t a = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);  // lanes 1,0,3,2
    v = v > a ? v : a;
    const uint32_t b = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true);  // lanes 2,3,0,1
    return v > b ? v : b;
}

// One lane's eight values of a block that a quad shares: their codes, and
// the block's scale byte.
__device__ __forceinline__ uint32_t quantise8(const float (&x)[8], uint32_t& byte) {
    uint32_t key = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t a = mag_key(x[i]);
        key = key > a ? key : a;
    }
    byte = scale_byte(quad_max(key));
    const uint32_t w = encode8(x, cvt_scale(byte));
    return byte == kNanByte ? 0u : w;
}

// Element types of the reading-back kernels' outputs (rz_dtype).
enum OutType { kF32 = 0, kF16 = 1, kBF16 = 2 };

// Eight values to out[at .. at + 7] in type DT (fp16 and bf16: one rounding,
// to nearest even); at is a multiple of 8.
template <int DT>
__device__ __forceinline__ void store8(void* __restrict__ out, uint64_t at, const float (&v)[8]) {
    if constexpr (DT == kF32) {
        f32x4* o = reinterpret_cast<f32x4*>(static_cast<float*>(out) + at);
        o[0] = (f32x4){v[0], v[1], v[2], v[3]};
        o[1] = (f32x4){v[4], v[5], v[6], v[7]};
    } else if constexpr (DT == kF16) {
        typedef _Float16 h8 __attribute__((ext_vector_type(8)));
        h8 h;
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = (_Float16)v[i];
        *reinterpret_cast<h8*>(static_cast<_Float16*>(out) + at) = h;
    } else {
        typedef __bf16 b8 __attribute__((ext_vector_type(8)));
        b8 h;
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = (__bf16)v[i];
        *reinterpret_cast<b8*>(static_cast<__bf16*>(out) + at) = h;
    }
}

// silu(g) = g / (1 + e^-g) with the hardware exponential and reciprocal
// (each within 1 ulp; the rounding of g log2(e) adds |g| half ulps).
__device__ __forceinline__ float silu(float g) {
    return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504088896341f));
}

// ---- tiled layout

__host__ __device__ __forceinline__ uint32_t pad32(uint32_t rows) { return (rows + 31u) & ~31u; }

// A wave of the tiled quantisers covers 8 rows x 64 columns at a time: lane
// 8 r + 4 h + p holds columns 32 h + 8 p .. + 7 of row r, so eight lanes read
// 256 consecutive bytes of fp32, and a quad holds one block.
struct TileLane {
    uint32_t row, half, part;
    __device__ __forceinline__ TileLane() {
        const uint32_t t = threadIdx.x;
        row = t >> 3;  // 0..31 over the four waves of a workgroup
        half = (t >> 2) & 1u;
        part = t & 3u;
    }
    // byte offset of this lane's word of codes in a 1 KB slab
    __device__ __forceinline__ uint32_t code() const { return half * 512u + row * 16u + part * 4u; }
    // byte offset of the dword of scales in a 256-byte slab
    __device__ __forceinline__ uint32_t scale() const { return half * 128u + row * 4u; }
};

}  // namespace mx
}  // namespace rz
