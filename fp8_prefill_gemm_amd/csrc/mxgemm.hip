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
// dwords.  The rows of the result (registers) are the first operand's.
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
    bool nt;  // every row of y starts on 64 bytes
};

enum Out { kOutF32 = 0, kOutMX = 1 };

__host__ __device__ __forceinline__ uint32_t min_u32(uint32_t a, uint32_t b) { return a < b ? a : b; }

// Workgroup -> tile: the dispatcher sends workgroup w to XCD w % 8; each XCD
// takes a contiguous run of tiles, m fastest in groups of group_m, so the
// workgroups that run together on one share rows through its L2.
__device__ __forceinline__ void tile_of(const Args& P, uint32_t& tm, uint32_t& tn) {
    const uint32_t T = P.tiles_m * P.tiles_n, x = blockIdx.x % kXcds;
    const uint32_t t = x * (T / kXcds) + min_u32(x, T % kXcds) + blockIdx.x / kXcds;
    const uint32_t per = P.group_m * P.tiles_n, first = t / per * P.group_m;
    const uint32_t gm = min_u32(P.group_m, P.tiles_m - first), in = t % per;
    tn = in / gm;
    tm = first + in % gm;
}

// f(integral_constant<0>) ... f(integral_constant<N - 1>).
template <int N, int I = 0, typename F>
__device__ __forceinline__ void for_each_index(F&& f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        for_each_index<N, I + 1>(f);
    }
}

// A row group's codes or scales as a buffer: `per` bytes for each 256-column slab.
__device__ __forceinline__ const uint8_t* group_base(const uint8_t* base, uint32_t grp, uint32_t slabs, uint32_t per) {
    return base + (uint64_t)grp * slabs * per;
}

// `count` row groups from `grp` on as a buffer (k <= RZ_MAX_GEMM_K keeps it
// under 2^31 bytes), and loads at a lane's offset plus a uniform one.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t group_rsrc(const uint8_t* base, uint32_t grp, uint32_t slabs, uint32_t per,
                                                             uint32_t count) {
    return gemm::tile_rsrc(group_base(base, grp, slabs, per), count * slabs * per);
}
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t rs, uint32_t vo, uint32_t so) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, vo, so, 0));
}
__device__ __forceinline__ uint32_t load4(__amdgpu_buffer_rsrc_t rs, uint32_t vo, uint32_t so) {
    return __builtin_amdgcn_raw_buffer_load_b32(rs, vo, so, 0);
}

// The 32 x 32 block v (v[e]: row 8 (e/4) + 4 (lane/32) + e%4, column lane%32)
// of row group grp and columns col0 .. + 31 to y; rows and columns outside
// [0, m) x [0, n) are dropped (rows by the buffer's range).  NT: non-temporal,
// the output is not kept in the caches.
template <bool NT>
__device__ __forceinline__ void store_rows(const Args& P, const float (&v)[16], uint32_t grp, uint32_t col0, uint32_t lane) {
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
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[e]), rs, (row * P.n + col) * 4u, 0, NT ? kNonTemporal : 0);
    }
}

// Non-temporal where every row of y starts on 64 bytes (2048 x 18944 x 3584:
// 77 us, 99 with ordinary stores); other widths leave parts of lines that the
// L2 has to put together first (2048 x 9000 x 3584: 47 us, non-temporal 59;
// 4096 x 9000 x 512: 46 and 81).  Wider runs store no faster: with a quad's values
// transposed for 16 bytes a lane, 128 of eight rows a store, the first shape
// takes 86 us, with the wave's halves swapped for 256 bytes of one row 81.
__device__ __forceinline__ void store_f32(const Args& P, const float (&v)[16], uint32_t grp, uint32_t col0, uint32_t lane) {
    if (P.nt)
        store_rows<true>(P, v, grp, col0, lane);
    else
        store_rows<false>(P, v, grp, col0, lane);
}

// Where the 16 bytes of codes and the scale byte of token row 0 of group grp,
// columns col0 .. + 31 of the MXFP4 output lie; row r's are 16 r and 4 r on.
struct MxBlock {
    uint8_t *codes, *scales;
    __device__ __forceinline__ MxBlock(const Args& P, uint32_t grp, uint32_t col0) {
        const uint32_t blk = col0 / 32u;
        codes = P.h_codes + ((uint64_t)grp * (P.n / 64u) + blk / 2u) * 1024u + (blk & 1u) * 512u;
        scales = P.h_scales + ((uint64_t)grp * (P.n / 256u) + blk / 8u) * 256u + (blk & 1u) * 128u + (blk / 2u) % 4u;
    }
};

// A 32 x 32 block in LDS (tokens x columns) quantised by one wave: a quad of
// lanes holds a row's block.  Pad rows become zeros whatever they hold (their
// products are zeros but for a NaN weight's).
__device__ __forceinline__ void quantise_block(const Args& P, uint32_t grp, uint32_t col0, uint32_t lane, const float* lds) {
    if (grp * 32u >= P.m) return;
    const uint32_t part = lane & 3u;
    const MxBlock o(P, grp, col0);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t row = 16u * i + (lane >> 2);
        float x[8];
        *reinterpret_cast<f32x4*>(x) = *reinterpret_cast<const f32x4*>(lds + row * 32 + part * 8);
        *reinterpret_cast<f32x4*>(x + 4) = *reinterpret_cast<const f32x4*>(lds + row * 32 + part * 8 + 4);
        uint32_t byte;
        uint32_t c = quantise8(x, byte);
        if (grp * 32u + row >= P.m) c = byte = 0u;
        *reinterpret_cast<uint32_t*>(o.codes + row * 16u + part * 4u) = c;
        if (part == 0) o.scales[row * 4u] = (uint8_t)byte;
    }
}

// A block with the tokens along the lanes quantised in registers: v[e] is
// token lane%32, column 8 (e/4) + 4 (lane/32) + e%4, so a lane and its
// partner 32 on hold a token's block.  They share its largest value, and each
// gets the other's codes of the eight bytes it stores.  Pad rows as above.
__device__ __forceinline__ void quantise_lanes(const Args& P, const float (&v)[16], uint32_t grp, uint32_t col0, uint32_t lane) {
    if (grp * 32u >= P.m) return;
    uint32_t key = 0;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const uint32_t a = mag_key(v[e]);
        key = key > a ? key : a;
    }
    const uint32_t other = (uint32_t)__shfl_xor((int)key, 32, 64);
    uint32_t byte = scale_byte(key > other ? key : other);
    float lo[8], hi[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        lo[e] = v[e];
        hi[e] = v[8 + e];
    }
    // 16 bits of codes for each e/4: columns 0-3 of eight (lane < 32) or 4-7
    const uint32_t w0 = encode8(lo, cvt_scale(byte)), w1 = encode8(hi, cvt_scale(byte));
    const bool upper = lane >= 32u;  // stores bytes 8..15
    const uint32_t got = (uint32_t)__shfl_xor((int)(upper ? w0 : w1), 32, 64);
    const uint32_t a = upper ? got : w0, b = upper ? w1 : got;  // the lower and the upper lane's codes
    u32x2 c = {(a & 0xFFFFu) | (b << 16), (a >> 16) | (b & 0xFFFF0000u)};
    if (byte == kNanByte) c = (u32x2){0u, 0u};
    if (grp * 32u + (lane & 31u) >= P.m) {
        c = (u32x2){0u, 0u};
        byte = 0u;
    }
    const MxBlock o(P, grp, col0);
    *reinterpret_cast<u32x2*>(o.codes + (lane & 31u) * 16u + (lane >> 5) * 8u) = c;
    if (!upper) o.scales[lane * 4u] = (uint8_t)byte;
}

// ---------------------------------------------------------------------------
// Tile kernel: 32 TM tokens (64 to 192) x 256 weight rows a workgroup (gated:
// 128 gate and 128 up rows of the same columns), four waves along the weight
// rows, each 32 TM x 64: TM activation blocks x kWN weight blocks.
//
// The four waves read the same activation blocks, so those go through LDS
// (two 16 KB stages of 256 columns, one barrier each); a weight block is
// used by one wave only and goes from the L2 straight to registers, a step
// ahead.  At 128 tokens, with 242 registers and 32 KB of LDS, two workgroups
// share a CU: while one stores its tile or waits, the other computes.
//
// Measured (random codes, M = 2048): gated N=18944 K=3584 133 us, 4.2
// PFLOP/s, of it 11 us that a copy without the store does not take, with MXFP4
// output 128; down N=3584 K=18944 64 us, 4.3 PFLOP/s.  What bounds it is the
// power limit: the socket draws its cap of 1400 W at 1.52 GHz (down 1.68), and
// with every code 1.0 the gated launches run at 6.0 and 6.6 PFLOP/s, at 2.35
// GHz.  The MFMA alone, on random register operands, reaches 6.6 (9.4 on
// constant ones).  Left to the compiler's own order, which moves
// the loads next to their use, 156 and 82 us.  A 256 x 256 tile of eight
// waves reads a third less through the L2 but has one workgroup a CU: 138
// and 85 us; one of four waves of 128 x 128, with half the LDS reads, takes 91
// us where this takes 73 (2048 x 18944 x 3584, not gated).  Three weight
// buffers, one workgroup a CU: 68 us for the down product.
// ---------------------------------------------------------------------------
constexpr int kWN = 2, kNW = 4;

template <int TM, bool GATED, int OUT>
__global__ __launch_bounds__(64 * kNW, TM > 4 ? 1 : 2) void mx_gemm_tile_kernel(Args P) {
    constexpr int kCols = GATED ? kWN / 2 : kWN;  // output blocks of a wave
    constexpr int kSides = GATED ? 2 : 1;
    static_assert(64 * kNW == 256, "a thread stages 16 of a row group's 4096 bytes");
    __shared__ __attribute__((aligned(16))) uint8_t smem[2][TM * 4096];
    const uint32_t tid = threadIdx.x, lane = tid & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t slabs = P.k / 256u;
    uint32_t tn, tm;
    tile_of(P, tm, tn);

    // Offsets (in slabs) of the row groups from the tile's or the wave's first
    // one, all uniform.  A group past the tensor's last is replaced by the
    // last: what it gives is not stored.
    const uint32_t a_groups = pad32(P.m) / 32u, w_groups = pad32(P.n) / 32u;
    const uint32_t g0 = tm * TM, w0 = (tn * kNW + wave) * kCols, wb = min_u32(w0, w_groups - 1u);
    const __amdgpu_buffer_rsrc_t arc = group_rsrc(P.a_codes, g0, slabs, 4096u, TM);
    const __amdgpu_buffer_rsrc_t ars = group_rsrc(P.a_scales, g0, slabs, 256u, TM);
    __amdgpu_buffer_rsrc_t wrc[kSides], wrs[kSides];
#pragma unroll
    for (int g = 0; g < kSides; ++g) {
        wrc[g] = group_rsrc(P.w.codes[g], wb, slabs, 4096u, kCols);
        wrs[g] = group_rsrc(P.w.scales[g], wb, slabs, 256u, kCols);
    }
    uint32_t ag[TM], wg[kCols];
#pragma unroll
    for (int j = 0; j < TM; ++j) ag[j] = (min_u32(g0 + j, a_groups - 1u) - g0) * slabs;
#pragma unroll
    for (int i = 0; i < kCols; ++i) wg[i] = (min_u32(wb + i, w_groups - 1u) - wb) * slabs;
    const uint32_t avo = tid * 16u, wvo = lane * 16u, svo = lane * 4u;

    v16f acc[kWN][TM] = {};
    u32x4 st[TM];       // activation rows on their way to LDS
    u32x4 w[2][kWN][4];  // weight blocks of this step and the next
    uint32_t sa[2][TM], sw[2][kWN];

    auto load_a = [&](int j, uint32_t s) { st[j] = load16(arc, avo, (ag[j] + s) * 4096u); };
    auto put_a = [&](uint8_t* dst, int j) { *reinterpret_cast<u32x4*>(dst + j * 4096 + avo) = st[j]; };
    auto load_w = [&](int b, int i, int q, uint32_t s) {
        w[b][i][q] = load16(wrc[i / kCols], wvo + q * 1024u, (wg[i % kCols] + s) * 4096u);
    };
    auto load_sw = [&](int b, int i, uint32_t s) { sw[b][i] = load4(wrs[i / kCols], svo, (wg[i % kCols] + s) * 256u); };
    auto load_sa = [&](int b, int j, uint32_t s) { sa[b][j] = load4(ars, svo, (ag[j] + s) * 256u); };

    // One 256-column step: 4 TM pieces (64-column slab q, activation block j)
    // of two MFMAs each, their order kept by the barriers to the scheduler.  In
    // the shadow of a piece's MFMAs: the read of the activation block two
    // pieces on; in the first eight the loads of the next step's weights and
    // scales; in TM of them from kPut on the write of an activation block to
    // the other stage and the load of the one two steps on.  So every load has
    // a whole step to land.
    auto step = [&](auto bc, uint32_t s) {
        constexpr int b = decltype(bc)::value;
        constexpr int kPieces = 4 * TM, kPut = 4 + TM;
        static_assert(4 * kWN == 8 && kPieces >= 8 && kPut + TM <= kPieces, "the loads' places below");
        const uint8_t* cur = smem[b] + wvo;
        uint8_t* nxt = smem[b ^ 1];
        const uint32_t s1 = min_u32(s + 1u, slabs - 1u), s2 = min_u32(s + 2u, slabs - 1u);
        __syncthreads();
        u32x4 a[3];
        a[0] = *reinterpret_cast<const u32x4*>(cur);
        a[1] = *reinterpret_cast<const u32x4*>(cur + 4096);
        __builtin_amdgcn_sched_barrier(0);
        for_each_index<kPieces>([&](auto pc) {
            constexpr int p = decltype(pc)::value, q = p / TM, j = p % TM;
            if constexpr (p < kPieces - 2) {
                constexpr int pn = p + 2;
                a[pn % 3] = *reinterpret_cast<const u32x4*>(cur + (pn % TM) * 4096 + (pn / TM) * 1024);
            }
            if constexpr (p < 8) load_w(b ^ 1, p % kWN, p / kWN, s1);
            if constexpr (p >= 2 && p < 4) load_sw(b ^ 1, p - 2, s1);
            if constexpr (p >= 4 && p < kPut) load_sa(b ^ 1, p - 4, s1);
            if constexpr (p >= kPut && p < kPut + TM) {
                put_a(nxt, p - kPut);
                load_a(p - kPut, s2);
            }
#pragma unroll
            for (int i = 0; i < kWN; ++i) {
                if constexpr (OUT == kOutMX)  // tokens along the lanes
                    acc[i][j] = mma<q>(w[b][i][q], a[p % 3], acc[i][j], sw[b][i], sa[b][j]);
                else
                    acc[i][j] = mma<q>(a[p % 3], w[b][i][q], acc[i][j], sa[b][j], sw[b][i]);
            }
            __builtin_amdgcn_sched_barrier(0);
        });
    };
#pragma unroll
    for (int j = 0; j < TM; ++j) load_a(j, 0);
#pragma unroll
    for (int j = 0; j < TM; ++j) load_sa(0, j, 0);
#pragma unroll
    for (int i = 0; i < kWN; ++i) {
        load_sw(0, i, 0);
#pragma unroll
        for (int q = 0; q < 4; ++q) load_w(0, i, q, 0);
    }
#pragma unroll
    for (int j = 0; j < TM; ++j) {
        put_a(smem[0], j);
        load_a(j, min_u32(1u, slabs - 1u));
    }
    for (uint32_t s = 0; s < slabs; s += 2) {
        step(std::integral_constant<int, 0>{}, s);
        if (s + 1 < slabs) step(std::integral_constant<int, 1>{}, s + 1);
    }

#pragma unroll
    for (int j = 0; j < TM; ++j)
#pragma unroll
        for (int i = 0; i < kCols; ++i) {
            float v[16];
            const uint32_t col = (w0 + i) * 32u;
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = GATED ? silu(acc[i][j][e]) * acc[kWN - kCols + i][j][e] : acc[i][j][e];
            if constexpr (OUT == kOutMX) {
                if (col < P.n) quantise_lanes(P, v, g0 + j, col, lane);
            } else {
                store_f32(P, v, g0 + j, col, lane);
            }
        }
}

// ---------------------------------------------------------------------------
// Split kernel, for few tiles: 32 TM tokens x 32 WN weight rows (gated: WN/2
// gate and WN/2 up blocks) a workgroup, whose KS waves share the K range (256
// columns a turn) and add their sums through LDS in a fixed order.  Every
// operand goes straight from the L2 to registers; a 64-column slab's next
// turn is loaded as soon as its MFMAs are issued.
// ---------------------------------------------------------------------------
template <int TM, int WN, int KS, bool GATED, int OUT>
__global__ __launch_bounds__(64 * KS, 2) void mx_gemm_split_kernel(Args P) {
    constexpr int kCols = GATED ? WN / 2 : WN;
    constexpr int kPair = GATED ? 2 : 1;
    constexpr int kRound = 16 / KS < kPair ? kPair : (16 / KS > TM * WN ? TM * WN : 16 / KS);  // blocks added at a time
    constexpr int kOutBlocks = kRound / kPair;
    constexpr int kPer = kOutBlocks * 16 / KS;         // register rows a wave adds
    static_assert(TM * WN % kRound == 0 && kPer >= 1 && kPer * KS == kOutBlocks * 16, "rounds");
    __shared__ __attribute__((aligned(16))) float sums[KS][kRound][16][64];
    const uint32_t tid = threadIdx.x, lane = tid & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t slabs = P.k / 256u;
    uint32_t tn, tm;
    tile_of(P, tm, tn);
    const uint32_t a_groups = pad32(P.m) / 32u, w_groups = pad32(P.n) / 32u;
    const uint32_t g0 = tm * TM, w0 = tn * kCols;
    const __amdgpu_buffer_rsrc_t arc = group_rsrc(P.a_codes, g0, slabs, 4096u, TM), ars = group_rsrc(P.a_scales, g0, slabs, 256u, TM);
    __amdgpu_buffer_rsrc_t wrc[kPair], wrs[kPair];
#pragma unroll
    for (int g = 0; g < kPair; ++g) {
        wrc[g] = group_rsrc(P.w.codes[g], w0, slabs, 4096u, kCols);
        wrs[g] = group_rsrc(P.w.scales[g], w0, slabs, 256u, kCols);
    }
    uint32_t ag[TM], wg[kCols];
#pragma unroll
    for (int j = 0; j < TM; ++j) ag[j] = (min_u32(g0 + j, a_groups - 1u) - g0) * slabs;
#pragma unroll
    for (int i = 0; i < kCols; ++i) wg[i] = (min_u32(w0 + i, w_groups - 1u) - w0) * slabs;
    const uint32_t cvo = lane * 16u, svo = lane * 4u;
    v16f acc[WN][TM] = {};
    u32x4 a[TM][4], w[WN][4];
    uint32_t sa[2][TM], sw[2][WN];
    auto load_q = [&](int q, uint32_t s) {
#pragma unroll
        for (int i = 0; i < WN; ++i) w[i][q] = load16(wrc[i / kCols], cvo + q * 1024u, (wg[i % kCols] + s) * 4096u);
#pragma unroll
        for (int j = 0; j < TM; ++j) a[j][q] = load16(arc, cvo + q * 1024u, (ag[j] + s) * 4096u);
    };
    auto load_s = [&](int b, uint32_t s) {
#pragma unroll
        for (int i = 0; i < WN; ++i) sw[b][i] = load4(wrs[i / kCols], svo, (wg[i % kCols] + s) * 256u);
#pragma unroll
        for (int j = 0; j < TM; ++j) sa[b][j] = load4(ars, svo, (ag[j] + s) * 256u);
    };
    auto turn = [&](auto bc, uint32_t s) {
        constexpr int b = decltype(bc)::value;
        const uint32_t next = min_u32(s + KS, slabs - 1u);
        load_s(b ^ 1, next);
        for_each_index<4>([&](auto qc) {
            constexpr int q = decltype(qc)::value;
#pragma unroll
            for (int j = 0; j < TM; ++j)
#pragma unroll
                for (int i = 0; i < WN; ++i) acc[i][j] = mma<q>(a[j][q], w[i][q], acc[i][j], sa[b][j], sw[b][i]);
            load_q(q, next);
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    if (wave < slabs) {
        load_s(0, wave);
#pragma unroll
        for (int q = 0; q < 4; ++q) load_q(q, wave);
        for (uint32_t s = wave; s < slabs; s += 2 * KS) {
            turn(std::integral_constant<int, 0>{}, s);
            if (s + KS < slabs) turn(std::integral_constant<int, 1>{}, s + KS);
        }
    }
    // rounds of kRound blocks; block b of a round is output block b / kPair
    // (gate before up)
    for_each_index<TM * WN / kRound>([&](auto rc) {
        constexpr int r = decltype(rc)::value;
        auto block = [&](int b) { return r * kOutBlocks + b / kPair; };  // output block i + kCols j
        if constexpr (r > 0) __syncthreads();
        for_each_index<kRound>([&](auto bc) {
            constexpr int b = decltype(bc)::value, o = r * kOutBlocks + b / kPair, i = o % kCols + (b % kPair) * kCols, j = o / kCols;
#pragma unroll
            for (int e = 0; e < 16; ++e) sums[wave][b][e][lane] = acc[i][j][e];
        });
        __syncthreads();
        float v[kPer];
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int e = (int)wave * kPer + u, b = (e / 16) * kPair;
            float s[kPair];
#pragma unroll
            for (int g = 0; g < kPair; ++g) {
                s[g] = 0.0f;
#pragma unroll
                for (int z = 0; z < KS; ++z) s[g] += sums[z][b + g][e % 16][lane];
            }
            v[u] = GATED ? silu(s[0]) * s[kPair - 1] : s[0];
        }
        if constexpr (OUT == kOutF32) {
#pragma unroll
            for (int u = 0; u < kPer; ++u) {
                const uint32_t e = wave * kPer + u, o = block((e / 16u) * kPair);
                const uint32_t row = (g0 + o / kCols) * 32u + 8u * ((e & 15u) >> 2) + 4u * (lane >> 5) + (e & 3u);
                const uint32_t col = (w0 + o % kCols) * 32u + (lane & 31u);
                if (row < P.m && col < P.n) P.y[(uint64_t)row * P.n + col] = v[u];
            }
        } else {
            __syncthreads();
            float* blk = &sums[0][0][0][0];  // the output blocks as 32 x 32 rows
#pragma unroll
            for (int u = 0; u < kPer; ++u) {
                const uint32_t e = wave * kPer + u;
                blk[(e / 16u) * 1024u + (8u * ((e & 15u) >> 2) + 4u * (lane >> 5) + (e & 3u)) * 32u + (lane & 31u)] = v[u];
            }
            __syncthreads();
            if (wave < kOutBlocks) {  // one block a wave
                const uint32_t o = block((int)wave * kPair);
                if ((w0 + o % kCols) * 32u < P.n) quantise_block(P, g0 + o / kCols, (w0 + o % kCols) * 32u, lane, blk + wave * 1024);
            }
        }
    });
}

// Row groups of a tile: those with the least cost, turns of the 256 CUs times
// what a turn of that height takes.  Two 128-token tiles on a CU do the most
// work a second; lower ones fill the CUs and waste less of a ragged batch
// where there are few, higher ones (one workgroup a CU, 278 and 316 registers,
// 330 to 426 gated) save a second turn that would be mostly idle, where a long
// K outweighs their slower start and end.  Measured (us, by tokens a tile, the
// one taken in brackets; the others with the same choice of everything else):
//                                 64     96    128    160    192
//   640 x 3584 x 3584          [10.0]          11.9
//   gated 160 x 18944 x 3584   [18.9]   24.7   28.7   18.1   19.3
//   2048 x 4608 x 3584          26.5  [22.6]   29.7   22.5   23.7
//   1280 x 3584 x 3584          18.1    13.2 [14.1]   15.2   16.6
//   1024 x 3584 x 18944        [43.1]          47.6
//   2048 x 4608 x 18944        114      95    107   [81.9]   87.7
//   2300 x 4608 x 18944                 98    111    138   [94.3]
//   1500 x 3584 x 18944               [52.8]   57.7   63.3   64.7
//   2048 x 3584 x 18944         78            [65]            72
//   2048 x 18944 x 3584         90            [76]            89
//   gated 160 x 18944 x 4608    29.1   33.0   35.3  [24.4]   25.2
//   gated 384 x 14336 x 4608    32.1   27.4   30.9   39.7  [27.1]
//   gated 1024 x 4608 x 8192    49.4   44.1   47.3  [39.7]   42.0
//   gated 1536 x 3584 x 8192    55.0   45.2   49.5   61.9  [43.2]
// (the MXFP4 output's within 3% of these).
// A 96-token tile alone on a CU is not surely faster than a 128-token one
// unless the batch is ragged or K long: its time depends on where the operands
// lie, by a cause that was not found (1280 x 3584 with K = 2048: 9.8 in one
// process and 11.5 in the next, 128 tokens 10.0 to 10.4 in both; 1500 x 3584
// 10.4 and 11.2, 128 tokens 10.9 to 11.1).  Tiles of 224 and 256 tokens: 94
// and 90 for 2048 x 4608 x 18944, 110 and 128 (of 118 and 127) for 3500 x 3584
// and 3400 x 4608, and the gated ones spill registers.
uint32_t tile_height(uint32_t a_groups, uint32_t tiles_n, uint32_t k) {
    auto tiles = [&](uint32_t tm) { return (a_groups + tm - 1) / tm * tiles_n; };
    auto cost = [&](uint32_t tm, uint32_t turn) { return (tiles(tm) + 255u) / 256u * turn; };
    const bool deep = k > 4096u;
    uint32_t best = 4, least = cost(4, 32);
    auto consider = [&](uint32_t tm, uint32_t turn) {
        if (cost(tm, turn) < least) {
            best = tm;
            least = cost(tm, turn);
        }
    };
    consider(2, 22);
    if (deep || tiles(3) > 256u || tiles(3) == tiles(4)) consider(3, 28);
    if (deep && tiles(5) <= 256u) consider(5, 36);
    if (deep && tiles(6) <= 256u) consider(6, 40);
    return best;
}

// The kernel goes by the number of 32 x 32 block products of a K step, the
// gate's and the up's counted: few blocks take small workgroups with K split
// eight ways, then larger ones split four ways, many the tile kernel.  The
// splits' times are nearly linear in K like the tile kernel's, so K does not
// matter between them; a 64-token tile starts and ends sooner than a four-way
// split but takes longer a step, so short K moves to it earlier.
// Measured, K = 3584 (us: 1x1 / 2x1 / 2x2 blocks / 64-token tile):
//   256 blocks (512 x 512)     3.9 /  4.7 /  5.5 /
//   288        (37 x 4608)     5.1 /  4.7 /  5.6 /
//   448        (128 x 3584)    5.4 /  5.0 /  5.8 /
//   896        (256 x 3584)    8.5 /  7.3 /  6.4 /  9.6
//   1024       (2048 x 512)   10.2 /  9.7 /  8.3 /  9.5
//   1792       (512 x 3584)   13.2 / 12.3 /  9.6 /  9.7
//   2304       (512 x 4608)           /     / 13.1 / 10.0
// and (2x2 blocks / tile) 256 x 4608, 1152 blocks, with K = 1024 5.7 / 4.5,
// 2048 6.8 / 5.9, 2560 7.5 / 7.7, 18944 28.5 / 37; 512 x 3584 with K = 1024
// 6.1 / 4.6, 2560 8.2 / 7.9, 18944 29.6 / 36.6.  Gated (1x2 / 2x2): 1152
// blocks (128 x 4608) 10.0 / 9.5.  A single row group keeps the 1-high
// workgroups until the tile (16 x 18944 gated, 1184 blocks: 13.9, 15.3 with
// 2x2, 12.8 the tile).  An odd number of row groups counts as the even one
// that 2x2 blocks and tiles compute (96 x 18944: 13.1 / 10.3).
MxPlan plan(uint32_t m, uint32_t n, uint32_t k, bool gated) {
    const uint32_t a_groups = pad32(m) / 32u, w_groups = pad32(n) / 32u;
    const uint64_t row = (uint64_t)w_groups * (gated ? 2 : 1), blocks = a_groups * row;
    const uint64_t paired = a_groups == 1 ? row : ((a_groups + 1u) & ~1u) * row;
    auto of = [&](uint32_t tm, uint32_t cols, uint32_t ways) {
        return MxPlan{tm, cols, ways, (a_groups + tm - 1) / tm * ((w_groups + cols - 1) / cols)};
    };
    if (paired > (a_groups == 1 || k <= 2048u ? 1100u : 2100u)) {
        const uint32_t cols = (gated ? kWN / 2 : kWN) * kNW;
        return of(tile_height(a_groups, (w_groups + cols - 1) / cols, k), cols, 1);
    }
    if (a_groups > 1 && blocks > (gated ? 600u : 800u)) return of(2, gated ? 1 : 2, 4);
    if (!gated && a_groups > 1 && blocks > 272u) return of(2, 1, 8);
    return of(1, 1, 8);
}

template <int TM, int WN, int KS, bool GATED, int OUT>
void launch_split(Args& P, const MxPlan& p, hipStream_t st) {
    P.tiles_m = P.group_m = (pad32(P.m) / 32u + TM - 1) / TM;
    P.tiles_n = p.workgroups / P.tiles_m;
    mx_gemm_split_kernel<TM, WN, KS, GATED, OUT><<<p.workgroups, 64 * KS, 0, st>>>(P);
}

template <int TM, bool GATED, int OUT>
void launch_tile(Args& P, const MxPlan& p, hipStream_t st) {
    P.tiles_m = (pad32(P.m) / 32u + TM - 1) / TM;
    P.tiles_n = p.workgroups / P.tiles_m;
    P.group_m = min_u32(P.tiles_m, 32u / TM);
    mx_gemm_tile_kernel<TM, GATED, OUT><<<p.workgroups, 64 * kNW, 0, st>>>(P);
}

template <bool GATED, int OUT>
void launch_as(Args P, hipStream_t st) {
    const MxPlan p = plan(P.m, P.n, P.k, GATED);
    if (p.ways == 1) {
        switch (p.row_groups) {
            case 2: return launch_tile<2, GATED, OUT>(P, p, st);
            case 3: return launch_tile<3, GATED, OUT>(P, p, st);
            case 5: return launch_tile<5, GATED, OUT>(P, p, st);
            case 6: return launch_tile<6, GATED, OUT>(P, p, st);
            default: return launch_tile<4, GATED, OUT>(P, p, st);
        }
    } else if (p.ways == 4) {
        launch_split<2, 2, 4, GATED, OUT>(P, p, st);
    } else if constexpr (GATED) {
        launch_split<1, 2, 8, GATED, OUT>(P, p, st);
    } else if (p.row_groups == 2) {
        launch_split<2, 1, 8, GATED, OUT>(P, p, st);
    } else {
        launch_split<1, 1, 8, GATED, OUT>(P, p, st);
    }
}

}  // namespace

MxPlan plan_mx_gemm(uint32_t m, uint32_t n, uint32_t k, bool gated) { return plan(m, n, k, gated); }

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
    P.nt = ((reinterpret_cast<uintptr_t>(y) | (uintptr_t)n * 4u) & 63u) == 0;
    if (!gated)
        launch_as<false, kOutF32>(P, st);
    else if (h_codes)
        launch_as<true, kOutMX>(P, st);
    else
        launch_as<true, kOutF32>(P, st);
    return hipGetLastError();
}

}  // namespace rz
