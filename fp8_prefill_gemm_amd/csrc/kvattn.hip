// Attention of one new token a sequence over the quantised, paged cache:
//   out[b][h] = sum_p w_p v_p,  w = softmax(scale q[b][h] . k_p),
// one pass over the rows with the running maximum and sum of the softmax.
//
// A step reads each cached row once for all the queries of its key head; what
// bounds it beside memory is the instructions a row takes, so both products
// run on the fp16 matrix cores, whose operands hold E4M3 and E2M1 codes
// exactly.  Both put positions or columns of the cache in the rows of the
// result and query heads in its columns (16 of them), so that a lane has the
// same head throughout:
//   scores  S[32 positions][16 heads] = K q^T, a lane reads 8 columns of a row
//           a step as they lie; which columns those are is the same for both
//           operands, so 16-byte loads serve two steps (four in MXFP4);
//   output  O[16 columns][16 heads] += V^T P, contraction over 32 positions:
//           lane l holds the weights of positions 4 (l/16) + i and those + 16
//           for head l % 16, which is where S leaves them, and reads V's rows
//           of these eight positions.  Nothing moves between lanes but the
//           maximum.
// q and the weights count to 22 bits, as two fp16 parts each (the second the
// first's rounding, rounded: 2^-22 at most).  With up to 8 queries a key head
// the parts lie side by side in the 16 columns, one product for both.  What
// fp16's range does not hold is kept outside it: a head's q, times scale and
// log2(e), is brought to 2^14 <= max |q| < 2^15 by a power of two, so that a
// score's way back is exact and the largest one's difference to itself 0 however
// large it is; a row's scale (MXFP4: its largest block's) multiplies scores and
// weights in fp32, and weights are taken times 2^14 over a power of two above
// the scales of the wave's values so far, so that what is lost lies 2^-38 below
// the largest value times its weight.  A block's scale is a factor of its codes
// relative to the row's largest one: exact down to 2^-23 of that, and below it
// fp16's steps are 2^-27 of the row's largest value or less.
//
// Workgroups take nearly equal units of the batch's blocks of 128 positions,
// whatever the sequences' lengths, one key head (and 16 of its queries) each;
// the heads of the same blocks go to one XCD, so that a page's lines, which hold
// rows of several heads, are fetched once (24 sequences of 131072 positions in
// all, MXFP4 rows of 64 bytes: 46 -> 42 us).  What is not the whole of a sequence
// goes to the workspace, and a second launch joins it.
//
// Measured (4 key heads of 128 columns, 7 queries each; MXFP4 8): 131072
// positions of one sequence E4M3 34.4 us, 4.0 TB/s of its rows, the loop itself
// at 7 TB/s; 64 sequences of 65536 in all 20.9; 24 sequences of 131072 in all
// MXFP4 24.3, 2.9 TB/s.  E4M3 is bound by memory in the loop and by what comes
// before and after it (lengths, tables, rows and scales are loads that wait for
// each other, 6 us; the join's launch, 4), MXFP4 by its vector instructions
// (about 245 a wave and 32 positions, half of them to widen codes).  Wider rows
// are bound by registers: 131072 positions of 128 columns, and fewer of more, of
// one sequence and with the join take E4M3 at 128, 192, 256, 384 and 512 columns
// 39, 46, 46, 51 and 89 us (memory: 28), MXFP4 26, 41, 38, 47 and 52 (15).  Beyond
// 128 columns (MXFP4: 160) a compute unit holds one workgroup of the two that a
// launch has for it, so the chain before the loop is paid twice, and from 416 on
// E4M3 keeps 130 to 480 bytes a lane of its two tiles of rows in memory.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "kv_steps.h"
#include "mx_device.h"
#include "rz_device.h"
#include "rz_internal.h"

namespace rz {
namespace {
using namespace mx;

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr uint32_t kTile = 32;               // positions a wave takes at a time
constexpr uint32_t kBlock = kTile * kWaves;  // and a workgroup
constexpr uint32_t kChunk = 8 * kBlock;      // positions whose rows are looked up at a time
constexpr uint32_t kHeads = 16;              // queries of a key head that a workgroup serves
constexpr uint32_t kPacked = 8;              // up to so many: both parts of theirs at a time

// A value that all lanes hold, in a scalar register.
__device__ __forceinline__ uint32_t scalar(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }
__device__ __forceinline__ uint32_t lane_value(uint32_t v, int lane) { return (uint32_t)__builtin_amdgcn_readlane((int)v, lane); }

// What the launch adds to its arguments.
struct Grid {
    uint32_t R;          // workers a key head (and 16 queries)
    uint32_t group;      // queries a key head
    uint32_t tiles;      // and 16 of them at a time
    uint32_t part_rows;  // queries that a part has room for
    uint32_t most;       // positions that a sequence's pages hold at most
    uint32_t magic, shift;  // v / page_len is v * magic >> 31 + shift for v < 2^31
    bool whole;          // workers take whole sequences
    bool near;           // a worker's key heads go to one XCD
    int dtype;
    uint64_t info;       // floats before the workspace's record of who holds which sequence
};

// Positions that sequence b attends (those of a choice may hold gaps, and count as many as the budget has: units are cut by
// these, so a short sequence's choice is shared out, and staged, like a full one).
__device__ __forceinline__ uint32_t length_of(const KvAttend& A, const Grid& G, uint32_t b) {
    const int32_t len = A.lens[b];
    if (len <= 0 || A.num_slots == 0) return 0;
    return A.pages || (uint32_t)len > G.most ? G.most : (uint32_t)len;
}
__device__ __forceinline__ uint32_t blocks_of(const KvAttend& A, const Grid& G, uint32_t b) { return (length_of(A, G, b) + kBlock - 1) / kBlock; }

// Sum and maximum over a wave's lanes, in a scalar register.
template <typename F>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t v, F&& f) {
    auto ror = [](uint32_t x, auto n) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x120 + decltype(n)::value, 0xF, 0xF, true); };
    v = f(v, ror(v, std::integral_constant<int, 8>{}));
    v = f(v, ror(v, std::integral_constant<int, 4>{}));
    v = f(v, ror(v, std::integral_constant<int, 2>{}));
    v = f(v, ror(v, std::integral_constant<int, 1>{}));
    const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = f(a[0], a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return scalar(f(b[0], b[1]));
}
__device__ __forceinline__ uint32_t wave_total(uint32_t v) {
    return wave_reduce(v, [](uint32_t a, uint32_t b) { return a + b; });
}

// Sum of the values of the lanes up to and with this one.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
    // lanes 1, 2, 4, 8 before in a row of 16, then the last lane of the row and of the half before
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, true);
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, true);
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, true);
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, true);
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false);
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false);
    return v;
}

// The batch as units of work, as every wave finds it for itself: sequence b of
// n blocks is ceil(n / per) units of nearly equal size.  Sequences are looked
// at 64 at a time, a lane each.
//
// A unit costs about four blocks' time beside its blocks (its lookups, the
// first loads, the join of its waves), so a worker should have one, or where
// there are many sequences two: `per` is the least that makes R units (2 R
// where more than R / 2 sequences have something), found by halving where one
// look holds all sequences, and bounded by T / (2 R - S) otherwise.  That bound
// goes to T as S nears 2 R, so just below that many sequences a long one among
// short ones stays whole (4 key heads, R = 128, one of 131072 positions among
// ones of 100: 200 sequences 58 us, 250 334, 255 1576, 256 58).  (A run of equal
// length for each worker instead, cut where sequences end, took 37 us on 64
// sequences of 65536 positions: two or three pieces for the last worker.)
struct Batch {
    uint32_t per = 1, units = 0;
    uint32_t b0 = 0;                      // the 64 that the lanes' values are of
    uint32_t base = 0, split_base = 0;    // units, and units that are not whole sequences, before b0
    uint32_t blocks = 0, sum = 0, split = 0;  // a lane's sequence's blocks; units up to and with it; those of them not whole sequences

    __device__ __forceinline__ uint32_t parts(uint32_t n) const { return (n + per - 1) / per; }
    __device__ __forceinline__ void look(const KvAttend& A, const Grid& G) {
        const uint32_t lane = threadIdx.x % kWave, b = b0 + lane;
        blocks = b < A.seqs ? blocks_of(A, G, b) : 0;
    }
    __device__ __forceinline__ void scan() {
        const uint32_t n = parts(blocks);
        sum = wave_scan(n);
        split = wave_scan(n > 1 ? n : 0);
    }
    __device__ __forceinline__ void begin(const KvAttend& A, const Grid& G) {
        look(A, G);
        uint32_t n = blocks, some = blocks != 0;
        for (uint32_t b = kWave + threadIdx.x % kWave; b < A.seqs; b += kWave) {
            const uint32_t k = blocks_of(A, G, b);
            n += k;
            some += k != 0;
        }
        const uint32_t T = wave_total(n), S = wave_total(some), R = G.R;
        const uint32_t most = 2u * S > R ? 2u * R : R;
        uint32_t low = (T + most - 1) / most, high = S < most ? (T + (most - S) - 1) / (most - S) : (T + R - 1) / R;
        low = low ? low : 1;
        per = high > low ? high : low;
        if (A.seqs <= kWave && S <= most) {
            while (low < per) {  // parts of `per` are few enough
                const uint32_t was = per, mid = (low + per) / 2;
                per = mid;
                if (wave_total(parts(blocks)) > most) {
                    low = mid + 1;
                    per = was;
                }
            }
        }
        per = scalar(per);
        scan();
        units = lane_value(sum, kWave - 1);
        if (A.seqs > kWave) {
            uint32_t u = 0;
            for (uint32_t b = kWave + threadIdx.x % kWave; b < A.seqs; b += kWave) u += parts(blocks_of(A, G, b));
            units += wave_total(u);
        }
    }
    // The first block of part i of n blocks' `count` parts.
    static __device__ __forceinline__ uint32_t cut(uint32_t n, uint32_t i, uint32_t count) {
        const uint32_t each = n / count, more = n - each * count;
        return each * i + (i < more ? i : more);
    }
    // Unit u < units, not below the last one asked for: blocks [first, last) of sequence b, which is all of it or `part` of `count`,
    // the workspace's `at`.
    struct Unit {
        uint32_t b, first, last, part, count, at;
    };
    __device__ __forceinline__ Unit find(const KvAttend& A, const Grid& G, uint32_t u) {
        for (;;) {
            const uint64_t past = __ballot(base + sum > u);
            if (past) {
                const int l = __ffsll((unsigned long long)past) - 1;
                const uint32_t n = lane_value(blocks, l), count = scalar(parts(n)), part = u - (base + lane_value(sum, l) - count);
                return {b0 + l, scalar(cut(n, part, count)), scalar(cut(n, part + 1, count)), part, count,
                        split_base + lane_value(split, l) - count + part};
            }
            base += lane_value(sum, kWave - 1);
            split_base += lane_value(split, kWave - 1);
            b0 += kWave;
            look(A, G);
            scan();
        }
    }
};

// ---- rows of the cache in registers

__device__ __forceinline__ uint32_t bits(f16x2 v) { return __builtin_bit_cast(uint32_t, v); }

// Eight consecutive codes as fp16 (times `scale`, a power of two, for MXFP4).
template <int FMT>
__device__ __forceinline__ u32x4 widen8(uint32_t w0, uint32_t w1, float scale) {
    if constexpr (FMT == kKvE4M3) {
        return (u32x4){bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.0f, false)), bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.0f, true)),
                       bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.0f, false)), bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.0f, true))};
    } else {
        return (u32x4){bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w0, scale, 0)), bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w0, scale, 1)),
                       bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w0, scale, 2)), bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w0, scale, 3))};
    }
}

// The columns of step s (32 columns) that lane group g (0..3) holds: eight
// from this one on.  Loads of 16 bytes serve two steps in E4M3, four in MXFP4.
template <int FMT, int C>
__device__ __forceinline__ constexpr uint32_t k_column(int s, uint32_t g) {
    constexpr int per = FMT == kKvE4M3 ? 2 : 4;
    int n = per, first = s / per * per;  // steps of the load that holds s, and its first
    while (first + n > C) n >>= 1;       // the last loads are halved until they fit
    if (s >= first + n) {                // (a remainder of three: two and one)
        first += n;
        n = 1;
    }
    return 32 * first + 8 * n * g + 8 * (s - first);
}

// Words of a lane's share of a K row: two a step (E4M3) or one.
template <int FMT, int C>
constexpr int kKWords = FMT == kKvE4M3 ? 2 * C : C;

template <int FMT, int C>
__device__ __forceinline__ void load_k(const uint8_t* row, uint32_t g, uint32_t (&w)[kKWords<FMT, C>]) {
    constexpr int per = FMT == kKvE4M3 ? 2 : 4, words = FMT == kKvE4M3 ? 2 : 1;  // a step
    constexpr uint32_t bytes = FMT == kKvE4M3 ? 32 : 16;                         // of a step's columns
    int s = 0;
#pragma unroll
    for (; s + per <= C; s += per) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(row + s * bytes + 16 * g);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[s * words + i] = v[i];
    }
    if constexpr (FMT == kKvE4M3 ? (C & 1) != 0 : (C & 2) != 0) {
        const u32x2 v = *reinterpret_cast<const u32x2*>(row + s * bytes + 8 * g);
        w[s * words] = v.x;
        w[s * words + 1] = v.y;
        s += per / 2;
    }
    if constexpr (FMT == kKvMXFP4 && (C & 1) != 0) w[s] = *reinterpret_cast<const uint32_t*>(row + s * bytes + 4 * g);
}

// V's columns: lane n (0..15) of a lane group holds `wide` consecutive ones of
// each of these runs, as 16 n to 2 n are the widest loads that fit.
template <int C>
struct VRuns {
    static constexpr int n256 = C / 8, n128 = (C >> 2) & 1, n64 = (C >> 1) & 1, n32 = C & 1;
    static constexpr int count = n256 + n128 + n64 + n32;
    static constexpr int wide(int r) { return r < n256 ? 16 : r < n256 + n128 ? 8 : r < n256 + n128 + n64 ? 4 : 2; }
    static constexpr int column(int r) {
        int c = 0;
        for (int i = 0; i < r; ++i) c += 16 * wide(i);
        return c;
    }
    // first word of run r in a lane's share of a row; words of E4M3 hold four columns, of MXFP4 eight
    template <int FMT>
    static constexpr int words(int r) {
        const int per = FMT == kKvE4M3 ? 4 : 8;
        return (wide(r) + per - 1) / per;
    }
    template <int FMT>
    static constexpr int word(int r) {
        int w = 0;
        for (int i = 0; i < r; ++i) w += words<FMT>(i);
        return w;
    }
    // first of the run's products of 16 columns
    static constexpr int product(int r) {
        int j = 0;
        for (int i = 0; i < r; ++i) j += wide(i);
        return j;
    }
};

// Calls f(integral_constant<0>) .. f(integral_constant<N - 1>).
template <int N, int I = 0, typename F>
__device__ __forceinline__ void unrolled(F&& f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        unrolled<N, I + 1>(f);
    }
}

template <int FMT, int C>
constexpr int kVWords = VRuns<C>::template word<FMT>(VRuns<C>::count);

template <int FMT, int C>
__device__ __forceinline__ void load_v(const uint8_t* row, uint32_t n, uint32_t (&w)[kVWords<FMT, C>]) {
    using R = VRuns<C>;
    unrolled<R::count>([&](auto r_) {
        constexpr int r = decltype(r_)::value, at = R::template word<FMT>(r), wide = R::wide(r);
        constexpr int bytes = FMT == kKvE4M3 ? wide : wide / 2, first = FMT == kKvE4M3 ? R::column(r) : R::column(r) / 2;
        const uint8_t* p = row + first + bytes * n;
        if constexpr (bytes == 16) {
            const u32x4 v = *reinterpret_cast<const u32x4*>(p);
            for (int i = 0; i < 4; ++i) w[at + i] = v[i];
        } else if constexpr (bytes == 8) {
            const u32x2 v = *reinterpret_cast<const u32x2*>(p);
            w[at] = v.x;
            w[at + 1] = v.y;
        } else if constexpr (bytes == 4)
            w[at] = *reinterpret_cast<const uint32_t*>(p);
        else if constexpr (bytes == 2)
            w[at] = *reinterpret_cast<const uint16_t*>(p);
        else
            w[at] = *p;
    });
}

// Maximum and sum over the four lanes of a head (l, l + 16, l + 32, l + 48).
__device__ __forceinline__ float head_max(float v) {
    const uint32_t u = __float_as_uint(v);
    const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const uint32_t x = __float_as_uint(fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1])));
    const auto b = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float head_sum(float v) {
    const uint32_t u = __float_as_uint(v);
    const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const uint32_t x = __float_as_uint(__uint_as_float(a[0]) + __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

__device__ __forceinline__ void put(void* out, int dtype, uint64_t at, float v) {
    if (dtype == kF32)
        static_cast<float*>(out)[at] = v;
    else if (dtype == kF16)
        static_cast<_Float16*>(out)[at] = (_Float16)v;
    else
        static_cast<__bf16*>(out)[at] = (__bf16)v;
}

// log of the sum l of 2^(x - m), in natural units; l == 0: of nothing.
__device__ __forceinline__ float lse_of(float m, float l) { return l == 0.0f ? -INFINITY : m * 0.693147180559945309f + logf(l); }

// Where a running maximum is -inf nothing has been added: any base will do.
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.0f : m; }

// Two fp16 parts of two values.
struct Parts {
    uint32_t part[2];
};
__device__ __forceinline__ Parts split2(float a, float b) {
    uint32_t first = bits((f16x2){(_Float16)a, (_Float16)b});
    float minus = -1.0f;
    // `first` as it is (of a product, the compiler would round it for its own use and, fused, once more for the difference: another
    // value at a tie); -1 kept a factor, so that one instruction widens and subtracts
    asm("" : "+v"(first), "+s"(minus));
    const f16x2 h = __builtin_bit_cast(f16x2, first);
    const f16x2 l = {(_Float16)__builtin_fmaf((float)h.x, minus, a), (_Float16)__builtin_fmaf((float)h.y, minus, b)};
    return {{bits(h), bits(l)}};
}

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Sum over lanes l and l ^ 8, where the two parts of packed heads lie.
__device__ __forceinline__ float part_sum(float v) {
    return v + __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), 0x128, 0xF, 0xF, true));  // row_ror:8
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float power(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// A wave's running state: o[j][i] is column VRuns' product j, row 4 g + i, of
// head l % 16 (or part l / 8 of head l % 8).  m is the largest score as the
// products give it, and m c = `base` in powers of two; l is the sum of
// 2^(score - base), o that of these times the values, in their unit.
template <int C>
struct State {
    f32x4 o[2 * C];
    float m, base, l;
};

// Floats of one part in the workspace: [rows][dim], then m [rows], l [rows]; the next begins on 16 bytes.
__host__ __device__ __forceinline__ uint64_t part_floats(uint32_t rows, uint32_t dim) { return ((uint64_t)rows * (dim + 2u) + 3u) & ~3ull; }

// Zeros for sequence b's rows of (h, z).
template <int C>
__device__ __forceinline__ void empty(const KvAttend& A, const Grid& G, uint32_t b, uint32_t h, uint32_t z) {
    const uint32_t group = G.group, rows = group - z * kHeads < kHeads ? group - z * kHeads : kHeads;
    const uint64_t head0 = (uint64_t)b * A.q_heads + h * group + z * kHeads;
    for (uint32_t i = threadIdx.x; i < rows * 32u * C; i += kThreads) {
        if (G.dtype == kF32)
            static_cast<float*>(A.out)[head0 * 32u * C + i] = 0.0f;
        else
            static_cast<uint16_t*>(A.out)[head0 * 32u * C + i] = 0;
    }
    if (A.lse && threadIdx.x < rows) A.lse[head0 + threadIdx.x] = -INFINITY;
}

template <int FMT, int C, bool PACK>
struct Kernel {
    static constexpr uint32_t D = 32 * C;
    static constexpr int kParts = PACK ? 1 : 2;              // products for a q or a weight
    static constexpr uint32_t kRow = FMT == kKvE4M3 ? D : D / 2;  // bytes

    struct Chunk {
        u32x4 q[kParts][C][kWave];  // the queries' parts as the matrix cores take them
        // a chunk of positions, every wave's tiles by itself: rows of the cache (row 0's for what is none), which of a tile's
        // count, their scales
        uint32_t row[kChunk + kBlock];  // behind them a wave's first one, a tile of it
        uint32_t live[kChunk / kTile];
        float scale[2][kChunk];  // keys, values
        float q_largest[kWaves][16];  // |q| of a head
        uint8_t byte[FMT == kKvE4M3 ? 1 : 2][FMT == kKvE4M3 ? 1 : C][FMT == kKvE4M3 ? 4 : kChunk];
    };
    union Shared {
        Chunk c;
        struct {
            float o[kWaves][8 * C][kWave], m[kWaves][kWave], l[kWaves][kWave];
        } w;  // the waves' results
    };

    // Where position v lies, as far as the length need not be known: its page's number in the cache (-1: none), its place in it
    // and in the sequence (no length reaches 2^32 - 1).
    struct Spot {
        int32_t id;
        uint32_t at, place;
    };
    static __device__ __forceinline__ Spot spot(const KvAttend& A, const Grid& G, uint32_t b, uint32_t h, uint32_t v) {
        uint32_t column = __umulhi(2u * v, G.magic) >> G.shift;
        Spot s = {-1, v - column * A.page_len, 0};
        if (A.pages) column = column < A.budget ? (uint32_t)A.pages[((uint64_t)b * A.heads + h) * A.budget + column] : ~0u;
        const uint64_t place = (uint64_t)column * A.page_len + s.at;
        s.place = place >> 32 ? ~0u : (uint32_t)place;
        if (v < G.most && column < A.max_pages) s.id = A.page_table[(uint64_t)b * A.max_pages + column];
        return s;
    }
    static __device__ __forceinline__ int32_t slot_of(const KvAttend& A, const Spot& s, uint32_t len) {
        const uint64_t slot = (uint64_t)(uint32_t)s.id * A.page_len + s.at;
        return s.id >= 0 && s.place < len && slot < A.num_slots ? (int32_t)slot : -1;
    }

    // A row's scales: fp32 of its key and value; MXFP4: their largest blocks', and the blocks' bytes relative to those.
    struct Scales2 {
        float row[2];
        uint32_t byte[FMT == kKvE4M3 ? 1 : 2 * C];
    };
    static __device__ __forceinline__ void load_scales(const KvAttend& A, uint64_t row, Scales2& s) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if constexpr (FMT == kKvE4M3) {
                s.row[c] = static_cast<const float*>(A.scales[c])[row];
            } else {
                const uint8_t* p = static_cast<const uint8_t*>(A.scales[c]) + row * C;
                uint32_t* x = s.byte + c * C;
                if constexpr (C % 4 == 0) {
#pragma unroll
                    for (int i = 0; i < C / 4; ++i) x[i] = reinterpret_cast<const uint32_t*>(p)[i];
                } else if constexpr (C % 2 == 0) {
#pragma unroll
                    for (int i = 0; i < C / 2; ++i) x[i] = reinterpret_cast<const uint16_t*>(p)[i];
                } else {
#pragma unroll
                    for (int i = 0; i < C; ++i) x[i] = p[i];
                }
            }
        }
    }
    static __device__ __forceinline__ void ready(bool live, Scales2& s) {
        if constexpr (FMT == kKvMXFP4) {
            constexpr int per = C % 4 == 0 ? 4 : C % 2 == 0 ? 2 : 1;  // bytes that were loaded at a time
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t* x = s.byte + c * C;
                uint32_t top = 0;
#pragma unroll
                for (int i = C - 1; i >= 0; --i) {
                    x[i] = x[i / per] >> (8 * (i % per)) & 255u;
                    top = x[i] != kNanByte && x[i] > top ? x[i] : top;
                }
                s.row[c] = __uint_as_float(top ? top << 23 : 0x00400000u);
#pragma unroll
                for (int i = 0; i < C; ++i) x[i] = x[i] == kNanByte ? kNanByte : x[i] + 127u > top ? x[i] + 127u - top : 0u;
            }
        }
        if (!live) {
            s.row[0] = s.row[1] = 0.0f;
            if constexpr (FMT == kKvMXFP4)
#pragma unroll
                for (int i = 0; i < 2 * C; ++i) s.byte[i] = 0;
        }
    }

    // A wave's lanes find the positions of its own tiles of a chunk, kTurns each; `blocks` of it are used.
    static constexpr int kTurns = kChunk / kThreads;
    static __device__ __forceinline__ uint32_t place(int turn) {
        const uint32_t lane = threadIdx.x % kWave;
        return (kWave / kTile * turn + lane / kTile) * kBlock + threadIdx.x / kWave * kTile + lane % kTile;
    }
    struct Spots {
        Spot s[kTurns];
    };
    static __device__ __forceinline__ void find(const KvAttend& A, const Grid& G, uint32_t b, uint32_t h, uint32_t block, Spots& x) {
#pragma unroll
        for (int i = 0; i < kTurns; ++i) x.s[i] = spot(A, G, b, h, block * kBlock + place(i));
    }
    // What a wave has staged, its lanes may read.
    static __device__ __forceinline__ void staged_by_wave() {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    // First the rows, whose scales are then on their way, and once those are here the scales.
    struct Staged {
        Scales2 sc[kTurns];
        uint32_t live;
    };
    static __device__ __forceinline__ void stage_rows(const KvAttend& A, Chunk& S, uint32_t h, uint32_t blocks, uint32_t len, const Spots& x, Staged& y) {
        y.live = 0;
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
            const uint32_t at = place(i), lane = threadIdx.x % kWave;
            const int32_t slot = at < blocks * kBlock ? slot_of(A, x.s[i], len) : -1;
            const uint32_t row = (uint32_t)(slot < 0 ? 0 : slot) * A.heads + h;  // below 2^31
            load_scales(A, row, y.sc[i]);
            const uint64_t on = __ballot(slot >= 0);
            S.row[at] = row;
            if (i == 0 && lane < kTile) S.row[kChunk + threadIdx.x / kWave * kTile + lane] = scalar(row);
            if (lane % kTile == 0) S.live[at / kTile] = (uint32_t)(on >> lane);
            y.live |= (slot >= 0 ? 1u : 0u) << i;
        }
    }
    // Whether the values of a row are zeros: E4M3's have the scale of a row whose largest magnitude is 1, so it is looked at
    // where that is met, and then staged as 0.
    static __device__ __forceinline__ bool zeros(const KvAttend& A, uint32_t row) {
        const u32x4* p = reinterpret_cast<const u32x4*>(A.codes[1] + (uint64_t)row * kRow);
        uint32_t any = 0;
#pragma unroll 1
        for (uint32_t i = 0; i < kRow / 16 && any == 0; ++i) any = (p[i].x | p[i].y | p[i].z | p[i].w) & 0x7F7F7F7Fu;
        return any == 0;
    }
    // The scales of values are staged in a unit of their own, 2^(e - 14) with e the exponent of a power of two over them, at
    // least the one before, which is returned.  (Times the weights instead, it would be an addend of the exponential's argument,
    // and its rounding the scores'.)
    static __device__ __forceinline__ int stage_scales(const KvAttend& A, Chunk& S, Staged& y, int e) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
            const uint32_t at = place(i);
            ready(y.live >> i & 1, y.sc[i]);
            S.scale[0][at] = y.sc[i].row[0];
            if constexpr (FMT == kKvMXFP4)
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int k = 0; k < C; ++k) S.byte[c][k][at] = (uint8_t)y.sc[i].byte[c * C + k];
        }
        if constexpr (FMT == kKvE4M3) {
            bool one = false;
#pragma unroll
            for (int i = 0; i < kTurns; ++i) one |= y.sc[i].row[1] == 1.0f / 448.0f;
            if (__builtin_expect(__any(one), 0)) {  // rare
#pragma unroll
                for (int i = 0; i < kTurns; ++i)
                    if (y.sc[i].row[1] == 1.0f / 448.0f && zeros(A, S.row[place(i)])) y.sc[i].row[1] = 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
            const uint32_t key = __float_as_uint(y.sc[i].row[1]) & 0x7FFFFFFFu;
            top = key < 0x7F800000u && key > top ? key : top;
        }
        top = wave_reduce(top, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
        const int over = (int)(top >> 23) - 126;
        e = over > e ? over < 127 ? over : 127 : e;
        const float unit = power(14 - e);
#pragma unroll
        for (int i = 0; i < kTurns; ++i) S.scale[1][place(i)] = y.sc[i].row[1] * unit;
        return e;
    }

    // kRow as a factor that the compiler does not know: one multiply-add an address, not a shift and two additions.
    static __device__ __forceinline__ uint32_t row_bytes() {
        uint32_t x = kRow;
        asm("" : "+s"(x));
        return x;
    }

    // A tile's rows as they are loaded; `row` its 32 rows of the cache.
    static __device__ __forceinline__ void load_keys(const KvAttend& A, const uint32_t* row, uint32_t (&k)[2][kKWords<FMT, C>]) {
        const uint32_t n = threadIdx.x % 16, g = threadIdx.x % kWave / 16;
#pragma unroll
        for (int t = 0; t < 2; ++t) load_k<FMT, C>(A.codes[0] + (uint64_t)row[16 * t + n] * row_bytes(), g, k[t]);
    }
    static __device__ __forceinline__ void load_values(const KvAttend& A, const uint32_t* row, uint32_t (&v)[8][kVWords<FMT, C>]) {
        const uint32_t n = threadIdx.x % 16, g = threadIdx.x % kWave / 16;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const u32x4 at = *reinterpret_cast<const u32x4*>(row + 16 * t + 4 * g);
#pragma unroll
            for (int i = 0; i < 4; ++i) load_v<FMT, C>(A.codes[1] + (uint64_t)at[i] * row_bytes(), n, v[4 * t + i]);
        }
    }

    // Scores of the tile at `at` of the chunk, in units of c powers of two: p[4 t + i] of position 16 t + 4 g + i.
    static __device__ __forceinline__ void scores(const Chunk& S, uint32_t at, const uint32_t (&k)[2][kKWords<FMT, C>], float (&p)[8]) {
        const uint32_t lane = threadIdx.x % kWave, n = lane % 16, g = lane / 16;
        f32x4 sum[2] = {};
#pragma unroll
        for (int s = 0; s < C; ++s) {
            u32x4 a[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if constexpr (FMT == kKvE4M3)
                    a[t] = widen8<FMT>(k[t][2 * s], k[t][2 * s + 1], 1.0f);
                else
                    a[t] = widen8<FMT>(k[t][s], 0u, cvt_scale(S.byte[0][k_column<FMT, C>(s, g) / 32][at + 16 * t + n]));
            }
#pragma unroll
            for (int i = kParts - 1; i >= 0; --i) {
                const u32x4 q = S.q[i][s][lane];
#pragma unroll
                for (int t = 0; t < 2; ++t) sum[t] = mfma(a[t], q, sum[t]);
            }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const f32x4 sc = *reinterpret_cast<const f32x4*>(&S.scale[0][at + 16 * t + 4 * g]);
#pragma unroll
            for (int i = 0; i < 4; ++i) p[4 * t + i] = (PACK ? part_sum(sum[t][i]) : sum[t][i]) * sc[i];
        }
    }

    // Scores into weights relative to the running maximum times the values' scales, `live` the positions that count.
    static __device__ __forceinline__ void weigh(const Chunk& S, uint32_t at, uint32_t live, float c, float (&p)[8], State<C>& st) {
        const uint32_t g = threadIdx.x % kWave / 16;
        if (live != 0xFFFFFFFFu) {
            asm volatile("" : "+s"(live));  // its bits are looked at here alone
#pragma unroll
            for (int e = 0; e < 8; ++e) p[e] = live >> (16 * (e / 4) + 4 * g + e % 4) & 1 ? p[e] : -INFINITY;
        }
        float top = fmaxf(fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3])), fmaxf(fmaxf(p[4], p[5]), fmaxf(p[6], p[7])));
        top = head_max(top);
        if (__any(top > st.m)) {  // rarely, after the first tiles
            top = fmaxf(top, st.m);
            const float base = base_of(top) * c;
            const float f = st.m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(st.base - base);
#pragma unroll
            for (int j = 0; j < 2 * C; ++j) st.o[j] *= f;
            st.l *= f;
            st.m = top;
            st.base = base;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(p[e], c, -st.base));
        st.l += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const f32x4 sc = *reinterpret_cast<const f32x4*>(&S.scale[1][at + 16 * t + 4 * g]);
#pragma unroll
            for (int i = 0; i < 4; ++i) p[4 * t + i] *= sc[i];  // 0 where there is no row
        }
    }

    // o += the tile's values times its weights.
    static __device__ __forceinline__ void add_values(const Chunk& S, uint32_t at, uint32_t live, const float (&p)[8],
                                                      uint32_t (&v)[8][kVWords<FMT, C>], State<C>& st) {
        const uint32_t n = threadIdx.x % 16, g = threadIdx.x % kWave / 16;
        u32x4 w[kParts];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const Parts s = split2(p[2 * e], p[2 * e + 1]);
            if constexpr (PACK) {
                w[0][e] = n < kPacked ? s.part[0] : s.part[1];
            } else {
                w[0][e] = s.part[0];
                w[1][e] = s.part[1];
            }
        }
        if (live != 0xFFFFFFFFu) {  // what lies in no row's place must not meet a weight of 0
            asm volatile("" : "+s"(live));
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const bool on = live >> (16 * (e / 4) + 4 * g + e % 4) & 1;
#pragma unroll
                for (int i = 0; i < kVWords<FMT, C>; ++i) v[e][i] = on ? v[e][i] : 0u;
            }
        }
        using R = VRuns<C>;
        unrolled<R::count>([&](auto r_) {
            constexpr int r = decltype(r_)::value, w0 = R::template word<FMT>(r), wide = R::wide(r), j0 = R::product(r);
            constexpr int step = wide < 4 ? wide : 4;  // columns at a time
            [[maybe_unused]] float sc[8];
            if constexpr (FMT == kKvMXFP4) {  // a lane's columns lie in one block of 32
                const uint8_t* by = S.byte[1][(R::column(r) + wide * n) / 32] + at;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const uint32_t four = *reinterpret_cast<const uint32_t*>(by + 16 * t + 4 * g);
#pragma unroll
                    for (int i = 0; i < 4; ++i) sc[4 * t + i] = __uint_as_float(i < 3 ? four << (23 - 8 * i) : four >> 1);  // the exponent field alone counts
                }
            }
            unrolled<wide / step>([&](auto k_) {
                constexpr int k = decltype(k_)::value;
                u32x4 a[step];  // positions e and e + 1 side by side, a column at a time
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (FMT == kKvE4M3) {
                        const uint32_t x0 = v[2 * e][w0 + k], x1 = v[2 * e + 1][w0 + k];
                        const uint32_t y0 = __builtin_amdgcn_perm(x1, x0, 0x05010400u);
                        a[0][e] = bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(y0, 1.0f, false));
                        a[1][e] = bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(y0, 1.0f, true));
                        if constexpr (step == 4) {
                            const uint32_t y1 = __builtin_amdgcn_perm(x1, x0, 0x07030602u);
                            a[2][e] = bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(y1, 1.0f, false));
                            a[3][e] = bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(y1, 1.0f, true));
                        }
                    } else {
                        unrolled<step / 2>([&](auto c_) {
                            constexpr int c = decltype(c_)::value, two = step / 2 * k + c;  // columns 2 two and 2 two + 1
                            const uint32_t x0 = bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(v[2 * e][w0 + two / 4], sc[2 * e], two % 4));
                            const uint32_t x1 = bits(__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(v[2 * e + 1][w0 + two / 4], sc[2 * e + 1], two % 4));
                            a[2 * c][e] = __builtin_amdgcn_perm(x1, x0, 0x05040100u);
                            a[2 * c + 1][e] = __builtin_amdgcn_perm(x1, x0, 0x07060302u);
                        });
                    }
                }
#pragma unroll
                for (int i = 0; i < kParts; ++i)
#pragma unroll
                    for (int j = 0; j < step; ++j) st.o[j0 + step * k + j] = mfma(a[j], w[i], st.o[j0 + step * k + j]);
            });
        });
    }

    struct Rows {
        uint32_t k[2][kKWords<FMT, C>], v[8][kVWords<FMT, C>];
    };
    static __device__ __forceinline__ void load(const KvAttend& A, const uint32_t* row, Rows& x) {
        load_keys(A, row, x.k);
        load_values(A, row, x.v);
    }
    static __device__ __forceinline__ void tile(const Chunk& S, uint32_t at, uint32_t live, float c, Rows& x, State<C>& st) {
        float p[8];
        scores(S, at, x.k, p);
        weigh(S, at, live, c, p, st);
        add_values(S, at, live, p, x.v, st);
    }

    // `blocks` blocks of the chunk, by the workgroup: every wave's own tiles of 32 into `st`, the next one's rows on their way;
    // x0: the first one's.  A load that may be left out makes the wait for the tile before it one for all loads, as the
    // compiler counts them.  So behind the last tile of MXFP4 the wave's first row is loaded instead (24 sequences of 131072
    // positions in all 28.4 -> 27.3 us, units of one tile 11.5 -> 12.0); E4M3, which waits for memory all the same, gains no
    // more in long units than it loses in short ones (131072 positions of one 34.1 -> 33.1, 37 positions 5.9 -> 6.3).
    static constexpr bool kAlways = FMT == kKvMXFP4;
    static __device__ __forceinline__ void chunk(const KvAttend& A, const Chunk& S, uint32_t blocks, float c, Rows& x0, State<C>& st) {
        Rows x1;
        uint32_t at = scalar(threadIdx.x / kWave) * kTile;
        const uint32_t spare = kChunk + at;
#pragma unroll 1
        for (uint32_t i = 0; i < blocks; i += 2, at += 2 * kBlock) {
            if (kAlways || i + 1 < blocks) load(A, S.row + (i + 1 < blocks ? at + kBlock : spare), x1);
            const uint32_t on = scalar(S.live[at / kTile]);
            if (on) tile(S, at, on, c, x0, st);
            if (kAlways || i + 2 < blocks) load(A, S.row + (i + 2 < blocks ? at + 2 * kBlock : spare), x0);
            if (i + 1 < blocks) {
                const uint32_t then = scalar(S.live[(at + kBlock) / kTile]);
                if (then) tile(S, at + kBlock, then, c, x1, st);
            }
        }
    }

    // A lane's columns in row i of each product, from element `at` on, times f.
    template <int DT>
    static __device__ __forceinline__ void store(void* out, uint64_t at, uint32_t row, float f, const float (&o)[2 * C]) {
        using T = std::conditional_t<DT == kF32, float, std::conditional_t<DT == kF16, _Float16, __bf16>>;
        using R = VRuns<C>;
        unrolled<R::count>([&](auto r_) {
            constexpr int r = decltype(r_)::value, wide = R::wide(r), j0 = R::product(r), most = wide < 4 ? wide : 4;
            typedef T vec __attribute__((ext_vector_type(most)));
#pragma unroll
            for (int j = 0; j < wide; j += most) {  // `wide` consecutive columns
                vec x;
#pragma unroll
                for (int e = 0; e < most; ++e) x[e] = (T)(o[j0 + j + e] * f);
                *reinterpret_cast<vec*>(static_cast<T*>(out) + at + R::column(r) + wide * row + j) = x;
            }
        });
    }

    // Blocks [first, last) of (b, h, tile z), all of them if `last` is 0; `part`: where they go if they are not the whole of
    // a sequence.  What needs no length is loaded beside it.
    static __device__ __forceinline__ void piece(const KvAttend& A, const Grid& G, Shared& shared, uint32_t b, uint32_t h, uint32_t z, uint32_t first,
                                                 uint32_t last, float* part) {
        Chunk& S = shared.c;
        const uint32_t lane = threadIdx.x % kWave, wave = scalar(threadIdx.x / kWave), n = lane % 16, g = lane / 16;
        const uint32_t group = G.group, rows = group - z * kHeads < kHeads ? group - z * kHeads : kHeads;
        const uint64_t head0 = (uint64_t)b * A.q_heads + h * group + z * kHeads;
        Spots spots;
        find(A, G, b, h, first, spots);
        constexpr int kSteps = (C + kWaves - 1) / kWaves;
        const uint32_t head = PACK ? n % kPacked : n;
        f32x4 q[kSteps][2] = {};
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const uint32_t s = i * kWaves + wave;
            if (s < C && head < rows) {
                const float* p = A.q + b * A.q_stride + (uint64_t)(h * group + z * kHeads + head) * D + k_column<FMT, C>(s, g);
                q[i][0] = *reinterpret_cast<const f32x4*>(p);
                q[i][1] = *reinterpret_cast<const f32x4*>(p + 4);
            }
        }
        const uint32_t len = length_of(A, G, b);
        if (last == 0) {
            last = (len + kBlock - 1) / kBlock;
            if (last == 0) return empty<C>(A, G, b, h, z);
        }
        const uint32_t until = A.pages ? (uint32_t)A.lens[b] : len;
        __syncthreads();  // the last piece's results have been read
        Staged staged;
        stage_rows(A, S, h, last - first, until, spots, staged);
        const float scale = A.scale * 1.44269504088896341f;
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            q[i][0] *= scale;
            q[i][1] *= scale;
#pragma unroll
            for (int e = 0; e < 4; ++e) top = fmaxf(top, fmaxf(fabsf(q[i][0][e]), fabsf(q[i][1][e])));
        }
        top = head_max(top);
        if (g == 0) S.q_largest[wave][n] = top;
        __syncthreads();
        Rows x0;
        load(A, S.row + wave * kTile, x0);
        int e = stage_scales(A, S, staged, -112);
#pragma unroll
        for (int i = 0; i < kWaves; ++i) top = fmaxf(top, S.q_largest[i][n]);
        // a head's power of two, which brings its scores back to powers of two
        int up = 141 - (int)(__float_as_uint(top) >> 23);
        up = up < -112 ? -112 : up > 126 ? 126 : up;
        const float c = power(-up), by = power(up);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const uint32_t s = i * kWaves + wave;
            u32x4 w[2];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const f32x4 x = q[i][e / 2] * by;
                const Parts p = split2(x[2 * (e % 2)], x[2 * (e % 2) + 1]);
                w[0][e] = p.part[0];
                w[1][e] = p.part[1];
            }
            if (s < C) {
                if constexpr (PACK) {
                    S.q[0][s][lane] = n < kPacked ? w[0] : w[1];
                } else {
                    S.q[0][s][lane] = w[0];
                    S.q[1][s][lane] = w[1];
                }
            }
        }
        __syncthreads();
        State<C> st;
#pragma unroll
        for (int j = 0; j < 2 * C; ++j) st.o[j] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
        st.m = -INFINITY;
        st.base = st.l = 0.0f;
        for (uint32_t at = first;;) {
            const uint32_t count = last - at < kChunk / kBlock ? last - at : kChunk / kBlock;
            chunk(A, S, count, c, x0, st);
            at += count;
            if (at >= last) break;
            find(A, G, b, h, at, spots);
            staged_by_wave();  // and has read: its tiles are done
            stage_rows(A, S, h, last - at, until, spots, staged);
            staged_by_wave();
            load(A, S.row + wave * kTile, x0);
            const int then = stage_scales(A, S, staged, e);
            if (then != e) {  // larger values to come: the sums' unit grows (past 2^126 what there was is nothing to them)
                const float f = power(e - then < -126 ? -126 : e - then);
#pragma unroll
                for (int j = 0; j < 2 * C; ++j) st.o[j] *= f;
            }
            staged_by_wave();
            e = then;
        }
        const float unit = power(e - 14);
        __syncthreads();  // the chunk and q are no longer read
        auto& W = shared.w;
#pragma unroll
        for (int j = 0; j < 2 * C; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) W.o[wave][4 * j + i][lane] = st.o[j][i] * unit;
        W.m[wave][lane] = st.m == -INFINITY ? -INFINITY : st.base;  // in powers of two
        W.l[wave][lane] = head_sum(st.l);
        __syncthreads();
        // wave i joins row i of every product
        float m = W.m[0][lane];
#pragma unroll
        for (int i = 1; i < kWaves; ++i) m = fmaxf(m, W.m[i][lane]);
        float l = 0.0f, f[kWaves], o[2 * C];
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
            f[i] = __builtin_amdgcn_exp2f(W.m[i][lane] - base_of(m));
            l += W.l[i][lane] * f[i];
        }
#pragma unroll
        for (int j = 0; j < 2 * C; ++j) {
            o[j] = W.o[0][4 * j + wave][lane] * f[0];
#pragma unroll
            for (int i = 1; i < kWaves; ++i) o[j] += W.o[i][4 * j + wave][lane] * f[i];
            if constexpr (PACK) o[j] = part_sum(o[j]);
        }
        if (n >= rows) return;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const uint32_t row = 4 * g + wave;
        if (part)
            store<kF32>(part, n * D, row, 1.0f, o);
        else if (G.dtype == kF32)
            store<kF32>(A.out, (head0 + n) * D, row, inv, o);
        else if (G.dtype == kF16)
            store<kF16>(A.out, (head0 + n) * D, row, inv, o);
        else
            store<kBF16>(A.out, (head0 + n) * D, row, inv, o);
        if (g == 0 && wave == 0) {
            if (part) {
                part[G.part_rows * D + n] = m;
                part[G.part_rows * (D + 1) + n] = l;
            } else if (A.lse)
                A.lse[head0 + n] = lse_of(m, l);
        }
    }
};

template <int FMT, int C, bool PACK>
__global__ __launch_bounds__(kThreads, C <= 4 ? 2 : 1) void attend_kernel(KvAttend A, Grid G) {
    using K = Kernel<FMT, C, PACK>;
    __shared__ typename K::Shared S;
    // the heads of a run of blocks on one XCD (workgroups go to the eight in turn): they share the lines of its L2
    const uint32_t lanes = A.heads * G.tiles, turn = G.near ? blockIdx.x >> 3 : blockIdx.x, run = scalar(turn / lanes);
    const uint32_t r = G.near ? run * 8u + (blockIdx.x & 7u) : run, hz = turn - run * lanes, h = scalar(hz / G.tiles), z = hz - h * G.tiles;
    if (r >= G.R) return;
    uint32_t* info = reinterpret_cast<uint32_t*>(static_cast<float*>(A.ws) + G.info);
    Batch batch;
    uint32_t end = A.seqs;  // whole sequences, or units
    if (!G.whole) {
        batch.begin(A, G);
        end = batch.units;
    }
    for (uint32_t u = r; u < end; u += G.R) {
        Batch::Unit x = {u, 0, 0, 0, 1, 0};
        if (!G.whole) {
            x = batch.find(A, G, u);
            if (x.part == 0 && threadIdx.x == 0) {  // the same from every key head's worker
                info[2 * x.b] = x.count > 1 ? x.at : 0;
                info[2 * x.b + 1] = x.count > 1 ? x.count : 0;
            }
        }
        K::piece(A, G, S, x.b, h, z, x.first, x.last,
                 x.count > 1 ? static_cast<float*>(A.ws) + (uint64_t)(x.at * lanes + hz) * part_floats(G.part_rows, K::D) : nullptr);
    }
    if (!G.whole)
        for (uint32_t b = r; b < A.seqs; b += G.R)
            if (blocks_of(A, G, b) == 0) {
                empty<C>(A, G, b, h, z);
                if (threadIdx.x == 0) info[2 * b] = info[2 * b + 1] = 0;
            }
}

// A part's, or several parts', sums of 2^(score - m), four columns of them.
struct Sums {
    float m = -INFINITY, l = 0.0f;
    f32x4 o = {};
    __device__ __forceinline__ void add(float m1, float l1, f32x4 o1) {
        const float top = fmaxf(m, m1), base = base_of(top);
        const float f = __builtin_amdgcn_exp2f(m - base), e = __builtin_amdgcn_exp2f(m1 - base);
        o = o * f + o1 * e;
        l = l * f + l1 * e;
        m = top;
    }
    // Those of the lanes whose numbers differ in the bits from `off` on.
    __device__ __forceinline__ void across(uint32_t off) {
        for (; off < (uint32_t)kWave; off <<= 1) {
            f32x4 x;
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = __shfl_xor(o[i], (int)off, kWave);
            add(__shfl_xor(m, (int)off, kWave), __shfl_xor(l, (int)off, kWave), x);
        }
    }
};

// Joins the parts of a sequence that several workers hold: kWays waves a query
// head and run of 32 columns, four columns a lane and eight parts a wave at a
// time, a running maximum each.  Few sequences are in many parts each: 16 waves
// a run (131072 positions of one sequence 4.9 us; 16 waves a head and all its
// columns 6.9).  Many: one, four a workgroup (64 sequences, with the attention
// 24.4 us; two waves a run and as many workgroups as runs 25.9).
constexpr uint32_t kManyWays = 16;
template <uint32_t kWays>
__global__ __launch_bounds__(kWays == 1 ? kThreads : kWays* kWave) void join_kernel(KvAttend A, Grid G) {
    const uint32_t lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const uint32_t runs = A.dim / 32u, job = kWays == 1 ? scalar(blockIdx.x * kWaves + wave) : blockIdx.x;
    const uint32_t bh = job / runs, run = job % runs, b = bh / A.q_heads, qh = bh % A.q_heads;
    if (b >= A.seqs) return;
    const uint32_t h = qh / G.group, z = qh % G.group / kHeads, row = qh % G.group % kHeads, lanes = A.heads * G.tiles;
    const uint32_t* info = reinterpret_cast<const uint32_t*>(static_cast<const float*>(A.ws) + G.info);
    const uint32_t first = info[2 * b], count = info[2 * b + 1];
    if (count == 0) return;
    const uint64_t floats = part_floats(G.part_rows, A.dim);
    const uint32_t col = 32u * run + lane % 8u * 4u;
    Sums x;
#pragma unroll 2
    for (uint32_t i = kWays == 1 ? lane / 8u : threadIdx.x / 8u; i < count; i += 8u * kWays) {
        const float* p = static_cast<const float*>(A.ws) + (uint64_t)((first + i) * lanes + h * G.tiles + z) * floats;
        x.add(p[G.part_rows * A.dim + row], p[G.part_rows * (A.dim + 1u) + row], *reinterpret_cast<const f32x4*>(p + row * A.dim + col));
    }
    x.across(8);
    if constexpr (kWays > 1) {
        __shared__ f32x4 o_of[kWays][8];
        __shared__ float m_of[kWays][8], l_of[kWays][8];
        if (lane < 8) {
            o_of[wave][lane] = x.o;
            m_of[wave][lane] = x.m;
            l_of[wave][lane] = x.l;
        }
        __syncthreads();
        if (wave != 0) return;
        x = Sums();
#pragma unroll
        for (uint32_t w = lane / 8; w < kWays; w += 8) x.add(m_of[w][lane % 8], l_of[w][lane % 8], o_of[w][lane % 8]);
        x.across(8);
    }
    if (lane >= 8) return;
    const float inv = x.l == 0.0f ? 0.0f : 1.0f / x.l;
    const uint64_t head = (uint64_t)b * A.q_heads + qh;
#pragma unroll
    for (int i = 0; i < 4; ++i) put(A.out, G.dtype, head * A.dim + col + i, x.l == 0.0f ? 0.0f : x.o[i] * inv);
    if (A.lse && lane == 0 && run == 0) A.lse[head] = lse_of(x.m, x.l);
}

// Workgroups of a launch: two a compute unit, which is what it holds up to 128 columns (MXFP4 160), and one at a time beyond.
uint32_t workers(int cus) { return 2u * (uint32_t)cus; }

uint32_t part_rows(uint32_t q_heads, uint32_t heads) {
    const uint32_t group = q_heads / heads;
    return group < kHeads ? group : kHeads;
}

// Workers a key head and 16 queries of it.
uint32_t split(uint32_t q_heads, uint32_t heads, int cus) {
    const uint32_t lanes = heads * ((q_heads / heads + kHeads - 1) / kHeads);
    const uint32_t r = workers(cus) / lanes;
    return r >= 8u ? r / 8u * 8u : r ? r : 1;
}

// Floats of all parts: a sequence in more than one has fewer than 2 n / per of them, and per is at least T / (2 R).
uint64_t part_total(uint32_t q_heads, uint32_t heads, uint32_t dim, int cus) {
    const uint64_t lanes = (uint64_t)heads * ((q_heads / heads + kHeads - 1) / kHeads);
    return split(q_heads, heads, cus) * lanes * 4u * part_floats(part_rows(q_heads, heads), dim);
}

}  // namespace

size_t kv_attend_ws_bytes(uint32_t seqs, uint32_t q_heads, uint32_t heads, uint32_t dim, int cus) {
    return (part_total(q_heads, heads, dim, cus) + 2u * (uint64_t)seqs) * 4u;
}

hipError_t launch_kv_attend(int format, const KvAttend& A, int dtype, int cus, hipStream_t st) {
    Grid G;
    G.group = A.q_heads / A.heads;
    G.tiles = (G.group + kHeads - 1) / kHeads;
    G.part_rows = part_rows(A.q_heads, A.heads);
    G.dtype = dtype;
    G.info = part_total(A.q_heads, A.heads, A.dim, cus);
    // one block a sequence at most: nothing to split
    const uint64_t most = (uint64_t)(A.pages ? A.budget : A.max_pages) * A.page_len;
    G.most = (uint32_t)(most < 0x7FFFFFFFu ? most : 0x7FFFFFFFu);
    G.shift = A.page_len == 1 || A.page_len >= 0x80000000u ? 0 : 32 - (uint32_t)__builtin_clz(A.page_len - 1);  // of 2^shift >= page_len
    G.magic = A.page_len >= 0x80000000u ? 0 : (uint32_t)((((uint64_t)1 << (31 + G.shift)) + A.page_len - 1) / A.page_len);
    G.whole = !A.ws || most <= kBlock || (uint64_t)A.seqs * A.q_heads >= 0x400000u;
    const uint32_t lanes = A.heads * G.tiles;
    G.R = split(A.q_heads, A.heads, cus);
    if (G.whole) {
        const uint32_t limit = 0x800000u / lanes;  // workgroups of 256 lanes, which are counted in 32 bits
        G.R = A.seqs < limit ? A.seqs : limit ? limit : 1;
    }
    G.near = G.R >= 8u;
    const uint32_t grid = (G.near ? (G.R + 7u) / 8u * 8u : G.R) * lanes;
    const bool known = with_steps(A.dim / 32u, [&](auto c_) {
        constexpr int C = decltype(c_)::value;
        auto launch = [&](auto pack_) {
            constexpr bool PACK = decltype(pack_)::value;
            if (format == kKvE4M3)
                attend_kernel<kKvE4M3, C, PACK><<<grid, kThreads, 0, st>>>(A, G);
            else
                attend_kernel<kKvMXFP4, C, PACK><<<grid, kThreads, 0, st>>>(A, G);
        };
        if (G.group <= kPacked)
            launch(std::true_type{});
        else
            launch(std::false_type{});
    });
    if (!known) return hipErrorInvalidValue;
    if (!G.whole) {
        const uint32_t jobs = A.seqs * A.q_heads * (A.dim / 32u);
        if (A.seqs < 8u && jobs <= 0x10000u)  // lanes of a launch are counted in 32 bits
            join_kernel<kManyWays><<<jobs, kManyWays * kWave, 0, st>>>(A, G);
        else
            join_kernel<1><<<(jobs + kWaves - 1) / kWaves, kThreads, 0, st>>>(A, G);
    }
    return hipGetLastError();
}

}  // namespace rz
