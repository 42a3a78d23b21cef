// Attention of one new token a sequence over the quantised, paged cache:
//   out[b][h] = sum_p w_p v_p,  w = softmax(scale q[b][h] . k_p),
// one pass over the rows with the running maximum and sum of the softmax.
//
// A step reads each cached row once for all the queries of its key head, so
// it is bound by memory; the products run on the bf16 matrix cores, whose
// operands hold E4M3 and E2M1 codes exactly.  Both products put positions or
// columns of the cache in the rows of the result and query heads in its
// columns (16 of them), so that a lane has the same head throughout:
//   scores  S[32 positions][16 heads] = K q^T, a lane reads 8 columns of a row
//           a step as they lie; which columns those are is the same for both
//           operands, so 16-byte loads serve two steps (four in MXFP4);
//   output  O[16 columns][16 heads] += V^T P, contraction over 32 positions:
//           lane l holds the weights of positions 4 (l/16) + i and those + 16
//           for head l % 16, which is where S leaves them, and reads V's rows
//           of these eight positions.  Nothing moves between lanes but the
//           maximum.
// q and the weights stay fp32: each is the exact sum of three bf16 parts (8
// bits each, cut, not rounded), multiplied one after another into fp32.
//
// Workgroups take equal shares of all blocks of 128 positions, whatever the
// sequences' lengths: worker r of R reads blocks [T r / R, T (r + 1) / R) of
// the T that the batch has, for one key head (and 16 of its queries); the
// heads of the same blocks are neighbours in the grid, so a page is read by
// all of them at a time.  What is not the whole of a sequence goes to the
// workspace, at most two parts a worker, and a second launch joins them.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "mx_device.h"
#include "rz_device.h"
#include "rz_internal.h"

namespace rz {
namespace {
using namespace mx;

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr uint32_t kTile = 32;               // positions a wave takes at a time
constexpr uint32_t kBlock = kTile * kWaves;  // and a workgroup
constexpr uint32_t kHeads = 16;              // queries of a key head that a workgroup serves

// Positions that sequence b attends (those of a choice may hold gaps).
__device__ __forceinline__ uint32_t length_of(const KvAttend& A, uint32_t b) {
    const int32_t len = A.lens[b];
    if (len <= 0 || A.num_slots == 0) return 0;
    if (A.pages) return A.budget * A.page_len;
    const uint64_t most = (uint64_t)A.max_pages * A.page_len;
    return (uint32_t)((uint64_t)len < most ? len : most);
}
__device__ __forceinline__ uint32_t blocks_of(const KvAttend& A, uint32_t b) { return (length_of(A, b) + kBlock - 1) / kBlock; }

__device__ __forceinline__ int64_t wave_sum(int64_t v) {
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) v += __shfl_xor(v, off, kWave);
    return v;
}

// Where the batch's blocks lie, as every wave finds it for itself: sequences
// are looked at 64 at a time, a lane each.
struct Batch {
    int64_t total = 0;        // blocks of all sequences
    uint32_t b0 = 0;          // the 64 that `count` is of
    uint32_t count = 0, sum = 0;  // a lane's sequence's blocks, and those of the lanes before it and its own
    int64_t base = 0;         // blocks before b0

    __device__ __forceinline__ void look(const KvAttend& A) {
        const uint32_t lane = threadIdx.x % kWave, b = b0 + lane;
        count = b < A.seqs ? blocks_of(A, b) : 0;
        sum = count;  // 64 of at most 2^24
#pragma unroll
        for (int off = 1; off < kWave; off <<= 1) {
            const uint32_t o = __shfl_up(sum, off, kWave);
            if (lane >= off) sum += o;
        }
    }
    __device__ __forceinline__ void begin(const KvAttend& A) {
        look(A);
        total = (uint32_t)__shfl((int)sum, kWave - 1, kWave);
        if (A.seqs > kWave) {
            int64_t n = 0;
            for (uint32_t b = kWave + threadIdx.x % kWave; b < A.seqs; b += kWave) n += blocks_of(A, b);
            total += wave_sum(n);
        }
    }
    // A block's sequence, the blocks before that and in it; g < total, not below the last one asked for.
    struct Place {
        uint32_t b, count;
        int64_t first;
    };
    __device__ __forceinline__ Place find(const KvAttend& A, int64_t g) {
        for (;;) {
            const uint64_t past = __ballot(base + sum > g);
            if (past) {
                const int l = __ffsll((unsigned long long)past) - 1;
                const uint32_t n = (uint32_t)__shfl((int)count, l, kWave);
                return {b0 + l, n, base + (uint32_t)__shfl((int)sum, l, kWave) - n};
            }
            base += (uint32_t)__shfl((int)sum, kWave - 1, kWave);
            b0 += kWave;
            look(A);
        }
    }
};

// Workers that get a block: each of them does.  The share of worker r: blocks [T r / R, T (r + 1) / R); and the worker of block g.
__device__ __forceinline__ uint32_t workers_of(int64_t T, uint32_t R) { return T < R ? (uint32_t)T : R; }
__device__ __forceinline__ int64_t share(int64_t T, uint32_t r, uint32_t R) { return T * r / R; }
__device__ __forceinline__ uint32_t worker_of(int64_t T, int64_t g, uint32_t R) { return (uint32_t)(((g + 1) * R - 1) / T); }

// ---- rows of the cache in registers

__device__ __forceinline__ uint32_t bits(bf16x2 v) { return __builtin_bit_cast(uint32_t, v); }

// Eight consecutive codes as bf16 (times `scale`, a power of two, for MXFP4).
template <int FMT>
__device__ __forceinline__ u32x4 widen8(uint32_t w0, uint32_t w1, float scale) {
    if constexpr (FMT == kKvE4M3) {
        return (u32x4){bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, false)), bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, true)),
                       bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, false)), bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, true))};
    } else {
        return (u32x4){bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w0, scale, 0)), bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w0, scale, 1)),
                       bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w0, scale, 2)), bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w0, scale, 3))};
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

// Three bf16 parts of two values, which they sum to exactly (24 bits in all).
struct Parts {
    uint32_t part[3];
};
__device__ __forceinline__ Parts split2(float a, float b) {
    Parts s;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        s.part[i] = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
        a -= __uint_as_float(__float_as_uint(a) & 0xFFFF0000u);
        b -= __uint_as_float(__float_as_uint(b) & 0xFFFF0000u);
    }
    return s;
}

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// A wave's running state: o[j][i] is column VRuns' product j, row 4 g + i, of head l % 16.
template <int C>
struct State {
    f32x4 o[2 * C];
    float m, l;
};

// Floats of one part in the workspace: [rows][dim], then m [rows], l [rows]; the next begins on 16 bytes.
__host__ __device__ __forceinline__ uint64_t part_floats(uint32_t rows, uint32_t dim) { return ((uint64_t)rows * (dim + 2u) + 3u) & ~3ull; }

struct Grid {
    uint32_t R;          // workers a key head (and 16 queries)
    uint32_t tiles;      // groups of 16 queries a key head
    uint32_t part_rows;  // queries that a part has room for
    bool whole;          // workers take whole sequences
    uint64_t info;       // floats before the workspace's record of who holds which sequence
    int dtype;
};

// Zeros for sequence b's rows of (h, z).
template <int C>
__device__ __forceinline__ void empty(const KvAttend& A, const Grid& G, uint32_t b, uint32_t h, uint32_t z) {
    const uint32_t group = A.q_heads / A.heads, rows = group - z * kHeads < kHeads ? group - z * kHeads : kHeads;
    const uint64_t head0 = (uint64_t)b * A.q_heads + h * group + z * kHeads;
    for (uint32_t i = threadIdx.x; i < rows * 32u * C; i += kThreads) {
        if (G.dtype == kF32)
            static_cast<float*>(A.out)[head0 * 32u * C + i] = 0.0f;
        else
            static_cast<uint16_t*>(A.out)[head0 * 32u * C + i] = 0;
    }
    if (A.lse && threadIdx.x < rows) A.lse[head0 + threadIdx.x] = -INFINITY;
}

template <int FMT, int C>
struct Kernel {
    static constexpr uint32_t D = 32 * C;
    static constexpr uint32_t kRow = FMT == kKvE4M3 ? D : D / 2;  // bytes

    struct Shared {
        union {
            u32x4 q[3][C][kWave];       // the query's parts as the matrix cores take them
            float o[2][8 * C][kWave];   // two waves' results
        };
        float m[2][kWave], l[2][kWave];
        // two tiles a wave at a time, twice
        uint32_t row[kWaves][2][kWave];  // rows of the cache; row 0's stands in for what is none
        float scale[FMT == kKvE4M3 ? kWaves : 1][2][2][FMT == kKvE4M3 ? kWave : 1];  // keys, values
        uint8_t byte[FMT == kKvE4M3 ? 1 : kWaves][2][2][FMT == kKvE4M3 ? 1 : C][FMT == kKvE4M3 ? 4 : kWave];
    };

    // Where position v of (b, h) lies, as far as the length need not be known: its page's number in the cache (-1: none)
    // and its place in the sequence.
    struct Spot {
        int32_t id;
        uint32_t at;    // in the page
        uint64_t place;
    };
    static __device__ __forceinline__ Spot spot(const KvAttend& A, uint32_t b, uint32_t h, uint32_t v) {
        uint32_t page = v / A.page_len;
        Spot s = {-1, v - page * A.page_len, 0};
        if (A.pages) page = page < A.budget ? (uint32_t)A.pages[((uint64_t)b * A.heads + h) * A.budget + page] : ~0u;
        s.place = (uint64_t)page * A.page_len + s.at;
        if (page < A.max_pages) s.id = A.page_table[(uint64_t)b * A.max_pages + page];
        return s;
    }
    static __device__ __forceinline__ int32_t slot_of(const KvAttend& A, const Spot& s, uint32_t len) {
        const uint64_t slot = (uint64_t)(uint32_t)s.id * A.page_len + s.at;
        return s.id >= 0 && s.place < len && slot < A.num_slots ? (int32_t)slot : -1;
    }

    // A tile's rows as they are loaded; `row` its 32 rows of the cache.
    static __device__ __forceinline__ void load_keys(const KvAttend& A, const uint32_t* row, uint32_t (&k)[2][kKWords<FMT, C>]) {
        const uint32_t n = threadIdx.x % 16, g = threadIdx.x % kWave / 16;
#pragma unroll
        for (int t = 0; t < 2; ++t) load_k<FMT, C>(A.codes[0] + (uint64_t)row[16 * t + n] * kRow, g, k[t]);
    }
    static __device__ __forceinline__ void load_values(const KvAttend& A, const uint32_t* row, uint32_t (&v)[8][kVWords<FMT, C>]) {
        const uint32_t n = threadIdx.x % 16, g = threadIdx.x % kWave / 16;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const u32x4 at = *reinterpret_cast<const u32x4*>(row + 16 * t + 4 * g);
#pragma unroll
            for (int i = 0; i < 4; ++i) load_v<FMT, C>(A.codes[1] + (uint64_t)at[i] * kRow, n, v[4 * t + i]);
        }
    }

    // Scores of a tile, in powers of two: p[4 t + i] of position 16 t + 4 g + i.
    static __device__ __forceinline__ void scores(const Shared& S, int wave, int buf, int half, const uint32_t (&k)[2][kKWords<FMT, C>], float (&p)[8]) {
        const uint32_t lane = threadIdx.x % kWave, n = lane % 16, g = lane / 16;
        f32x4 hi[2] = {}, lo[2] = {};
#pragma unroll
        for (int s = 0; s < C; ++s) {
            const u32x4 q0 = S.q[0][s][lane], q1 = S.q[1][s][lane], q2 = S.q[2][s][lane];
            u32x4 a[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if constexpr (FMT == kKvE4M3)
                    a[t] = widen8<FMT>(k[t][2 * s], k[t][2 * s + 1], 1.0f);
                else
                    a[t] = widen8<FMT>(k[t][s], 0u, cvt_scale(S.byte[wave][buf][0][k_column<FMT, C>(s, g) / 32][half * 32 + 16 * t + n]));
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) hi[t] = mfma(a[t], q0, hi[t]);
#pragma unroll
            for (int t = 0; t < 2; ++t) lo[t] = mfma(a[t], q1, lo[t]);
#pragma unroll
            for (int t = 0; t < 2; ++t) lo[t] = mfma(a[t], q2, lo[t]);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            f32x4 sc = hi[t] + lo[t];
            if constexpr (FMT == kKvE4M3) sc *= *reinterpret_cast<const f32x4*>(&S.scale[wave][buf][0][half * 32 + 16 * t + 4 * g]);
#pragma unroll
            for (int i = 0; i < 4; ++i) p[4 * t + i] = sc[i];
        }
    }

    // Scores into weights relative to the running maximum, `live` the positions that count; E4M3: times the values' scales.
    static __device__ __forceinline__ void weigh(const Shared& S, int wave, int buf, int half, uint32_t live, float (&p)[8], State<C>& st) {
        const uint32_t g = threadIdx.x % kWave / 16;
        if (live != 0xFFFFFFFFu) {
#pragma unroll
            for (int e = 0; e < 8; ++e) p[e] = live >> (16 * (e / 4) + 4 * g + e % 4) & 1 ? p[e] : -INFINITY;
        }
        float top = fmaxf(fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3])), fmaxf(fmaxf(p[4], p[5]), fmaxf(p[6], p[7])));
        top = fmaxf(head_max(top), st.m);
        const float base = base_of(top);
        if (__any(top > st.m)) {  // rarely, after the first tiles
            const float f = __builtin_amdgcn_exp2f(st.m - base);
#pragma unroll
            for (int j = 0; j < 2 * C; ++j) st.o[j] *= f;
            st.l *= f;
            st.m = top;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = __builtin_amdgcn_exp2f(p[e] - base);
        st.l += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
        if constexpr (FMT == kKvE4M3) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const f32x4 sc = *reinterpret_cast<const f32x4*>(&S.scale[wave][buf][1][half * 32 + 16 * t + 4 * g]);
#pragma unroll
                for (int i = 0; i < 4; ++i) p[4 * t + i] *= sc[i];  // 0 where there is no row
            }
        }
    }

    // o += the tile's values times its weights.
    static __device__ __forceinline__ void add_values(const Shared& S, int wave, int buf, int half, uint32_t live, const float (&p)[8],
                                                      uint32_t (&v)[8][kVWords<FMT, C>], State<C>& st) {
        const uint32_t n = threadIdx.x % 16, g = threadIdx.x % kWave / 16;
        u32x4 w[3];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const Parts s = split2(p[2 * e], p[2 * e + 1]);
#pragma unroll
            for (int i = 0; i < 3; ++i) w[i][e] = s.part[i];
        }
        if (live != 0xFFFFFFFFu) {  // what lies in no row's place must not meet a weight of 0
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const bool on = live >> (16 * (e / 4) + 4 * g + e % 4) & 1;
#pragma unroll
                for (int i = 0; i < kVWords<FMT, C>; ++i) v[e][i] = on ? v[e][i] : 0u;
            }
        }
        using R = VRuns<C>;
        unrolled<R::count>([&](auto r_) {
            constexpr int r = decltype(r_)::value, at = R::template word<FMT>(r), wide = R::wide(r), j0 = R::product(r);
            constexpr int step = wide < 4 ? wide : 4;  // columns at a time
            [[maybe_unused]] float sc[8];
            if constexpr (FMT == kKvMXFP4) {  // a lane's columns lie in one block of 32
                const uint8_t* by = S.byte[wave][buf][1][(R::column(r) + wide * n) / 32] + half * 32;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const uint32_t four = *reinterpret_cast<const uint32_t*>(by + 16 * t + 4 * g);
#pragma unroll
                    for (int i = 0; i < 4; ++i) sc[4 * t + i] = cvt_scale(four >> (8 * i) & 255u);
                }
            }
            unrolled<wide / step>([&](auto k_) {
                constexpr int k = decltype(k_)::value;
                u32x4 a[step];  // positions e and e + 1 side by side, a column at a time
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (FMT == kKvE4M3) {
                        const uint32_t x0 = v[2 * e][at + k], x1 = v[2 * e + 1][at + k];
                        const uint32_t y0 = __builtin_amdgcn_perm(x1, x0, 0x05010400u);
                        a[0][e] = bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(y0, 1.0f, false));
                        a[1][e] = bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(y0, 1.0f, true));
                        if constexpr (step == 4) {
                            const uint32_t y1 = __builtin_amdgcn_perm(x1, x0, 0x07030602u);
                            a[2][e] = bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(y1, 1.0f, false));
                            a[3][e] = bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(y1, 1.0f, true));
                        }
                    } else {
                        unrolled<step / 2>([&](auto c_) {
                            constexpr int c = decltype(c_)::value, two = step / 2 * k + c;  // columns 2 two and 2 two + 1
                            const uint32_t x0 = bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[2 * e][at + two / 4], sc[2 * e], two % 4));
                            const uint32_t x1 = bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[2 * e + 1][at + two / 4], sc[2 * e + 1], two % 4));
                            a[2 * c][e] = __builtin_amdgcn_perm(x1, x0, 0x05040100u);
                            a[2 * c + 1][e] = __builtin_amdgcn_perm(x1, x0, 0x07060302u);
                        });
                    }
                }
#pragma unroll
                for (int i = 0; i < 3; ++i)
#pragma unroll
                    for (int j = 0; j < step; ++j) st.o[j0 + step * k + j] = mfma(a[j], w[i], st.o[j0 + step * k + j]);
            });
        });
    }

    // This lane's row's scales: fp32 of its key and value, or C bytes each.
    struct Scales2 {
        uint32_t x[FMT == kKvE4M3 ? 2 : 2 * C];
    };
    static __device__ __forceinline__ void load_scales(const KvAttend& A, uint64_t row, bool live, Scales2& s) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if constexpr (FMT == kKvE4M3) {
                s.x[c] = static_cast<const uint32_t*>(A.scales[c])[row];
                if (!live) s.x[c] = 0;
            } else {
                const uint8_t* p = static_cast<const uint8_t*>(A.scales[c]) + row * C;
                if constexpr (C % 4 == 0) {
#pragma unroll
                    for (int i = 0; i < C / 4; ++i) {
                        const uint32_t w = reinterpret_cast<const uint32_t*>(p)[i];
#pragma unroll
                        for (int j = 0; j < 4; ++j) s.x[c * C + 4 * i + j] = w >> (8 * j) & 255u;
                    }
                } else if constexpr (C % 2 == 0) {
#pragma unroll
                    for (int i = 0; i < C / 2; ++i) {
                        const uint32_t w = reinterpret_cast<const uint16_t*>(p)[i];
                        s.x[c * C + 2 * i] = w & 255u;
                        s.x[c * C + 2 * i + 1] = w >> 8;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < C; ++i) s.x[c * C + i] = p[i];
                }
                if (!live)
#pragma unroll
                    for (int i = 0; i < C; ++i) s.x[c * C + i] = 0;
            }
        }
    }
    static __device__ __forceinline__ void keep_scales(Shared& S, int wave, int buf, const Scales2& s) {
        const uint32_t lane = threadIdx.x % kWave;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if constexpr (FMT == kKvE4M3)
                S.scale[wave][buf][c][lane] = __uint_as_float(s.x[c]);
            else
#pragma unroll
                for (int i = 0; i < C; ++i) S.byte[wave][buf][c][i][lane] = (uint8_t)s.x[c * C + i];
        }
    }

    // LDS of one wave, written and read by its own lanes.
    static __device__ __forceinline__ void wave_sync() {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }

    // Two blocks at a time: lanes 0..31 take a wave's tile of the first, 32..63 that of the second.
    static __device__ __forceinline__ Spot spot_in(const KvAttend& A, uint32_t b, uint32_t h, uint32_t block) {
        const uint32_t lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
        return spot(A, b, h, (block + lane / 32) * kBlock + wave * kTile + lane % 32);
    }

    // Blocks [first, last) of sequence b, by the workgroup: every wave's own tiles of 32 into `st`.  `begin`: the first ones' spots.
    static __device__ __forceinline__ void blocks(const KvAttend& A, Shared& S, uint32_t b, uint32_t h, const Spot& begin, uint32_t len, uint32_t first,
                                                  uint32_t last, State<C>& st) {
        const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
        auto slot_in = [&](const Spot& s, uint32_t block) { return block + lane / 32 < last ? slot_of(A, s, len) : -1; };
        Scales2 sc;
        // the rows of two blocks' spots into buffer `buf`, their scales on their way
        auto rows_of = [&](const Spot& s, uint32_t block, int buf) {
            const int32_t slot = slot_in(s, block);
            const uint32_t row = (uint32_t)((slot < 0 ? 0 : slot) * A.heads + h);  // below 2^31
            S.row[wave][buf][lane] = row;
            load_scales(A, row, slot >= 0, sc);
            return __ballot(slot >= 0);
        };
        uint64_t live = rows_of(begin, first, 0);
        wave_sync();
        uint32_t k[2][kKWords<FMT, C>], v[8][kVWords<FMT, C>];
        load_keys(A, S.row[wave][0], k);
        load_values(A, S.row[wave][0], v);
        keep_scales(S, wave, 0, sc);
        wave_sync();
        int buf = 0;
        for (uint32_t at = first; at < last; at += 2) {
            Spot s = {-1, 0, 0};
            if (at + 2 < last) s = spot_in(A, b, h, at + 2);
            uint64_t next = 0;
#pragma unroll
            for (int half = 0; half < 2; ++half) {  // the next tile's keys are loaded once this one's are used, its values likewise
                const uint32_t on = (uint32_t)(live >> (32 * half));
                const uint32_t* then = half ? S.row[wave][buf ^ 1] : S.row[wave][buf] + 32;
                float p[8];
                if (on) scores(S, wave, buf, half, k, p);
                load_keys(A, then, k);
                if (on) {
                    weigh(S, wave, buf, half, on, p, st);
                    add_values(S, wave, buf, half, on, p, v, st);
                }
                load_values(A, then, v);
                if (half == 0) next = rows_of(s, at + 2, buf ^ 1);
                if (half == 1) keep_scales(S, wave, buf ^ 1, sc);
                wave_sync();
            }
            live = next;
            buf ^= 1;
        }
    }

    // Adds the state that lane, by lane, lies in set `c` of the workgroup's LDS.
    static __device__ __forceinline__ void give(Shared& S, int c, const State<C>& st) {
        const int lane = threadIdx.x % kWave;
#pragma unroll
        for (int j = 0; j < 2 * C; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) S.o[c][4 * j + i][lane] = st.o[j][i];
        S.m[c][lane] = st.m;
        S.l[c][lane] = st.l;
    }
    static __device__ __forceinline__ void take(const Shared& S, int c, State<C>& st) {
        const int lane = threadIdx.x % kWave;
        const float m = fmaxf(st.m, S.m[c][lane]), base = base_of(m);
        const float f = __builtin_amdgcn_exp2f(st.m - base), e = __builtin_amdgcn_exp2f(S.m[c][lane] - base);
#pragma unroll
        for (int j = 0; j < 2 * C; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) st.o[j][i] = st.o[j][i] * f + S.o[c][4 * j + i][lane] * e;
        st.l = st.l * f + S.l[c][lane] * e;
        st.m = m;
    }

    // A lane's columns of its head, from element `at` on, times f.
    template <int DT>
    static __device__ __forceinline__ void store(void* out, uint64_t at, uint32_t g, float f, const State<C>& st) {
        using T = std::conditional_t<DT == kF32, float, std::conditional_t<DT == kF16, _Float16, __bf16>>;
        using R = VRuns<C>;
        unrolled<R::count>([&](auto r_) {
            constexpr int r = decltype(r_)::value, wide = R::wide(r), j0 = R::product(r);
            typedef T vec __attribute__((ext_vector_type(wide < 4 ? wide : 4)));
#pragma unroll
            for (int i = 0; i < 4; ++i)  // `wide` consecutive columns
#pragma unroll
                for (int j = 0; j < wide; j += 4) {
                    vec x;
#pragma unroll
                    for (int e = 0; e < (wide < 4 ? wide : 4); ++e) x[e] = (T)(st.o[j0 + j + e][i] * f);
                    *reinterpret_cast<vec*>(static_cast<T*>(out) + at + R::column(r) + wide * (4 * g + i) + j) = x;
                }
        });
    }

    // Blocks [first, last) of (b, h, tile z), all of them if `last` is 0; `part`: where they go if they are not the whole of
    // a sequence.  What needs no length is loaded beside it.
    static __device__ __forceinline__ void piece(const KvAttend& A, const Grid& G, Shared& S, uint32_t b, uint32_t h, uint32_t z, uint32_t first, uint32_t last,
                                                 float* part) {
        const uint32_t lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, n = lane % 16, g = lane / 16;
        const uint32_t group = A.q_heads / A.heads, rows = group - z * kHeads < kHeads ? group - z * kHeads : kHeads;
        const uint64_t head0 = (uint64_t)b * A.q_heads + h * group + z * kHeads;
        const Spot begin = spot_in(A, b, h, first);
        constexpr int kTurns = (C + kWaves - 1) / kWaves;
        f32x4 q[kTurns][2] = {};
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
            const uint32_t s = i * kWaves + wave;
            if (s < C && n < rows) {
                const float* p = A.q + b * A.q_stride + (uint64_t)(h * group + z * kHeads + n) * D + k_column<FMT, C>(s, g);
                q[i][0] = *reinterpret_cast<const f32x4*>(p);
                q[i][1] = *reinterpret_cast<const f32x4*>(p + 4);
            }
        }
        const uint32_t len = length_of(A, b);
        if (last == 0) {
            last = (len + kBlock - 1) / kBlock;
            if (last == 0) return empty<C>(A, G, b, h, z);
        }
        __syncthreads();  // the last piece's results have been read
        const float unit = A.scale * 1.44269504088896341f;  // scores in powers of two
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
            const uint32_t s = i * kWaves + wave;
            u32x4 w[3];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const f32x4 x = q[i][e / 2] * unit;
                const Parts p = split2(x[2 * (e % 2)], x[2 * (e % 2) + 1]);
#pragma unroll
                for (int k = 0; k < 3; ++k) w[k][e] = p.part[k];
            }
            if (s < C)
#pragma unroll
                for (int k = 0; k < 3; ++k) S.q[k][s][lane] = w[k];
        }
        __syncthreads();
        State<C> st;
#pragma unroll
        for (int j = 0; j < 2 * C; ++j) st.o[j] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
        st.m = -INFINITY;
        st.l = 0.0f;
        blocks(A, S, b, h, begin, A.pages ? (uint32_t)A.lens[b] : len, first, last, st);
        st.l = head_sum(st.l);
        __syncthreads();  // q is no longer read
        if (wave >= 2) give(S, wave - 2, st);
        __syncthreads();
        if (wave < 2) take(S, wave, st);
        __syncthreads();
        if (wave == 1) give(S, 0, st);
        __syncthreads();
        if (wave != 0) return;
        take(S, 0, st);
        if (n >= rows) return;
        const float inv = st.l == 0.0f ? 0.0f : 1.0f / st.l;
        if (part)
            store<kF32>(part, n * D, g, 1.0f, st);
        else if (G.dtype == kF32)
            store<kF32>(A.out, (head0 + n) * D, g, inv, st);
        else if (G.dtype == kF16)
            store<kF16>(A.out, (head0 + n) * D, g, inv, st);
        else
            store<kBF16>(A.out, (head0 + n) * D, g, inv, st);
        if (g == 0) {
            if (part) {
                part[G.part_rows * D + n] = st.m;
                part[G.part_rows * (D + 1) + n] = st.l;
            } else if (A.lse)
                A.lse[head0 + n] = lse_of(st.m, st.l);
        }
    }
};

template <int FMT, int C>
__global__ __launch_bounds__(kThreads, C <= 4 ? 2 : 1) void attend_kernel(KvAttend A, Grid G) {
    using K = Kernel<FMT, C>;
    __shared__ typename K::Shared S;
    const uint32_t lanes = A.heads * G.tiles, r = blockIdx.x / lanes, h = blockIdx.x % lanes / G.tiles, z = blockIdx.x % G.tiles;
    uint32_t* info = reinterpret_cast<uint32_t*>(static_cast<float*>(A.ws) + G.info);
    float* part = static_cast<float*>(A.ws) + (uint64_t)blockIdx.x * 2u * part_floats(G.part_rows, K::D);
    Batch batch;
    uint32_t R = G.R;
    int64_t at = r, end = A.seqs;  // whole sequences r, r + R, ..; or blocks
    if (!G.whole) {
        for (uint32_t b = r; b < A.seqs; b += G.R)
            if (blocks_of(A, b) == 0) {
                empty<C>(A, G, b, h, z);
                if (threadIdx.x == 0) info[2 * b] = info[2 * b + 1] = 0;
            }
        batch.begin(A);
        R = workers_of(batch.total, G.R);
        if (r >= R) return;
        at = share(batch.total, r, R);
        end = share(batch.total, r + 1, R);
    }
    while (at < end) {
        uint32_t b = (uint32_t)at, first = 0, last = 0;
        float* to = nullptr;
        if (!G.whole) {
            const Batch::Place p = batch.find(A, at);
            b = p.b;
            first = (uint32_t)(at - p.first);
            last = end - p.first < p.count ? (uint32_t)(end - p.first) : p.count;
            if (first != 0 || last != p.count) to = part + (first == 0 ? part_floats(G.part_rows, K::D) : 0);
            if (first == 0 && threadIdx.x == 0) {  // the same from every key head's worker
                info[2 * b] = r;
                info[2 * b + 1] = worker_of(batch.total, p.first + p.count - 1, R);
            }
        }
        K::piece(A, G, S, b, h, z, first, last, to);
        at += G.whole ? R : last - first;
    }
}

// Joins the parts of a sequence that several workers hold: a workgroup a query
// head.  Four columns a lane, and the parts shared among the rows of lanes,
// each with a running maximum of its own.
constexpr int kJoin = 1024;
__global__ __launch_bounds__(kJoin) void join_kernel(KvAttend A, Grid G) {
    const uint32_t b = blockIdx.x / A.q_heads, qh = blockIdx.x % A.q_heads, group = A.q_heads / A.heads;
    const uint32_t h = qh / group, z = qh % group / kHeads, row = qh % group % kHeads, lanes = A.heads * G.tiles;
    const uint32_t* info = reinterpret_cast<const uint32_t*>(static_cast<const float*>(A.ws) + G.info);
    const uint32_t r0 = info[2 * b], r1 = info[2 * b + 1];
    if (r0 == r1) return;
    const uint64_t floats = part_floats(G.part_rows, A.dim);
    const uint32_t cols = A.dim / 4u, ways = kJoin / cols, way = threadIdx.x / cols, col = threadIdx.x % cols * 4u;
    float m = -INFINITY, l = 0.0f;
    f32x4 o = {};
    if (way < ways) {
#pragma unroll 4
        for (uint32_t r = r0 + way; r <= r1; r += ways) {
            // worker r0 began the sequence: its second part; the others hold it from their start: their first
            const uint32_t block = r * lanes + h * G.tiles + z;
            const float* p = static_cast<const float*>(A.ws) + ((uint64_t)block * 2u + (r == r0 ? 1u : 0u)) * floats;
            const f32x4 v = *reinterpret_cast<const f32x4*>(p + row * A.dim + col);
            const float mp = p[G.part_rows * A.dim + row], lp = p[G.part_rows * (A.dim + 1u) + row];
            const float top = fmaxf(m, mp), base = base_of(top);
            const float f = __builtin_amdgcn_exp2f(m - base), e = __builtin_amdgcn_exp2f(mp - base);
            o = o * f + v * e;
            l = l * f + lp * e;
            m = top;
        }
    }
    __shared__ f32x4 o_of[kJoin];
    __shared__ float m_of[kJoin], l_of[kJoin];
    o_of[threadIdx.x] = o;
    m_of[threadIdx.x] = m;
    l_of[threadIdx.x] = l;
    __syncthreads();
    if (way != 0) return;
    float top = m;
    for (uint32_t w = 1; w < ways; ++w) top = fmaxf(top, m_of[w * cols + threadIdx.x]);
    const float base = base_of(top);
    o = (f32x4){};
    l = 0.0f;
    for (uint32_t w = 0; w < ways; ++w) {
        const float e = __builtin_amdgcn_exp2f(m_of[w * cols + threadIdx.x] - base);
        o += o_of[w * cols + threadIdx.x] * e;
        l += l_of[w * cols + threadIdx.x] * e;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const uint64_t head = (uint64_t)b * A.q_heads + qh;
#pragma unroll
    for (int i = 0; i < 4; ++i) put(A.out, G.dtype, head * A.dim + col + i, l == 0.0f ? 0.0f : o[i] * inv);
    if (A.lse && threadIdx.x == 0) A.lse[head] = lse_of(top, l);
}

// Workgroups of a launch: two a compute unit.
uint32_t workers(int cus) { return 2u * (uint32_t)cus; }

uint32_t part_rows(uint32_t q_heads, uint32_t heads) {
    const uint32_t group = q_heads / heads;
    return group < kHeads ? group : kHeads;
}

template <typename F>
void with_steps(uint32_t c, F&& f) {
    switch (c) {
#define RZ_C(n) case n: f(std::integral_constant<int, n>{}); break;
        RZ_C(1) RZ_C(2) RZ_C(3) RZ_C(4) RZ_C(5) RZ_C(6) RZ_C(7) RZ_C(8)
        RZ_C(9) RZ_C(10) RZ_C(11) RZ_C(12) RZ_C(13) RZ_C(14) RZ_C(15) RZ_C(16)
#undef RZ_C
    }
}

// Workers a key head and 16 queries of it.
uint32_t split(uint32_t q_heads, uint32_t heads, int cus) {
    const uint32_t lanes = heads * ((q_heads / heads + kHeads - 1) / kHeads);
    const uint32_t r = workers(cus) / lanes;
    return r ? r : 1;
}

// Floats of all workers' parts.
uint64_t part_total(uint32_t q_heads, uint32_t heads, uint32_t dim, int cus) {
    const uint64_t lanes = (uint64_t)heads * ((q_heads / heads + kHeads - 1) / kHeads);
    return split(q_heads, heads, cus) * lanes * 2u * part_floats(part_rows(q_heads, heads), dim);
}

}  // namespace

size_t kv_attend_ws_bytes(uint32_t seqs, uint32_t q_heads, uint32_t heads, uint32_t dim, int cus) {
    return (part_total(q_heads, heads, dim, cus) + 2u * (uint64_t)seqs) * 4u;
}

hipError_t launch_kv_attend(int format, const KvAttend& A, int dtype, int cus, hipStream_t st) {
    Grid G;
    G.tiles = (A.q_heads / A.heads + kHeads - 1) / kHeads;
    G.part_rows = part_rows(A.q_heads, A.heads);
    G.dtype = dtype;
    G.info = part_total(A.q_heads, A.heads, A.dim, cus);
    // one block a sequence at most: nothing to split
    const uint64_t most = (uint64_t)(A.pages ? A.budget : A.max_pages) * A.page_len;
    G.whole = !A.ws || most <= kBlock || (uint64_t)A.seqs * A.q_heads >= 0x400000u;
    const uint32_t lanes = A.heads * G.tiles;
    G.R = split(A.q_heads, A.heads, cus);
    if (G.whole) {
        const uint32_t limit = 0x800000u / lanes;  // workgroups of 256 lanes, which are counted in 32 bits
        G.R = A.seqs < limit ? A.seqs : limit ? limit : 1;
    }
    with_steps(A.dim / 32u, [&](auto c_) {
        constexpr int C = decltype(c_)::value;
        if (format == kKvE4M3)
            attend_kernel<kKvE4M3, C><<<G.R * lanes, kThreads, 0, st>>>(A, G);
        else
            attend_kernel<kKvMXFP4, C><<<G.R * lanes, kThreads, 0, st>>>(A, G);
    });
    if (!G.whole) join_kernel<<<A.seqs * A.q_heads, kJoin, 0, st>>>(A, G);
    return hipGetLastError();
}

}  // namespace rz
