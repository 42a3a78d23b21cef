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

// Blocks of all sequences, by each wave for itself.
__device__ __forceinline__ int64_t total_blocks(const KvAttend& A) {
    int64_t n = 0;
    for (uint32_t b = threadIdx.x % kWave; b < A.seqs; b += kWave) n += blocks_of(A, b);
    return wave_sum(n);
}

// The sequence that holds block g, and the first block of it.
struct Place {
    uint32_t b;
    int64_t first;
};
__device__ __forceinline__ Place find_block(const KvAttend& A, int64_t g) {
    const int lane = threadIdx.x % kWave;
    int64_t base = 0;
    for (uint32_t b0 = 0; b0 < A.seqs; b0 += kWave) {
        const int64_t n = b0 + lane < A.seqs ? blocks_of(A, b0 + lane) : 0;
        int64_t sum = n;
#pragma unroll
        for (int off = 1; off < kWave; off <<= 1) {
            const int64_t o = __shfl_up(sum, off, kWave);
            if (lane >= off) sum += o;
        }
        const uint64_t past = __ballot(base + sum > g);
        if (past) {
            const int l = __ffsll((unsigned long long)past) - 1;
            return {b0 + l, base + __shfl(sum - n, l, kWave)};
        }
        base += __shfl(sum, kWave - 1, kWave);
    }
    return {A.seqs, base};
}

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

// Where partial results lie in the workspace: part s is fp32 [rows][dim], then m [rows], l [rows].
__device__ __forceinline__ uint64_t part_floats(uint32_t rows, uint32_t dim) { return (uint64_t)rows * (dim + 2u); }

struct Grid {
    uint32_t R;          // workers a key head (and 16 queries)
    uint32_t tiles;      // groups of 16 queries a key head
    uint32_t part_rows;  // queries that a part has room for
    bool whole;          // workers take whole sequences
    int dtype;
};

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
        int32_t slot[kWaves][2][kWave];
        float scale[FMT == kKvE4M3 ? kWaves : 1][2][2][FMT == kKvE4M3 ? kWave : 1];  // keys, values
        uint8_t byte[FMT == kKvE4M3 ? 1 : kWaves][2][2][FMT == kKvE4M3 ? 1 : C][FMT == kKvE4M3 ? 4 : kWave];
    };

    // Slot of position v of (b, h), -1: none.
    static __device__ __forceinline__ int32_t slot_at(const KvAttend& A, uint32_t b, uint32_t h, uint32_t v, uint32_t n, uint32_t len) {
        if (v >= n) return -1;
        uint32_t page = v / A.page_len;
        const uint32_t at = v - page * A.page_len;
        if (A.pages) page = (uint32_t)A.pages[((uint64_t)b * A.heads + h) * A.budget + page];
        if (page >= A.max_pages || (uint64_t)page * A.page_len + at >= len) return -1;
        const int32_t id = A.page_table[(uint64_t)b * A.max_pages + page];
        const uint64_t slot = (uint64_t)(uint32_t)id * A.page_len + at;
        return id >= 0 && slot < A.num_slots ? (int32_t)slot : -1;
    }

    // A tile's rows as they are loaded.
    struct Rows {
        uint32_t k[2][kKWords<FMT, C>], v[8][kVWords<FMT, C>];
    };

    // Loads the rows of a tile: `slot` its 32 slots, `live` those that are slots (others read row 0).
    static __device__ __forceinline__ void load(const KvAttend& A, uint32_t h, const int32_t* slot, uint32_t live, Rows& x) {
        const uint32_t lane = threadIdx.x % kWave, n = lane % 16, g = lane / 16;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint32_t p = 16 * t + n, s = live >> p & 1 ? (uint32_t)slot[p] : 0u;
            load_k<FMT, C>(A.codes[0] + ((uint64_t)s * A.heads + h) * kRow, g, x.k[t]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t p = 16 * (e / 4) + 4 * g + e % 4, s = live >> p & 1 ? (uint32_t)slot[p] : 0u;
            load_v<FMT, C>(A.codes[1] + ((uint64_t)s * A.heads + h) * kRow, n, x.v[e]);
        }
    }

    static __device__ __forceinline__ void compute(const Shared& S, int wave, int buf, int half, uint32_t live, Rows& x, State<C>& st) {
        const uint32_t lane = threadIdx.x % kWave, n = lane % 16, g = lane / 16;
        f32x4 hi[2] = {}, lo[2] = {};
#pragma unroll
        for (int s = 0; s < C; ++s) {
            const u32x4 q0 = S.q[0][s][lane], q1 = S.q[1][s][lane], q2 = S.q[2][s][lane];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                u32x4 a;
                if constexpr (FMT == kKvE4M3)
                    a = widen8<FMT>(x.k[t][2 * s], x.k[t][2 * s + 1], 1.0f);
                else
                    a = widen8<FMT>(x.k[t][s], 0u, cvt_scale(S.byte[wave][buf][0][k_column<FMT, C>(s, g) / 32][half * 32 + 16 * t + n]));
                hi[t] = mfma(a, q0, hi[t]);
                lo[t] = mfma(a, q1, lo[t]);
                lo[t] = mfma(a, q2, lo[t]);
            }
        }
        // a lane's eight positions: 16 t + 4 g + i
        float p[8], top = -INFINITY;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            f32x4 sc = hi[t] + lo[t];
            if constexpr (FMT == kKvE4M3) sc *= *reinterpret_cast<const f32x4*>(&S.scale[wave][buf][0][half * 32 + 16 * t + 4 * g]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[4 * t + i] = live >> (16 * t + 4 * g + i) & 1 ? sc[i] : -INFINITY;
                top = fmaxf(top, p[4 * t + i]);
            }
        }
        top = fmaxf(head_max(top), st.m);
        if (__any(top > st.m)) {  // rarely, after the first tiles
            const float f = __builtin_amdgcn_exp2f(st.m - base_of(top));
#pragma unroll
            for (int j = 0; j < 2 * C; ++j) st.o[j] *= f;
            st.l *= f;
            st.m = top;
        }
        const float base = base_of(top);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            p[e] = __builtin_amdgcn_exp2f(p[e] - base);
            st.l += p[e];
        }
        if constexpr (FMT == kKvE4M3) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const f32x4 sc = *reinterpret_cast<const f32x4*>(&S.scale[wave][buf][1][half * 32 + 16 * t + 4 * g]);
#pragma unroll
                for (int i = 0; i < 4; ++i) p[4 * t + i] *= sc[i];  // 0 where there is no row
            }
        }
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
                for (int i = 0; i < kVWords<FMT, C>; ++i) x.v[e][i] = on ? x.v[e][i] : 0u;
            }
        }
        using R = VRuns<C>;
        unrolled<R::count>([&](auto r_) {
            constexpr int r = decltype(r_)::value, at = R::template word<FMT>(r), wide = R::wide(r), j0 = R::product(r);
            // positions e and e + 1 side by side, a column at a time
            auto go = [&](int j, const u32x4& a) {
#pragma unroll
                for (int i = 0; i < 3; ++i) st.o[j] = mfma(a, w[i], st.o[j]);
            };
            if constexpr (FMT == kKvE4M3) {
                constexpr int step = wide < 4 ? wide : 4;
                unrolled<wide / step>([&](auto k_) {
                    constexpr int k = decltype(k_)::value;
                    u32x4 a[step];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t x0 = x.v[2 * e][at + k], x1 = x.v[2 * e + 1][at + k];
                        const uint32_t y0 = __builtin_amdgcn_perm(x1, x0, 0x05010400u);
                        a[0][e] = bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(y0, 1.0f, false));
                        a[1][e] = bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(y0, 1.0f, true));
                        if constexpr (step == 4) {
                            const uint32_t y1 = __builtin_amdgcn_perm(x1, x0, 0x07030602u);
                            a[2][e] = bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(y1, 1.0f, false));
                            a[3][e] = bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(y1, 1.0f, true));
                        }
                    }
#pragma unroll
                    for (int i = 0; i < step; ++i) go(j0 + step * k + i, a[i]);
                });
            } else {
                // a lane's columns lie in one block of 32
                float sc[8];
                const uint8_t* by = S.byte[wave][buf][1][(R::column(r) + wide * n) / 32] + half * 32;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const uint32_t four = *reinterpret_cast<const uint32_t*>(by + 16 * t + 4 * g);
#pragma unroll
                    for (int i = 0; i < 4; ++i) sc[4 * t + i] = cvt_scale(four >> (8 * i) & 255u);
                }
                unrolled<wide / 2>([&](auto c_) {
                    constexpr int c = decltype(c_)::value;  // columns 2 c and 2 c + 1
                    u32x4 a[2];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t x0 = bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x.v[2 * e][at + c / 4], sc[2 * e], c % 4));
                        const uint32_t x1 = bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x.v[2 * e + 1][at + c / 4], sc[2 * e + 1], c % 4));
                        a[0][e] = __builtin_amdgcn_perm(x1, x0, 0x05040100u);
                        a[1][e] = __builtin_amdgcn_perm(x1, x0, 0x07060302u);
                    }
                    go(j0 + 2 * c, a[0]);
                    go(j0 + 2 * c + 1, a[1]);
                });
            }
        });
    }

    // This lane's row's scales: fp32 of its key and value, or C bytes each.
    struct Scales2 {
        uint32_t x[FMT == kKvE4M3 ? 2 : 2 * C];
    };
    static __device__ __forceinline__ void load_scales(const KvAttend& A, uint32_t h, int32_t slot, Scales2& s) {
        const uint64_t row = (uint64_t)(uint32_t)(slot < 0 ? 0 : slot) * A.heads + h;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if constexpr (FMT == kKvE4M3) {
                s.x[c] = static_cast<const uint32_t*>(A.scales[c])[row];
                if (slot < 0) s.x[c] = 0;
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
                if (slot < 0)
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

    // Blocks [first, last) of sequence b, by the workgroup: every wave's own tiles of 32 into `st`.
    static __device__ __forceinline__ void blocks(const KvAttend& A, Shared& S, uint32_t b, uint32_t h, uint32_t first, uint32_t last, State<C>& st) {
        const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
        const uint32_t n = length_of(A, b), len = (uint32_t)A.lens[b];
        // two blocks at a time: lanes 0..31 take the tile of the first, 32..63 that of the second
        auto find = [&](uint32_t block) {
            const uint32_t at = block + lane / 32;
            return at < last ? slot_at(A, b, h, at * kBlock + wave * kTile + lane % 32, n, len) : -1;
        };
        int buf = 0;
        int32_t slot = find(first);
        uint64_t live = __ballot(slot >= 0);
        S.slot[wave][0][lane] = slot;
        Scales2 sc;
        load_scales(A, h, slot, sc);
        wave_sync();
        Rows x0, x1;
        load(A, h, S.slot[wave][0], (uint32_t)live, x0);
        keep_scales(S, wave, 0, sc);
        wave_sync();
        for (uint32_t at = first; at < last; at += 2) {
            int32_t ahead = at + 2 < last ? find(at + 2) : -1;  // uniform branch
            load(A, h, S.slot[wave][buf] + 32, (uint32_t)(live >> 32), x1);
            if ((uint32_t)live) compute(S, wave, buf, 0, (uint32_t)live, x0, st);
            const uint64_t next = __ballot(ahead >= 0);
            S.slot[wave][buf ^ 1][lane] = ahead;
            load_scales(A, h, ahead, sc);
            wave_sync();
            load(A, h, S.slot[wave][buf ^ 1], (uint32_t)next, x0);
            if ((uint32_t)(live >> 32)) compute(S, wave, buf, 1, (uint32_t)(live >> 32), x1, st);
            keep_scales(S, wave, buf ^ 1, sc);
            wave_sync();
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

    // Blocks [first, last) of (b, h, tile z); `part`: where they go if they are not the whole of a sequence.
    static __device__ void piece(const KvAttend& A, const Grid& G, Shared& S, uint32_t b, uint32_t h, uint32_t z, uint32_t first, uint32_t last, float* part) {
        const uint32_t lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, n = lane % 16, g = lane / 16;
        const uint32_t group = A.q_heads / A.heads, rows = group - z * kHeads < kHeads ? group - z * kHeads : kHeads;
        const uint64_t head0 = (uint64_t)b * A.q_heads + h * group + z * kHeads;
        __syncthreads();  // the last piece's results have been read
        const float unit = A.scale * 1.44269504088896341f;  // scores in powers of two
        for (uint32_t s = wave; s < C; s += kWaves) {
            u32x4 w[3] = {};
            if (n < rows) {
                const float* q = A.q + b * A.q_stride + (uint64_t)(h * group + z * kHeads + n) * D + k_column<FMT, C>(s, g);
                const f32x4 a = *reinterpret_cast<const f32x4*>(q) * unit, c = *reinterpret_cast<const f32x4*>(q + 4) * unit;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const Parts p = e < 2 ? split2(a[2 * e], a[2 * e + 1]) : split2(c[2 * e - 4], c[2 * e - 3]);
#pragma unroll
                    for (int i = 0; i < 3; ++i) w[i][e] = p.part[i];
                }
            }
#pragma unroll
            for (int i = 0; i < 3; ++i) S.q[i][s][lane] = w[i];
        }
        __syncthreads();
        State<C> st;
#pragma unroll
        for (int j = 0; j < 2 * C; ++j) st.o[j] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
        st.m = -INFINITY;
        st.l = 0.0f;
        blocks(A, S, b, h, first, last, st);
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
        const float inv = 1.0f / st.l;
        using R = VRuns<C>;
        unrolled<R::count>([&](auto r_) {
            constexpr int r = decltype(r_)::value, wide = R::wide(r), j0 = R::product(r);
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // `wide` consecutive columns
                const uint32_t col = R::column(r) + wide * (4 * g + i);
                if (part) {
#pragma unroll
                    for (int j = 0; j < wide; ++j) part[n * D + col + j] = st.o[j0 + j][i];
                } else {
#pragma unroll
                    for (int j = 0; j < wide; ++j) {
                        const float v = st.l == 0.0f ? 0.0f : st.o[j0 + j][i] * inv;
                        const uint64_t at = (head0 + n) * D + col + j;
                        if (G.dtype == kF32)
                            static_cast<float*>(A.out)[at] = v;
                        else if (G.dtype == kF16)
                            static_cast<_Float16*>(A.out)[at] = (_Float16)v;
                        else
                            static_cast<__bf16*>(A.out)[at] = (__bf16)v;
                    }
                }
            }
        });
        if (g == 0) {
            if (part) {
                part[G.part_rows * D + n] = st.m;
                part[G.part_rows * (D + 1) + n] = st.l;
            } else if (A.lse)
                A.lse[head0 + n] = st.l == 0.0f ? -INFINITY : st.m * 0.693147180559945309f + logf(st.l);
        }
    }
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
__global__ __launch_bounds__(kThreads, C <= 4 ? 2 : 1) void attend_kernel(KvAttend A, Grid G) {
    using K = Kernel<FMT, C>;
    __shared__ typename K::Shared S;
    const uint32_t lanes = A.heads * G.tiles, r = blockIdx.x / lanes, h = blockIdx.x % lanes / G.tiles, z = blockIdx.x % G.tiles;
    if (G.whole) {
        for (uint32_t b = r; b < A.seqs; b += G.R) {
            const uint32_t n = blocks_of(A, b);
            if (n)
                K::piece(A, G, S, b, h, z, 0, n, nullptr);
            else
                empty<C>(A, G, b, h, z);
        }
        return;
    }
    for (uint32_t b = r; b < A.seqs; b += G.R)
        if (blocks_of(A, b) == 0) empty<C>(A, G, b, h, z);
    const int64_t T = total_blocks(A);
    const uint32_t R = workers_of(T, G.R);
    if (r >= R) return;
    int64_t at = share(T, r, R);
    const int64_t end = share(T, r + 1, R);
    Place p = find_block(A, at);
    float* part = static_cast<float*>(A.ws) + (uint64_t)blockIdx.x * 2u * part_floats(G.part_rows, K::D);
    while (at < end) {
        const uint32_t n = blocks_of(A, p.b), first = (uint32_t)(at - p.first);
        if (n == 0) {
            ++p.b;
            continue;
        }
        const uint32_t last = end - p.first < n ? (uint32_t)(end - p.first) : n;
        K::piece(A, G, S, p.b, h, z, first, last, first == 0 && last == n ? nullptr : part + (first == 0 ? part_floats(G.part_rows, K::D) : 0));
        at += last - first;
        p.first += n;
        ++p.b;
    }
}

// Joins the parts of sequences that several workers hold: a workgroup a query.
__global__ __launch_bounds__(kThreads) void join_kernel(KvAttend A, Grid G) {
    const uint32_t b = blockIdx.x / A.q_heads, qh = blockIdx.x % A.q_heads, group = A.q_heads / A.heads;
    const uint32_t h = qh / group, z = qh % group / kHeads, row = qh % group % kHeads, lanes = A.heads * G.tiles;
    const uint32_t n = blocks_of(A, b);
    if (n == 0) return;
    int64_t T = 0, g0 = 0;
    for (uint32_t i = threadIdx.x % kWave; i < A.seqs; i += kWave) {
        const uint32_t k = blocks_of(A, i);
        T += k;
        if (i < b) g0 += k;
    }
    T = wave_sum(T);
    g0 = wave_sum(g0);
    const uint32_t R = workers_of(T, G.R), r0 = worker_of(T, g0, R), r1 = worker_of(T, g0 + n - 1, R);
    if (r0 == r1) return;
    const uint64_t floats = part_floats(G.part_rows, A.dim);
    // worker r0 began the sequence: its second part; the others hold it from their start: their first
    auto part = [&](uint32_t r) {
        const uint32_t block = r * lanes + h * G.tiles + z;
        return static_cast<const float*>(A.ws) + ((uint64_t)block * 2u + (r == r0 ? 1u : 0u)) * floats;
    };
    __shared__ float top_of[kWaves], sum_of[kWaves];
    float top = -INFINITY;
    for (uint32_t r = r0 + threadIdx.x; r <= r1; r += kThreads) top = fmaxf(top, part(r)[G.part_rows * A.dim + row]);
    for (int off = 1; off < kWave; off <<= 1) top = fmaxf(top, __shfl_xor(top, off, kWave));
    if (threadIdx.x % kWave == 0) top_of[threadIdx.x / kWave] = top;
    __syncthreads();
    for (int i = 0; i < kWaves; ++i) top = fmaxf(top, top_of[i]);
    const float base = base_of(top);
    float sum = 0.0f;
    for (uint32_t r = r0 + threadIdx.x; r <= r1; r += kThreads) {
        const float* p = part(r) + G.part_rows * A.dim + row;
        sum += p[G.part_rows] * __builtin_amdgcn_exp2f(p[0] - base);
    }
    for (int off = 1; off < kWave; off <<= 1) sum += __shfl_xor(sum, off, kWave);
    if (threadIdx.x % kWave == 0) sum_of[threadIdx.x / kWave] = sum;
    __syncthreads();
    sum = 0.0f;
    for (int i = 0; i < kWaves; ++i) sum += sum_of[i];
    const float inv = 1.0f / sum;
    const uint64_t head = (uint64_t)b * A.q_heads + qh;
    for (uint32_t d = threadIdx.x; d < A.dim; d += kThreads) {
        float o = 0.0f;
        for (uint32_t r = r0; r <= r1; ++r) {
            const float* p = part(r);
            o += p[row * A.dim + d] * __builtin_amdgcn_exp2f(p[G.part_rows * A.dim + row] - base);
        }
        const float v = sum == 0.0f ? 0.0f : o * inv;
        if (G.dtype == kF32)
            static_cast<float*>(A.out)[head * A.dim + d] = v;
        else if (G.dtype == kF16)
            static_cast<_Float16*>(A.out)[head * A.dim + d] = (_Float16)v;
        else
            static_cast<__bf16*>(A.out)[head * A.dim + d] = (__bf16)v;
    }
    if (A.lse && threadIdx.x == 0) A.lse[head] = sum == 0.0f ? -INFINITY : top * 0.693147180559945309f + logf(sum);
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

}  // namespace

size_t kv_attend_ws_bytes(uint32_t q_heads, uint32_t heads, uint32_t dim, int cus) {
    const uint64_t lanes = (uint64_t)heads * ((q_heads / heads + kHeads - 1) / kHeads);
    return split(q_heads, heads, cus) * lanes * 2u * (uint64_t)part_rows(q_heads, heads) * (dim + 2u) * 4u;
}

hipError_t launch_kv_attend(int format, const KvAttend& A, int dtype, int cus, hipStream_t st) {
    Grid G;
    G.tiles = (A.q_heads / A.heads + kHeads - 1) / kHeads;
    G.part_rows = part_rows(A.q_heads, A.heads);
    G.dtype = dtype;
    // one block a sequence at most: nothing to split
    const uint64_t most = (uint64_t)(A.pages ? A.budget : A.max_pages) * A.page_len;
    G.whole = !A.ws || most <= kBlock || (uint64_t)A.seqs * A.q_heads >= 0x1000000u;
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
    if (!G.whole) join_kernel<<<A.seqs * A.q_heads, kThreads, 0, st>>>(A, G);
    return hipGetLastError();
}

}  // namespace rz
