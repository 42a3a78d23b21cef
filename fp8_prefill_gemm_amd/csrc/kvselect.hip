// Bounds of the keys in a page, and the choice of pages by them.
//
// A page and head's bounds are the largest and smallest value of each column
// over the page's filled rows, as int8 multiples of one scale, rounded away
// from the middle; a query is held as int8 too, so that
//   sum_d max(n_d hi_d, n_d lo_d) = sum_d max(n_d, 0) hi_d + min(n_d, 0) lo_d
// is a product of whole numbers on the matrix cores (below 2^24 for 512
// columns: exact in fp32 as well), the same in any order, and the choice by it
// has no rounding to depend on.  To its roundings it is an upper bound of n . k
// for every key k of the page.
//
// Few bytes are moved for each launch, so latency counts: the loads that wait for
// each other (slots, rows; lengths, tables, bounds; keys) and the barriers of
// the choice.  4 key heads of 128 columns: bounds of 64 pages of 64 rows 6.2 us, of a
// 32768-token prompt 8.6 (1.2 TB/s); scores of 8192 pages of 32 sequences 7.5
// and their choice 6.0; of 8192 pages of one 5.8 and 8.9, the choice on as many
// compute units as there are key heads.
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

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr float kTiny = 0x1p-100f;

// f over the lanes whose numbers differ in the bits from kFrom to below kTo.
template <int kFrom, int kTo, typename T, typename F>
__device__ __forceinline__ T across(T v, F&& f) {
    auto bits = [](T x) { return __builtin_bit_cast(uint32_t, x); };
    auto value = [](uint32_t x) { return __builtin_bit_cast(T, x); };
    auto lane = [&](auto c) { return value((uint32_t)__builtin_amdgcn_update_dpp(0, (int)bits(v), decltype(c)::value, 0xF, 0xF, true)); };
    if constexpr (kFrom <= 1 && kTo > 1) v = f(v, lane(std::integral_constant<int, 0xB1>{}));  // 1 0 3 2
    if constexpr (kFrom <= 2 && kTo > 2) v = f(v, lane(std::integral_constant<int, 0x4E>{}));  // 2 3 0 1
    static_assert(kFrom == 1 || kFrom >= 8);
    if constexpr (kFrom == 1 && kTo > 4) v = f(v, lane(std::integral_constant<int, 0x141>{}));  // 7 - l, alike in fours
    if constexpr (kFrom <= 8 && kTo > 8) v = f(v, lane(std::integral_constant<int, 0x128>{}));  // l + 8 of 16
    if constexpr (kFrom <= 16 && kTo > 16) {
        const auto x = __builtin_amdgcn_permlane16_swap(bits(v), bits(v), false, false);
        v = f(value(x[0]), value(x[1]));
    }
    if constexpr (kFrom <= 32 && kTo > 32) {
        const auto x = __builtin_amdgcn_permlane32_swap(bits(v), bits(v), false, false);
        v = f(value(x[0]), value(x[1]));
    }
    return v;
}
__device__ __forceinline__ uint32_t greater(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ float smaller(float a, float b) { return fminf(a, b); }

// What a largest magnitude a stands for: 1 where there is next to nothing.
__device__ __forceinline__ float sized(float a) { return a >= kTiny ? a : 1.0f; }

// ---- bounds

// Eight fp32 values of a row of keys, as the cache's read gives them.
template <int FMT>
struct Eight {
    u32x2 w;
    uint32_t sc;  // the row's fp32 scale, or the block's byte
    __device__ __forceinline__ void load(const KvBounds& A, uint64_t row, uint32_t part) {
        if constexpr (FMT == kKvE4M3) {
            w = *reinterpret_cast<const u32x2*>(A.codes + row * A.dim + part * 8u);
            sc = static_cast<const uint32_t*>(A.scales)[row];
        } else {
            w.x = *reinterpret_cast<const uint32_t*>(A.codes + row * (A.dim / 2u) + part * 4u);
            sc = static_cast<const uint8_t*>(A.scales)[row * (A.dim / 32u) + part / 4u];
        }
    }
    __device__ __forceinline__ void values(float (&x)[8]) const {
        if constexpr (FMT == kKvE4M3) {
            const float s = __uint_as_float(sc);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[j], false);
                const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[j], true);
                x[4 * j] = a.x * s;
                x[4 * j + 1] = a.y * s;
                x[4 * j + 2] = b.x * s;
                x[4 * j + 3] = b.y * s;
            }
        } else {
            decode8(w.x, x, cvt_scale(sc));
        }
    }
};

// Largest and smallest values of eight columns over some rows.
struct Ends {
    float hi[8], lo[8], bad;  // bad: not 0 where a value is none
    __device__ __forceinline__ Ends() : bad(0.0f) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            hi[j] = -INFINITY;
            lo[j] = INFINITY;
        }
    }
    // rows `way`, way + ways, .. below `filled` of a page whose first row (of `head`) is row0; kTurn of them in flight
    template <int FMT, int kTurn>
    __device__ __forceinline__ void rows(const KvBounds& A, uint64_t row0, uint32_t part, uint32_t way, uint32_t ways, uint32_t filled) {
        for (uint32_t r0 = way; r0 < filled; r0 += kTurn * ways) {
            Eight<FMT> x[kTurn];
#pragma unroll
            for (int u = 0; u < kTurn; ++u) {
                const uint32_t r = r0 + u * ways < filled ? r0 + u * ways : r0;  // a row twice changes nothing
                x[u].load(A, row0 + (uint64_t)r * A.heads, part);
            }
#pragma unroll
            for (int u = 0; u < kTurn; ++u) {
                float v[8];
                x[u].values(v);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    bad = fabsf(v[j]) < INFINITY ? bad : 1.0f;
                    hi[j] = fmaxf(hi[j], v[j]);
                    lo[j] = fminf(lo[j], v[j]);
                }
            }
        }
    }
    __device__ __forceinline__ float largest() const {
        float a = bad != 0.0f ? INFINITY : 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) a = fmaxf(a, fmaxf(fabsf(hi[j]), fabsf(lo[j])));
        return a;
    }
    // This lane's columns of (page, head) `dst`, a the largest magnitude of all of them (infinite: a value is none).
    __device__ __forceinline__ void write(const KvBounds& A, uint64_t dst, uint32_t part, float a) const {
        const bool fine = a < INFINITY;
        a = sized(a);
        const float inv = 127.0f / a;
        u32x2 up, down;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t u = 0, d = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float p = fine ? ceilf(hi[4 * j + e] * inv) : 127.0f, n = fine ? floorf(lo[4 * j + e] * inv) : -127.0f;
                u |= ((uint32_t)(int)__builtin_amdgcn_fmed3f(p, -127.0f, 127.0f) & 255u) << (8 * e);
                d |= ((uint32_t)(int)__builtin_amdgcn_fmed3f(n, -127.0f, 127.0f) & 255u) << (8 * e);
            }
            up[j] = u;
            down[j] = d;
        }
        *reinterpret_cast<u32x2*>(A.bounds + dst * 2u * A.dim + part * 8u) = up;
        *reinterpret_cast<u32x2*>(A.bounds + (dst * 2u + 1u) * A.dim + part * 8u) = down;
        if (part == 0) A.bound_scales[dst] = fine ? a / 127.0f : INFINITY;
    }
};

// Slots and pages count below 2^31 (a cache holds at most 2^36 values, 32 a
// row): a token's slot, or none.
constexpr uint32_t kNone = 0xFFFFFFFFu;
__device__ __forceinline__ uint32_t slot_at(const KvBounds& A, uint64_t t) {
    const int64_t s = t < A.tokens ? A.slots[t] : -1;
    return s < 0 || (uint64_t)s >= A.num_slots ? kNone : (uint32_t)s;
}

// How far `page` is filled by token t + l and those that follow it there, the
// lanes holding the slots of tokens t on: the largest of them counts.
__device__ __forceinline__ uint32_t filled_from(const KvBounds& A, uint64_t t, uint32_t s, int l, uint32_t page) {
    const uint32_t lane = threadIdx.x % kWave, row0 = page * A.page_len;
    uint32_t top = 0;
    for (;;) {
        const uint64_t out = ~__ballot(s - row0 < A.page_len) >> l << l;
        const uint32_t n = out ? (uint32_t)__ffsll((unsigned long long)out) - 1 : kWave;  // lanes l to n - 1 follow on
        const uint32_t at = lane >= (uint32_t)l && lane < n ? s - row0 + 1 : 0;
        top = top > at ? top : at;
        if (n < kWave) break;
        t += kWave;
        l = 0;
        s = slot_at(A, t + lane);
    }
    return across<1, kWave>(top, greater);
}

// A decoding step: a workgroup a (token, head).  A token whose predecessor lies
// in another page leads; the page's rows are shared among the rows of lanes,
// eight columns a lane (L lanes a row).
template <int FMT, int L>
__global__ __launch_bounds__(kThreads) void bounds_step_kernel(KvBounds A) {
    constexpr uint32_t ways = kThreads / L;
    __shared__ float of[17][kThreads];  // column first: no two lanes in a bank
    const uint32_t t = blockIdx.x / A.heads, head = blockIdx.x % A.heads, part = threadIdx.x % L, way = threadIdx.x / L;
    const uint32_t next = slot_at(A, (uint64_t)t + threadIdx.x % kWave), prior = t ? slot_at(A, t - 1) : kNone;
    const uint32_t s = (uint32_t)__builtin_amdgcn_readfirstlane((int)next);
    if (s == kNone) return;
    const uint32_t page = s / A.page_len;
    if (page >= A.num_pages || (prior != kNone && prior / A.page_len == page)) return;
    const uint32_t filled = filled_from(A, t, next, 0, page);
    Ends x;
    const bool live = part * 8u < A.dim;
    if (live) x.template rows<FMT, 4>(A, (uint64_t)page * A.page_len * A.heads + head, part, way, ways, filled);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        of[j][threadIdx.x] = x.hi[j];
        of[8 + j][threadIdx.x] = x.lo[j];
    }
    of[16][threadIdx.x] = x.bad;
    __syncthreads();
    if (way != 0) return;
#pragma unroll 4
    for (uint32_t w = 1; w < ways; ++w) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x.hi[j] = fmaxf(x.hi[j], of[j][w * L + part]);
            x.lo[j] = fminf(x.lo[j], of[8 + j][w * L + part]);
        }
        x.bad = fmaxf(x.bad, of[16][w * L + part]);
    }
    const float a = across<1, L>(live ? x.largest() : 0.0f, larger);
    if (live) x.write(A, (uint64_t)page * A.heads + head, part, a);
}

// Prompts: a workgroup looks `per` tokens over for those that lead, and its
// waves take the (page, head) pairs in turn, each by itself.
template <int FMT, int L>
__global__ __launch_bounds__(kThreads) void bounds_prompt_kernel(KvBounds A, uint32_t per) {
    constexpr uint32_t ways = kWave / L;
    const uint32_t lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, part = lane % L, way = lane / L;
    const uint64_t t0 = (uint64_t)blockIdx.x * per;
    const uint32_t s = slot_at(A, t0 + lane), prior = t0 + lane ? slot_at(A, t0 + lane - 1) : kNone;
    const uint32_t mine = s == kNone ? kNone : s / A.page_len;
    const bool leads = lane < per && mine < A.num_pages && !(prior != kNone && prior / A.page_len == mine);
    const bool live = part * 8u < A.dim;
    uint32_t turn = 0;
    for (uint64_t todo = __ballot(leads); todo; todo &= todo - 1) {
        const int l = __ffsll((unsigned long long)todo) - 1;
        const uint32_t page = (uint32_t)__builtin_amdgcn_readlane((int)mine, l);
        uint32_t filled = 0;
        for (uint32_t head = 0; head < A.heads; ++head, ++turn) {
            if (turn % (kThreads / kWave) != wave) continue;
            if (filled == 0) filled = filled_from(A, t0, s, l, page);
            Ends x;
            if (live) x.template rows<FMT, 4>(A, (uint64_t)page * A.page_len * A.heads + head, part, way, ways, filled);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x.hi[j] = across<L, kWave>(x.hi[j], larger);
                x.lo[j] = across<L, kWave>(x.lo[j], smaller);
            }
            x.bad = across<L, kWave>(x.bad, larger);
            const float a = across<1, L>(live ? x.largest() : 0.0f, larger);
            if (live && way == 0) x.write(A, (uint64_t)page * A.heads + head, part, a);
        }
    }
}

// ---- scores

// Scores as ordered integers: 0 for a page that cannot be taken.
__device__ __forceinline__ uint32_t order_key(float s) {
    s = s != s ? INFINITY : s + 0.0f;  // -0 counts as 0
    const uint32_t u = __float_as_uint(s);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr uint32_t kInfinite = 0xFF800000u;  // that of +inf, the largest score
constexpr uint32_t kEnd = kInfinite + 1;     // a sequence's first and last page

__device__ __forceinline__ uint32_t used_pages(const KvSelect& A, uint32_t b) {
    const int64_t len = A.lens[b] > 0 ? A.lens[b] : 0, n = (len + A.page_len - 1) / A.page_len;
    return (uint32_t)(n < A.max_pages ? n : A.max_pages);
}

// 16 queries of a key head at a time, as the matrix cores take them: lane 16 g
// + m holds bytes 64 s + 16 g .. + 15 of query m's 2 dim bytes max(n, 0), min(n,
// 0).  C steps of 64 bytes cover them, as they do a page's hi, lo.
constexpr uint32_t kQueries = 16;
constexpr uint32_t kMaxSteps = 16;
struct Queries {
    i32x4 n[kMaxSteps][kWave];
    float scale[kQueries];
    uint32_t top[kQueries];
};

// Fills `Q` with the queries from q0 on (`rows` of them; zeros behind), by a workgroup of T lanes; barriers at both ends.
template <int T>
__device__ __forceinline__ void hold_queries(const float* q0, uint32_t rows, uint32_t dim, Queries& Q) {
    constexpr uint32_t kLanes = T / kQueries;  // a query
    const uint32_t m = threadIdx.x / kLanes, part = threadIdx.x % kLanes;
    static_assert(kLanes >= 16 && kWave % 16 == 0);
    __syncthreads();
    const float* q = q0 + (uint64_t)m * dim;
    uint32_t top = 0;
    if (m < rows)
        for (uint32_t d = part * 4u; d < dim; d += kLanes * 4u) {
            const f32x4 x = *reinterpret_cast<const f32x4*>(q + d);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t k = abs_key(x[i]);
                top = top > k ? top : k;
            }
        }
    constexpr uint32_t kIn = kLanes < (uint32_t)kWave ? kLanes : kWave;  // of them in a wave
    top = across<1, (int)kIn>(top, greater);
    const float a = sized(__uint_as_float(top)), inv = 127.0f / a;
    if (part == 0) Q.scale[m] = a / 127.0f;
    for (uint32_t d = part * 4u; d < dim; d += kLanes * 4u) {
        uint32_t plus = 0, minus = 0;
        if (m < rows) {
            const f32x4 x = *reinterpret_cast<const f32x4*>(q + d);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float y = x[i] * inv;
                const int n = y != y ? 0 : (int)__builtin_amdgcn_fmed3f(rintf(y), -127.0f, 127.0f);
                plus |= (uint32_t)(n > 0 ? n : 0) << (8 * i);
                minus |= ((uint32_t)(n < 0 ? n : 0) & 255u) << (8 * i);
            }
        }
        // byte k of the 2 dim: step k / 64, lane group k / 16 % 4, byte k % 16
        uint32_t* out = reinterpret_cast<uint32_t*>(Q.n);
        const uint32_t k0 = d, k1 = dim + d;
        out[(k0 / 64u * kWave + k0 / 16u % 4u * 16u + m) * 4u + k0 / 4u % 4u] = plus;
        out[(k1 / 64u * kWave + k1 / 16u % 4u * 16u + m) * 4u + k1 / 4u % 4u] = minus;
    }
    __syncthreads();
}

// 16 pages' bounds as the matrix cores take them, lane 16 g + n those of page n.
template <int C>
struct Pages {
    i32x4 b[C];
    float scale;
    int32_t id;  // -1: not a page

    __device__ __forceinline__ void load(const KvSelect& A, uint32_t b0, uint32_t h, uint32_t page, uint32_t last) {
        const uint32_t g = threadIdx.x % kWave / 16;
        id = page < last ? A.page_table[(uint64_t)b0 * A.max_pages + page] : -1;
        if ((uint32_t)id >= A.num_pages) id = -1;
        if (A.num_pages == 0) return;
        const uint64_t at = (uint64_t)(id < 0 ? 0 : id) * A.heads + h;
        scale = A.bound_scales[at];
#pragma unroll
        for (int s = 0; s < C; ++s) b[s] = *reinterpret_cast<const i32x4*>(A.bounds + at * (64u * C) + 64 * s + 16 * g);
    }
    // The largest key of their scores with the queries held in Q: every lane 16 g + n gets that of page n.
    __device__ __forceinline__ uint32_t key(const Queries& Q, uint32_t rows) const {
        const uint32_t lane = threadIdx.x % kWave, g = lane / 16;
        i32x4 sum = {0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < C; ++s) sum = __builtin_amdgcn_mfma_i32_16x16x64_i8(Q.n[s][lane], b[s], sum, 0, 0, 0);
        uint32_t key = 0;  // of queries 4 g + i
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t k = 4 * g + i < rows ? order_key((float)sum[i] * scale * Q.scale[4 * g + i]) : 0u;
            key = key > k ? key : k;
        }
        const auto x = __builtin_amdgcn_permlane16_swap(key, key, false, false);
        key = x[0] > x[1] ? x[0] : x[1];
        const auto y = __builtin_amdgcn_permlane32_swap(key, key, false, false);
        return y[0] > y[1] ? y[0] : y[1];
    }
};

// Keys of pages [first, last) of (b, h), by a workgroup of T lanes, to out[0 ..
// last - first); the first pages' bounds are loaded before the queries are
// held, the next ones' before a tile is scored.
template <int C, int T>
__device__ __forceinline__ void score_pages(const KvSelect& A, Queries& Q, uint32_t b, uint32_t h, uint32_t first, uint32_t last, uint32_t used, uint32_t* out) {
    const uint32_t group = A.q_heads / A.heads, lane = threadIdx.x % kWave, n = lane % 16;
    const uint32_t begin = first + threadIdx.x / kWave * 16u;
    for (uint32_t q0 = 0; q0 < group; q0 += kQueries) {
        const uint32_t rows = group - q0 < kQueries ? group - q0 : kQueries;
        Pages<C> x, next;
        x.load(A, b, h, begin + n, last);
        hold_queries<T>(A.q + b * A.q_stride + (uint64_t)(h * group + q0) * A.dim, rows, A.dim, Q);
        for (uint32_t p0 = begin; p0 < last; p0 += T / kWave * 16u) {
            const uint32_t page = p0 + n;
            if (p0 + T / kWave * 16u < last) next.load(A, b, h, page + T / kWave * 16u, last);
            uint32_t key = x.key(Q, rows);
            if (page == 0 || page == used - 1) key = kEnd;
            if (x.id < 0) key = 0;
            if (lane < 16 && page < last) out[page - first] = q0 && out[page - first] > key ? out[page - first] : key;
            x = next;
        }
    }
}

// ---- the choice

constexpr int kPick = 1024;
constexpr int kPickWaves = kPick / kWave;
constexpr uint32_t kBins = 2048;

struct Pick {
    uint32_t count[kBins];
    uint32_t part[2][2][kPickWaves];
    uint32_t bin, above, in, low, high, some, first;
};

// Sum of v over the wave's lanes up to and with this one.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, true);
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, true);
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, true);
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, true);
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false);
    v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false);
    return v;
}

// Of each wave's value, the sum of those before this wave's and of all.
__device__ __forceinline__ void wave_sums(const uint32_t* part, uint32_t& before, uint32_t& all) {
    const uint32_t wave = threadIdx.x / kWave;
    before = all = 0;
#pragma unroll
    for (uint32_t i = 0; i < kPickWaves; ++i) {
        const uint32_t n = part[i];
        before += i < wave ? n : 0;
        all += n;
    }
}

// The `budget` largest of keys[0 .. n), ascending by place, ties to the lower
// one; then -1.  The key of the last one taken is found from counts of 2048
// equal bins between the smallest and the largest key that can be it, then
// between that bin's ends, and so on: two or three rounds, whose counts fall on
// many bins (counts by a key's upper bits fall on a few, as scores are alike).
// A sequence's ends and infinite scores come first, and are counted apart: they
// would stretch the bins.  A wave has a run of 64 HELD places at most in its registers (HELD 0: of
// any length, where they lie).
template <int HELD>
__device__ __forceinline__ void pick(Pick& P, const uint32_t* keys, uint32_t n, uint32_t budget, int32_t* out) {
    const uint32_t lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const uint32_t turns = (n + kPick - 1) / kPick, first = wave * turns * kWave + lane;
    uint32_t held[HELD ? HELD : 1];
    if constexpr (HELD != 0) {
#pragma unroll
        for (int j = 0; j < HELD; ++j) held[j] = (uint32_t)j < turns && first + j * kWave < n ? keys[first + j * kWave] : 0u;
    }
    auto each = [&](auto&& f) {  // f(place, key) of all of the lane's places, 0 for the keys behind the last; whole waves
        if constexpr (HELD != 0) {
#pragma unroll
            for (int j = 0; j < HELD; ++j)
                if ((uint32_t)j < turns) f(first + j * kWave, held[j]);
        } else {
            for (uint32_t j = 0; j < turns; ++j) f(first + j * kWave, first + j * kWave < n ? keys[first + j * kWave] : 0u);
        }
    };
    for (uint32_t i = threadIdx.x; i < kBins; i += kPick) P.count[i] = 0;
    if (threadIdx.x == 0) {
        P.low = 0xFFFFFFFFu;
        P.high = P.some = P.first = 0;
    }
    __syncthreads();
    // key - 1 and key + 2^23 put those that cannot be taken behind the smallest, the first ones before the largest
    static_assert((uint32_t)(kInfinite + 0x00800000u) == 0u);
    uint32_t low = 0xFFFFFFFFu, high = 0, some = 0, first_ones = 0;  // the counts are the wave's
    each([&](uint32_t, uint32_t k) {
        first_ones += (uint32_t)__popcll(__ballot(k >= kInfinite));
        some += (uint32_t)__popcll(__ballot(k != 0));
        low = k - 1u < low ? k - 1u : low;
        high = k + 0x00800000u > high ? k + 0x00800000u : high;
    });
    some -= first_ones;
    high = across<1, kWave>(high, greater);
    low = ~across<1, kWave>(~low, greater);
    if (lane == 0) {
        if (some) {
            atomicMin(&P.low, low + 1u);
            atomicMax(&P.high, high - 0x00800000u);
            atomicAdd(&P.some, some);
        }
        if (first_ones) atomicAdd(&P.first, first_ones);
    }
    __syncthreads();
    low = P.low;
    high = P.high;
    const uint32_t total = P.some, always = P.first;
    // the threshold: every key above it is taken, and `left` of those equal to it
    uint32_t threshold = 0, left = 0;
    if (always >= budget) {
        const uint32_t ends = (keys[0] == kEnd) + (n > 1 && keys[n - 1] == kEnd);  // always > 0: there is a page
        threshold = ends < budget ? kInfinite : kEnd;
        left = ends < budget ? budget - ends : budget;
    } else if (total > budget - always) {
        left = budget - always;
        for (uint32_t round = 0;; ++round) {
            const uint32_t span = high - low, shift = span < kBins ? 0 : 21 - (uint32_t)__builtin_clz(span);  // span >> shift < 2048
            each([&](uint32_t, uint32_t k) {
                if (k >= low && k <= high) atomicAdd(&P.count[(k - low) >> shift], 1u);
            });
            __syncthreads();
            // lane t holds the bins 2047 - 2 t and 2046 - 2 t: sums run from the largest keys down
            uint32_t* bins = &P.count[kBins - 2 - 2 * threadIdx.x];
            const uint32_t x = bins[1], y = bins[0], sum = wave_scan(x + y);
            bins[0] = bins[1] = 0;  // for the next round
            uint32_t* part = P.part[round & 1][0];
            if (lane == kWave - 1) part[wave] = sum;
            __syncthreads();
            uint32_t above, all;
            wave_sums(part, above, all);
            above += sum - (x + y);
            if (above < left && above + x >= left) {
                P.bin = kBins - 1 - 2 * threadIdx.x;
                P.above = above;
                P.in = x;
            } else if (above + x < left && above + x + y >= left) {
                P.bin = kBins - 2 - 2 * threadIdx.x;
                P.above = above + x;
                P.in = y;
            }
            __syncthreads();
            left -= P.above;
            low += P.bin << shift;
            if (shift == 0) break;
            if (P.in == left) {  // the whole bin is taken: its lower end will do, and nothing equals what lies below that
                left = 0;
                low -= 1;
                break;
            }
            const uint32_t end = low + (1u << shift) - 1;
            high = end < high ? end : high;
        }
        threshold = low;
    }
    // where each wave's taken ones go
    uint32_t over = 0, equal = 0;
    each([&](uint32_t, uint32_t k) {
        over += (uint32_t)__popcll(__ballot(k > threshold));
        equal += (uint32_t)__popcll(__ballot(k != 0 && k == threshold));
    });
    __syncthreads();
    if (lane == 0) {
        P.part[0][0][wave] = over;
        P.part[0][1][wave] = equal;
    }
    __syncthreads();
    uint32_t at, rank, overs, equals;
    wave_sums(P.part[0][0], at, overs);
    wave_sums(P.part[0][1], rank, equals);
    at += rank < left ? rank : left;
    const uint32_t taken = overs + (equals < left ? equals : left);
    const uint64_t below = ((uint64_t)1 << lane) - 1;
    each([&](uint32_t place, uint32_t k) {
        const bool same = k != 0 && k == threshold;
        const uint64_t sames = __ballot(same);
        const bool mine = k > threshold || (same && rank + (uint32_t)__popcll(sames & below) < left);
        const uint64_t all = __ballot(mine);
        if (mine) out[at + (uint32_t)__popcll(all & below)] = (int32_t)place;
        rank += (uint32_t)__popcll(sames);
        at += (uint32_t)__popcll(all);
    });
    for (uint32_t i = taken + threadIdx.x; i < budget; i += kPick) out[i] = -1;
}

// Few pages a sequence: a workgroup scores all pages of its (sequence, key
// head) into its LDS and picks from there.  Its 1024 lanes have 128 registers
// each: from 288 columns on the next tile's bounds do not fit beside this one's
// (60 to 428 bytes a lane in memory).
constexpr uint32_t kOnePages = 512;
template <int C>
__global__ __launch_bounds__(kPick) void select_kernel(KvSelect A) {
    __shared__ uint32_t keys[kOnePages];
    __shared__ union {
        Queries q;
        Pick p;
    } S;
    const uint32_t b = blockIdx.x / A.heads, h = blockIdx.x % A.heads, used = used_pages(A, b);
    score_pages<C, kPick>(A, S.q, b, h, 0, used, used, keys);
    __syncthreads();
    pick<1>(S.p, keys, used, A.budget, A.pages + (uint64_t)blockIdx.x * A.budget);
}

// Otherwise workgroups of their own score `span` pages each, and a second launch picks.
template <int C>
__global__ __launch_bounds__(kThreads) void score_kernel(KvSelect A, uint32_t* keys, uint32_t span, uint32_t spans) {
    __shared__ Queries Q;
    const uint32_t bh = blockIdx.x / spans, b = bh / A.heads, h = bh % A.heads, first = blockIdx.x % spans * span, used = used_pages(A, b);
    if (first >= used) return;
    const uint32_t last = used - first < span ? used : first + span;
    score_pages<C, kThreads>(A, Q, b, h, first, last, used, keys + (uint64_t)bh * A.max_pages + first);
}

template <int HELD>
__global__ __launch_bounds__(kPick) void pick_kernel(KvSelect A, const uint32_t* keys) {
    __shared__ Pick P;
    const uint32_t used = used_pages(A, blockIdx.x / A.heads);
    pick<HELD>(P, keys + (uint64_t)blockIdx.x * A.max_pages, used, A.budget, A.pages + (uint64_t)blockIdx.x * A.budget);
}

// Scoring workgroups are more only where a tile a wave is not: each holds the queries once (2048 instead: 25.6 and 23.4 us).
constexpr uint32_t kScorers = 1024;

// 4 key heads, 7 queries each, 128 columns, us in one launch and in two: 16
// sequences of 256 pages 9.6, 10.4; of 512 12.0, 11.2; of 1024 16.3, 12.9; 64 of
// 512 13.8, 16.9; 32 of 2048 26.3, 23.4; one of 4096 39.9, 11.7.
bool one_launch(uint32_t max_pages) { return max_pages <= kOnePages; }

}  // namespace

hipError_t launch_kv_bounds(int format, const KvBounds& A, hipStream_t st) {
    const uint32_t lanes = A.dim <= 64 ? 8 : A.dim <= 128 ? 16 : A.dim <= 256 ? 32 : 64;
    // up to 2048 (token, head) pairs a workgroup each; more: as many tokens a workgroup as 1024 of them need, as each costs its
    // launch (32768 tokens, us: 8 a workgroup 15.4, 16 11.5, 32 8.6, 64 10.6; with 8 rows a lane in flight instead of 4 9.3)
    const bool step = (uint64_t)A.tokens * A.heads <= 2048u;
    const uint32_t per = A.tokens / 1024u < 1u ? 1u : A.tokens / 1024u < 64u ? A.tokens / 1024u : 64u;
    const uint32_t grid = step ? A.tokens * A.heads : (A.tokens + per - 1) / per;
    auto launch = [&](auto l_) {
        constexpr int L = decltype(l_)::value;
        auto go = [&](auto f_) {
            constexpr int FMT = decltype(f_)::value;
            if (step)
                bounds_step_kernel<FMT, L><<<grid, kThreads, 0, st>>>(A);
            else
                bounds_prompt_kernel<FMT, L><<<grid, kThreads, 0, st>>>(A, per);
        };
        if (format == kKvE4M3)
            go(std::integral_constant<int, kKvE4M3>{});
        else
            go(std::integral_constant<int, kKvMXFP4>{});
    };
    if (lanes == 8)
        launch(std::integral_constant<int, 8>{});
    else if (lanes == 16)
        launch(std::integral_constant<int, 16>{});
    else if (lanes == 32)
        launch(std::integral_constant<int, 32>{});
    else
        launch(std::integral_constant<int, 64>{});
    return hipGetLastError();
}

size_t kv_select_ws_bytes(uint32_t seqs, uint32_t heads, uint32_t max_pages) {
    return one_launch(max_pages) ? 0 : (size_t)seqs * heads * max_pages * 4u;
}

hipError_t launch_kv_select(const KvSelect& A, hipStream_t st) {
    const uint32_t pairs = A.seqs * A.heads;
    const bool known = with_steps(A.dim / 32u, [&](auto c_) {
        constexpr int C = decltype(c_)::value;
        if (one_launch(A.max_pages)) {
            select_kernel<C><<<pairs, kPick, 0, st>>>(A);
            return;
        }
        uint32_t* keys = static_cast<uint32_t*>(A.ws);
        // a tile a wave, or more where that is more than eight workgroups a compute unit: each holds the queries once
        const uint64_t tiles = (uint64_t)pairs * ((A.max_pages + 63u) / 64u) / kScorers;
        const uint32_t span = 64u * (uint32_t)(tiles < 1 ? 1 : tiles < 16 ? tiles : 16), spans = (A.max_pages + span - 1) / span;
        score_kernel<C><<<pairs * spans, kThreads, 0, st>>>(A, keys, span, spans);
        if (A.max_pages <= 8u * kPick)
            pick_kernel<8><<<pairs, kPick, 0, st>>>(A, keys);
        else if (A.max_pages <= 32u * kPick)
            pick_kernel<32><<<pairs, kPick, 0, st>>>(A, keys);
        else
            pick_kernel<0><<<pairs, kPick, 0, st>>>(A, keys);
    });
    if (!known) return hipErrorInvalidValue;
    return hipGetLastError();
}

}  // namespace rz
