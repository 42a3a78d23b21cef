// Bounds of the keys in a page, and the choice of pages by them.
//
// A page and head's bounds are the largest and smallest value of each column
// over the page's filled rows, as int8 multiples of one scale, rounded away
// from the middle; a query is held as int8 too, so that
//   sum_d max(n_d hi_d, n_d lo_d)
// is a sum of whole numbers (below 2^24 for 512 columns: exact in fp32 as
// well), the same in any order, and the choice by it has no rounding to
// depend on.  To its roundings it is an upper bound of n . k for every key k
// of the page.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_device.h"
#include "rz_device.h"
#include "rz_internal.h"

namespace rz {
namespace {
using namespace mx;

constexpr int kThreads = 256;
constexpr float kTiny = 0x1p-100f;

// a / 127 and 127 / a of a largest magnitude a.
__device__ __forceinline__ float sized(float a) { return a >= kTiny ? a : 1.0f; }

// One wave a (token, head): the first token of a page in `slots` takes the
// page, eight columns a lane.
template <int FMT>
__global__ __launch_bounds__(kThreads) void bounds_kernel(KvBounds A) {
    const uint64_t item = (uint64_t)blockIdx.x * (kThreads / kWave) + threadIdx.x / kWave;
    const uint32_t lane = threadIdx.x % kWave;
    if (item >= (uint64_t)A.tokens * A.heads) return;
    const uint32_t t = (uint32_t)(item / A.heads), h = (uint32_t)(item % A.heads);
    auto page_of = [&](uint32_t i) -> int64_t {
        const int64_t s = A.slots[i];
        return s < 0 || (uint64_t)s >= A.num_slots ? -1 : s / A.page_len;
    };
    const int64_t page = page_of(t);
    if (page < 0 || (uint64_t)page >= A.num_pages || (t > 0 && page_of(t - 1) == page)) return;
    uint32_t filled = 0;
    for (uint32_t i = t; i < A.tokens && page_of(i) == page; ++i) {
        const uint32_t at = (uint32_t)(A.slots[i] % A.page_len) + 1;
        filled = filled > at ? filled : at;
    }
    const bool live = lane * 8u < A.dim;
    float hi[8], lo[8];
    bool fine = true;
    for (int i = 0; i < 8; ++i) {
        hi[i] = -INFINITY;
        lo[i] = INFINITY;
    }
    for (uint32_t r = 0; r < filled && live; ++r) {
        const uint64_t row = ((uint64_t)page * A.page_len + r) * A.heads + h;
        float x[8];
        if constexpr (FMT == kKvE4M3) {
            const u32x2 w = *reinterpret_cast<const u32x2*>(A.codes + row * A.dim + lane * 8u);
            const float s = static_cast<const float*>(A.scales)[row];
            for (int j = 0; j < 2; ++j) {
                const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[j], false);
                const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[j], true);
                x[4 * j] = a.x * s;
                x[4 * j + 1] = a.y * s;
                x[4 * j + 2] = b.x * s;
                x[4 * j + 3] = b.y * s;
            }
        } else {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(A.codes + row * (A.dim / 2u) + lane * 4u);
            decode8(w, x, cvt_scale(static_cast<const uint8_t*>(A.scales)[row * (A.dim / 32u) + lane / 4u]));
        }
        for (int i = 0; i < 8; ++i) {
            fine = fine && fabsf(x[i]) < INFINITY;
            hi[i] = fmaxf(hi[i], x[i]);
            lo[i] = fminf(lo[i], x[i]);
        }
    }
    float a = 0.0f;
    if (live)
        for (int i = 0; i < 8; ++i) a = fmaxf(a, fmaxf(fabsf(hi[i]), fabsf(lo[i])));
    for (int off = 1; off < kWave; off <<= 1) a = fmaxf(a, __shfl_xor(a, off, kWave));
    fine = __ballot(!fine) == 0;
    a = sized(a);
    const float inv = 127.0f / a;
    const uint64_t dst = (uint64_t)page * A.heads + h;
    if (live) {
        u32x2 up, down;
        for (int j = 0; j < 2; ++j) {
            uint32_t u = 0, d = 0;
            for (int i = 0; i < 4; ++i) {
                const float p = fine ? ceilf(hi[4 * j + i] * inv) : 127.0f, n = fine ? floorf(lo[4 * j + i] * inv) : -127.0f;
                u |= ((uint32_t)(int)__builtin_amdgcn_fmed3f(p, -127.0f, 127.0f) & 255u) << (8 * i);
                d |= ((uint32_t)(int)__builtin_amdgcn_fmed3f(n, -127.0f, 127.0f) & 255u) << (8 * i);
            }
            up[j] = u;
            down[j] = d;
        }
        *reinterpret_cast<u32x2*>(A.bounds + dst * 2u * A.dim + lane * 8u) = up;
        *reinterpret_cast<u32x2*>(A.bounds + (dst * 2u + 1u) * A.dim + lane * 8u) = down;
    }
    if (lane == 0) A.bound_scales[dst] = fine ? a / 127.0f : INFINITY;
}

// Scores as ordered integers: 0 for a page that cannot be taken.
__device__ __forceinline__ uint32_t order_key(float s) {
    s = s != s ? INFINITY : s + 0.0f;  // -0 counts as 0
    const uint32_t u = __float_as_uint(s);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ uint32_t used_pages(const KvSelect& A, uint32_t b) {
    const int64_t len = A.lens[b] > 0 ? A.lens[b] : 0, n = (len + A.page_len - 1) / A.page_len;
    return (uint32_t)(n < A.max_pages ? n : A.max_pages);
}

// keys[b][h][page]; a workgroup takes 4 pages of (b, h), one a wave.
__global__ __launch_bounds__(kThreads) void score_kernel(KvSelect A, uint32_t* keys, uint32_t groups) {
    const uint64_t bh = blockIdx.x / groups;
    const uint32_t b = (uint32_t)(bh / A.heads), h = (uint32_t)(bh % A.heads), lane = threadIdx.x % kWave;
    const uint32_t page = (blockIdx.x % groups) * (kThreads / kWave) + threadIdx.x / kWave, used = used_pages(A, b);
    if (page >= A.max_pages) return;
    uint32_t key = 0;
    const int32_t id = page < used ? A.page_table[(uint64_t)b * A.max_pages + page] : -1;
    if (id >= 0 && (uint32_t)id < A.num_pages) {
        const uint64_t at = (uint64_t)id * A.heads + h;
        const uint32_t group = A.q_heads / A.heads;
        for (uint32_t g = 0; g < group; ++g) {
            const float* q = A.q + b * A.q_stride + (uint64_t)(h * group + g) * A.dim;
            uint32_t top = 0;
            for (uint32_t d = lane; d < A.dim; d += kWave) {
                const uint32_t k = abs_key(q[d]);
                top = top > k ? top : k;
            }
            const float a = sized(__uint_as_float(wave_max_u32(top))), inv = 127.0f / a, qs = a / 127.0f;
            int sum = 0;
            for (uint32_t d = lane; d < A.dim; d += kWave) {
                const float x = q[d] * inv;
                const int n = x != x ? 0 : (int)__builtin_amdgcn_fmed3f(rintf(x), -127.0f, 127.0f);
                const int u = n * A.bounds[at * 2 * A.dim + d], l = n * A.bounds[(at * 2 + 1) * A.dim + d];
                sum += u > l ? u : l;
            }
            for (int off = 1; off < kWave; off <<= 1) sum += __shfl_xor(sum, off, kWave);
            const uint32_t k = order_key((float)sum * A.bound_scales[at] * qs);
            key = key > k ? key : k;
        }
        if (page == 0 || page == used - 1) key = order_key(INFINITY);
    }
    if (lane == 0) keys[bh * A.max_pages + page] = key;
}

// The `budget` largest keys of each row, ascending by page: the key of the
// last one taken is found 8 bits at a time from counts.
constexpr int kPick = 1024;
__global__ __launch_bounds__(kPick) void pick_kernel(KvSelect A, const uint32_t* keys) {
    __shared__ uint32_t count[256], part[kPick / kWave], found[2];
    const uint64_t bh = blockIdx.x;
    const uint32_t used = used_pages(A, (uint32_t)(bh / A.heads)), lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    keys += bh * A.max_pages;
    int32_t* out = A.pages + bh * A.budget;
    uint32_t prefix = 0, left = A.budget;  // the threshold's upper bits so far; how many of those that share them are taken
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (threadIdx.x < 256) count[threadIdx.x] = 0;
        if (threadIdx.x == 0) found[0] = 0, found[1] = left;
        __syncthreads();
        const uint32_t mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
        for (uint32_t i = threadIdx.x; i < used; i += kPick)
            if ((keys[i] & mask) == prefix) atomicAdd(&count[keys[i] >> shift & 255u], 1u);
        __syncthreads();
        if (threadIdx.x < 256) {
            uint32_t above = 0;
            for (uint32_t i = threadIdx.x + 1; i < 256; ++i) above += count[i];
            if (above < left && above + count[threadIdx.x] >= left) {
                found[0] = threadIdx.x;
                found[1] = left - above;
            }
        }
        __syncthreads();
        prefix |= found[0] << shift;
        left = found[1];
        __syncthreads();
    }
    // fewer than `budget` pages: the threshold is 0, and every key above it is taken
    uint32_t taken = 0, same = 0;
    for (uint32_t i0 = 0; i0 < used; i0 += kPick) {
        const uint32_t i = i0 + threadIdx.x, key = i < used ? keys[i] : 0;
        const uint64_t eq = __ballot(key == prefix && key != 0);
        if (lane == 0) part[wave] = (uint32_t)__popcll(eq);
        __syncthreads();
        uint32_t before = same + (uint32_t)__popcll(eq & ((1ull << lane) - 1));
        for (uint32_t w = 0; w < kPick / kWave; ++w) {
            if (w < wave) before += part[w];
            same += part[w];
        }
        __syncthreads();
        const bool take = key != 0 && (key > prefix || (key == prefix && before < left));
        const uint64_t all = __ballot(take);
        if (lane == 0) part[wave] = (uint32_t)__popcll(all);
        __syncthreads();
        uint32_t at = taken + (uint32_t)__popcll(all & ((1ull << lane) - 1));
        for (uint32_t w = 0; w < kPick / kWave; ++w) {
            if (w < wave) at += part[w];
            taken += part[w];
        }
        __syncthreads();
        if (take) out[at] = (int32_t)i;
    }
    for (uint32_t i = taken + threadIdx.x; i < A.budget; i += kPick) out[i] = -1;
}

}  // namespace

hipError_t launch_kv_bounds(int format, const KvBounds& A, hipStream_t st) {
    const uint64_t items = (uint64_t)A.tokens * A.heads;
    const uint32_t grid = (uint32_t)((items + kThreads / kWave - 1) / (kThreads / kWave));
    if (format == kKvE4M3)
        bounds_kernel<kKvE4M3><<<grid, kThreads, 0, st>>>(A);
    else
        bounds_kernel<kKvMXFP4><<<grid, kThreads, 0, st>>>(A);
    return hipGetLastError();
}

size_t kv_select_ws_bytes(uint32_t seqs, uint32_t heads, uint32_t max_pages) { return (size_t)seqs * heads * max_pages * 4u; }

hipError_t launch_kv_select(const KvSelect& A, hipStream_t st) {
    uint32_t* keys = static_cast<uint32_t*>(A.ws);
    const uint32_t groups = (A.max_pages + kThreads / kWave - 1) / (kThreads / kWave);
    if (groups) score_kernel<<<A.seqs * A.heads * groups, kThreads, 0, st>>>(A, keys, groups);
    pick_kernel<<<A.seqs * A.heads, kPick, 0, st>>>(A, keys);
    return hipGetLastError();
}

}  // namespace rz
