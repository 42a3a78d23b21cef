// Quantised key/value cache: written from the K and V projections' fp32
// outputs, read back for attention.
//
// A cache row is one head of one token: `dim` values, in one of two formats:
//   E4M3   the FP8 path's conversion with a row's own absmax a (NaN ignored):
//          a' = a or 1 when a == 0, codes E4M3(RN(x * RN(448/a'))), scale
//          RN(a'/448) in fp32; a value reads back as RN(code * scale);
//   MXFP4  blocks of 32 as in mx_device.h, rows in plain order: codes
//          [slot][head][dim/2], scale bytes [slot][head][dim/32].
// Both directions are bound by memory (a decoding step by its launch).  A
// lane holds eight values, 8..64 lanes a row; keys and values share a launch
// (grid y).  Measured, 4 heads of 128: writing 131072 tokens 134 us (E4M3) and
// 121 us (MXFP4), both 5.0 TB/s, 64 tokens 3 us; reading 131072 tokens back in
// bf16 82 us (E4M3, 5.0 TB/s) and 67 us (MXFP4, 5.1 TB/s), in fp32 171 and 161
// us (3.9 TB/s), 4096 tokens 5 us.  With one row a lane in flight E4M3 took 88.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_device.h"
#include "rz_device.h"
#include "rz_internal.h"

namespace rz {
namespace {
using namespace mx;

constexpr int kThreads = 256;

template <int L>
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
#pragma unroll
    for (int off = 1; off < L; off <<= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)v, off, kWave);
        v = v > o ? v : o;
    }
    return v;
}

// L lanes a row (a power of two, 8 L >= dim; lanes past dim are idle).
template <int FMT, int L>
__global__ __launch_bounds__(kThreads) void kv_write_kernel(KvWrite A) {
    const uint32_t part = threadIdx.x % L;
    const uint64_t row = (uint64_t)blockIdx.x * (kThreads / L) + threadIdx.x / L;
    if (row >= (uint64_t)A.tokens * A.heads) return;  // whole rows: the shuffles below stay inside a row
    const uint32_t token = (uint32_t)(row / A.heads), head = (uint32_t)(row % A.heads);
    const int64_t slot = A.slots[token];
    if (slot < 0 || (uint64_t)slot >= A.num_slots) return;  // not a slot: this token is not kept
    const int c = blockIdx.y;
    const bool live = part * 8u < A.dim;
    float x[8] = {};
    if (live) {
        const float* p = A.x[c] + (uint64_t)token * A.stride[c] + head * A.dim + part * 8u;
        const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = a[i];
            x[4 + i] = b[i];
        }
    }
    const uint64_t dst = (uint64_t)slot * A.heads + head;
    if constexpr (FMT == kKvE4M3) {
        uint32_t key = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t a = abs_key(x[i]);
            key = key > a ? key : a;
        }
        const Scales s = scales_from_key(row_max<L>(key));
        if (live) {
            u32x2 w;
            w.x = e4m3_pack4(x[0] * s.q, x[1] * s.q, x[2] * s.q, x[3] * s.q);
            w.y = e4m3_pack4(x[4] * s.q, x[5] * s.q, x[6] * s.q, x[7] * s.q);
            *reinterpret_cast<u32x2*>(A.codes[c] + dst * A.dim + part * 8u) = w;
        }
        if (part == 0) static_cast<float*>(A.scales[c])[dst] = s.dq;
    } else {
        uint32_t byte;
        const uint32_t w = quantise8(x, byte);
        if (live) {
            *reinterpret_cast<uint32_t*>(A.codes[c] + dst * (A.dim / 2u) + part * 4u) = w;
            if ((part & 3u) == 0) static_cast<uint8_t*>(A.scales[c])[dst * (A.dim / 32u) + part / 4u] = (uint8_t)byte;
        }
    }
}

// A workgroup reads `per` consecutive output rows (tokens): one lane a token
// finds its sequence (binary search in the offsets) and slot, then the
// workgroup copies the tokens' heads, kTurn of them a lane at a time so that
// their loads are in flight together.
constexpr int kMaxRows = 64;
constexpr int kTurn = 4;

template <int FMT, int DT, int L>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvRead A, uint32_t per) {
    __shared__ int64_t slot_of[kMaxRows];  // -1: zeros, -2: not a row of any sequence
    const uint32_t row0 = blockIdx.x * per;
    if (threadIdx.x < per) {
        const uint32_t row = row0 + threadIdx.x;
        int64_t slot = -2;
        if (row < A.rows && (int64_t)row >= A.offsets[0] && (int64_t)row < A.offsets[A.seqs]) {
            uint32_t lo = 0, hi = A.seqs;  // offsets[lo] <= row < offsets[hi]
            while (hi - lo > 1) {
                const uint32_t mid = (lo + hi) >> 1;
                if ((int64_t)row >= A.offsets[mid]) lo = mid; else hi = mid;
            }
            const uint32_t pos = row - (uint32_t)A.offsets[lo];
            const uint32_t page = pos / A.page_len;
            slot = -1;
            if (page < A.max_pages) {
                const int32_t id = A.page_table[(uint64_t)lo * A.max_pages + page];
                const uint64_t s = (uint64_t)(uint32_t)id * A.page_len + pos % A.page_len;
                if (id >= 0 && s < A.num_slots) slot = (int64_t)s;
            }
        }
        slot_of[threadIdx.x] = slot;
    }
    __syncthreads();
    const int c = blockIdx.y;
    const uint32_t part = threadIdx.x % L, end = per * A.heads;
    if (part * 8u >= A.dim) return;
    for (uint32_t i0 = threadIdx.x / L; i0 < end; i0 += kTurn * (kThreads / L)) {
        int64_t slot[kTurn];
        u32x2 w[kTurn];
        uint32_t sc[kTurn];  // the row's fp32 scale, or the block's byte
#pragma unroll
        for (int u = 0; u < kTurn; ++u) {
            const uint32_t i = i0 + u * (kThreads / L), t = i / A.heads;
            slot[u] = i < end ? slot_of[t] : -2;
            w[u] = (u32x2){0u, 0u};
            sc[u] = 0;  // zeros, where nothing is read
            if (slot[u] >= 0) {
                const uint64_t src = (uint64_t)slot[u] * A.heads + (i - t * A.heads);
                if constexpr (FMT == kKvE4M3) {
                    w[u] = *reinterpret_cast<const u32x2*>(A.codes[c] + src * A.dim + part * 8u);
                    sc[u] = static_cast<const uint32_t*>(A.scales[c])[src];
                } else {
                    w[u].x = *reinterpret_cast<const uint32_t*>(A.codes[c] + src * (A.dim / 2u) + part * 4u);
                    sc[u] = static_cast<const uint8_t*>(A.scales[c])[src * (A.dim / 32u) + part / 4u];
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kTurn; ++u) {
            if (slot[u] == -2) continue;
            float v[8];
            if constexpr (FMT == kKvE4M3) {
                const float s = __uint_as_float(sc[u]);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[u][j], false);
                    const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[u][j], true);
                    v[4 * j] = a.x * s;
                    v[4 * j + 1] = a.y * s;
                    v[4 * j + 2] = b.x * s;
                    v[4 * j + 3] = b.y * s;
                }
            } else {
                decode8(w[u].x, v, cvt_scale(sc[u]));
            }
            const uint64_t i = i0 + u * (kThreads / L);  // (row - row0) * heads + head
            store8<DT>(A.out[c], ((uint64_t)row0 * A.heads + i) * A.dim + part * 8u, v);
        }
    }
}

// Tokens a reading workgroup takes: one turn of its lanes (1024 items of
// eight values), halved while that leaves fewer than 512 workgroups a tensor
// (E4M3, heads 4 x dim 128, us at 8 / 16 / 32 tokens: 4096 rows 4.7 / 4.9 /
// 6.2; 16384 rows 10.8 / 9.7 / 10.9; 131072 rows 100 / 81 / 84, of which 81
// is 5.0 TB/s).
uint32_t rows_per_group(const KvRead& A, uint32_t lanes) {
    uint32_t per = kMaxRows;
    while (per > 4u && (uint64_t)per * A.heads * lanes > 1024u) per >>= 1;
    while (per > 8u && A.rows / per < 512u) per >>= 1;
    return per;
}

template <int FMT, int L>
void read_as(const KvRead& A, int dtype, uint32_t per, hipStream_t st) {
    const dim3 grid((A.rows + per - 1) / per, 2);
    if (dtype == kF32)
        kv_read_kernel<FMT, kF32, L><<<grid, kThreads, 0, st>>>(A, per);
    else if (dtype == kF16)
        kv_read_kernel<FMT, kF16, L><<<grid, kThreads, 0, st>>>(A, per);
    else
        kv_read_kernel<FMT, kBF16, L><<<grid, kThreads, 0, st>>>(A, per);
}

// Calls f(integral_constant<L>) with the fewest lanes that hold dim values.
template <typename F>
void with_lanes(uint32_t dim, F&& f) {
    if (dim <= 64)
        f(std::integral_constant<int, 8>{});
    else if (dim <= 128)
        f(std::integral_constant<int, 16>{});
    else if (dim <= 256)
        f(std::integral_constant<int, 32>{});
    else
        f(std::integral_constant<int, 64>{});
}

}  // namespace

hipError_t launch_kv_write(int format, const KvWrite& A, hipStream_t st) {
    with_lanes(A.dim, [&](auto l) {
        constexpr int L = decltype(l)::value;
        const uint64_t rows = (uint64_t)A.tokens * A.heads;
        const dim3 grid((uint32_t)((rows + kThreads / L - 1) / (kThreads / L)), 2);
        if (format == kKvE4M3)
            kv_write_kernel<kKvE4M3, L><<<grid, kThreads, 0, st>>>(A);
        else
            kv_write_kernel<kKvMXFP4, L><<<grid, kThreads, 0, st>>>(A);
    });
    return hipGetLastError();
}

hipError_t launch_kv_read(int format, const KvRead& A, int dtype, hipStream_t st) {
    with_lanes(A.dim, [&](auto l) {
        constexpr int L = decltype(l)::value;
        const uint32_t per = rows_per_group(A, L);
        if (format == kKvE4M3)
            read_as<kKvE4M3, L>(A, dtype, per, st);
        else
            read_as<kKvMXFP4, L>(A, dtype, per, st);
    });
    return hipGetLastError();
}

}  // namespace rz
