// Attention of one new token a sequence over the quantised, paged cache:
//   out[b][h] = sum_p w_p v_p,  w = softmax(scale q[b][h] . k_p),
// one pass over the rows with the running maximum and sum of the softmax.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_device.h"
#include "rz_device.h"
#include "rz_internal.h"

namespace rz {
namespace {
using namespace mx;

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / kWave;

// Slot of the v-th position that (sequence b, key head h) attends, -1: none.
__device__ __forceinline__ int64_t slot_at(const KvAttend& A, uint32_t b, uint32_t h, uint32_t v, uint32_t len) {
    uint32_t page = v / A.page_len;
    const uint32_t at = v - page * A.page_len;
    if (A.pages) {
        const int32_t p = A.pages[((uint64_t)b * A.heads + h) * A.budget + page];
        if (p < 0) return -1;
        page = (uint32_t)p;
    }
    if (page >= A.max_pages || (uint64_t)page * A.page_len + at >= len) return -1;
    const int32_t id = A.page_table[(uint64_t)b * A.max_pages + page];
    const uint64_t slot = (uint64_t)(uint32_t)id * A.page_len + at;
    return id >= 0 && slot < A.num_slots ? (int64_t)slot : -1;
}

// Eight fp32 values of a row from column 8 part on.
template <int FMT>
__device__ __forceinline__ void load8(const KvAttend& A, int c, uint64_t row, uint32_t part, float (&x)[8]) {
    if constexpr (FMT == kKvE4M3) {
        const u32x2 w = *reinterpret_cast<const u32x2*>(A.codes[c] + row * A.dim + part * 8u);
        const float s = static_cast<const float*>(A.scales[c])[row];
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
        const uint32_t w = *reinterpret_cast<const uint32_t*>(A.codes[c] + row * (A.dim / 2u) + part * 4u);
        decode8(w, x, cvt_scale(static_cast<const uint8_t*>(A.scales[c])[row * (A.dim / 32u) + part / 4u]));
    }
}

__device__ __forceinline__ void store1(const KvAttend& A, int dtype, uint64_t at, float v) {
    if (dtype == kF32)
        static_cast<float*>(A.out)[at] = v;
    else if (dtype == kF16)
        static_cast<_Float16*>(A.out)[at] = (_Float16)v;
    else
        static_cast<__bf16*>(A.out)[at] = (__bf16)v;
}

// A workgroup computes one query head of one sequence: its waves share the
// positions, a lane holds eight columns.
template <int FMT>
__global__ __launch_bounds__(kThreads) void attend_kernel(KvAttend A, int dtype) {
    __shared__ float acc_of[kWaves][512], m_of[kWaves], l_of[kWaves];
    const uint32_t b = blockIdx.x / A.q_heads, qh = blockIdx.x % A.q_heads, h = qh / (A.q_heads / A.heads);
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const bool live = lane * 8u < A.dim;
    float q[8] = {}, acc[8] = {}, m = -INFINITY, l = 0.0f;
    if (live)
        for (int i = 0; i < 8; ++i) q[i] = A.q[b * A.q_stride + (uint64_t)qh * A.dim + lane * 8 + i] * A.scale;
    const uint32_t len = A.lens[b] > 0 ? (uint32_t)A.lens[b] : 0u;
    const uint64_t most = (uint64_t)(A.pages ? A.budget : A.max_pages) * A.page_len;
    const uint32_t n = A.pages ? (uint32_t)most : (uint32_t)(len < most ? len : most);
    for (uint32_t v = wave; v < n; v += kWaves) {
        const int64_t slot = slot_at(A, b, h, v, len);
        if (slot < 0) continue;
        const uint64_t row = (uint64_t)slot * A.heads + h;
        float x[8] = {}, s = 0.0f;
        if (live) load8<FMT>(A, 0, row, lane, x);
        for (int i = 0; i < 8; ++i) s += q[i] * x[i];
        for (int off = 1; off < kWave; off <<= 1) s += __shfl_xor(s, off, kWave);
        if (live) load8<FMT>(A, 1, row, lane, x);
        const float top = s > m || s != s ? s : m, base = top == -INFINITY ? 0.0f : top;
        const float old = __expf(m - base), w = __expf(s - base);
        m = top;
        l = l * old + w;
        for (int i = 0; i < 8; ++i) acc[i] = acc[i] * old + w * x[i];
    }
    if (lane == 0) {
        m_of[wave] = m;
        l_of[wave] = l;
    }
    if (live)
        for (int i = 0; i < 8; ++i) acc_of[wave][lane * 8 + i] = acc[i];
    __syncthreads();
    float top = -INFINITY, sum = 0.0f, f[kWaves];
    for (int i = 0; i < kWaves; ++i) top = m_of[i] > top || m_of[i] != m_of[i] ? m_of[i] : top;
    for (int i = 0; i < kWaves; ++i) {
        f[i] = __expf(m_of[i] - (top == -INFINITY ? 0.0f : top));
        sum += l_of[i] * f[i];
    }
    for (uint32_t d = threadIdx.x; d < A.dim; d += kThreads) {
        float o = 0.0f;
        for (int i = 0; i < kWaves; ++i) o += acc_of[i][d] * f[i];
        store1(A, dtype, ((uint64_t)b * A.q_heads + qh) * A.dim + d, sum == 0.0f ? 0.0f : o / sum);
    }
    if (A.lse && threadIdx.x == 0) A.lse[(uint64_t)b * A.q_heads + qh] = sum == 0.0f ? -INFINITY : top + __logf(sum);
}

}  // namespace

size_t kv_attend_ws_bytes(uint32_t, uint32_t, uint32_t, int) { return 0; }

hipError_t launch_kv_attend(int format, const KvAttend& A, int dtype, int, hipStream_t st) {
    const uint32_t grid = A.seqs * A.q_heads;
    if (format == kKvE4M3)
        attend_kernel<kKvE4M3><<<grid, kThreads, 0, st>>>(A, dtype);
    else
        attend_kernel<kKvMXFP4><<<grid, kThreads, 0, st>>>(A, dtype);
    return hipGetLastError();
}

}  // namespace rz
