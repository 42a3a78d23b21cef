// A step's pages and slots from the sequences' lengths.
//
// Sequence b keeps keep[b] of its lens[b] tokens and adds new[b]; with
// held = ceil(lens / page_len) and need = ceil((keep + new) / page_len) it
// gives max(held - need, 0) pages to a stack, then takes max(need - held, 0).
// The i-th page given lies at stack[count + i], the i-th taken comes from
// stack[count + given - 1 - i], so two prefix sums over the sequences say
// where every page goes, in any order of execution.
//
// One workgroup does the sums and moves the pages; where a step has more
// tokens than it serves well, a second launch gives every token its slot.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "rz_device.h"
#include "rz_internal.h"

namespace rz {
namespace {

constexpr int kThreads = 1024;

// What a sequence does in this step.
struct Row {
    int64_t first;  // position of its first new token
    int64_t held, need;
    bool ok;
    __device__ __forceinline__ Row(const KvPlan& A, uint32_t b) {
        const int64_t len = A.lens[b], keep = A.keep ? A.keep[b] : len;
        const int64_t fresh = (int64_t)A.offsets[b + 1] - A.offsets[b];
        first = keep;
        ok = keep >= 0 && keep <= len && fresh >= 0 && keep + fresh <= INT32_MAX;
        held = ok ? (len + A.page_len - 1) / A.page_len : 0;
        need = ok ? (keep + fresh + A.page_len - 1) / A.page_len : 0;
        ok = ok && held <= A.max_pages && need <= A.max_pages;
    }
    __device__ __forceinline__ int64_t give() const { return ok && held > need ? held - need : 0; }
    __device__ __forceinline__ int64_t take() const { return ok && need > held ? need - held : 0; }
};

// Sum of v over the threads before this one, and over all of them.
struct Scan {
    int64_t before, all;
};
__device__ __forceinline__ Scan scan(int64_t v, int64_t* smem) {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    int64_t sum = v;
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
        const int64_t o = __shfl_up(sum, off, kWave);
        if (lane >= off) sum += o;
    }
    if (lane == kWave - 1) smem[wave] = sum;
    __syncthreads();
    Scan s = {sum - v, 0};
    for (int i = 0; i < kThreads / kWave; ++i) {
        if (i < wave) s.before += smem[i];
        s.all += smem[i];
    }
    __syncthreads();
    return s;
}

// Calls f(lane, n of that lane) for each lane whose n is not 0, with the whole
// wave: f may shuffle before it loops.
template <typename F>
__device__ __forceinline__ void each(int64_t n, F&& f) {
    for (uint64_t todo = __ballot(n > 0); todo; todo &= todo - 1) {
        const int l = __ffsll((unsigned long long)todo) - 1;
        f(l, __shfl(n, l, kWave));
    }
}

// The slot of token t: `first` holds each sequence's first new position (-1: refused).
__device__ __forceinline__ int64_t slot_of(const KvPlan& A, const int32_t* first, uint32_t t) {
    if (A.seqs == 0 || (int64_t)t < A.offsets[0] || (int64_t)t >= A.offsets[A.seqs]) return -1;
    uint32_t lo = 0, hi = A.seqs;  // offsets[lo] <= t < offsets[hi]
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) >> 1;
        if ((int64_t)t >= A.offsets[mid]) lo = mid; else hi = mid;
    }
    if (first[lo] < 0) return -1;
    const uint64_t pos = (uint64_t)first[lo] + (t - (uint32_t)A.offsets[lo]);
    if (pos / A.page_len >= A.max_pages) return -1;  // offsets that decrease
    const int64_t page = A.page_table[(uint64_t)lo * A.max_pages + pos / A.page_len];
    return page < 0 ? -1 : page * A.page_len + (int64_t)(pos % A.page_len);
}

__global__ __launch_bounds__(kThreads) void plan_kernel(KvPlan A, int32_t* first, bool with_slots) {
    __shared__ int64_t smem[kThreads / kWave];
    const int lane = threadIdx.x & (kWave - 1);
    const uint32_t rounds = (A.seqs + kThreads - 1) / kThreads;
    int64_t have = A.free_count[0];
    have = have < 0 ? 0 : have > A.num_pages ? A.num_pages : have;
    for (uint32_t r = 0; r < rounds; ++r) {
        const uint32_t b = r * kThreads + threadIdx.x, wave0 = b & ~(kWave - 1u);
        int64_t give = 0, need = 0;
        if (b < A.seqs) {
            const Row row(A, b);
            give = row.give();
            need = row.need;
        }
        const Scan s = scan(give, smem);
        const int64_t at = have + s.before;
        each(give, [&](int l, int64_t n) {
            const int64_t to = __shfl(at, l, kWave);
            const int32_t* from = A.page_table + (uint64_t)(wave0 + l) * A.max_pages + __shfl(need, l, kWave);
            for (int64_t i = lane; i < n; i += kWave)
                if (to + i < A.num_pages) A.free_pages[to + i] = from[i];
        });
        have += s.all;
    }
    have = have > A.num_pages ? A.num_pages : have;
    __syncthreads();  // what was given may be taken below
    int64_t taken = 0, used = 0;
    for (uint32_t r = 0; r < rounds; ++r) {
        const uint32_t b = r * kThreads + threadIdx.x, wave0 = b & ~(kWave - 1u);
        int64_t take = 0, held = 0;
        bool ok = false;
        int64_t len = 0, then = 0, pos = 0;
        if (b < A.seqs) {
            const Row row(A, b);
            take = row.take();
            held = row.held;
            ok = row.ok;
            pos = row.first;
            len = A.lens[b];
            then = row.first + A.offsets[b + 1] - A.offsets[b];
        }
        const Scan s = scan(take, smem);
        const int64_t before = taken + s.before;
        const bool fits = ok && (take == 0 || before + take <= have);
        if (b < A.seqs) {
            first[b] = fits ? (int32_t)pos : -1;
            A.lens_out[b] = (int32_t)(fits ? then : len);
        }
        each(fits ? take : 0, [&](int l, int64_t n) {
            const int32_t* from = A.free_pages + (have - 1 - __shfl(before, l, kWave));
            int32_t* to = A.page_table + (uint64_t)(wave0 + l) * A.max_pages + __shfl(held, l, kWave);
            for (int64_t i = lane; i < n; i += kWave) to[i] = from[-i];
        });
        const Scan u = scan(fits ? take : 0, smem);
        taken += s.all;
        used += u.all;
    }
    __syncthreads();
    if (threadIdx.x == 0) A.count_out[0] = (int32_t)(have - used);
    if (with_slots)
        for (uint32_t t = threadIdx.x; t < A.tokens; t += kThreads) A.slots[t] = slot_of(A, first, t);
}

__global__ __launch_bounds__(256) void slots_kernel(KvPlan A, const int32_t* first) {
    const uint32_t t = blockIdx.x * 256u + threadIdx.x;
    if (t < A.tokens) A.slots[t] = slot_of(A, first, t);
}

constexpr uint32_t kOneLaunch = 4096;  // tokens

}  // namespace

size_t kv_plan_ws_bytes(uint32_t seqs, uint32_t) { return (size_t)seqs * 4u; }

hipError_t launch_kv_plan(const KvPlan& A, hipStream_t st) {
    int32_t* first = static_cast<int32_t*>(A.ws);
    const bool one = A.tokens <= kOneLaunch;
    plan_kernel<<<1, kThreads, 0, st>>>(A, first, one);
    if (!one) slots_kernel<<<(A.tokens + 255u) / 256u, 256, 0, st>>>(A, first);
    return hipGetLastError();
}

}  // namespace rz
