// A step's pages and slots from the sequences' lengths.
//
// Sequence b keeps keep[b] of its lens[b] tokens and adds new[b]; with
// held = ceil(lens / page_len) and need = ceil((keep + new) / page_len) it
// gives max(held - need, 0) pages to a stack, then takes max(need - held, 0).
// The i-th page given lies at stack[count + i], the i-th taken comes from
// stack[count + given - 1 - i], so two prefix sums over the sequences say
// where every page goes, in any order of execution.
//
// A few hundred bytes are read and written, so what counts is the chain of
// loads and barriers.  One workgroup does the sums, a lane a sequence, and for
// a decoding step everything else; where a step has more tokens than its
// lanes serve in four turns, a second launch gives every token its slot and
// writes the new pages' numbers as it meets their first tokens.  64 sequences'
// step 5.0 us; 131072 tokens of 96 prompts 5.4 and
// 4.4 us (the second alone moves 1.1 MB, 0.2 us of memory time).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "rz_device.h"
#include "rz_internal.h"

namespace rz {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / kWave;
constexpr uint32_t kOneLaunch = 4u * kThreads;  // tokens

// What the second launch (and the slots of the first) know of a sequence.
struct Row {
    int32_t first;  // position of its first new token, -1: refused
    uint32_t held;  // pages
    uint32_t top;   // place of its first new page in the stack; the next ones lie below
};

// Saturating sums: page counts of any input stay in order, and none wraps.
__device__ __forceinline__ uint32_t add(uint32_t a, uint32_t b) { return __builtin_elementwise_add_sat(a, b); }

// Sums over the lanes before this one, and over all of them, of two values.
struct Scan {
    uint32_t before[2], all[2];
};
__device__ __forceinline__ Scan scan(uint32_t x, uint32_t y, uint32_t (*smem)[2]) {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    uint32_t v[2] = {x, y};
#pragma unroll
    for (int c = 0; c < 2; ++c) {  // lanes 1, 2, 4, 8 before in a row of 16, then the last lane of the row and of the half before
        v[c] = add(v[c], (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v[c], 0x111, 0xF, 0xF, true));
        v[c] = add(v[c], (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v[c], 0x112, 0xF, 0xF, true));
        v[c] = add(v[c], (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v[c], 0x114, 0xF, 0xF, true));
        v[c] = add(v[c], (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v[c], 0x118, 0xF, 0xF, true));
        v[c] = add(v[c], (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v[c], 0x142, 0xA, 0xF, false));
        v[c] = add(v[c], (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v[c], 0x143, 0xC, 0xF, false));
    }
    Scan s = {{0, 0}, {0, 0}};
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const uint32_t up = (uint32_t)__shfl_up((int)v[c], 1, kWave);
        s.before[c] = lane ? up : 0;
        if (lane == kWave - 1) smem[wave][c] = v[c];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWaves; ++i)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const uint32_t n = smem[i][c];
            if (i < wave) s.before[c] = add(s.before[c], n);
            s.all[c] = add(s.all[c], n);
        }
    __syncthreads();
    return s;
}

// Calls f(lane, n of that lane) for each lane whose n is not 0, with the whole
// wave: f may shuffle before it loops.
template <typename F>
__device__ __forceinline__ void each(uint32_t n, F&& f) {
    for (uint64_t todo = __ballot(n > 0); todo; todo &= todo - 1) {
        const int l = __ffsll((unsigned long long)todo) - 1;
        f(l, (uint32_t)__shfl((int)n, l, kWave));
    }
}

// A step's demand of sequence b.
struct Step {
    int32_t len = 0;
    int64_t first = 0, then = 0;  // tokens kept, and with the new ones
    uint32_t held = 0, need = 0;
    bool ok = false, falls = false;  // falls: its offsets decrease
    __device__ __forceinline__ Step(const KvPlan& A, uint32_t b) {
        if (b >= A.seqs) return;
        len = A.lens[b];
        first = A.keep ? A.keep[b] : len;
        const int64_t fresh = (int64_t)A.offsets[b + 1] - A.offsets[b];
        then = first + fresh;
        falls = fresh < 0;
        ok = first >= 0 && first <= len && !falls && then <= INT32_MAX;
        held = ok ? ((uint32_t)len + (A.page_len - 1ull)) / A.page_len : 0;
        need = ok ? ((uint32_t)then + (A.page_len - 1ull)) / A.page_len : 0;
        ok = ok && held <= A.max_pages && need <= A.max_pages;
    }
    __device__ __forceinline__ uint32_t give() const { return ok && held > need ? held - need : 0; }
    __device__ __forceinline__ uint32_t take() const { return ok && need > held ? need - held : 0; }
};

// The sequence among [lo, hi) that token t belongs to, offsets[lo] <= t < offsets[hi].
__device__ __forceinline__ uint32_t sequence_of(const int32_t* offsets, uint32_t lo, uint32_t hi, uint32_t t) {
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) >> 1;
        if ((int64_t)t >= offsets[mid]) lo = mid; else hi = mid;
    }
    return lo;
}

// The slot of token t of sequence b.  A new page's number is taken from
// the stack and, at the page's first token, written to the table.
__device__ __forceinline__ int64_t slot_of(const KvPlan& A, const Row& row, uint32_t b, uint32_t t, int32_t offset) {
    if (row.first < 0) return -1;
    const uint64_t pos = (uint64_t)(uint32_t)row.first + (t - (uint32_t)offset), page = pos / A.page_len;
    if (page >= A.max_pages) return -1;  // a write stays in the row, and a read in the stack, whatever the lengths say
    const uint32_t at = (uint32_t)(pos - page * A.page_len);
    int32_t* entry = A.page_table + (uint64_t)b * A.max_pages + page;
    int64_t id;
    if (page >= row.held) {
        const uint64_t below = page - row.held;
        if (below > row.top || row.top - below >= A.num_pages) return -1;
        id = A.free_pages[row.top - below];
        if (at == 0) *entry = (int32_t)id;
    } else {
        id = *entry;
    }
    return id < 0 ? -1 : id * A.page_len + at;
}

// The row whose run of a prefix sum place i lies in: sums[b] <= i < sums[b + 1].
__device__ __forceinline__ uint32_t row_of_place(const uint32_t* sums, uint32_t rows, uint32_t i) {
    uint32_t lo = 0, hi = rows;
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) >> 1;
        if (i >= sums[mid]) lo = mid; else hi = mid;
    }
    return lo;
}

// `few`: up to 1024 sequences, a lane each, whose pages the lanes move one a
// lane; otherwise rounds of 1024, whose waves move a sequence's at a time.
__global__ __launch_bounds__(kThreads) void plan_kernel(KvPlan A, Row* rows, bool one) {
    __shared__ uint32_t smem[kWaves][2];
    __shared__ uint32_t used_of;
    __shared__ Row row_of[kThreads];
    __shared__ int32_t offset_of[kThreads + 1];
    __shared__ uint32_t sums[kThreads], need_of[kThreads];
    __shared__ bool falls_of;
    const int lane = threadIdx.x & (kWave - 1);
    const uint32_t rounds = (A.seqs + kThreads - 1) / kThreads;
    const bool few = rounds <= 1;
    const int32_t count = A.free_count[0];
    uint32_t have = count < 0 ? 0 : (uint32_t)count > A.num_pages ? A.num_pages : (uint32_t)count;
    if (threadIdx.x == 0) used_of = 0;
    Step step(A, threadIdx.x);
    if (few && A.seqs)
        for (uint32_t i = threadIdx.x; i <= A.seqs; i += kThreads) offset_of[i] = A.offsets[i];
    // new pages are written here unless their tokens do that (those that `tokens` leaves out have pages too)
    const bool fill = A.seqs != 0 && (A.offsets[A.seqs] > (int64_t)A.tokens || A.offsets[0] < 0);
    uint32_t before_take = 0, taken = 0;
    if (few) {
        // offsets that decrease leave no sequence its tokens: a sum at its limit, which no cache's pages reach, says so
        const Scan s = scan(step.falls ? ~0u : step.give(), step.take(), smem);
        const uint32_t given = s.all[0] == ~0u ? 0 : s.all[0];
        step.ok = step.ok && s.all[0] != ~0u;
        before_take = s.before[1];
        sums[threadIdx.x] = s.before[0];
        need_of[threadIdx.x] = step.need;
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < given && add(have, i) < A.num_pages; i += kThreads) {
            const uint32_t b = row_of_place(sums, A.seqs, i);
            A.free_pages[have + i] = A.page_table[(uint64_t)b * A.max_pages + need_of[b] + (i - sums[b])];
        }
        have = add(have, given);
    }
    bool falls = false;
    if (!few) {
        if (threadIdx.x == 0) falls_of = false;
        __syncthreads();
        for (uint32_t b = threadIdx.x; b < A.seqs; b += kThreads)
            if (A.offsets[b + 1] < A.offsets[b]) falls_of = true;
        __syncthreads();
        falls = falls_of;
    }
    for (uint32_t r = 0; r < rounds && !few && !falls; ++r) {
        step = Step(A, r * kThreads + threadIdx.x);
        const uint32_t give = step.give(), wave0 = (r * kThreads + threadIdx.x) & ~(kWave - 1u);
        const Scan s = scan(give, 0, smem);
        const uint32_t at = add(have, s.before[0]);
        each(give, [&](int l, uint32_t n) {
            const uint32_t to = (uint32_t)__shfl((int)at, l, kWave);
            const int32_t* from = A.page_table + (uint64_t)(wave0 + l) * A.max_pages + (uint32_t)__shfl((int)step.need, l, kWave);
            for (uint32_t i = lane; i < n && add(to, i) < A.num_pages; i += kWave) A.free_pages[to + i] = from[i];
        });
        have = add(have, s.all[0]);
    }
    have = have > A.num_pages ? A.num_pages : have;
    __syncthreads();  // what was given may be taken below
    for (uint32_t r = 0; r < rounds; ++r) {
        const uint32_t b = r * kThreads + threadIdx.x, wave0 = b & ~(kWave - 1u);
        if (!few) {
            step = Step(A, b);
            step.ok = step.ok && !falls;
            const Scan s = scan(step.take(), 0, smem);
            before_take = add(taken, s.before[0]);
            taken = add(taken, s.all[0]);
        }
        const uint32_t take = step.take(), after = add(before_take, take);
        const bool fits = step.ok && (take == 0 || after <= have);
        if (b < A.seqs) {
            const Row row = {fits ? (int32_t)step.first : -1, step.held, have - 1 - before_take};
            if (one && few) row_of[b] = row; else rows[b] = row;
            A.lens_out[b] = (int32_t)(fits ? step.then : step.len);
        }
        if (fits && take) atomicMax(&used_of, after);
        each(fits && fill ? take : 0, [&](int l, uint32_t n) {
            const int32_t* from = A.free_pages + (have - 1 - (uint32_t)__shfl((int)before_take, l, kWave));
            int32_t* to = A.page_table + (uint64_t)(wave0 + l) * A.max_pages + (uint32_t)__shfl((int)step.held, l, kWave);
            for (uint32_t i = lane; i < n; i += kWave) to[i] = from[-(int64_t)i];
        });
    }
    __syncthreads();
    if (threadIdx.x == 0) A.count_out[0] = (int32_t)(have - used_of);
    if (!one) return;
    const int32_t* offsets = few ? offset_of : A.offsets;
    const int64_t begin = A.seqs ? offsets[0] : 0, end = A.seqs ? offsets[A.seqs] : 0;
    for (uint32_t t = threadIdx.x; t < A.tokens; t += kThreads) {
        int64_t slot = -1;
        if (t >= begin && t < end) {
            const uint32_t b = sequence_of(offsets, 0, A.seqs, t);
            slot = slot_of(A, few ? row_of[b] : rows[b], b, t, offsets[b]);
        }
        A.slots[t] = slot;
    }
}

// The sequences of a workgroup's first and last token narrow down those of the others.
__global__ __launch_bounds__(256) void slots_kernel(KvPlan A, const Row* rows) {
    const uint32_t t = blockIdx.x * 256u + threadIdx.x;
    if (t >= A.tokens) return;
    int64_t slot = -1;
    if (A.seqs != 0 && (int64_t)t >= A.offsets[0] && (int64_t)t < A.offsets[A.seqs]) {
        const int64_t begin = A.offsets[0], end = A.offsets[A.seqs], first = blockIdx.x * 256ll, last = first + 255;
        const uint32_t lo = sequence_of(A.offsets, 0, A.seqs, (uint32_t)(first < begin ? begin : first));
        const uint32_t hi = sequence_of(A.offsets, lo, A.seqs, (uint32_t)(last < end ? last : end - 1)) + 1;
        const uint32_t b = sequence_of(A.offsets, lo, hi, t);
        slot = slot_of(A, rows[b], b, t, A.offsets[b]);
    }
    A.slots[t] = slot;
}

}  // namespace

size_t kv_plan_ws_bytes(uint32_t seqs, uint32_t tokens) {
    return seqs <= (uint32_t)kThreads && tokens <= kOneLaunch ? 0 : (size_t)seqs * sizeof(Row);  // 0: the rows stay in LDS
}

hipError_t launch_kv_plan(const KvPlan& A, hipStream_t st) {
    Row* rows = static_cast<Row*>(A.ws);
    const bool one = A.tokens <= kOneLaunch;
    plan_kernel<<<1, kThreads, 0, st>>>(A, rows, one);
    if (!one) slots_kernel<<<(A.tokens + 255u) / 256u, 256, 0, st>>>(A, rows);
    return hipGetLastError();
}

}  // namespace rz
