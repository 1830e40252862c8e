// A step's page tables, positions and cache slots from the requests' lengths
// (tq_plan_step), and the way back of finished requests' pages
// (tq_release_pages).
//
// With n_b new tokens behind len_b cached ones, request b needs want_b =
// ceil((len_b + n_b) / page) pages and takes grow_b = max(want_b - owned_b, 0)
// from the top of the free stack.  Two running sums over the requests, of n and
// of grow, say which request a row or a new page belongs to.
//
// Bound: latency (lengths -> sums -> request of a row -> page -> slot).  Every
// workgroup forms the sums for itself, a request a thread and 1024 at a time,
// up to the rows it writes; so one launch does it, whatever the lengths are, and
// nothing is handed from one workgroup to another.  Rows, and new pages, find
// their request by bisection in LDS, so a prompt's rows and pages spread over
// all threads.  64 requests of a token: 3.6 us; 511 requests of 190 thousand tokens
// in all, whose positions and slots are 1.5 MB: 6.2 us.
#include <algorithm>

#include "block_ops.h"

namespace tq {
namespace {

constexpr int WAVES = 16, THREADS = 64 * WAVES;
constexpr int ROWS = THREADS;                    // rows (tokens) of a workgroup
constexpr int64_t MAX_LEN = int64_t(1) << 30;    // positions of a request

// What is known of the 1024 requests in hand.
struct Shared {
    uint32_t row0[THREADS];                      // first row of each
    uint64_t page0[THREADS];                     // new pages before each
    int len[THREADS], owned[THREADS];
    uint64_t scan[2][WAVES];
};

// Last i of 0 .. n - 1 with start[i] <= x (start[0] <= x); empty ones are passed over.
template <typename T> __device__ __forceinline__ int find(const T *start, int n, T x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__global__ __launch_bounds__(THREADS) void k_plan(PlanArgs a)
{
    __shared__ Shared s;
    const int tid = threadIdx.x;
    const int64_t P = int64_t(1) << a.log_page;
    const int64_t count = min(max((int64_t)*a.free_count, (int64_t)0), a.free_capacity);
    const int64_t row_begin = (int64_t)blockIdx.x * ROWS, row = row_begin + tid;
    uint64_t rows = 0, pages = 0;                // before the requests in hand
    for (int64_t base = 0, turn = 0; base < a.batch; base += THREADS, turn++) {
        const int64_t b = base + tid;
        const int in_hand = (int)min((int64_t)THREADS, a.batch - base);
        int64_t len = 0, n = 0, owned = 0;
        if (b < a.batch) {
            len = min(max((int64_t)a.lens[b], (int64_t)0), MAX_LEN);
            n = min(max((int64_t)a.new_tokens[b], (int64_t)0), a.tokens);
            owned = min(max((int64_t)a.owned[b], (int64_t)0), a.table_pages);
        }
        // tokens that there are no rows for are left out
        uint64_t all_rows, all_pages;
        const uint64_t r = rows + scan_before<WAVES, uint64_t>((uint64_t)n, s.scan[0], all_rows);
        const int64_t r0 = min((int64_t)r, a.tokens);
        n = min(n, a.tokens - r0);
        const int64_t want = min((len + n + P - 1) >> a.log_page, a.table_pages);
        const int64_t grow = max(want - owned, (int64_t)0);
        const uint64_t p0 =
            pages + scan_before<WAVES, uint64_t>((uint64_t)grow, s.scan[1], all_pages);
        rows += all_rows;
        pages += all_pages;
        s.row0[tid] = (uint32_t)r0;
        s.page0[tid] = p0;
        s.len[tid] = (int)len;
        s.owned[tid] = (int)owned;
        if (b < a.batch && turn % gridDim.x == blockIdx.x) {
            const int64_t got = min(max(count - (int64_t)p0, (int64_t)0), grow);
            a.starts[b] = (int32_t)r0;
            a.new_lens[b] = (int32_t)(len + n);
            a.new_owned[b] = (int32_t)(owned + got);
            if (b == a.batch - 1) {
                a.starts[a.batch] = (int32_t)(r0 + n);
                const int64_t left = count - (int64_t)pages;
                *a.free_left = (int32_t)max(left, -(int64_t(1) << 31));
            }
        }
        __syncthreads();
        const int64_t end = min((int64_t)rows, a.tokens);
        // new pages, every gridDim-th thousand of them
        const uint64_t first = s.page0[0];
        for (uint64_t i = first + (uint64_t)blockIdx.x * THREADS + tid; i < pages;
             i += (uint64_t)gridDim.x * THREADS) {
            const int k = find(s.page0, in_hand, i);
            const int64_t at = count - 1 - (int64_t)i;
            a.table[(base + k) * a.table_stride + s.owned[k] + (int64_t)(i - s.page0[k])] =
                at >= 0 ? a.free_pages[at] : -1;
        }
        if (row >= s.row0[0] && row < end) {
            const int k = find(s.row0, in_hand, (uint32_t)row);
            const int64_t pos = s.len[k] + (row - s.row0[k]), j = pos >> a.log_page;
            int64_t id = -1;
            if (j < s.owned[k]) {
                id = a.table[(base + k) * a.table_stride + j];
            } else if (j < a.table_pages) {
                const int64_t at = count - 1 - (int64_t)(s.page0[k] + (uint64_t)(j - s.owned[k]));
                id = at >= 0 ? a.free_pages[at] : -1;
            }
            const int64_t slot = (id << a.log_page) + (pos & (P - 1));
            a.positions[row] = (int32_t)pos;
            a.slots[row] = id >= 0 && slot < (int64_t(1) << 31) ? (int32_t)slot : -1;
        }
        __syncthreads();
    }
    if (row < a.tokens && row >= min((int64_t)rows, a.tokens)) {
        a.positions[row] = 0;
        a.slots[row] = -1;
    }
    if (a.batch == 0 && blockIdx.x == 0 && tid == 0) {
        a.starts[0] = 0;
        *a.free_left = (int32_t)count;
    }
}

__global__ __launch_bounds__(THREADS) void k_release(ReleaseArgs a)
{
    __shared__ uint64_t page0[THREADS], scan[WAVES];
    const int tid = threadIdx.x;
    const int64_t count = min(max((int64_t)*a.free_count, (int64_t)0), a.free_capacity);
    uint64_t pages = 0;
    for (int64_t base = 0, turn = 0; base < a.batch; base += THREADS, turn++) {
        const int64_t b = base + tid;
        const int in_hand = (int)min((int64_t)THREADS, a.batch - base);
        int64_t owned = 0;
        bool done = false;
        if (b < a.batch) {
            owned = min(max((int64_t)a.owned[b], (int64_t)0), a.table_pages);
            done = a.done[b] != 0;
            if (turn % gridDim.x == blockIdx.x)
                a.new_owned[b] = done ? 0 : (int32_t)owned;
        }
        const uint64_t first = pages;
        uint64_t all;
        page0[tid] = pages + scan_before<WAVES, uint64_t>(done ? (uint64_t)owned : 0, scan, all);
        pages += all;
        __syncthreads();
        for (uint64_t i = first + (uint64_t)blockIdx.x * THREADS + tid; i < pages;
             i += (uint64_t)gridDim.x * THREADS) {
            const int k = find(page0, in_hand, i);
            int32_t *entry = a.table + (base + k) * a.table_stride + (int64_t)(i - page0[k]);
            const int64_t at = count + (int64_t)i;
            if (at < a.free_capacity)
                a.free_pages[at] = *entry;
            *entry = -1;
        }
        __syncthreads();
    }
    if (blockIdx.x == 0 && tid == 0)
        *a.free_left = (int32_t)min(count + (int64_t)pages, a.free_capacity);
}

}  // namespace

hipError_t launch_plan(const PlanArgs &a, hipStream_t s)
{
    const int64_t blocks = std::max<int64_t>(1, (a.tokens + ROWS - 1) / ROWS);
    if (!grid_fits(blocks, THREADS))
        return hipErrorInvalidConfiguration;
    k_plan<<<dim3((unsigned)blocks), THREADS, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_release(const ReleaseArgs &a, hipStream_t s)
{
    // a request a thread; its pages, some thousands at most, spread over a few
    const int64_t blocks = std::min<int64_t>(16, std::max<int64_t>(1, (a.batch + 63) / 64));
    k_release<<<dim3((unsigned)blocks), THREADS, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace tq
