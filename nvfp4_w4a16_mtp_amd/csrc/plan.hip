// kv8_plan: block tables, positions and slots of a step, built on the device from
// request lengths (definition in nvfp4_mtp.h).
//
// One workgroup walks the requests a thread each, blockDim.x at a time, in three
// passes: prefix sums of the new rows (cu_rows, lengths); pages that go, pushed on the
// stack of free pages; pages that come, popped from it.  A chunk's pages are spread
// over all threads: page i belongs to the request whose prefix sums enclose it, found
// by bisection in LDS.  A decode step is all latency: a few KB, through a chain of loads,
// scans and barriers.  Few rows' positions and slots are written here,
// many by a second launch.  64 requests that give back 1530 pages: 8 us a launch.  700 with
// 166 k rows of prompts that give back 19.6 k pages and take 2.6 k: 25 us, the throughput of one
// CU (a round of 1024 pages costs a bisection and a chain of scattered loads and stores), and
// 5 us for the rows.
#include "common.hpp"

namespace nvfp4 {

constexpr int kPlanThreads = 1024;

struct PlanArgs {
    int32_t *table, *held, *free_pages, *free_count;
    int batch, max_pages, num_pages, lp;
    const int32_t *kept, *fresh;
    int rows;
    int32_t *cu, *lens, *positions;
    int64_t *slots;
    int32_t *missing;
};

// Sums that stop at 2^32 - 1 (only states that make no sense come near it).
__device__ __forceinline__ uint32_t add_sat(uint32_t a, uint32_t b) { return __builtin_elementwise_add_sat(a, b); }

// Prefix sums of N values a thread over the workgroup: v becomes the sum of the threads
// before this one, total the sum of all.  The caller's last reads of `waves` lie before
// a barrier.
template <int N>
__device__ __forceinline__ void scan_group(uint32_t (&v)[N], uint32_t (*waves)[N], uint32_t (&total)[N]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = blockDim.x >> 6;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        uint32_t run = v[k];
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t o = __shfl_up(run, d, 64);
            if (lane >= d) run = add_sat(run, o);
        }
        if (lane == 63) waves[wave][k] = run;
        v[k] = __shfl_up(run, 1, 64);
        if (lane == 0) v[k] = 0;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
        uint32_t before = 0;
        total[k] = 0;
        for (int i = 0; i < n; ++i) {
            if (i == wave) before = total[k];
            total[k] = add_sat(total[k], waves[i][k]);
        }
        v[k] = add_sat(before, v[k]);
    }
}

// First i with ends[i] > x (ascending; x < ends[n - 1]).
__device__ __forceinline__ int owner(const uint32_t *ends, int n, uint32_t x) {
    int lo = -1, hi = n - 1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (ends[mid] > x) hi = mid; else lo = mid;
    }
    return hi;
}

// Position and slot of row r, the i-th new one of request b.
__device__ __forceinline__ void write_row(const PlanArgs &a, int b, int kept, int r, int i) {
    const int pos = kept + i;
    if (a.positions) a.positions[r] = pos;
    if (a.slots) {
        const int page = a.table[(int64_t)b * a.max_pages + (pos >> a.lp)];
        a.slots[r] = page >= 0 && page < a.num_pages ? ((int64_t)page << a.lp) + (pos & ((1 << a.lp) - 1)) : -1;
    }
}

__global__ __launch_bounds__(kPlanThreads) void k_plan(PlanArgs a, int rows_here) {
    constexpr int W = kPlanThreads / 64;
    __shared__ uint32_t row_sums[W][1], page_sums[2][W][2], ends[3][kPlanThreads];
    __shared__ int32_t from[3][kPlanThreads];
    const int tid = threadIdx.x, step = blockDim.x;
    const int cap = (int)min((int64_t)a.max_pages << a.lp, (int64_t)0x7FFFFF00);
    const int64_t count = min(max(*a.free_count, 0), a.num_pages);
    const int chunks = (a.batch + step - 1) / step;

    // this thread's request of a chunk: pages held and needed
    int h = 0, need = 0;
    auto pages = [&](int c) {
        const int b = c * step + tid;
        h = need = 0;
        if (b < a.batch) {
            h = min(max(a.held[b], 0), a.max_pages);
            need = (a.lens[b] + (1 << a.lp) - 1) >> a.lp;
        }
    };
    uint32_t before[2], total[2], rows_before[1], rows_total[1];   // pages that go, that come; rows
    int64_t rows = 0, given = 0;
    if (tid == 0) a.cu[0] = 0;
    for (int c = 0; c < chunks; ++c) {
        const int b = c * step + tid;
        int kept = 0, n = 0;
        h = need = 0;
        if (b < a.batch) {
            kept = min(max(a.kept[b], 0), cap);
            n = min(max(a.fresh[b], 0), cap - kept);
            h = min(max(a.held[b], 0), a.max_pages);
        }
        rows_before[0] = n;
        scan_group<1>(rows_before, row_sums, rows_total);
        const int64_t start = rows + rows_before[0];
        rows += rows_total[0];
        const int lo = (int)min(start, (int64_t)a.rows), hi = (int)min(start + n, (int64_t)a.rows), len = kept + hi - lo;
        if (b < a.batch) {
            a.cu[b + 1] = hi;
            a.lens[b] = len;                          // (may be a.kept itself)
            need = (len + (1 << a.lp) - 1) >> a.lp;
        }
        ends[2][tid] = hi;                            // for the rows, where this chunk is the only one
        from[2][tid] = len;
        before[0] = max(h - need, 0);
        before[1] = max(need - h, 0);
        scan_group<2>(before, page_sums[c & 1], total);
        given += total[0];
    }
    // the pages that go, the first of them on top of the stack
    const int64_t top = count + given;
    int64_t moved = 0;
    for (int c = 0; c < chunks && given > 0; ++c) {
        if (chunks > 1) {
            __syncthreads();
            pages(c);
            before[0] = max(h - need, 0);
            before[1] = max(need - h, 0);
            scan_group<2>(before, page_sums[0], total);
        }
        ends[0][tid] = add_sat(before[0], max(h - need, 0));
        from[0][tid] = need;
        __syncthreads();
        for (uint32_t i = tid; i < total[0]; i += step) {
            const int o = owner(ends[0], step, i);
            int32_t *e = a.table + (int64_t)(c * step + o) * a.max_pages + from[0][o] + (i - (o ? ends[0][o - 1] : 0));
            const int64_t at = top - 1 - moved - i;
            if (at < a.num_pages) a.free_pages[at] = *e;
            *e = -1;
        }
        moved += total[0];
    }
    // the pages that come, from the top on
    const int64_t have = min(top, (int64_t)a.num_pages);
    int64_t taken = 0;
    for (int c = 0; c < chunks; ++c) {
        const int b = c * step + tid;
        if (chunks > 1) {
            __syncthreads();
            pages(c);
            before[0] = max(h - need, 0);
            before[1] = max(need - h, 0);
            scan_group<2>(before, page_sums[0], total);
        }
        const int want = max(need - h, 0);
        ends[1][tid] = add_sat(before[1], want);
        from[1][tid] = h;
        if (b < a.batch) a.held[b] = min(need, h) + (int)min(max(have - (taken + before[1]), (int64_t)0), (int64_t)want);
        __syncthreads();                              // (and the pages given back are in place)
        for (uint32_t i = tid; i < total[1]; i += step) {
            const int o = owner(ends[1], step, i);
            const int64_t at = have - 1 - taken - i;
            a.table[(int64_t)(c * step + o) * a.max_pages + from[1][o] + (i - (o ? ends[1][o - 1] : 0))] = at >= 0 ? a.free_pages[at] : -1;
        }
        taken += total[1];
    }
    if (tid == 0) {
        *a.free_count = (int)max(have - taken, (int64_t)0);
        *a.missing = (int)min(max(taken - have, (int64_t)0), (int64_t)0x7FFFFFFF);
    }
    if (!rows_here) return;
    __syncthreads();                                  // (the tables and cu are this workgroup's own stores)
    for (int c = 0; c < chunks; ++c) {
        const int b = c * step + tid, n = min(a.batch - c * step, step);
        int first = 0;
        if (chunks > 1) {
            __syncthreads();
            first = a.cu[c * step];
            ends[2][tid] = b < a.batch ? a.cu[b + 1] : 0;
            from[2][tid] = b < a.batch ? a.lens[b] : 0;
            __syncthreads();
        }
        for (int r = first + tid; r < (int)ends[2][n - 1]; r += step) {
            const int o = owner(ends[2], n, r);
            // (the request's last row is its last token)
            write_row(a, c * step + o, from[2][o] - (int)ends[2][o], r, r);
        }
    }
}

// The rows' positions and slots, a thread a row.
__global__ __launch_bounds__(256) void k_plan_rows(PlanArgs a) {
    const int r = blockIdx.x * 256 + threadIdx.x;
    if (r >= a.cu[a.batch]) return;
    int lo = 0, hi = a.batch;                         // cu[lo] <= r < cu[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu[mid] > r) hi = mid; else lo = mid;
    }
    write_row(a, lo, a.lens[lo] - a.cu[lo + 1], r, r);
}

// Rows written by the planning workgroup itself, without another launch: 64 requests, 2048
// rows 6.6 us a call (8.0 with the launch), 4096 rows 8.0 (7.9); 700 requests 7.4 (9.2) and 9.2
// (9.2).
constexpr int kRowsHere = 2048;

// Threads of the planning workgroup.  Fewer wavefronts pass their barriers sooner, more walk the
// requests and rows in fewer steps: 64 requests, 512 rows 5.1 us with 256 threads (5.8 with
// 1024), 1024 rows 6.3 (5.9); 200 requests, 800 rows 6.8 (6.0).
static int plan_threads(int batch, int rows) { return batch <= 64 && rows <= 512 ? 256 : kPlanThreads; }

}  // namespace nvfp4

using namespace nvfp4;

extern "C" int kv8_plan(const nvfp4_kv8_pool *pool, const int32_t *kept_lens, const int32_t *new_rows, int32_t rows,
                        int32_t *cu_rows, int32_t *kv_lens, int32_t *positions, int64_t *slots, int32_t *missing, void *stream) {
    const char *who = "kv8_plan";
    if (!pool) return fail(NVFP4_ERR_ARG, "%s: NULL pool", who);
    const int p = pool->page_tokens;
    if (p != 16 && p != 32 && p != 64 && p != 128)
        return fail(NVFP4_ERR_SHAPE, "%s: page_tokens=%d (need 16, 32, 64 or 128)", who, p);
    if (pool->batch < 0 || pool->max_pages < 1 || pool->num_pages < 1 || rows < 0)
        return fail(NVFP4_ERR_SHAPE, "%s: batch=%d max_pages=%d num_pages=%d rows=%d", who, pool->batch, pool->max_pages,
                    pool->num_pages, rows);
    if (!pool->free_pages || !pool->free_count || !cu_rows || !missing ||
        (pool->batch > 0 && (!pool->block_table || !pool->held || !kept_lens || !new_rows || !kv_lens)))
        return fail(NVFP4_ERR_ARG, "%s: NULL pointer", who);
    const void *all[] = {pool->block_table, pool->held, pool->free_pages, pool->free_count, kept_lens,
                         new_rows, cu_rows, kv_lens, positions, missing};
    for (const void *x : all)
        if (!aligned(x, 4)) return fail(NVFP4_ERR_ALIGN, "%s: a pointer is not 4-byte aligned", who);
    if (!aligned(slots, 8)) return fail(NVFP4_ERR_ALIGN, "%s: slots not 8-byte aligned", who);
    PlanArgs a{pool->block_table, pool->held, pool->free_pages, pool->free_count, pool->batch, pool->max_pages, pool->num_pages,
               __builtin_ctz((unsigned)p), kept_lens, new_rows, rows, cu_rows, kv_lens, positions, slots, missing};
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const bool write = rows > 0 && pool->batch > 0 && (positions || slots), here = write && rows <= kRowsHere;
    hipLaunchKernelGGL(k_plan, dim3(1), dim3(plan_threads(pool->batch, rows)), 0, s, a, here ? 1 : 0);
    if (write && !here) hipLaunchKernelGGL(k_plan_rows, dim3((unsigned)(((int64_t)rows + 255) / 256)), dim3(256), 0, s, a);
    return check_launch(who);
}
