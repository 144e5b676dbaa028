// kv8_plan: block tables, positions and slots of a step, built on the device from
// request lengths (definition in nvfp4_mtp.h).
//
// One workgroup walks the requests a thread each, blockDim.x at a time, in three
// passes: prefix sums of the new rows (cu_rows, lengths); pages that go, pushed on the
// stack of free pages; pages that come, popped from it.  A chunk's pages are spread
// over all threads: page i belongs to the request whose prefix sums enclose it, found
// by bisection in LDS.  Nothing but latency: a decode step moves a few KB, through a
// chain of loads, scans and barriers.  Few rows' positions and slots are written here,
// many by a second launch.
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

// Prefix sum over the workgroup's threads, this thread's value included; total: all.
__device__ __forceinline__ int64_t scan_group(int64_t v, int64_t *waves, int64_t &total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = blockDim.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t o = __shfl_up(v, d, 64);
        if (lane >= d) v += o;
    }
    __syncthreads();                                  // the last scan's reads of waves are over
    if (lane == 63) waves[wave] = v;
    __syncthreads();
    int64_t before = 0;
    total = 0;
    for (int i = 0; i < n; ++i) {
        if (i < wave) before += waves[i];
        total += waves[i];
    }
    return v + before;
}

// First i with ends[i] > x (ascending; x < ends[n - 1]).
__device__ __forceinline__ int owner(const int64_t *ends, int n, int64_t x) {
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
    __shared__ int64_t waves[kPlanThreads / 64], ends[kPlanThreads];
    __shared__ int32_t from[kPlanThreads];
    const int tid = threadIdx.x, step = blockDim.x;
    const int cap = (int)min((int64_t)a.max_pages << a.lp, (int64_t)0x7FFFFF00);
    const int64_t count = min(max(*a.free_count, 0), a.num_pages);
    const int chunks = (a.batch + step - 1) / step;

    // this thread's request of the present chunk: pages held and needed
    int h = 0, need = 0;
    auto pages = [&](int c) {
        const int b = c * step + tid;
        h = need = 0;
        if (b < a.batch) {
            h = min(max(a.held[b], 0), a.max_pages);
            need = (a.lens[b] + (1 << a.lp) - 1) >> a.lp;
        }
    };
    int64_t rows = 0, given = 0, total;
    if (tid == 0) a.cu[0] = 0;
    for (int c = 0; c < chunks; ++c) {
        const int b = c * step + tid;
        int kept = 0, n = 0;
        if (b < a.batch) {
            kept = min(max(a.kept[b], 0), cap);
            n = min(max(a.fresh[b], 0), cap - kept);
        }
        const int64_t end = rows + scan_group(n, waves, total);
        rows += total;
        const int lo = (int)min(end - n, (int64_t)a.rows), hi = (int)min(end, (int64_t)a.rows);
        if (b < a.batch) {
            a.cu[b + 1] = hi;
            a.lens[b] = kept + hi - lo;               // (may be a.kept itself)
        }
        pages(c);                                     // (this thread's own store)
        scan_group(max(h - need, 0), waves, total);
        given += total;
    }
    // the pages that go, the first of them on top of the stack
    const int64_t top = count + given;
    int64_t moved = 0;
    if (given > 0) {
        for (int c = 0; c < chunks; ++c) {
            if (chunks > 1) pages(c);
            ends[tid] = scan_group(max(h - need, 0), waves, total);   // (its barriers follow the last reads of ends)
            from[tid] = need;
            __syncthreads();
            for (int64_t i = tid; i < total; i += step) {
                const int o = owner(ends, step, i);
                int32_t *e = a.table + (int64_t)(c * step + o) * a.max_pages + from[o] + (i - (o ? ends[o - 1] : 0));
                const int64_t at = top - 1 - moved - i;
                if (at < a.num_pages) a.free_pages[at] = *e;
                *e = -1;
            }
            moved += total;
        }
    }
    // the pages that come, from the top on
    const int64_t have = min(top, (int64_t)a.num_pages);
    int64_t taken = 0;
    for (int c = 0; c < chunks; ++c) {
        const int b = c * step + tid;
        if (chunks > 1) pages(c);
        const int want = max(need - h, 0);
        const int64_t last = scan_group(want, waves, total);
        ends[tid] = last;
        from[tid] = h;
        if (b < a.batch) a.held[b] = min(need, h) + (int)min(max(have - (taken + last - want), (int64_t)0), (int64_t)want);
        __syncthreads();
        for (int64_t i = tid; i < total; i += step) {
            const int o = owner(ends, step, i);
            const int64_t at = have - 1 - taken - i;
            a.table[(int64_t)(c * step + o) * a.max_pages + from[o] + (i - (o ? ends[o - 1] : 0))] = at >= 0 ? a.free_pages[at] : -1;
        }
        taken += total;
    }
    if (tid == 0) {
        *a.free_count = (int)max(have - taken, (int64_t)0);
        *a.missing = (int)min(max(taken - have, (int64_t)0), (int64_t)0x7FFFFFFF);
    }
    if (!rows_here) return;
    __syncthreads();                                  // (the tables and cu are this workgroup's own stores)
    for (int c = 0; c < chunks; ++c) {
        const int b = c * step + tid, n = min(a.batch - c * step, step);
        __syncthreads();
        const int first = a.cu[c * step];
        if (b < a.batch) {
            ends[tid] = a.cu[b + 1];
            from[tid] = a.lens[b];
        }
        __syncthreads();
        for (int r = first + tid; r < (int)ends[n - 1]; r += step) {
            const int o = owner(ends, n, r);
            // (the request's last row is its last token)
            write_row(a, c * step + o, from[o] - (int)ends[o], r, r);
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

constexpr int kRowsHere = 2048;

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
    hipLaunchKernelGGL(k_plan, dim3(1), dim3(pool->batch <= 256 && rows <= 1024 ? 256 : kPlanThreads), 0, s, a, here ? 1 : 0);
    if (write && !here) hipLaunchKernelGGL(k_plan_rows, dim3((unsigned)(((int64_t)rows + 255) / 256)), dim3(256), 0, s, a);
    return check_launch(who);
}
