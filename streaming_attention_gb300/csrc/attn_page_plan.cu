// Block tables and slots of a serving step, built on the device from the
// requests' lengths: which pages each request's new keys go to, the row of the
// pool that each new row of the batch is written to, and the lengths the paged
// calls read.
//
// With c_b keys cached and n_b new ones, request b holds old_b = ceil(c_b / ps)
// pages and takes need_b = ceil((c_b + n_b) / ps) - old_b more. Two exclusive
// sums over the requests place everything: start_b = sum n gives its rows in
// the batch, first_b = sum need its pages in the free list. The sums run over
// at most a few thousand requests, which one block does in a microsecond or
// two, so there is one launch: every block computes them for itself, a chunk of
// 1024 requests at a time, and takes its share of the chunk's rows and pages,
// whose request it finds by bisection in shared memory. No block reads a table
// entry that another one writes: entries below old_b are only read, the others
// only written (their page is computed from the free list instead).
#include <cuda_runtime.h>
#include <stdint.h>

#include "attn.h"
#include "attn_internal.h"

namespace attn {
namespace {

constexpr int kPlanThreads = 1024;  // requests of a chunk, one per thread
constexpr int64_t kI32Max = 2147483647LL;

struct PlanArgs {
    const int* cached;
    const int* fresh;
    const int* free_pages;
    int* table;
    int* seq_lens;
    int* row_starts;
    int* slots;
    int* stats;
    int B, page_size, max_pages, num_free, num_rows;
};

__device__ __forceinline__ int saturate(long long x) { return (int)(x < kI32Max ? x : kI32Max); }

// Exclusive sum over the block of x, plus the block's total. `part` holds 32 values.
__device__ __forceinline__ long long block_sum(long long x, long long* part, long long* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long s = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += y;
    }
    __syncthreads();  // the last use of `part` is done
    if (lane == 31) part[warp] = s;
    __syncthreads();
    if (warp == 0) {
        long long w = part[lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, w, d);
            if (lane >= d) w += y;
        }
        part[lane] = w;
    }
    __syncthreads();
    *total = part[31];
    return s - x + (warp > 0 ? part[warp - 1] : 0);
}

// The last entry e of the ascending a[0..n) with a[e] <= x; a[0] <= x.
__device__ __forceinline__ int last_not_above(const long long* a, int n, long long x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const PlanArgs a) {
    __shared__ long long start[kPlanThreads], first[kPlanThreads], part[32];
    __shared__ int have[kPlanThreads], old[kPlanThreads];
    const long long mine = (long long)blockIdx.x * kPlanThreads + threadIdx.x;
    const long long step = (long long)gridDim.x * kPlanThreads;
    long long rows = 0, pages = 0, lost = 0;  // of the requests before this chunk
    for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
        const int b = b0 + threadIdx.x;
        const bool in = b < a.B;
        const long long c = in ? max(__ldg(a.cached + b), 0) : 0;
        const long long n = in ? max(__ldg(a.fresh + b), 0) : 0;
        const long long ps = a.page_size;
        const int had = (int)min((c + ps - 1) / ps, (long long)a.max_pages);
        const int need = (int)min((c + n + ps - 1) / ps, (long long)a.max_pages) - had;
        long long chunk_rows, chunk_pages, chunk_lost = 0;
        const long long s = rows + block_sum(n, part, &chunk_rows);
        const long long f = pages + block_sum(need, part, &chunk_pages);
        if (blockIdx.x == 0) {
            // rows without a place: behind the pages this request could get, or behind slot_map
            const long long got = had + min(max(a.num_free - f, 0LL), (long long)need);
            const long long kept = min(max(min(c + n, got * ps) - c, 0LL), max(a.num_rows - s, 0LL));
            block_sum(n - kept, part, &chunk_lost);
            if (in) {
                a.seq_lens[b] = saturate(c + n);
                a.row_starts[b] = saturate(s);
            }
        }
        start[threadIdx.x] = s;
        first[threadIdx.x] = f;
        have[threadIdx.x] = (int)c;
        old[threadIdx.x] = had;
        __syncthreads();
        const int live = min(a.B - b0, kPlanThreads);
        for (long long x = pages + mine; x < pages + chunk_pages; x += step) {
            const int e = last_not_above(first, live, x);
            const long long k = old[e] + (x - first[e]);
            a.table[(size_t)(b0 + e) * a.max_pages + k] = x < a.num_free ? __ldg(a.free_pages + x) : -1;
        }
        const long long end = min(rows + chunk_rows, (long long)a.num_rows);
        for (long long r = rows + mine; r < end; r += step) {
            const int e = last_not_above(start, live, r);
            const long long pos = have[e] + (r - start[e]);
            const long long k = pos / a.page_size;
            int page = -1;
            if (k < old[e]) {
                page = a.table[(size_t)(b0 + e) * a.max_pages + k];
            } else if (k < a.max_pages) {
                const long long x = first[e] + (k - old[e]);
                if (x < a.num_free) page = __ldg(a.free_pages + x);
            }
            const long long slot = (long long)page * a.page_size + pos % a.page_size;
            a.slots[r] = page >= 0 && slot <= kI32Max ? (int)slot : -1;
        }
        rows += chunk_rows;
        pages += chunk_pages;
        lost += chunk_lost;
        __syncthreads();  // the chunk's arrays are read
    }
    for (long long r = rows + mine; r < a.num_rows; r += step) a.slots[r] = -1;
    if (mine == 0) {
        a.row_starts[a.B] = saturate(rows);
        a.stats[0] = saturate(rows);
        a.stats[1] = saturate(pages < a.num_free ? pages : a.num_free);
        a.stats[2] = saturate(lost);
    }
}

bool overlap(const void* p, int64_t np, const void* q, int64_t nq) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(p), y = reinterpret_cast<uintptr_t>(q);
    return np > 0 && nq > 0 && x < y + 4 * (uintptr_t)nq && y < x + 4 * (uintptr_t)np;
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" {

int attn_page_plan(const int* cached_lens, const int* new_lens, const int* free_pages, int* block_table, int* seq_lens,
                   int* row_starts, int* slot_map, int* stats, int B, int page_size, int max_pages, int num_free,
                   int num_rows, void* stream) {
    if (B < 0 || page_size < 1 || max_pages < 0 || num_free < 0 || num_rows < 0) return ATTN_ERR_SHAPE;
    if ((int64_t)B * max_pages > kI32Max || B > kI32Max - kPlanThreads) return ATTN_ERR_OVERFLOW;
    if (!row_starts || !stats || (B > 0 && (!cached_lens || !new_lens || !seq_lens)) ||
        ((int64_t)B * max_pages > 0 && !block_table) || (num_free > 0 && !free_pages) || (num_rows > 0 && !slot_map))
        return ATTN_ERR_NULL;
    const void* in[] = {cached_lens, new_lens, free_pages, block_table};
    void* out[] = {block_table, seq_lens, row_starts, slot_map, stats};
    const int64_t nin[] = {B, B, num_free, (int64_t)B * max_pages};
    const int64_t nout[] = {(int64_t)B * max_pages, B, (int64_t)B + 1, num_rows, 3};
    for (int i = 0; i < 4; ++i)
        if (reinterpret_cast<uintptr_t>(in[i]) & 3u) return ATTN_ERR_ALIGN;
    for (int j = 0; j < 5; ++j)
        if (reinterpret_cast<uintptr_t>(out[j]) & 3u) return ATTN_ERR_ALIGN;
    // blocks read the inputs while others write the outputs
    for (int j = 0; j < 5; ++j) {
        for (int i = 0; i < 4; ++i)
            if (!(i == 3 && j == 0) && overlap(in[i], nin[i], out[j], nout[j])) return ATTN_ERR_ALIAS;
        for (int i = 0; i < j; ++i)
            if (overlap(out[i], nout[i], out[j], nout[j])) return ATTN_ERR_ALIAS;
    }
    // one row per thread, on at most one block per SM; a step of a few hundred rows is one block
    int sms = device_sm_count();
    if (sms <= 0) sms = 148;
    int64_t grid = ((int64_t)(num_rows > B ? num_rows : B) + kPlanThreads - 1) / kPlanThreads;
    if (grid > sms) grid = sms;
    if (grid < 1) grid = 1;
    const PlanArgs a{cached_lens, new_lens, free_pages, block_table, seq_lens, row_starts, slot_map, stats,
                     B, page_size, max_pages, num_free, num_rows};
    page_plan_kernel<<<(unsigned)grid, kPlanThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // extern "C"
