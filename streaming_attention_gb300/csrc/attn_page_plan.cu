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
// one or two requests per thread at a time, and takes its share of the chunk's rows and
// pages, whose request it finds by bisection in shared memory. No block reads a
// table entry that another one writes: entries below old_b are only read, the
// others only written (their page is computed from the free list instead). One more block
// writes what there is per request and counts the rows without a slot: per request those
// behind the pages it gets and behind slot_map, and those on the page its cached keys end in,
// if that is none; per page taken, those on a page that is none.
// Latency bounds it: loads, sums, bisection, loads, stores. 64 requests of one new key
// take 2.7 us, 2000 of 97 new keys each 6.5.
#include <cuda_runtime.h>
#include <stdint.h>

#include "attn.h"
#include "attn_internal.h"
#include "attn_kv4.h"

namespace attn {
namespace {

constexpr int kPlanMost = 2048;  // requests of a chunk, at most
constexpr int kPlanLoads = 16;   // entries of the free list that a counting thread has in flight
constexpr long long kI32Max = 2147483647LL;

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
    uint32_t last_page;  // all slots of the pages 0 .. last_page fit 32 bits
};

__device__ __forceinline__ int saturate(long long x) { return (int)(x < kI32Max ? x : kI32Max); }

// Exclusive sums over the block of x and y, and their totals. `part` holds a pair per warp.
template <int N>
__device__ __forceinline__ void block_sums(long long& x, long long& y, longlong2* part, long long* all_x,
                                           long long* all_y) {
    constexpr int kWarps = N / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long sx = x, sy = y;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long tx = __shfl_up_sync(0xffffffffu, sx, d), ty = __shfl_up_sync(0xffffffffu, sy, d);
        if (lane >= d) {
            sx += tx;
            sy += ty;
        }
    }
    if (lane == 31) part[warp] = make_longlong2(sx, sy);
    __syncthreads();
    // every warp sums the warps' totals for itself
    longlong2 w = lane < kWarps ? part[lane] : make_longlong2(0, 0);
#pragma unroll
    for (int d = 1; d < kWarps; d <<= 1) {
        const long long tx = __shfl_up_sync(0xffffffffu, w.x, d), ty = __shfl_up_sync(0xffffffffu, w.y, d);
        if (lane >= d) {
            w.x += tx;
            w.y += ty;
        }
    }
    *all_x = __shfl_sync(0xffffffffu, w.x, kWarps - 1);
    *all_y = __shfl_sync(0xffffffffu, w.y, kWarps - 1);
    const long long bx = __shfl_sync(0xffffffffu, w.x, (warp + 31) & 31), by = __shfl_sync(0xffffffffu, w.y, (warp + 31) & 31);
    x = sx - x + (warp > 0 ? bx : 0);
    y = sy - y + (warp > 0 ? by : 0);
}

// The last entry e of the ascending a[0..n) with a[e] <= x; a[0] <= x.
__device__ __forceinline__ int last_not_above(const int* a, int n, int x) {
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

// Pages of x keys, x below 2^32, at most `most`.
__device__ __forceinline__ int pages_of(uint32_t x, uint32_t page_size, int most) {
    const uint32_t n = x / page_size + (x % page_size != 0);
    return (int)min(n, (uint32_t)most);
}

// How many of `rows` keys from offset `off` on of a page have no slot: all if it is no page (below 0), else those whose
// slot passes 2^31 - 1.
__device__ __forceinline__ long long without_slot(int page, int page_size, long long off, long long rows) {
    const long long past = (long long)page * page_size + off + rows - 1 - kI32Max;
    return max(page < 0 ? rows : min(past, rows), 0LL);
}

// N threads, K requests of a chunk to a thread.
template <int N, int K>
__global__ void __launch_bounds__(N) page_plan_kernel(PlanArgs a) {
    // a request's first row of the batch and first page of the free list (2^31 - 1 for all behind that), its keys in
    // the cache and its pages
    __shared__ int start[N * K], first[N * K], have[N * K], old[N * K];
    __shared__ longlong2 part[N / 32];
    // launched while the kernel in front of it may still run: nothing in memory is touched before that has ended
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // the last block writes what there is per request and the counts, the others share the pages and rows
    const bool counts = blockIdx.x == gridDim.x - 1;
    const long long mine = (long long)blockIdx.x * N + threadIdx.x;
    const long long step = (long long)(gridDim.x - 1) * N;
    long long rows = 0, pages = 0;  // of the requests before this chunk
    long long lost = 0;             // rows without a place of this thread's requests
    for (int b0 = 0; b0 < a.B; b0 += N * K) {
        const int b = b0 + (int)threadIdx.x * K;
        uint32_t c[K], n[K];
        int had[K], need[K];
        int begun[K];  // the table's entry for the page that the request's first new key goes to, if it has one already
        long long s = 0, f = 0;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            c[k] = b + k < a.B ? (uint32_t)max(load_global(a.cached + b + k), 0) : 0;
            n[k] = b + k < a.B ? (uint32_t)max(load_global(a.fresh + b + k), 0) : 0;
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            had[k] = pages_of(c[k], a.page_size, a.max_pages);
            need[k] = pages_of(c[k] + n[k], a.page_size, a.max_pages) - had[k];
            const uint32_t at = c[k] / (uint32_t)a.page_size;
            begun[k] = counts && n[k] > 0 && at < (uint32_t)had[k]
                           ? load_global(a.table + (size_t)(b + k) * a.max_pages + at)
                           : 0;
            s += n[k];
            f += need[k];
        }
        long long chunk_rows, chunk_pages;
        block_sums<N>(s, f, part, &chunk_rows, &chunk_pages);
        s += rows;
        f += pages;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int e = (int)threadIdx.x * K + k;
            start[e] = saturate(s);
            first[e] = saturate(f);
            have[e] = (int)c[k];
            old[e] = had[k];
            if (counts && b + k < a.B) {
                const long long len = (long long)c[k] + n[k];
                a.seq_lens[b + k] = saturate(len);
                a.row_starts[b + k] = saturate(s);
                // kept: the rows on pages that this request could get, and not behind slot_map
                const long long got = had[k] + min(max(a.num_free - f, 0LL), (long long)need[k]);
                const long long kept =
                    min(max(min(len, got * a.page_size) - c[k], 0LL), max(a.num_rows - s, 0LL));
                const long long off = c[k] % (uint32_t)a.page_size;
                lost += n[k] - kept + without_slot(begun[k], a.page_size, off, min(kept, a.page_size - off));
            }
            s += n[k];
            f += need[k];
        }
        __syncthreads();
        const int live = min(a.B - b0, N * K);
        const long long page_end = min(pages + chunk_pages, kI32Max);
        const long long row_end = min(rows + chunk_rows, (long long)a.num_rows);
        if (counts) {
            // rows on entries of the free list that are no pages
            const long long listed = min(page_end, (long long)a.num_free);
            for (long long x0 = pages + threadIdx.x; x0 < listed; x0 += kPlanLoads * N) {
                int page[kPlanLoads];
                bool none = false;
#pragma unroll
                for (int i = 0; i < kPlanLoads; ++i) {
                    page[i] = x0 + i * N < listed ? load_global(a.free_pages + x0 + i * N) : 0;
                    none |= (uint32_t)page[i] > a.last_page;
                }
                if (!none) continue;
#pragma unroll
                for (int i = 0; i < kPlanLoads; ++i) {
                    if ((uint32_t)page[i] <= a.last_page) continue;
                    const int x = (int)(x0 + i * N);
                    const int e = last_not_above(first, live, x);
                    const long long next = e + 1 < live ? start[e + 1] : min(rows + chunk_rows, kI32Max);
                    const long long r =
                        start[e] + ((long long)(old[e] + (x - first[e])) * a.page_size - (uint32_t)have[e]);
                    const long long on = min(min(next, (long long)a.num_rows) - r, (long long)a.page_size);
                    lost += without_slot(page[i], a.page_size, 0, max(on, 0LL));
                }
            }
        } else {
            for (long long x = pages + mine; x < page_end; x += step) {
                const int e = last_not_above(first, live, (int)x);
                const int k = old[e] + ((int)x - first[e]);
                a.table[(size_t)(b0 + e) * a.max_pages + k] = x < a.num_free ? load_global(a.free_pages + x) : -1;
            }
            for (long long r = rows + mine; r < row_end; r += step) {
                const int e = last_not_above(start, live, (int)r);
                const uint32_t pos = (uint32_t)have[e] + (uint32_t)((int)r - start[e]);
                const uint32_t k = pos / (uint32_t)a.page_size;
                int page = -1;
                if (k < (uint32_t)old[e]) {
                    page = a.table[(size_t)(b0 + e) * a.max_pages + k];
                } else if (k < (uint32_t)a.max_pages) {
                    const long long x = (long long)first[e] + (k - (uint32_t)old[e]);
                    if (x < a.num_free) page = load_global(a.free_pages + x);
                }
                const long long slot = (long long)page * a.page_size + (pos - k * (uint32_t)a.page_size);
                a.slots[r] = page >= 0 && slot <= kI32Max ? (int)slot : -1;
            }
        }
        rows += chunk_rows;
        pages += chunk_pages;
        __syncthreads();  // the chunk's arrays are read
    }
    if (!counts) {
        for (long long r = rows + mine; r < a.num_rows; r += step) a.slots[r] = -1;
        return;
    }
    long long none = 0, all, all_none;
    block_sums<N>(lost, none, part, &all, &all_none);
    if (threadIdx.x == 0) {
        a.row_starts[a.B] = saturate(rows);
        a.stats[0] = saturate(rows);
        a.stats[1] = saturate(pages < a.num_free ? pages : a.num_free);
        a.stats[2] = saturate(all);
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
    if ((int64_t)B * max_pages > kI32Max || B > kI32Max - kPlanMost) return ATTN_ERR_OVERFLOW;
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
    const PlanArgs a{cached_lens, new_lens, free_pages, block_table, seq_lens, row_starts, slot_map, stats,
                     B, page_size, max_pages, num_free, num_rows, (uint32_t)((kI32Max - (page_size - 1)) / page_size)};
    // one row per thread, on at most one block per SM, and the block that counts. Few requests take smaller blocks, whose
    // sums are quicker; many take larger ones, and so fewer chunks one after the other: 64 requests 2.7 us in blocks of 256
    // threads and 4.2 in blocks of 1024, 256 3.0 and 4.4, 512 (two chunks) 4.8 and 4.8, 513 5.9 and 4.8, 2000 of 97 new
    // keys each 16.8 and 6.5.
    int sms = device_sm_count();
    if (sms <= 0) sms = 148;
    const int threads = B <= 512 ? 256 : 1024;
    int64_t grid = ((int64_t)(num_rows > B ? num_rows : B) + threads - 1) / threads;
    if (grid > sms - 1) grid = sms - 1;
    if (grid < 1) grid = 1;
    ++grid;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const dim3 g((unsigned)grid);
    const cudaError_t e = threads == 256
                              ? launch_programmatic(page_plan_kernel<256, 1>, g, threads, s, a)
                              : launch_programmatic(page_plan_kernel<1024, kPlanMost / 1024>, g, threads, s, a);
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // extern "C"
