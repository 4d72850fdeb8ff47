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
// one request per thread at a time, and takes its share of the chunk's rows and
// pages, whose request it finds by bisection in shared memory. No block reads a
// table entry that another one writes: entries below old_b are only read, the
// others only written (their page is computed from the free list instead).
// Latency bounds it: loads, sums, bisection, loads, stores.
#include <cuda_runtime.h>
#include <stdint.h>

#include "attn.h"
#include "attn_internal.h"

namespace attn {
namespace {

constexpr int kPlanMost = 1024;  // threads of a block, and requests of a chunk
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

template <int N>
__global__ void __launch_bounds__(N) page_plan_kernel(const PlanArgs a) {
    __shared__ long long start[N], first[N];
    __shared__ longlong2 part[N / 32];
    __shared__ int have[N], old[N];
    const long long mine = (long long)blockIdx.x * N + threadIdx.x;
    const long long step = (long long)gridDim.x * N;
    long long rows = 0, pages = 0;  // of the requests before this chunk
    long long lost = 0;             // rows without a place of this thread's requests
    int c32 = (int)threadIdx.x < a.B ? __ldg(a.cached + threadIdx.x) : 0;
    int n32 = (int)threadIdx.x < a.B ? __ldg(a.fresh + threadIdx.x) : 0;
    for (int b0 = 0; b0 < a.B; b0 += N) {
        const int b = b0 + threadIdx.x;
        const long long c = max(c32, 0), n = max(n32, 0), ps = a.page_size;
        if (b0 + N < a.B) {  // the next chunk's lengths are on their way while this one is worked on
            c32 = b + N < a.B ? __ldg(a.cached + b + N) : 0;
            n32 = b + N < a.B ? __ldg(a.fresh + b + N) : 0;
        }
        const int had = (int)min((c + ps - 1) / ps, (long long)a.max_pages);
        const int need = (int)min((c + n + ps - 1) / ps, (long long)a.max_pages) - had;
        long long s = n, f = need, chunk_rows, chunk_pages;
        block_sums<N>(s, f, part, &chunk_rows, &chunk_pages);
        s += rows;
        f += pages;
        start[threadIdx.x] = s;
        first[threadIdx.x] = f;
        have[threadIdx.x] = (int)c;
        old[threadIdx.x] = had;
        if (blockIdx.x == 0 && b < a.B) {
            a.seq_lens[b] = saturate(c + n);
            a.row_starts[b] = saturate(s);
            // kept: the rows on pages that this request could get, and not behind slot_map
            const long long got = had + min(max(a.num_free - f, 0LL), (long long)need);
            lost += n - min(max(min(c + n, got * ps) - c, 0LL), max(a.num_rows - s, 0LL));
        }
        __syncthreads();
        const int live = min(a.B - b0, N);
        for (long long x = pages + mine; x < pages + chunk_pages; x += step) {
            const int e = last_not_above(first, live, x);
            const long long k = old[e] + (x - first[e]);
            a.table[(size_t)(b0 + e) * a.max_pages + k] = x < a.num_free ? __ldg(a.free_pages + x) : -1;
        }
        const long long end = min(rows + chunk_rows, (long long)a.num_rows);
        for (long long r = rows + mine; r < end; r += step) {
            const int e = last_not_above(start, live, r);
            const long long pos = have[e] + (r - start[e]);
            // positions pass 32 bits only where no page is left
            const int k = pos <= kI32Max ? (int)((uint32_t)pos / (uint32_t)a.page_size) : a.max_pages;
            int page = -1;
            if (k < old[e]) {
                page = a.table[(size_t)(b0 + e) * a.max_pages + k];
            } else if (k < a.max_pages) {
                const long long x = first[e] + (k - old[e]);
                if (x < a.num_free) page = __ldg(a.free_pages + x);
            }
            const long long slot = (long long)page * a.page_size + ((uint32_t)pos - (uint32_t)k * (uint32_t)a.page_size);
            a.slots[r] = page >= 0 && slot <= kI32Max ? (int)slot : -1;
        }
        rows += chunk_rows;
        pages += chunk_pages;
        __syncthreads();  // the chunk's arrays are read
    }
    for (long long r = rows + mine; r < a.num_rows; r += step) a.slots[r] = -1;
    if (blockIdx.x != 0) return;
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
                     B, page_size, max_pages, num_free, num_rows};
    // one row per thread, on at most one block per SM. Few requests take smaller blocks, whose sums are quicker (64
    // requests); many take larger ones, and so fewer chunks one after the other (2000).
    int sms = device_sm_count();
    if (sms <= 0) sms = 148;
    const int threads = B <= 256 ? 256 : kPlanMost;
    int64_t grid = ((int64_t)(num_rows > B ? num_rows : B) + threads - 1) / threads;
    if (grid > sms) grid = sms;
    if (grid < 1) grid = 1;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (threads == 256)
        page_plan_kernel<256><<<(unsigned)grid, 256, 0, s>>>(a);
    else
        page_plan_kernel<kPlanMost><<<(unsigned)grid, kPlanMost, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // extern "C"
