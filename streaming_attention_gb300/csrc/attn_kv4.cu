// The 4-bit paged KV cache: the write of new rows into it and its read back into
// 16 bits (its format is in attn_kv4.h; the attention that reads it in
// attn_kv4_decode.cu).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attn.h"
#include "attn_internal.h"
#include "attn_kv4.h"

namespace attn {
namespace {

constexpr int64_t kI32Max = 2147483647LL;
constexpr int kThreads = 256;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
int cuda_status(cudaError_t e) { return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA; }

template <typename T>
__device__ __forceinline__ float2 to_float2(uint32_t w);
template <>
__device__ __forceinline__ float2 to_float2<__nv_bfloat16>(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float2 to_float2<__half>(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t from_float2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t from_float2<__nv_bfloat16>(float lo, float hi) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&t);
}
template <>
__device__ __forceinline__ uint32_t from_float2<__half>(float lo, float hi) {
    const __half2 t = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&t);
}

// log2 of a power of two, else -1
int shift_of(int ps) {
    int n = 0;
    while ((1 << n) < ps && n < 30) ++n;
    return (1 << n) == ps ? n : -1;
}
__device__ __forceinline__ int page_index(int x, int ps, int shift) { return shift >= 0 ? x >> shift : x / ps; }

__device__ __forceinline__ float e4m3_value(uint32_t byte) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3)));
}

// ---------------------------------------------------------------------------
// append: one thread takes 8 elements of a key row and the same 8 of the value
// row; the 4 threads of a group share its maximum. A thread takes kAppendRows such
// pieces, a block's width apart, with all their loads in flight at once: the chain
// slot -> row -> store is what a thread waits for, and with one piece a thread the
// kernel was bound by it. 16640 rows of 8 heads, D = 128, BF16 (68 MB read, 18 MB
// written): 17.8 us, 4.8 TB/s, 71 % of the measured copy bandwidth; bound by issue slots (79 % taken: per element two
// multiply-adds, a saturation and a product) and the ALU (64 % of its pipe); with
// one row a thread 19.9, with four 17.8 but 16 rows 2.2 us instead of 1.7.
// ---------------------------------------------------------------------------
constexpr int kAppendRows = 2;

struct AppendArgs {
    const void* k;
    const void* v;
    const int* slots;
    Kv4Cache c;
    long long k_stride, v_stride;  // elements from one row of the batch to the next
    int T, Hkv, ps_shift;
    float k_inv, v_inv;  // 1 / descale (a power of two)
};

// the larger one, NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
// max |x| of the 8 elements of four words, two halves at a time
template <typename T2>
__device__ __forceinline__ T2 as_pair(uint32_t w) {
    return *reinterpret_cast<const T2*>(&w);
}
template <typename T>
__device__ __forceinline__ float largest(const uint32_t (&w)[4]);
template <>
__device__ __forceinline__ float largest<__nv_bfloat16>(const uint32_t (&w)[4]) {
    using P = __nv_bfloat162;
    const P m = __hmax2_nan(__hmax2_nan(__habs2(as_pair<P>(w[0])), __habs2(as_pair<P>(w[1]))),
                        __hmax2_nan(__habs2(as_pair<P>(w[2])), __habs2(as_pair<P>(w[3]))));
    return max_nan(__low2float(m), __high2float(m));
}
template <>
__device__ __forceinline__ float largest<__half>(const uint32_t (&w)[4]) {
    using P = __half2;
    const P m = __hmax2_nan(__hmax2_nan(__habs2(as_pair<P>(w[0])), __habs2(as_pair<P>(w[1]))),
                        __hmax2_nan(__habs2(as_pair<P>(w[2])), __habs2(as_pair<P>(w[3]))));
    return max_nan(__low2float(m), __high2float(m));
}

// 8 elements -> 8 codes in one word (lowest element in the lowest bits) and the
// group's scale byte. Exact with respect to the format's definition:
//   max / 7.5 is one product and one correction by its remainder, which leaves a
//   quotient that lies on a border between two scales (5 bits) exactly there, and
//   others (the maximum has 11 bits) on their side of it.
//   x / s is x * r with r = (1 / s)(1 + 2^-16). A tie between two codes is pushed to
//   the larger magnitude (by at least 2^-17; the roundings of what follows add up to
//   less than 2^-19), and nothing else crosses a border: x has 11 significant bits
//   and s times a border 8, so a quotient that is not on a border is at least 2^-11
//   of it away.
//   The clamp to codes 0..15 is the saturation of (x / s + 8) / 15 to 0..1, which
//   comes with the multiply-add.
// inv, 1 / descale, is a power of two: x is scaled by way of r. A NaN or an infinity among
// the group's elements makes the scale NaN (the remainder of an infinite quotient is NaN).
template <typename T>
__device__ __forceinline__ uint32_t quantize8(const uint4& w, float inv, uint32_t* scale) {
    const uint32_t words[4] = {w.x, w.y, w.z, w.w};
    float top = largest<T>(words);
    top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // scales end at 448: nothing is lost here, and a large number over a small factor stays finite
    top = top < INFINITY ? fminf(top * inv, 2.0f * 7.5f * 448.0f) : top;
    const float q = top * (1.0f / 7.5f);
    const uint32_t s =
        __nv_cvt_float_to_fp8(fmaf(fmaf(-7.5f, q, top), 1.0f / 7.5f, q), __NV_SATFINITE, __NV_E4M3);
    const float sf = e4m3_value(s);
    const float r = sf > 0.f ? __fdividef((1.0f + 0x1p-16f) / 15.0f, sf) * inv : 0.f;
    // 1.5 * 2^23 + code has the code in its low bits, under bits that are always the same
    constexpr uint32_t kUnder = 0x4B400000u * 0x11111111u;
    uint32_t codes = 0;
#pragma unroll
    for (int i = 3; i >= 0; --i) {
        const float2 x = to_float2<T>(words[i]);
        codes = codes * 16 + __float_as_uint(fmaf(__saturatef(fmaf(x.y, r, 8.0f / 15.0f)), 15.0f, 12582912.0f));
        codes = codes * 16 + __float_as_uint(fmaf(__saturatef(fmaf(x.x, r, 8.0f / 15.0f)), 15.0f, 12582912.0f));
    }
    *scale = s;
    return codes - kUnder;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(AppendArgs a) {
    constexpr int NG = D / kKv4Group;
    constexpr int U = D / 8;  // threads of a row
    // launched while the kernel in front of it may still run: nothing in memory is touched before that has ended
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int u = threadIdx.x % U;
    const int i = u / 4, c = u % 4;  // group, and which 8 of its 32 elements
    // a block takes one head of consecutive rows, whose keys mostly lie side by side on a page
    const int h = (int)(blockIdx.x % a.Hkv);
    const int first = (int)(blockIdx.x / a.Hkv) * (kAppendRows * (kThreads / U)) + (int)threadIdx.x / U;
    const int ps = a.c.page_size;
    int slot[kAppendRows];
    uint4 wk[kAppendRows], wv[kAppendRows];
#pragma unroll
    for (int x = 0; x < kAppendRows; ++x) {
        const int t = first + x * (kThreads / U);
        const bool in = t < a.T;
        slot[x] = in ? load_global(a.slots + t) : -1;
        if (slot[x] >= (long long)a.c.num_pages * ps) slot[x] = -1;
        // read whether the row has a slot or not: the loads need not wait for it
        wk[x] = wv[x] = make_uint4(0, 0, 0, 0);
        if (in) {
            wk[x] = load_global(reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.k) + t * a.k_stride + h * D + u * 8));
            wv[x] = load_global(reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.v) + t * a.v_stride + h * D + u * 8));
        }
    }
#pragma unroll
    for (int x = 0; x < kAppendRows; ++x) {
        uint32_t sk, sv;
        const uint32_t ck = quantize8<T>(wk[x], a.k_inv, &sk);
        const uint32_t cv = quantize8<T>(wv[x], a.v_inv, &sv);
        // value units of 4 elements: two groups' units at one position make a word, so
        // the threads of groups i and i ^ 1 trade one unit each
        int vword = c;
        uint32_t vbits = cv;
        if (NG > 1) {
            const bool odd = i & 1;
            const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? (cv & 0xFFFFu) : (cv >> 16), 4);
            vbits = odd ? (got | (cv & 0xFFFF0000u)) : ((cv & 0xFFFFu) | (got << 16));
            vword = ((2 * c + (odd ? 1 : 0)) * NG + (i & ~1)) / 2;
        }
        if (NG == 4) {  // the row's four scales into one word, of K in its first and of V in its second thread
            uint32_t two = c == 0 ? sk : sv;
            two |= __shfl_down_sync(0xffffffffu, two, 4) << 8;
            two |= __shfl_down_sync(0xffffffffu, two, 8) << 16;
            sk = two;
        }
        if (slot[x] < 0) continue;
        const int page = page_index(slot[x], ps, a.ps_shift);
        const size_t at = ((size_t)page * a.Hkv + h) * ps + (slot[x] - page * ps);
        reinterpret_cast<uint32_t*>(a.c.k_codes + at * (D / 2))[c * NG + i] = ck;
        reinterpret_cast<uint32_t*>(a.c.v_codes + at * (D / 2))[vword] = vbits;
        if (NG == 4) {
            if (u < 2) reinterpret_cast<uint32_t*>(u == 0 ? a.c.k_scales : a.c.v_scales)[at] = sk;
        } else if (c == 0) {
            a.c.k_scales[at * NG + i] = (uint8_t)sk;
            a.c.v_scales[at * NG + i] = (uint8_t)sv;
        }
    }
}

// ---------------------------------------------------------------------------
// gather: one thread writes 8 elements of a key row and the same 8 of the value row,
// for kGatherRows rows a block's width apart, all their loads in flight at once. Bound
// by memory: 2 sequences of 32768 keys of 8 heads, D = 128 (340 MB): 54.1 us, 6.3 TB/s,
// 93 % of the measured copy bandwidth; with two or eight rows a thread 53.7 and 54.3.
// ---------------------------------------------------------------------------
constexpr int kGatherRows = 4;

struct GatherArgs {
    Kv4Cache c;
    const int* table;
    const int* lens;
    void* k;
    void* v;
    int Hkv, N, max_pages, ps_shift;
    float k_scale, v_scale;
};

// s (n - 8) of eight codes. Pairs: a byte b of the word times 0x1001 has its two nibbles at bits 0 and 16, where they
// are small whole numbers under the exponent of 128 (BF16) or 1024 (FP16); n - 8 and its product with the scale are
// exact in 16 bits (4 + 4 significant ones) where the scale times the factor is a normal number of T, which the caller
// has seen to. 5 operations a pair; in 32 bits, for other factors, 10 (54.7 us where this takes 54.1).
template <typename T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
    static constexpr uint32_t kBase = 0x43004300u;  // 128 + n
    static constexpr bool kAlways = true;           // every allowed factor is narrow
    static __device__ __forceinline__ uint32_t value(uint32_t h, uint32_t s2) {
        const __nv_bfloat162 x = __hsub2(as_pair<__nv_bfloat162>(h), __floats2bfloat162_rn(136.f, 136.f));
        const __nv_bfloat162 y = __hmul2(x, as_pair<__nv_bfloat162>(s2));
        return *reinterpret_cast<const uint32_t*>(&y);
    }
};
template <>
struct Pair<__half> {
    static constexpr uint32_t kBase = 0x64006400u;  // 1024 + n
    static constexpr bool kAlways = false;
    static __device__ __forceinline__ uint32_t value(uint32_t h, uint32_t s2) {
        const __half2 x = __hsub2(as_pair<__half2>(h), __floats2half2_rn(1032.f, 1032.f));
        const __half2 y = __hmul2(x, as_pair<__half2>(s2));
        return *reinterpret_cast<const uint32_t*>(&y);
    }
};
template <typename T, bool kNarrow>
__device__ __forceinline__ uint4 expand8(uint32_t codes, float s) {
    uint32_t w[4];
    const uint32_t s2 = from_float2<T>(s, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kNarrow) {
            const uint32_t two = __byte_perm(codes, 0, 0x4440 | i) * 0x1001u;
            w[i] = Pair<T>::value((two & 0x000F000Fu) | Pair<T>::kBase, s2);
        } else {
            const float lo = __uint_as_float(((codes >> (8 * i)) & 15u) | 0x4B000000u) - 8388616.0f;
            const float hi = __uint_as_float(((codes >> (8 * i + 4)) & 15u) | 0x4B000000u) - 8388616.0f;
            w[i] = from_float2<T>(lo * s, hi * s);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T, int D, bool kNarrow>
__global__ void __launch_bounds__(kThreads) kv4_gather_kernel(GatherArgs a) {
    constexpr int NG = D / kKv4Group;
    constexpr int U = D / 8;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int u = threadIdx.x % U;
    const int i = u / 4, c = u % 4;
    const bool odd = i & 1;
    const int h = blockIdx.y, b = blockIdx.z;
    const int first = (int)blockIdx.x * (kGatherRows * (kThreads / U)) + (int)threadIdx.x / U;
    const int ps = a.c.page_size;
    const int vword = NG > 1 ? ((2 * c + (odd ? 1 : 0)) * NG + (i & ~1)) / 2 : c;
    const int L = min(load_global(a.lens + b), a.N);
    int page[kGatherRows];
#pragma unroll
    for (int x = 0; x < kGatherRows; ++x) {
        const int j = first + x * (kThreads / U);
        const int n = page_index(j, ps, a.ps_shift);
        page[x] = j < L && n < a.max_pages ? load_global(a.table + (size_t)b * a.max_pages + n) : -1;
        if (page[x] >= a.c.num_pages) page[x] = -1;
    }
    // a row behind the sequence, or on a page outside the pool, is zeros: code 8 (code 0 would make negative ones)
    uint32_t ck[kGatherRows], cv[kGatherRows], sk[kGatherRows], sv[kGatherRows];
#pragma unroll
    for (int x = 0; x < kGatherRows; ++x) {
        ck[x] = cv[x] = 0x88888888u;
        sk[x] = sv[x] = 0;
        if (page[x] >= 0) {
            const int j = first + x * (kThreads / U);
            const size_t at = ((size_t)page[x] * a.Hkv + h) * ps + (j - page_index(j, ps, a.ps_shift) * ps);
            ck[x] = load_global(reinterpret_cast<const uint32_t*>(a.c.k_codes + at * (D / 2)) + c * NG + i);
            cv[x] = load_global(reinterpret_cast<const uint32_t*>(a.c.v_codes + at * (D / 2)) + vword);
            sk[x] = load_global(a.c.k_scales + at * NG + i);
            sv[x] = load_global(a.c.v_scales + at * NG + i);
        }
    }
#pragma unroll
    for (int x = 0; x < kGatherRows; ++x) {
        if (NG > 1) {  // the inverse of the append kernel's trade
            const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? (cv[x] & 0xFFFFu) : (cv[x] >> 16), 4);
            cv[x] = odd ? (got | (cv[x] & 0xFFFF0000u)) : ((cv[x] & 0xFFFFu) | (got << 16));
        }
        const int j = first + x * (kThreads / U);
        if (j >= a.N) continue;
        const size_t out = (((size_t)b * a.Hkv + h) * a.N + j) * U + u;
        reinterpret_cast<uint4*>(a.k)[out] = expand8<T, kNarrow>(ck[x], e4m3_value(sk[x]) * a.k_scale);
        reinterpret_cast<uint4*>(a.v)[out] = expand8<T, kNarrow>(cv[x], e4m3_value(sv[x]) * a.v_scale);
    }
}

template <typename T>
cudaError_t launch_append(const AppendArgs& a, int D, cudaStream_t s) {
    const int per = kAppendRows * (kThreads / (D / 8));
    const dim3 grid((unsigned)(((long long)a.T + per - 1) / per * a.Hkv));
    switch (D) {
        case 32: return launch_programmatic(kv4_append_kernel<T, 32>, grid, kThreads, s, a);
        case 64: return launch_programmatic(kv4_append_kernel<T, 64>, grid, kThreads, s, a);
        default: return launch_programmatic(kv4_append_kernel<T, 128>, grid, kThreads, s, a);
    }
}

template <typename T, int D>
cudaError_t launch_gather_d(const GatherArgs& a, dim3 grid, bool narrow, cudaStream_t s) {
    if constexpr (!Pair<T>::kAlways)
        if (!narrow) return launch_programmatic(kv4_gather_kernel<T, D, false>, grid, kThreads, s, a);
    return launch_programmatic(kv4_gather_kernel<T, D, true>, grid, kThreads, s, a);
}

// Whether every scale (2^-9 .. 448) times the factor is a normal FP16 number. In BF16 all are.
bool narrow_factor(float f) { return f >= 0x1p-5f && f <= 0x1p7f; }

template <typename T>
cudaError_t launch_gather(const GatherArgs& a, int B, int D, cudaStream_t s) {
    const int per = kGatherRows * (kThreads / (D / 8));
    const dim3 grid((unsigned)(((long long)a.N + per - 1) / per), (unsigned)a.Hkv, (unsigned)B);
    const bool narrow = narrow_factor(a.k_scale) && narrow_factor(a.v_scale);
    switch (D) {
        case 32: return launch_gather_d<T, 32>(a, grid, narrow, s);
        case 64: return launch_gather_d<T, 64>(a, grid, narrow, s);
        default: return launch_gather_d<T, 128>(a, grid, narrow, s);
    }
}

}  // namespace

// The pools hold 64-bit many bytes; their slots are numbered in 32 bits.
int kv4_validate_cache(const Kv4Cache& c, int Hkv, int D) {
    if (c.num_pages < 0 || Hkv < 0 || D <= 0) return ATTN_ERR_SHAPE;
    if (!kv4_page_size(c.page_size)) return ATTN_ERR_SHAPE;
    if (!kv4_head_dim(D)) return ATTN_ERR_HEADDIM;
    if ((int64_t)c.num_pages * c.page_size > kI32Max) return ATTN_ERR_OVERFLOW;
    if (c.num_pages > 0 && Hkv > 0 && (!c.k_codes || !c.k_scales || !c.v_codes || !c.v_scales)) return ATTN_ERR_NULL;
    if (!aligned(c.k_codes, 16) || !aligned(c.k_scales, 16) || !aligned(c.v_codes, 16) || !aligned(c.v_scales, 16))
        return ATTN_ERR_ALIGN;
    return ATTN_OK;
}

}  // namespace attn

using namespace attn;

extern "C" {

int attn_kv4_append(const void* k, const void* v, const int* slot_map, void* k_codes, void* k_scales, void* v_codes,
                    void* v_scales, int T, int Hkv, int D, long long k_stride, long long v_stride, int num_pages,
                    int page_size, float k_descale, float v_descale, attn_dtype_t dtype, void* stream) {
    if (dtype != ATTN_BF16 && dtype != ATTN_FP16) return ATTN_ERR_DTYPE;
    if (T < 0) return ATTN_ERR_SHAPE;
    const Kv4Cache c{static_cast<uint8_t*>(k_codes), static_cast<uint8_t*>(k_scales), static_cast<uint8_t*>(v_codes),
                     static_cast<uint8_t*>(v_scales), num_pages, page_size};
    const int rc = kv4_validate_cache(c, Hkv, D);
    if (rc != ATTN_OK) return rc;
    const int64_t row = (int64_t)Hkv * D;
    if (elements({T, Hkv, D}) > kI32Max) return ATTN_ERR_OVERFLOW;
    if (T > 1 && (k_stride < row || v_stride < row)) return ATTN_ERR_SHAPE;
    if (!kv4_descale(k_descale) || !kv4_descale(v_descale)) return ATTN_ERR_SCALE;
    if (T == 0 || Hkv == 0 || num_pages == 0) return ATTN_OK;
    if (!k || !v || !slot_map) return ATTN_ERR_NULL;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slot_map, 4) || (T > 1 && (k_stride % 8 || v_stride % 8)))
        return ATTN_ERR_ALIGN;
    const AppendArgs a{k, v, slot_map, c, k_stride, v_stride, T, Hkv, shift_of(page_size), 1.0f / k_descale, 1.0f / v_descale};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(dtype == ATTN_BF16 ? launch_append<__nv_bfloat16>(a, D, s) : launch_append<__half>(a, D, s));
}

int attn_kv4_gather(const void* k_codes, const void* k_scales, const void* v_codes, const void* v_scales,
                    const int* block_table, const int* seq_lens, void* k, void* v, int B, int Hkv, int N, int D,
                    int num_pages, int page_size, int max_pages, float k_descale, float v_descale, attn_dtype_t dtype,
                    void* stream) {
    if (dtype != ATTN_BF16 && dtype != ATTN_FP16) return ATTN_ERR_DTYPE;
    if (B < 0 || N < 0 || max_pages < 0) return ATTN_ERR_SHAPE;
    const auto mut = [](const void* p) { return static_cast<uint8_t*>(const_cast<void*>(p)); };
    const Kv4Cache c{mut(k_codes), mut(k_scales), mut(v_codes), mut(v_scales), num_pages, page_size};
    const int rc = kv4_validate_cache(c, Hkv, D);
    if (rc != ATTN_OK) return rc;
    // the grid holds a KV head per y and a sequence per z index
    if (elements({B, Hkv, N, D}) > kI32Max || elements({B, max_pages}) > kI32Max || B > 65535 || Hkv > 65535)
        return ATTN_ERR_OVERFLOW;
    if (!kv4_descale(k_descale) || !kv4_descale(v_descale)) return ATTN_ERR_SCALE;
    if (elements({B, Hkv, N}) == 0) return ATTN_OK;
    if (!k || !v || !seq_lens || (max_pages > 0 && !block_table)) return ATTN_ERR_NULL;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(seq_lens, 4) || !aligned(block_table, 4)) return ATTN_ERR_ALIGN;
    const GatherArgs a{c, block_table, seq_lens, k, v, Hkv, N, max_pages, shift_of(page_size), k_descale, v_descale};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(dtype == ATTN_BF16 ? launch_gather<__nv_bfloat16>(a, B, D, s)
                                          : launch_gather<__half>(a, B, D, s));
}

}  // extern "C"
