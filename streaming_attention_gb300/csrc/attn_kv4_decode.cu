// Decode attention over the 4-bit paged KV cache (format: attn_kv4.h).
//
// One block owns one split of a sequence's visible key tiles for one KV head and
// up to 8 * NT of its grouped query rows (query head h = g * G + r / M, row
// i = r % M); its four warps take 16 keys each of a 64-key tile and keep their own
// running (m, l, acc) per row, joined at the end by the common-maximum rule.
//
// A warp's products run transposed, on m16n8k16 matrix instructions with the
// cache as the left operand, so that a row of the cache is expanded once for all
// the query rows: S^T = K Q^T (16 keys by 8 rows) and O^T += V^T P^T (16 elements
// by 8 rows). Codes become FP16 in registers: a nibble in bits 4..7 of a half with
// exponent 0x54 is 64 + n, and one fused multiply-add with s and -72 s gives
// s (n - 8), exact in FP16 (s has 4 significant bits, n - 8 has 4).
// Rounded below 32 bits: Q to FP16 after scaling each row by a power of two to
// maximum 1..2 (exact for elements above 2^-14 of the maximum), and the
// probabilities to FP16, kept 64 times too large to stay clear of its small
// numbers; the row sum adds them unrounded.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attn.h"
#include "attn_internal.h"
#include "attn_kv4.h"
#include "sm100_ptx.cuh"

namespace attn {
namespace {

constexpr int kWarps = 4;
constexpr int kTile = 16 * kWarps;  // keys of a tile, 16 per warp
constexpr float kPShift = 6.0f;     // probabilities are kept times 2^6

struct DecodeArgs {
    const void* q;
    Kv4Cache c;
    const int* table;
    const int* lens;
    void* o;
    float *ws_m, *ws_l, *ws_acc;
    int Hq, Hkv, M, G;
    int max_pages, max_len;
    int causal, window, sinks;
    float scale_log2;  // logit scale and K factor, times log2(e)
    float v_scale;
    int per_split, S;  // tiles of a split, splits
};

template <int N>
struct Bytes;
template <>
struct Bytes<16> {
    using T = uint4;
};
template <>
struct Bytes<8> {
    using T = uint2;
};
template <>
struct Bytes<4> {
    using T = uint32_t;
};
template <>
struct Bytes<2> {
    using T = uint16_t;
};
template <>
struct Bytes<1> {
    using T = uint8_t;
};

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// transposes an 8 x 8 matrix of halves held by the warp (two per lane)
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// two E4M3 bytes -> two halves
__device__ __forceinline__ uint32_t e4m3x2(uint32_t two) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xFFFFu), __NV_E4M3);
    return (uint32_t)h.x | ((uint32_t)h.y << 16);
}
constexpr uint32_t kMinus72 = 0xD480D480u;  // -72 in both halves

// nibble x of each half of w, as s (n - 8): s and ns = -72 s per half
template <int x>
__device__ __forceinline__ uint32_t expand(uint32_t w, uint32_t s, uint32_t ns) {
    const uint32_t sh = x == 0 ? w << 4 : x == 1 ? w : x == 2 ? w >> 4 : w >> 8;
    return hfma2((sh & 0x00F000F0u) | 0x54005400u, s, ns);
}

template <typename T>
__device__ __forceinline__ float lo_of(uint32_t w);
template <>
__device__ __forceinline__ float lo_of<__nv_bfloat16>(uint32_t w) {
    return __uint_as_float(w << 16);
}
template <>
__device__ __forceinline__ float lo_of<__half>(uint32_t w) {
    return __half2float(__ushort_as_half((unsigned short)(w & 0xFFFFu)));
}
template <typename T>
__device__ __forceinline__ void put(void* o, size_t i, float x);
template <>
__device__ __forceinline__ void put<__nv_bfloat16>(void* o, size_t i, float x) {
    reinterpret_cast<__nv_bfloat16*>(o)[i] = __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ void put<__half>(void* o, size_t i, float x) {
    reinterpret_cast<__half*>(o)[i] = __float2half_rn(x);
}

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kWarps * 32) kv4_decode_kernel(const DecodeArgs a) {
    constexpr int NG = D / kKv4Group;
    constexpr int ROWS = 8 * NT;
    using KChunk = typename Bytes<4 * NG>::T;
    using VChunk = typename Bytes<2 * NG>::T;
    using Scales = typename Bytes<NG>::T;
    __shared__ float sm_m[kWarps][ROWS], sm_l[kWarps][ROWS];
    __shared__ float sm_acc[kWarps][ROWS][D];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gq = lane >> 2, cq = lane & 3;  // the lane's place in a matrix fragment
    const int split = blockIdx.x;
    const int b = blockIdx.y / a.Hkv, g = blockIdx.y % a.Hkv;
    const int R = a.G * a.M, r0 = blockIdx.z * ROWS;
    const int ps = a.c.page_size;

    // keys of this sequence and the tiles any of its rows may see: those of the
    // first `sinks` keys, then those of the window's union
    const int L = min(max(__ldg(a.lens + b), 0), a.max_len);
    int lo0, hi0, lo1, hi1;
    key_range(L - a.M, L, a.causal, a.window, &lo0, &hi0);
    key_range(L - 1, L, a.causal, a.window, &lo1, &hi1);
    const int t_end = hi1 / kTile + (hi1 % kTile != 0);
    const int t_win = min(lo0 / kTile, t_end);
    const int n_sink = min(min(a.sinks / kTile + (a.sinks % kTile != 0), t_win), t_end);
    const int tiles = n_sink + t_end - t_win;
    const int first = split * a.per_split, last = min(first + a.per_split, tiles);

    // Q^T fragments, each row scaled to maximum 1..2, and the visible range of the lane's own rows
    uint32_t qf[NT][NG][2][2];
    float sc[NT][2];
    int vis_lo[NT][2], vis_hi[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = r0 + nt * 8 + gq;
        float x[NG][8], top = 0.f;
        const bool row = r < R;
        const int h = g * a.G + (row ? r / a.M : 0), i = row ? r % a.M : 0;
        const uint32_t* qrow =
            reinterpret_cast<const uint32_t*>(a.q) + (((size_t)b * a.Hq + h) * a.M + i) * (D / 2) + cq * 4;
#pragma unroll
        for (int n = 0; n < NG; ++n) {
            const uint4 w = row ? __ldg(reinterpret_cast<const uint4*>(qrow + n * 16)) : make_uint4(0, 0, 0, 0);
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[n][2 * e] = lo_of<T>(ww[e]);
                x[n][2 * e + 1] = lo_of<T>(ww[e] >> 16);
                top = fmaxf(top, fmaxf(fabsf(x[n][2 * e]), fabsf(x[n][2 * e + 1])));
            }
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // biased exponent of the row's maximum, kept where 2^e and 2^-e are both normal
        int e = (int)(__float_as_uint(top) >> 23);
        e = top == 0.f ? 127 : min(max(e, 1), 253);
        const float down = __uint_as_float((uint32_t)(254 - e) << 23);
        const float up = __uint_as_float((uint32_t)e << 23) * a.scale_log2;
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    qf[nt][n][s][t] = ptx::pack_f16(x[n][2 * s + t] * down, x[n][4 + 2 * s + t] * down);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            sc[nt][t] = __shfl_sync(0xffffffffu, up, (2 * cq + t) * 4);
            const int rt = r0 + nt * 8 + 2 * cq + t;
            int p = rt < R ? rt % a.M + L - a.M : L - 1;
            key_range(p, L, a.causal, a.window, &vis_lo[nt][t], &vis_hi[nt][t]);
        }
    }

    float m[NT][2], l[NT][2], acc[NT][2 * NG][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            m[nt][t] = -INFINITY;
            l[nt][t] = 0.f;
        }
#pragma unroll
        for (int n = 0; n < 2 * NG; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[nt][n][e] = 0.f;
    }

    const int* trow = a.table + (size_t)b * a.max_pages;
    for (int tile = first; tile < last; ++tile) {
        const int j0 = (tile < n_sink ? tile : tile - n_sink + t_win) * kTile + warp * 16;
        if (j0 >= L) continue;
        const int page = __ldg(trow + j0 / ps);
        const bool held = page >= 0 && page < a.c.num_pages;  // a page outside the pool reads as zeros
        const size_t at = ((size_t)(held ? page : 0) * a.Hkv + g) * ps + j0 % ps;

        // ---- S^T = K Q^T ----
        float s[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
        if (held) {
            union {
                KChunk v;
                uint32_t w[NG];
            } k0, k1;
            k0.v = __ldg(reinterpret_cast<const KChunk*>(a.c.k_codes + (at + gq) * (D / 2)) + cq);
            k1.v = __ldg(reinterpret_cast<const KChunk*>(a.c.k_codes + (at + gq + 8) * (D / 2)) + cq);
            const uint32_t s0 = __ldg(reinterpret_cast<const Scales*>(a.c.k_scales + (at + gq) * NG));
            const uint32_t s1 = __ldg(reinterpret_cast<const Scales*>(a.c.k_scales + (at + gq + 8) * NG));
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                // the scale in both halves
                const uint32_t f0 = e4m3x2(((s0 >> (8 * n)) & 0xFFu) * 0x0101u);
                const uint32_t f1 = e4m3x2(((s1 >> (8 * n)) & 0xFFu) * 0x0101u);
                const uint32_t n0 = hmul2(f0, kMinus72), n1 = hmul2(f1, kMinus72);
                const uint32_t x0[4] = {expand<0>(k0.w[n], f0, n0), expand<0>(k1.w[n], f1, n1),
                                        expand<1>(k0.w[n], f0, n0), expand<1>(k1.w[n], f1, n1)};
                const uint32_t x1[4] = {expand<2>(k0.w[n], f0, n0), expand<2>(k1.w[n], f1, n1),
                                        expand<3>(k0.w[n], f0, n0), expand<3>(k1.w[n], f1, n1)};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma_16816(s[nt], x0, qf[nt][n][0][0], qf[nt][n][0][1]);
                    mma_16816(s[nt], x1, qf[nt][n][1][0], qf[nt][n][1][1]);
                }
            }
        }

        // ---- softmax: s[0..1] is key gq of rows 2 cq, 2 cq + 1; s[2..3] key gq + 8 ----
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float p[4];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                float x[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int j = j0 + gq + 8 * e;
                    const bool see = j < vis_hi[nt][t] && (j >= vis_lo[nt][t] || j < a.sinks);
                    x[e] = see ? s[nt][2 * e + t] * sc[nt][t] : -INFINITY;  // a masked key scores -inf
                }
                float mx = fmaxf(m[nt][t], fmaxf(x[0], x[1]));
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                // ghost-row pin: while every key so far is masked, 0 stands for the maximum
                const float use = mx == -INFINITY ? 0.f : mx;
                const float alpha = ptx::ex2(m[nt][t] - use);
                m[nt][t] = mx;
                p[t] = ptx::ex2(x[0] - use + kPShift);
                p[2 + t] = ptx::ex2(x[1] - use + kPShift);
                l[nt][t] = l[nt][t] * alpha + p[t] + p[2 + t];
#pragma unroll
                for (int n = 0; n < 2 * NG; ++n) {
                    acc[nt][n][t] *= alpha;
                    acc[nt][n][2 + t] *= alpha;
                }
            }
            pb[nt][0] = transpose8(ptx::pack_f16(p[0], p[1]));
            pb[nt][1] = transpose8(ptx::pack_f16(p[2], p[3]));
        }

        // ---- O^T += V^T P^T ----
        if (held) {
            union VWords {
                VChunk v;
                uint32_t w[(NG + 1) / 2];
            } v[4];
            uint32_t vs[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int k = 2 * cq + (e & 1) + 8 * (e >> 1);
                v[e].w[0] = 0;
                v[e].v = __ldg(reinterpret_cast<const VChunk*>(a.c.v_codes + (at + k) * (D / 2)) + gq);
                vs[e] = __ldg(reinterpret_cast<const Scales*>(a.c.v_scales + (at + k) * NG));
                if (j0 + k >= L) vs[e] = 0;  // whatever stands behind the sequence counts as zero
            }
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                const uint32_t pick = n & 1 ? 0x7632u : 0x5410u, byte = (uint32_t)(n | ((4 + n) << 4));
                const uint32_t u0 = __byte_perm(v[0].w[n / 2], v[1].w[n / 2], pick);
                const uint32_t u1 = __byte_perm(v[2].w[n / 2], v[3].w[n / 2], pick);
                const uint32_t f0 = e4m3x2(__byte_perm(vs[0], vs[1], byte));
                const uint32_t f1 = e4m3x2(__byte_perm(vs[2], vs[3], byte));
                const uint32_t n0 = hmul2(f0, kMinus72), n1 = hmul2(f1, kMinus72);
                const uint32_t x0[4] = {expand<0>(u0, f0, n0), expand<1>(u0, f0, n0), expand<0>(u1, f1, n1),
                                        expand<1>(u1, f1, n1)};
                const uint32_t x1[4] = {expand<2>(u0, f0, n0), expand<3>(u0, f0, n0), expand<2>(u1, f1, n1),
                                        expand<3>(u1, f1, n1)};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma_16816(acc[nt][2 * n], x0, pb[nt][0], pb[nt][1]);
                    mma_16816(acc[nt][2 * n + 1], x1, pb[nt][0], pb[nt][1]);
                }
            }
        }
    }

    // ---- join the warps ----
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) l[nt][t] += __shfl_xor_sync(0xffffffffu, l[nt][t], d);
            const int r = nt * 8 + 2 * cq + t;
            if (gq == 0) {
                sm_m[warp][r] = m[nt][t];
                sm_l[warp][r] = l[nt][t];
            }
            // element 32 n + 4 gq + x: accumulator 2 n + x / 2, its row gq (x even) or gq + 8
#pragma unroll
            for (int n = 0; n < NG; ++n)
                *reinterpret_cast<float4*>(&sm_acc[warp][r][32 * n + 4 * gq]) =
                    make_float4(acc[nt][2 * n][t], acc[nt][2 * n][2 + t], acc[nt][2 * n + 1][t],
                                acc[nt][2 * n + 1][2 + t]);
        }
    }
    __syncthreads();
    for (int x = threadIdx.x; x < ROWS * D; x += kWarps * 32) {
        const int r = x / D, d = x % D;
        if (r0 + r >= R) break;
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sm_m[w][r]);
        float lt = 0.f, y = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = sm_m[w][r] == -INFINITY ? 0.f : ptx::ex2(sm_m[w][r] - mx);
            lt = fmaf(f, sm_l[w][r], lt);
            y = fmaf(f, sm_acc[w][r][d], y);
        }
        const int h = g * a.G + (r0 + r) / a.M, i = (r0 + r) % a.M;
        const size_t row = ((size_t)b * a.Hq + h) * a.M + i;
        if (a.S == 1) {
            put<T>(a.o, row * D + d, lt > 0.f ? y * (a.v_scale / lt) : 0.f);
        } else {
            const size_t at = row * a.S + split;
            a.ws_acc[at * D + d] = y;
            if (d == 0) {
                a.ws_m[at] = mx;
                a.ws_l[at] = lt;
            }
        }
    }
}

struct Kv4Call {
    Problem p;
    Kv4Cache c;
    int max_pages, max_len, sinks;
    float k_descale, v_descale;
};

int rows_per_block(const Problem& p) { return (long long)p.G * p.M <= 8 ? 8 : 16; }

// Tiles of the longest range a sequence can have, in splits enough for about four blocks per SM.
void plan_splits(const Kv4Call& c, int* per_split, int* S) {
    const Problem& p = c.p;
    long long tiles = ((long long)c.max_len + kTile - 1) / kTile;
    if (p.window > 0) {
        const long long span = (long long)p.window + p.M - 1 + (kTile - 1);
        const long long wt = (span + kTile - 1) / kTile + ((long long)c.sinks + kTile - 1) / kTile;
        if (wt < tiles) tiles = wt;
    }
    if (tiles < 1) tiles = 1;
    const int rows = rows_per_block(p);
    const long long groups = (long long)p.B * p.Hkv * (((long long)p.G * p.M + rows - 1) / rows);
    int sms = device_sm_count();
    if (sms <= 0) sms = 148;
    long long s = (4LL * sms + groups - 1) / groups;
    if (s > tiles) s = tiles;
    if (s > 512) s = 512;
    const long long per = (tiles + s - 1) / s;
    *per_split = (int)per;
    *S = (int)((tiles + per - 1) / per);
}

template <typename T, int NT>
cudaError_t launch_d(const DecodeArgs& a, int D, dim3 grid, cudaStream_t s) {
    switch (D) {
        case 32: kv4_decode_kernel<T, 32, NT><<<grid, kWarps * 32, 0, s>>>(a); break;
        case 64: kv4_decode_kernel<T, 64, NT><<<grid, kWarps * 32, 0, s>>>(a); break;
        default: kv4_decode_kernel<T, 128, NT><<<grid, kWarps * 32, 0, s>>>(a); break;
    }
    return cudaGetLastError();
}

constexpr int64_t kI32Max = 2147483647LL;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int validate(const void* q, const Kv4Cache& cache, const int* table, const int* lens, const void* o, int B, int Hq,
             int Hkv, int M, int D, int max_pages, int max_seq_len, int causal, int window, int sinks, float scale,
             float k_descale, float v_descale, int dtype, Kv4Call* c) {
    if (dtype != ATTN_BF16 && dtype != ATTN_FP16) return ATTN_ERR_DTYPE;
    if (B < 0 || Hq < 0 || Hkv < 0 || M < 0 || max_pages < 0 || max_seq_len < 0) return ATTN_ERR_SHAPE;
    if (Hq > 0 && Hkv == 0) return ATTN_ERR_SHAPE;
    if (Hq > 0 && Hq % Hkv != 0) return ATTN_ERR_GQA;
    const int rc = kv4_validate_cache(cache, Hkv, D);
    if (rc != ATTN_OK) return rc;
    const int G = Hkv > 0 ? Hq / Hkv : 1;
    const int64_t nq = (int64_t)B * Hq * M * D, ntab = (int64_t)B * max_pages;
    if (nq > kI32Max || ntab > kI32Max || (int64_t)B * Hkv > 65535 || ((int64_t)G * M + 15) / 16 > 65535)
        return ATTN_ERR_OVERFLOW;
    if (!kv4_descale(k_descale) || !kv4_descale(v_descale)) return ATTN_ERR_SCALE;
    if ((nq > 0 && (!q || !o)) || (ntab > 0 && !table) || (B > 0 && !lens)) return ATTN_ERR_NULL;
    if (!aligned(q, 16) || !aligned(o, 16) || !aligned(table, 4) || !aligned(lens, 4)) return ATTN_ERR_ALIGN;
    const int64_t cover = (int64_t)max_pages * cache.page_size;
    const int max_len = (int)(cover < max_seq_len ? cover : max_seq_len);
    Problem& p = c->p;
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.M = M;
    p.N = max_len;
    p.D = D;
    p.causal = causal ? 1 : 0;
    // a window as long as every position of every row hides nothing more
    p.window = window <= 0 ? 0 : (int64_t)window < (int64_t)max_len + M ? window : 0;
    p.scale = (scale == 0.0f) ? (float)(1.0 / sqrt((double)D)) : scale;
    p.scale_log2 = (float)((double)p.scale * (double)k_descale * (double)kLog2e);
    p.dtype = dtype;
    p.G = G;
    p.klo = 0;
    p.khi = max_len;
    p.lse = nullptr;
    c->c = cache;
    c->max_pages = max_pages;
    c->max_len = max_len;
    c->sinks = sinks <= 0 ? 0 : sinks < max_len ? sinks : max_len;
    c->k_descale = k_descale;
    c->v_descale = v_descale;
    return ATTN_OK;
}

bool nothing_to_attend(const Kv4Call& c) { return c.max_len == 0 || c.c.num_pages == 0; }

size_t workspace_bytes(const Kv4Call& c) {
    int per = 0, S = 0;
    plan_splits(c, &per, &S);
    return S == 1 ? 0 : split_workspace_bytes(c.p.B * c.p.Hq * c.p.M, S, c.p.D);
}

int run(const Kv4Call& c, const void* q, const int* table, const int* lens, void* o, void* ws, size_t ws_bytes,
        cudaStream_t s) {
    const Problem& p = c.p;
    int per = 0, S = 0;
    plan_splits(c, &per, &S);
    const int rows = p.B * p.Hq * p.M;
    SplitWorkspace w{nullptr, nullptr, nullptr};
    if (S > 1) {
        if (!ws || ws_bytes < split_workspace_bytes(rows, S, p.D)) return ATTN_ERR_WORKSPACE;
        if (!aligned(ws, 16)) return ATTN_ERR_ALIGN;
        w = split_workspace(ws, rows, S, p.D);
    }
    const DecodeArgs a{q, c.c, table, lens, o, w.m, w.l, w.acc, p.Hq, p.Hkv, p.M, p.G, c.max_pages, c.max_len,
                       p.causal, p.window, c.sinks, p.scale_log2, c.v_descale, per, S};
    const int rb = rows_per_block(p);
    const dim3 grid((unsigned)S, (unsigned)(p.B * p.Hkv), (unsigned)((p.G * p.M + rb - 1) / rb));
    cudaError_t e;
    if (p.dtype == ATTN_BF16)
        e = rb == 8 ? launch_d<__nv_bfloat16, 1>(a, p.D, grid, s) : launch_d<__nv_bfloat16, 2>(a, p.D, grid, s);
    else
        e = rb == 8 ? launch_d<__half, 1>(a, p.D, grid, s) : launch_d<__half, 2>(a, p.D, grid, s);
    if (e == cudaSuccess && S > 1)
        e = launch_merge(w.m, w.l, w.acc, o, nullptr, nullptr, nullptr, rows, S, p.D, p.dtype, 1.0f, false, s,
                         c.v_descale);
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" {

size_t attn_decode_paged_kv4_workspace_bytes(int B, int Hq, int Hkv, int M, int D, int page_size, int max_pages,
                                             int max_seq_len, int causal, int window, int sinks) {
    static uint8_t dummy[16] __attribute__((aligned(16))) = {};
    const int* idummy = reinterpret_cast<const int*>(dummy);
    const Kv4Cache cache{dummy, dummy, dummy, dummy, 1, page_size};
    Kv4Call c;
    if (validate(dummy, cache, idummy, idummy, dummy, B, Hq, Hkv, M, D, max_pages, max_seq_len, causal, window, sinks,
                 0.f, 1.f, 1.f, ATTN_BF16, &c) != ATTN_OK)
        return 0;
    if ((int64_t)B * Hq * M == 0 || nothing_to_attend(c)) return 0;
    return workspace_bytes(c);
}

int attn_decode_paged_kv4(const void* q, const void* k_codes, const void* k_scales, const void* v_codes,
                          const void* v_scales, const int* block_table, const int* seq_lens, void* o, int B, int Hq,
                          int Hkv, int M, int D, int num_pages, int page_size, int max_pages, int max_seq_len,
                          int causal, int window, int sinks, float scale, float k_descale, float v_descale,
                          attn_dtype_t dtype, void* workspace, size_t ws_bytes, void* stream) {
    const auto mut = [](const void* p) { return static_cast<uint8_t*>(const_cast<void*>(p)); };
    const Kv4Cache cache{mut(k_codes), mut(k_scales), mut(v_codes), mut(v_scales), num_pages, page_size};
    Kv4Call c;
    int rc = validate(q, cache, block_table, seq_lens, o, B, Hq, Hkv, M, D, max_pages, max_seq_len, causal, window,
                      sinks, scale, k_descale, v_descale, dtype, &c);
    if (rc != ATTN_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if ((int64_t)B * Hq * M == 0) return ATTN_OK;
    if (nothing_to_attend(c))  // no sequence can hold a key: every row outputs 0
        return cudaMemsetAsync(o, 0, (size_t)B * Hq * M * D * 2, s) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
    const size_t bytes = workspace ? 0 : workspace_bytes(c);
    if (workspace || bytes == 0) return run(c, q, block_table, seq_lens, o, workspace, ws_bytes, s);
    void* ws = nullptr;
    if (cudaMallocAsync(&ws, bytes, s) != cudaSuccess) return ATTN_ERR_CUDA;
    rc = run(c, q, block_table, seq_lens, o, ws, bytes, s);
    if (cudaFreeAsync(ws, s) != cudaSuccess && rc == ATTN_OK) rc = ATTN_ERR_CUDA;
    return rc;
}

}  // extern "C"
