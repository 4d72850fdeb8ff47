// Decode attention over the 4-bit paged KV cache (format: attn_kv4.h).
//
// Work. A segment is the visible keys of one (sequence, KV head, block of 8 grouped
// query rows), in tiles; query head h = g * G + r / M, row i = r % M. The tiles of all
// segments in a row are cut into equal ranges, one per team of W warps, whose tiles are
// of 16 W keys; a block of 12 warps fills an SM, and the grid the GPU, once, whatever the
// lengths are: each block counts the tiles from seq_lens itself. A segment that lies
// inside a team's range is written to o there; of one that is cut, each team leaves
// its part's (m, l, acc) in the workspace (at most two parts a team: one begun before
// it, one that goes on behind it), and a second kernel joins them by the
// common-maximum rule. Ranges depend on the lengths and the grid alone, so the order
// of all sums does too. (Teams in one block and not one to a block: the schedulers then
// serve them alike; as blocks they ended one after the other, 135 us for 129.)
//
// A team is one warp where there are many segments (the rule is at Plan): it has no
// sums of other warps to wait for and reads a segment's query once instead of four
// times. It is four warps for few segments, which would be cut into many parts, and for
// segments that are left whole: the warps take 16 keys each of a tile and keep their own
// running (m, l, acc) per row, joined through shared memory at the end of a segment's
// part. Each warp copies its keys' codes and scales into a ring of its own (cp.async, a
// pair of tiles ahead, no barrier between warps); the next part's copies begin before
// the sums of the last one are joined.
//
// A warp's products run transposed, on m16n8k16 matrix instructions with the
// cache as the left operand, so that a row of the cache is expanded once for all
// the query rows: S^T = K Q^T (16 keys by 8 rows) and O^T += V^T P^T (16 elements
// by 8 rows). A nibble masked out of a 16-bit half is an FP16 number as it stands:
// below 2^11 a half's bits count units of 2^-24, so bits 0..3 are n 2^-24 and bits
// 4..7 are n 2^-20, exactly, and the matrix instructions take FP16's small numbers
// at full value. One AND per two elements is all the expansion there is; the factor
// 16 between the two kinds goes into Q (keys) or into the outputs (values), and the
// 8 of n - 8 is subtracted from sums: 8 times the groups' sums of Q, times the keys'
// scales, is where the logits start (one product more), and the sums of P, which a
// product with a matrix of ones gives in the accumulators' own layout, are taken off
// at the end. (Exact n - 8 in halves took one more addition per pair: 430 -> 350
// instructions per 16 keys.) The scales are applied where there are fewer numbers than
// elements: a key's to the sum of a group's 32 products, a value's to the
// probabilities, once per group.
// What bounds it: instructions that depend on each other. Of about 300 of a warp per 16
// keys of D = 128, 88 expand codes and 21 are matrix instructions, the rest loads, scales,
// softmax and sums; the three warps of a scheduler issue in 55 of 100 cycles, as each mostly
// waits for the instruction before (1.5 warps an issue) or for a busy pipe (0.8), hardly for
// memory (0.2). 64 sequences of up to 16384 keys, 8192 on average, 8 KV
// heads (580 MB): 112 us, 5.2 TB/s, 76 % of the measured copy bandwidth. (Without its
// copies a kernel of 122 us took 115.) 12 warps of 168 registers beat 16 of 128 (139 us
// where 12 took 122), 20 of 96 and 24 of 80: fewer registers leave the compiler less to
// overlap in a warp. 16 query rows to a team, for more than
// 8, need 255 registers and leave 8 warps: 44.6 us for 16 sequences of 8192 keys with 16
// rows each, and in two blocks of 8 rows 41.7. FP8 products (half the expansion) run at a
// quarter of the rate and lose (144 us). The time moves by up to 8 % with the order in
// which the compiler is given the same work.
// Rounded below 32 bits: Q to FP16 after scaling each row by a power of two to
// maximum 2^14..2^15 (exact for elements above 2^-20 of the maximum), the
// probabilities to FP16, kept 8 to 128 times too large to stay clear of its small
// numbers (the row sum adds them unrounded), and their products with the values' scales
// (2^-9 .. 448, so between 2^-6 and 57344 at the largest score) to FP16; with FP16
// outputs less is lost (kFine). A product is one of FP16's small numbers where the
// probability is below 2^-17 / scale of the largest one, and zero below 2^-28 / scale:
// the factor of the values says how much of that range a cache has.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "attn.h"
#include "attn_internal.h"
#include "attn_kv4.h"
#include "sm100_ptx.cuh"

namespace attn {
namespace {

constexpr int kWarps = 12;           // of a block, 168 registers a thread; one block per SM
constexpr int kThreads = 32 * kWarps;
// W warps make a team, 4 or 1, and share a tile of 16 keys per warp.
constexpr int teams_of(int W) { return kWarps / W; }
constexpr int tile_of(int W) { return 16 * W; }
constexpr int kStages = 4;           // tiles in a warp's ring, two pairs
constexpr int ROWS = 8;              // query rows of a team
constexpr int kPartCost = 6;         // what a segment costs beside its tiles, in tiles (see Part)
constexpr int kMinTiles = 4;         // a team's range is at least this long while there are teams to spare
// Probabilities are kept times 2^kPShift relative to a score that the largest one may exceed by kPSlack (base 2): times
// a scale of at most 448 they stay below 2^7 * 448 = 57344.
constexpr float kPShift = 3.0f, kPSlack = 4.0f;

struct DecodeArgs {
    const void* q;
    Kv4Cache c;
    const int* table;
    const int* lens;
    void* o;
    float *ws_m, *ws_l, *ws_acc;  // [places][2][ROWS], the same, [places][2][ROWS][D]
    int4* cut;  // segments that are in parts (b, head * Z + z, first and last place; b < 0: none): by segment,
                // [segments], or where there are more segments than places by the place that begins one, [places]
    int by_segment;
    int B, Hq, Hkv, M, G, Z;
    int max_pages, max_len;
    int causal, window, sinks;
    float scale_log2;  // logit scale and K factor, times log2(e)
    float v_scale;
};

// The tiles that any row of a sequence of L keys may see: those of the first `sinks` keys, then those of the
// window's union. At least one, so that every segment belongs to a block.
struct Tiles {
    int sink, win, n;  // tiles of the sinks, first tile of the window, all
    __device__ int at(int t) const { return t < sink ? t : t - sink + win; }
};
template <int W>
__device__ __forceinline__ Tiles tiles_of(const DecodeArgs& a, int L) {
    constexpr int kTile = tile_of(W);
    int lo0, hi0, lo1, hi1;
    key_range(L - a.M, L, a.causal, a.window, &lo0, &hi0);
    key_range(L - 1, L, a.causal, a.window, &lo1, &hi1);
    const int end = hi1 / kTile + (hi1 % kTile != 0);
    Tiles t;
    t.win = min(lo0 / kTile, end);
    t.sink = min(a.sinks / kTile + (a.sinks % kTile != 0), t.win);
    t.n = max(t.sink + end - t.win, 1);
    return t;
}
__device__ __forceinline__ int length_of(const DecodeArgs& a, int b) {
    return min(max(load_global(a.lens + b), 0), a.max_len);
}

// D = A B + C, FP16 in, FP32 out; the left operand's four registers one by one
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1, const float (&c)[4]) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
// transposes an 8 x 8 matrix of halves held by the warp (two per lane)
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
// four E4M3 bytes -> four halves
__device__ __forceinline__ void e4m3x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\tcvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
// pairs of floats in one instruction
__device__ __forceinline__ void fma2(float& x, float& y, const float (&a)[2], const float (&b)[2]) {
    ptx::f2_unpack(ptx::f2_fma(ptx::f2_pack(x, y), ptx::f2_pack(a[0], a[1]), ptx::f2_pack(b[0], b[1])), x, y);
}
__device__ __forceinline__ void add2(float& x, float& y, float a, float b) {
    ptx::f2_unpack(ptx::f2_add(ptx::f2_pack(x, y), ptx::f2_pack(a, b)), x, y);
}
__device__ __forceinline__ float2 halves(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

// Bits 0..3 and 4..7 of both halves: n 2^-24 and n 2^-20 as FP16.
constexpr uint32_t kLow = 0x000F000Fu, kHigh = 0x00F000F0u;
constexpr float kLowUnit = 0x1p-24f, kHighUnit = 0x1p-20f;
constexpr uint32_t kOnes = 0x3C003C00u, kMinus = 0x80008000u;

// shared memory by its 32-bit address
__device__ __forceinline__ void load_shared(uint32_t (&w)[4], uint32_t at) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void load_shared(uint32_t (&w)[2], uint32_t at) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at) : "memory");
}
__device__ __forceinline__ void load_shared(uint32_t (&w)[1], uint32_t at) {
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(at) : "memory");
}
// 1, 2 or 4 bytes, the rest zero
template <int N>
__device__ __forceinline__ uint32_t load_shared_small(uint32_t at) {
    uint32_t w;
    if constexpr (N == 4)
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(at) : "memory");
    else if constexpr (N == 2)
        asm volatile("{\n\t.reg .u16 t;\n\tld.shared.u16 t, [%1];\n\tcvt.u32.u16 %0, t;\n\t}" : "=r"(w) : "r"(at) : "memory");
    else
        asm volatile("ld.shared.u8 %0, [%1];" : "=r"(w) : "r"(at) : "memory");
    return w;
}
__device__ __forceinline__ const void* row_block(const uint8_t* pool, uint32_t block, uint32_t bytes) {
    uint64_t p;
    asm("mad.wide.u32 %0, %1, %2, %3;" : "=l"(p) : "r"(block), "r"(bytes), "l"(reinterpret_cast<uint64_t>(pool)));
    return reinterpret_cast<const void*>(p);
}

template <typename T>
constexpr bool is_half = false;
template <>
constexpr bool is_half<__half> = true;

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

// four elements y f from i on, i a multiple of 4
template <typename T>
__device__ __forceinline__ void put4(void* o, size_t i, const float4& y, float f);
template <>
__device__ __forceinline__ void put4<__nv_bfloat16>(void* o, size_t i, const float4& y, float f) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(y.x * f, y.y * f), hi = __floats2bfloat162_rn(y.z * f, y.w * f);
    *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(o) + i) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}
template <>
__device__ __forceinline__ void put4<__half>(void* o, size_t i, const float4& y, float f) {
    *reinterpret_cast<uint2*>(reinterpret_cast<__half*>(o) + i) =
        make_uint2(ptx::pack_f16(y.x * f, y.y * f), ptx::pack_f16(y.z * f, y.w * f));
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// x / n and x % n, in 32 bits where they suffice (a division in 64 takes a hundred instructions)
__device__ __forceinline__ long long divide(long long x, int n, int* rest) {
    if ((unsigned long long)x >> 32) {
        *rest = (int)(x % n);
        return x / n;
    }
    const uint32_t q = (uint32_t)x / (uint32_t)n;
    *rest = (int)((uint32_t)x - q * (uint32_t)n);
    return q;
}

// The tiles are shared out equally: `per` to a place, and one more to the first `more` of them. (Larger shares for the
// warps of a block that come first measured slower.)
struct Shares {
    long long per;
    int more;
    __device__ __forceinline__ long long begin(int i) const { return per * i + min(i, more); }
    __device__ __forceinline__ int place_of(long long tile) const {
        const long long first = (per + 1) * more;
        return (int)(tile < first ? tile / (per + 1) : more + (tile - first) / per);
    }
};

// The part of a segment that a block is at: tiles [t0, t1) of it. Kept in shared memory, so that what the warps need
// only before and after a part's tiles takes no registers while they run through them.
// Every segment counts kPartCost more than its tiles when the tiles are shared out, in front of its first one: that is
// what a team spends on starting its copies, its query and its sums. 256 ragged sequences of up to 1000 keys, 4 KV
// heads, D = 64: 22.5 us at a cost of 4, 21.7 at 5, 20.8 at 6, 20.9 at 8; 64 of up to 16384, 8 KV heads, D = 128:
// 113.0, 112.3, 112.1, 112.4.
struct Part {
    long long u, rem;      // before the part: of all, and of its sequence
    int b, L, hz, t0, t1;  // t0 == t1: no part
    int len;               // t1 - t0 and what of kPartCost goes with it
    Tiles tl;
};
// The part at p.u, p.rem of sequence p.b in a range that ends at `end`.
template <int W>
__device__ __forceinline__ void set_part(Part& p, const DecodeArgs& a, long long end) {
    p.t0 = p.t1 = 0;
    if (p.u >= end) return;
    p.L = length_of(a, p.b);
    p.tl = tiles_of<W>(a, p.L);
    const int n = p.tl.n + kPartCost;
    int from;
    p.hz = (int)divide(p.rem, n, &from);
    p.len = (int)min((long long)(n - from), end - p.u);
    p.t0 = max(from - kPartCost, 0);
    p.t1 = max(from + p.len - kPartCost, 0);
}
template <int W>
__device__ __forceinline__ void next_part(Part& p, const Part& q, const DecodeArgs& a, long long end) {
    p.t0 = p.t1 = 0;
    if (q.t0 == q.t1) return;
    p.u = q.u + q.len;
    p.rem = q.rem + q.len;
    p.b = q.b;
    if (p.rem == (long long)(q.tl.n + kPartCost) * a.Hkv * a.Z) {
        ++p.b;
        p.rem = 0;
    }
    set_part<W>(p, a, end);
}

template <bool B>
struct Flag {
    static constexpr bool value = B;
};
template <int N>
struct Number {
    static constexpr int value = N;
};

// One stage of a warp's ring: the codes and scales of 16 keys and values. Row `slot` of the S^T product's left
// operand is key (slot / 2) % 4 + 4 (slot % 2) + 8 (slot / 8), so that the four keys that a lane needs of the
// values (slots 2 cq, 2 cq + 1, 2 cq + 8, 2 cq + 9) are cq + 4 e. Key rows lie in the order of the slots and value
// rows in that of the keys, at D = 128 with the 16-byte chunks of every other pair of rows exchanged: both are read
// without bank conflicts.
template <int D>
struct Stage {
    static constexpr int NG = D / kKv4Group;
    static constexpr int kRow = D / 2;           // bytes of a row's codes
    static constexpr int kCodes = 16 * kRow;     // 64 chunks of 16 bytes at D = 128, 32, 16
    static constexpr int kScales = 16 * NG;
    static constexpr int kK = 0, kV = kCodes, kKs = 2 * kCodes, kVs = 2 * kCodes + kScales;
    static constexpr int kBytes = 2 * kCodes + 2 * kScales;

    static constexpr int Q = kRow / 16;     // chunks of a row's codes
    static constexpr int S = kScales / 16;  // chunks of 16 rows' scales
    // at 4 bytes a row the scales that a lane needs are brought together: those of keys j and j + 8, and those of
    // values j, j + 4, j + 8 and j + 12
    static constexpr bool kSpread = NG == 4;

    // Where a lane reads and writes; the pools' rows come in blocks of 16, numbered in 32 bits.
    const uint8_t *k, *v, *s;
    uint32_t to_k, to_v, to_s;
    bool codes, scales;
    __device__ __forceinline__ Stage(const Kv4Cache& c, int lane) {
        const int x = lane & (kCodes / 16 - 1), r = x / Q, q = x % Q;
        k = c.k_codes + x * 16;
        v = c.v_codes + x * 16;
        to_k = kK + ((r & 8) | ((r & 3) << 1) | ((r >> 2) & 1)) * kRow + q * 16;
        to_v = kV + r * kRow + (D == 128 ? q ^ (r & 2) : q) * 16;
        codes = lane < kCodes / 16;
        if (kSpread) {  // one key's or value's scales to a lane
            const int j = lane & 15;
            s = (lane < 16 ? c.k_scales : c.v_scales) + j * NG;
            to_s = lane < 16 ? kKs + ((j & 7) * 2 + (j >> 3)) * NG : kVs + ((j & 3) * 4 + (j >> 2)) * NG;
            scales = true;
        } else {
            const bool vs = lane >= S;
            s = (vs ? c.v_scales : c.k_scales) + (vs ? lane - S : lane) * 16;
            to_s = vs ? kVs + (lane - S) * 16 : kKs + lane * 16;
            scales = lane < 2 * S;
        }
    }
    // The lane's part of the copy of block `at`; -1, a page outside the pool, reads as zeros: scales of zero.
    __device__ __forceinline__ void load(uint32_t dst, int at) const {
        if (at >= 0) {
            if (kCodes >= 512 || codes) {
                const uint8_t* kp = static_cast<const uint8_t*>(row_block(k, (uint32_t)at, kCodes));
                const uint8_t* vp = static_cast<const uint8_t*>(row_block(v, (uint32_t)at, kCodes));
                copy16(dst + to_k, kp);
                copy16(dst + to_v, vp);
                if (kCodes == 1024) {  // rows 8 .. 15
                    copy16(dst + to_k + 512, kp + 512);
                    copy16(dst + to_v + 512, vp + 512);
                }
            }
            if (kSpread)
                copy4(dst + to_s, row_block(s, (uint32_t)at, kScales));
            else if (scales)
                copy16(dst + to_s, row_block(s, (uint32_t)at, kScales));
        } else if (kSpread) {
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst + to_s), "r"(0) : "memory");
        } else if (scales) {
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst + to_s), "r"(0) : "memory");
        }
    }
};

// What a team's warps share.
template <int W>
struct Shared {
    float m[W][ROWS], l[W][ROWS];  // of a part, by warp
    int2 vis[2][ROWS];             // the visible range of every row, of this part and of the last or next
    long long end;                 // of the team's range
    Part parts[2];
    Shares shares;
};

template <int W>
__device__ __forceinline__ void sync_team(int team) {
    if constexpr (W == 1)
        __syncwarp();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(32 * W) : "memory");
}

// Exclusive sum over a block's threads, and the total.
__device__ __forceinline__ long long block_sum(long long x, long long* part, long long* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long s = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += y;
    }
    if (lane == 31) part[warp] = s;
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += part[w];
        all += part[w];
    }
    *total = all;
    return s - x + before;
}

// Finds the ranges of the block's teams: the first part and the end of each. False: there is none for this team. The
// costs are summed a chunk of sequences at a time, one per thread; up to kThreads sequences take one pass.
template <int W, bool kWhole>
__device__ __forceinline__ bool find_range(const DecodeArgs& a, Shared<W>* teams, int team, int place, bool first) {
    constexpr int kTeams = teams_of(W);
    const int H = a.Hkv * a.Z;
    if (kWhole) {
        if (place >= a.B * H) return false;
        if (first) {
            Part& p = teams[team].parts[0];
            p.u = p.rem = 0;
            p.b = place / H;
            p.hz = place % H;
            p.L = length_of(a, p.b);
            p.tl = tiles_of<W>(a, p.L);
            p.t0 = 0;
            p.t1 = p.tl.n;
            p.len = 1;
            teams[team].end = 1;
        }
    } else {
        __shared__ long long sums[kWarps];
        const auto cost_of = [&](int b) {
            return b < a.B ? (long long)(tiles_of<W>(a, length_of(a, b)).n + kPartCost) * H : 0ll;
        };
        long long total = 0, cost = 0, before = 0;
        for (int b0 = 0; b0 < a.B; b0 += kThreads) {
            long long all;
            cost = cost_of(b0 + (int)threadIdx.x);
            if (b0 > 0) __syncthreads();
            before = block_sum(cost, sums, &all);
            total += all;
        }
        // a grid that is larger than the tiles need uses its first places only
        const int all_places = (int)gridDim.x * kTeams;
        const int places =
            total >= (long long)kMinTiles * all_places ? all_places : (int)((total + kMinTiles - 1) / kMinTiles);
        Shares shares;
        shares.per = divide(total, places, &shares.more);
        if (first && !a.by_segment) a.cut[place] = make_int4(-1, 0, 0, 0);
        if (first) teams[team].shares = shares;
        long long behind = 0;
        for (int b0 = 0; b0 < a.B; b0 += kThreads) {
            long long all = total;
            if (a.B > kThreads) {  // one chunk's sums are still at hand
                cost = cost_of(b0 + (int)threadIdx.x);
                __syncthreads();
                before = behind + block_sum(cost, sums, &all);
            }
            for (int t = 0; t < kTeams; ++t) {
                const int at = t * (int)gridDim.x + (int)blockIdx.x;
                const long long u0 = shares.begin(at);
                if (at < places && before <= u0 && u0 < before + cost) {
                    Part& p = teams[t].parts[0];
                    p.u = u0;
                    p.rem = u0 - before;
                    p.b = b0 + (int)threadIdx.x;
                    teams[t].end = shares.begin(at + 1);
                }
            }
            behind += all;
        }
        __syncthreads();
        if (place >= places) return false;
        if (first) set_part<W>(teams[team].parts[0], a, teams[team].end);
    }
    return true;
}

// the rings of a team's warps, and where there are more than one their sums of a part
template <int D, int W>
constexpr int kTeamBytes = W * (kStages * Stage<D>::kBytes + (W > 1 ? ROWS * D * (int)sizeof(float) : 0));

template <typename T, int D, int W, bool kWhole>
__global__ void __launch_bounds__(kThreads, 1) kv4_decode_kernel(const __grid_constant__ DecodeArgs a) {
    using St = Stage<D>;
    constexpr int NG = D / kKv4Group;
    // An output in FP16 shows the two roundings of a probability (1.7 times the error of the output's own rounding), one
    // in BF16 does not. For FP16 the first one's remainder is carried into the second (1.4 times, and 1 % of the time).
    // Whole segments, whose time is mostly latency, multiply the second one's remainder too (1.0 times: 300 keys 5.4 us
    // for 5.2, 8 sequences of up to 1000 keys, D = 128, 11.8 for 10.6); for 16 sequences of up to 8192 keys with 16 rows
    // each that would be 48.8 us for 40.2.
    constexpr bool kFine = is_half<T>, kFinest = kFine && kWhole;
    extern __shared__ __align__(16) uint8_t smem_of_block[];
    constexpr int kTile = tile_of(W);
    __shared__ Shared<W> shared_of_block[teams_of(W)];
    const int team = threadIdx.x / (32 * W), thread = threadIdx.x % (32 * W);
    Shared<W>& sh = shared_of_block[team];
    uint8_t* smem = smem_of_block + team * kTeamBytes<D, W>;  // the rings, then the warps' sums of a part
    [[maybe_unused]] float* sm_acc = reinterpret_cast<float*>(smem + W * kStages * St::kBytes);  // [W][ROWS][D]
    const auto team_sync = [&] { sync_team<W>(team); };
    const int place = team * (int)gridDim.x + (int)blockIdx.x;

    const int warp = thread >> 5, lane = thread & 31;
    const int gq = lane >> 2, cq = lane & 3;  // the lane's place in a matrix fragment
    const int key_slot = (gq >> 1) + 4 * (gq & 1);  // the key of slot gq; slot gq + 8: 8 more
    const uint32_t ring = ptx::smem_u32(smem) + warp * (kStages * St::kBytes);
    const St from(a.c, lane);
    // where the lane reads in a stage; the values' chunks of every other pair of rows are exchanged
    const int at_k = St::kK + gq * St::kRow + cq * (4 * NG), at_ks = St::kKs + key_slot * NG * (St::kSpread ? 2 : 1);
    const int at_v = St::kV + cq * St::kRow + (D == 128 ? (gq * 8) ^ ((cq & 2) * 16) : gq * (2 * NG));
    const int at_vs = St::kVs + cq * NG * (St::kSpread ? 4 : 1);
    const int R = a.G * a.M;
    const int ps = a.c.page_size;

    // The join kernel may be launched now (it waits for this one's end); and this kernel may itself have been launched
    // before the end of the one in front of it, so nothing in memory is touched before that has ended.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    if (!find_range<W, kWhole>(a, shared_of_block, team, place, thread == 0)) return;
    team_sync();

    // ---- the copies of a part ----
    // the pool's blocks of this warp's keys, for 32 tiles at a time: lane x has that of tile base + x
    int base, blocks_at, next_page, copy_end;
    uint32_t fill = 0;  // the half of the ring that is filled next, in bytes
    const auto page_of = [&](const Part& p, int t) {
        const int j = p.tl.at(t) * kTile + warp * 16;
        return t < p.t1 && j < p.L ? load_global(a.table + (size_t)p.b * a.max_pages + j / ps) : -1;
    };
    const auto block_of = [&](const Part& p, int page, int t) {  // -1: a page outside the pool, or nothing to read
        const int j = p.tl.at(t) * kTile + warp * 16, g = p.hz / a.Z;
        return page >= 0 && page < a.c.num_pages ? (page * a.Hkv + g) * (ps / 16) + j % ps / 16 : -1;
    };
    const auto issue = [&](const Part& p, int t) {  // the pair of tiles t, t + 1
        if (t < copy_end) {
            if (t - base == 32) {
                base = t;
                blocks_at = block_of(p, next_page, t + lane);
                next_page = page_of(p, t + 32 + lane);
            }
            from.load(ring + fill, __shfl_sync(0xffffffffu, blocks_at, t - base));
            if (t + 1 < copy_end) from.load(ring + fill + St::kBytes, __shfl_sync(0xffffffffu, blocks_at, t + 1 - base));
            fill ^= 2 * St::kBytes;
        }
        copy_commit();
    };
    // begins the copies of part p, whose first 64 tiles' pages are at hand
    const auto begin_copies = [&](const Part& p, int page0, int page1) {
        base = p.t0;
        copy_end = p.t1;
        blocks_at = block_of(p, page0, p.t0 + lane);
        next_page = page1;
        issue(p, p.t0);
    };
    begin_copies(sh.parts[0], page_of(sh.parts[0], sh.parts[0].t0 + lane), page_of(sh.parts[0], sh.parts[0].t0 + 32 + lane));
    if (thread == 0) next_part<W>(sh.parts[1], sh.parts[0], a, sh.end);
    team_sync();

    for (int turn = 0;; turn ^= 1) {
        const Part& part = sh.parts[turn];
        if (part.t0 == part.t1) return;
        const int t1 = part.t1, L = part.L;
        const Tiles tl = part.tl;
        // rows of q and o are [b][g][row of the group]: query head g * G + r / M, row r % M
        const int r0 = (part.hz % a.Z) * ROWS;
        const size_t first_row = ((size_t)part.b * a.Hq + part.hz / a.Z * a.G) * a.M;
        // what the next part begins with, asked for now: its pages, and its query rows into L1
        const Part& ahead = sh.parts[turn ^ 1];
        const int page0 = page_of(ahead, ahead.t0 + lane), page1 = page_of(ahead, ahead.t0 + 32 + lane);
        if (ahead.t0 < ahead.t1) {
            const int r = (ahead.hz % a.Z) * ROWS + gq;
            const size_t row = ((size_t)ahead.b * a.Hq + ahead.hz / a.Z * a.G) * a.M + r;
            if (r < R && cq * 128 < 2 * D)
                asm volatile("prefetch.global.L1 [%0];" ::"l"(reinterpret_cast<const uint8_t*>(a.q) + row * (2 * D) +
                                                           cq * 128));
        }

        // Q^T fragments, each row scaled to maximum 2^14..2^15 (the elements that meet high nibbles 2^-4 of that),
        // negated if the logit scale is negative.
        // start: minus 8 times the rows' sums by group, each as the sum of four halves, as the right operand of a
        // product with the keys' scales (column k of that product's left operand is the scale of group k % 4).
        uint32_t qf[NG][2][2], start[2];
        float sc[2];
        {
            const int r = r0 + gq;
            float x[NG][8], top = 0.f;
            const bool row = r < R;
            const uint32_t* qrow = reinterpret_cast<const uint32_t*>(a.q) + (first_row + (row ? r : 0)) * (D / 2) + cq * 4;
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                const uint4 w = row ? load_global(reinterpret_cast<const uint4*>(qrow + n * 16)) : make_uint4(0, 0, 0, 0);
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
            const float down = copysignf(__uint_as_float((uint32_t)(254 - e) << 23), a.scale_log2);
            const float up =
                fmaxf(__uint_as_float((uint32_t)e << 23) * fabsf(a.scale_log2) * (0x1p-14f / kLowUnit), FLT_MIN);
            float sums[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int n = 0; n < NG; ++n) {
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const float unit = t == 0 ? 0x1p14f : 0x1p14f * (kLowUnit / kHighUnit);
                        qf[n][s][t] =
                            ptx::pack_f16(x[n][2 * s + t] * down * unit, x[n][4 + 2 * s + t] * down * unit);
                        const float2 y = halves(qf[n][s][t]);
                        sums[n] += (y.x + y.y) * (t == 0 ? kLowUnit : kHighUnit);
                    }
                sums[n] += __shfl_xor_sync(0xffffffffu, sums[n], 1);
                sums[n] += __shfl_xor_sync(0xffffffffu, sums[n], 2);
            }
            // rows k of the right operand in this lane: 2 cq, 2 cq + 1 (term cq / 2 of two groups), and 8 further (term
            // 2 more)
            float two[2] = {-8.f * (cq & 1 ? sums[2] : sums[0]), -8.f * (cq & 1 ? sums[3] : sums[1])};
#pragma unroll
            for (int term = 0; term < 4; ++term) {
                const uint32_t w = ptx::pack_f16(two[0], two[1]);
                const float2 y = halves(w);
                two[0] -= y.x;
                two[1] -= y.y;
                if ((term & 1) == (cq >> 1)) start[term >> 1] = w;
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) sc[t] = __shfl_sync(0xffffffffu, up, (2 * cq + t) * 4);
        }
        if (lane < ROWS) {  // every warp writes the same
            const int p = r0 + lane < R ? (r0 + lane) % a.M + L - a.M : L - 1;
            int2 v;
            key_range(p, L, a.causal, a.window, &v.x, &v.y);
            sh.vis[turn][lane] = v;
        }
        // keys [all_lo, all_hi) are visible to every row
        int all_lo, all_hi, skip;
        key_range(L - 1, L, a.causal, a.window, &all_lo, &skip);
        key_range(L - a.M, L, a.causal, a.window, &skip, &all_hi);

        // m: the score that stands for the largest one so far, in units of sc: it is set anew only when a score exceeds
        // it by kPSlack in base 2 (else every few steps some row's would be); limit: that border; mu: kPShift less m in
        // base 2
        float m[2], limit[2], mu[2], l[2], acc[2 * NG][4];
        float psum[NG][2];  // of the probabilities times a group's scales, as rounded for the products
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            m[t] = limit[t] = -FLT_MAX;  // finite: a masked key's -inf less it is -inf, never NaN
            mu[t] = kPShift;
            l[t] = 0.f;
        }
#pragma unroll
        for (int n = 0; n < 2 * NG; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
#pragma unroll
        for (int n = 0; n < NG; ++n) psum[n][0] = psum[n][1] = 0.f;

        // One step: N blocks of 16 keys, the first at j0, from the stages at st. `edge`: some row does not see some of
        // them. Two blocks at a time wherever both are seen by every row: their products do not depend on each other, and
        // one test of the maximum serves both (64 ragged sequences of up to 16384 keys: 112 us, 123 one at a time).
        const auto step = [&](uint32_t st, auto n_tag, int j0, auto edge_tag) {
            constexpr bool edge = decltype(edge_tag)::value;
            constexpr int N = decltype(n_tag)::value;
            uint32_t v[N][4][(NG + 1) / 2], vs[N][4];
            const auto load_values = [&](int b) {  // the lane's are keys cq + 4 e
                const uint32_t at = st + b * St::kBytes;
                if constexpr (St::kSpread) load_shared(vs[b], at + at_vs);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (NG == 1)
                        v[b][e][0] = load_shared_small<2>(at + at_v + 4 * e * St::kRow);
                    else
                        load_shared(v[b][e], at + at_v + 4 * e * St::kRow);
                    if constexpr (!St::kSpread) vs[b][e] = load_shared_small<NG>(at + at_vs + 4 * e * NG);
                }
                // A value that the lane's row of P^T does not see counts as zero, whatever it holds (a probability of
                // zero would not hide a NaN): its scales are cleared.
                if constexpr (edge) {
                    const int2 vis = sh.vis[turn][gq];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = j0 + cq + 4 * e;
                        if (!(j < vis.y && (j >= vis.x || j < a.sinks))) vs[b][e] = 0;
                    }
                }
            };
            // of one block with the keys', ahead of the branch below; of two behind the keys' products, for the registers
            if constexpr (N == 1) load_values(0);
            // ---- S^T = K Q^T, a group at a time: its 32 products' sum times the key's scale ----
            float s[N][4];
#pragma unroll
            for (int b = 0; b < N; ++b) {
                const uint32_t at = st + b * St::kBytes;
                uint32_t k0[NG], k1[NG], e0[2], e1[2];
                load_shared(k0, at + at_k);
                load_shared(k1, at + at_k + 8 * St::kRow);
                uint32_t ks[2];
                if constexpr (St::kSpread) {
                    load_shared(ks, at + at_ks);
                } else {
                    ks[0] = load_shared_small<NG>(at + at_ks);
                    ks[1] = load_shared_small<NG>(at + at_ks + 8 * NG);
                }
                e4m3x4(ks[0], e0[0], e0[1]);
                e4m3x4(ks[1], e1[0], e1[1]);
                const float2 f0[2] = {halves(e0[0]), halves(e0[1])}, f1[2] = {halves(e1[0]), halves(e1[1])};
                const uint32_t g0 = cq & 1 ? e0[1] : e0[0], g1 = cq & 1 ? e1[1] : e1[0];
                const float zero[4] = {0.f, 0.f, 0.f, 0.f};
                mma_16816(s[b], g0, g1, g0, g1, start[0], start[1], zero);
#pragma unroll
                for (int n = 0; n < NG; ++n) {
                    const uint32_t h0 = k0[n] >> 8, h1 = k1[n] >> 8;
                    const float y0 = n & 1 ? f0[n / 2].y : f0[n / 2].x, y1 = n & 1 ? f1[n / 2].y : f1[n / 2].x;
                    float x[4];
                    mma_16816(x, k0[n] & kLow, k1[n] & kLow, k0[n] & kHigh, k1[n] & kHigh, qf[n][0][0], qf[n][0][1], zero);
                    mma_16816(x, h0 & kLow, h1 & kLow, h0 & kHigh, h1 & kHigh, qf[n][1][0], qf[n][1][1], x);
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[b][e] = fmaf(x[e], e < 2 ? y0 : y1, s[b][e]);
                }
            }
            uint32_t f0[N][4], f1[N][4];
            const auto convert = [&](int b) {  // the values' scales as halves, those of a pair of keys side by side
                e4m3x4(__byte_perm(vs[b][0], vs[b][1], 0x5140u), f0[b][0], f0[b][1]);
                e4m3x4(__byte_perm(vs[b][2], vs[b][3], 0x5140u), f1[b][0], f1[b][1]);
                e4m3x4(__byte_perm(vs[b][0], vs[b][1], 0x7362u), f0[b][2], f0[b][3]);
                e4m3x4(__byte_perm(vs[b][2], vs[b][3], 0x7362u), f1[b][2], f1[b][3]);
            };
            if constexpr (N == 1) {
                convert(0);
            } else {
#pragma unroll
                for (int b = 0; b < N; ++b) load_values(b);
            }

            // ---- softmax: s[b][0..1] is slot gq of rows 2 cq, 2 cq + 1; s[b][2..3] slot gq + 8 ----
            bool rises = false;
#pragma unroll
            for (int b = 0; b < N; ++b)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (edge) {
                        const int j = j0 + key_slot + 8 * (e >> 1);
                        const int2 vis = sh.vis[turn][2 * cq + (e & 1)];
                        if (!(j < vis.y && (j >= vis.x || j < a.sinks))) s[b][e] = -INFINITY;  // a masked key scores -inf
                    }
                    rises |= s[b][e] > limit[e & 1];
                }
            if (__any_sync(0xffffffffu, rises)) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = m[e];
#pragma unroll
                    for (int b = 0; b < N; ++b) mx = fmaxf(mx, fmaxf(s[b][e], s[b][2 + e]));
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                    const float alpha = ptx::ex2((m[e] - mx) * sc[e]);
                    m[e] = mx;
                    if (mx > -FLT_MAX) {
                        limit[e] = mx + kPSlack / sc[e];
                        mu[e] = fmaf(-mx, sc[e], kPShift);
                    }
                    l[e] *= alpha;
#pragma unroll
                    for (int n = 0; n < 2 * NG; ++n) {
                        acc[n][e] *= alpha;
                        acc[n][2 + e] *= alpha;
                    }
#pragma unroll
                    for (int n = 0; n < NG; ++n) psum[n][e] *= alpha;
                }
            }
            uint32_t pb0[N], pb1[N];
            [[maybe_unused]] uint32_t rest0[N], rest1[N];  // what the rounding of P left
#pragma unroll
            for (int b = 0; b < N; ++b) {
                fma2(s[b][0], s[b][1], sc, mu);
                fma2(s[b][2], s[b][3], sc, mu);
#pragma unroll
                for (int e = 0; e < 4; ++e) s[b][e] = ptx::ex2(s[b][e]);
                const uint32_t h0 = ptx::pack_f16(s[b][0], s[b][1]), h1 = ptx::pack_f16(s[b][2], s[b][3]);
                pb0[b] = transpose8(h0);
                pb1[b] = transpose8(h1);
                if constexpr (kFine) {
                    const float2 y0 = halves(h0), y1 = halves(h1);
                    rest0[b] = transpose8(ptx::pack_f16(s[b][0] - y0.x, s[b][1] - y0.y));
                    rest1[b] = transpose8(ptx::pack_f16(s[b][2] - y1.x, s[b][3] - y1.y));
                }
                add2(l[0], l[1], s[b][0], s[b][1]);
                add2(l[0], l[1], s[b][2], s[b][3]);
            }

            // ---- O^T += V^T (P s)^T ----
#pragma unroll
            for (int b = 0; b < N; ++b) {
                if constexpr (N > 1) {
                    convert(b);
                }
#pragma unroll
                for (int n = 0; n < NG; ++n) {
                    // the unit of group n of both keys of a pair: its low byte and its high byte
                    const uint32_t lo = n & 1 ? 0x7632u : 0x5410u, hi = n & 1 ? 0x0703u : 0x0501u;
                    const auto& w = v[b];
                    const uint32_t u0 = __byte_perm(w[0][n / 2], w[1][n / 2], lo), u1 = __byte_perm(w[2][n / 2], w[3][n / 2], lo);
                    const uint32_t h0 = __byte_perm(w[0][n / 2], w[1][n / 2], hi), h1 = __byte_perm(w[2][n / 2], w[3][n / 2], hi);
                    uint32_t p0, p1;
                    [[maybe_unused]] uint32_t left0, left1;  // what the rounding of P s left
                    if constexpr (kFine) {
                        p0 = hfma2(pb0[b], f0[b][n], hmul2(rest0[b], f0[b][n]));
                        p1 = hfma2(pb1[b], f1[b][n], hmul2(rest1[b], f1[b][n]));
                        if constexpr (kFinest) {
                            left0 = hfma2(rest0[b], f0[b][n], hfma2(pb0[b], f0[b][n], p0 ^ kMinus));
                            left1 = hfma2(rest1[b], f1[b][n], hfma2(pb1[b], f1[b][n], p1 ^ kMinus));
                        }
                    } else {
                        p0 = hmul2(pb0[b], f0[b][n]);
                        p1 = hmul2(pb1[b], f1[b][n]);
                    }
                    float (&lo_acc)[4] = acc[2 * n], (&hi_acc)[4] = acc[2 * n + 1];
                    mma_16816(lo_acc, u0 & kLow, u0 & kHigh, u1 & kLow, u1 & kHigh, p0, p1, lo_acc);
                    mma_16816(hi_acc, h0 & kLow, h0 & kHigh, h1 & kLow, h1 & kHigh, p0, p1, hi_acc);
                    const float zero[4] = {0.f, 0.f, 0.f, 0.f};
                    float x[4];
                    mma_16816(x, kOnes, kOnes, kOnes, kOnes, p0, p1, zero);
                    if constexpr (kFinest) {
                        mma_16816(lo_acc, u0 & kLow, u0 & kHigh, u1 & kLow, u1 & kHigh, left0, left1, lo_acc);
                        mma_16816(hi_acc, h0 & kLow, h0 & kHigh, h1 & kLow, h1 & kHigh, left0, left1, hi_acc);
                        mma_16816(x, kOnes, kOnes, kOnes, kOnes, left0, left1, x);
                    }
                    add2(psum[n][0], psum[n][1], x[0], x[1]);
                }
            }
        };

        const auto full = [&](int j0) { return j0 + 16 <= all_hi && (j0 >= all_lo || j0 + 16 <= a.sinks); };
        const auto any_step = [&](uint32_t st, int j0) {
            if (full(j0)) {
                step(st, Number<1>(), j0, Flag<false>());
            } else if (j0 < L) {
                step(st, Number<1>(), j0, Flag<true>());
            }
        };
        for (int t = part.t0; t < t1; t += 2) {
            const uint32_t st = ring + (fill ^ 2 * St::kBytes);  // the pair of tiles t, t + 1
            __syncwarp();
            issue(part, t + 2);  // into the half that was read in the last turn
            copy_wait<1>();
            __syncwarp();
            const int j0 = tl.at(t) * kTile + warp * 16, j1 = tl.at(t + 1) * kTile + warp * 16;
            if (t + 1 < t1 && full(j0) && full(j1)) {
                step(st, Number<2>(), j0, Flag<false>());
            } else {
                any_step(st, j0);
                if (t + 1 < t1) any_step(st + St::kBytes, j1);
            }
        }

        // ---- the next part's copies begin; then the warps' sums are joined ----
        begin_copies(ahead, page0, page1);
        const bool begun = part.t0 == 0, done = begun && t1 == tl.n;
        const size_t part_row = ((size_t)place * 2 + begun) * ROWS;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) l[t] += __shfl_xor_sync(0xffffffffu, l[t], d);
            const int r = 2 * cq + t;
            // element 32 n + 4 gq + x: accumulator 2 n + x / 2, its row gq (x even: low nibbles) or gq + 8
            float4 y[NG];
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                const float off = -8.f * psum[n][t];
                y[n] = make_float4(fmaf(acc[2 * n][t], 1.f / kLowUnit, off), fmaf(acc[2 * n][2 + t], 1.f / kHighUnit, off),
                                   fmaf(acc[2 * n + 1][t], 1.f / kLowUnit, off),
                                   fmaf(acc[2 * n + 1][2 + t], 1.f / kHighUnit, off));
            }
            if constexpr (W > 1) {
                if (gq == 0) {
                    sh.m[warp][r] = m[t] * sc[t];
                    sh.l[warp][r] = l[t];
                }
#pragma unroll
                for (int n = 0; n < NG; ++n)
                    *reinterpret_cast<float4*>(sm_acc + (warp * ROWS + r) * D + 32 * n + 4 * gq) = y[n];
            } else if (r0 + r < R) {
                if (done) {
                    const float f = l[t] != 0.f ? a.v_scale / l[t] : 0.f;
                    const size_t at = (first_row + r0 + r) * D + 4 * gq;
#pragma unroll
                    for (int n = 0; n < NG; ++n) put4<T>(a.o, at + 32 * n, y[n], f);
                } else {
#pragma unroll
                    for (int n = 0; n < NG; ++n)
                        *reinterpret_cast<float4*>(a.ws_acc + (part_row + r) * D + 32 * n + 4 * gq) = y[n];
                    if (gq == 0) {
                        a.ws_m[part_row + r] = m[t] * sc[t];
                        a.ws_l[part_row + r] = l[t];
                    }
                }
            }
        }
        team_sync();
        if constexpr (W > 1) {
            for (int x = thread; x < ROWS * D; x += 32 * W) {
                const int r = x / D, d = x % D;
                if (r0 + r >= R) break;
                float mx = -FLT_MAX;
#pragma unroll
                for (int w = 0; w < W; ++w) mx = fmaxf(mx, sh.m[w][r]);
                float lt = 0.f, y = 0.f;
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    const float f = ptx::ex2(sh.m[w][r] - mx);  // a warp that saw no key has sums of zero
                    lt = fmaf(f, sh.l[w][r], lt);
                    y = fmaf(f, sm_acc[(w * ROWS + r) * D + d], y);
                }
                if (done) {
                    put<T>(a.o, (first_row + r0 + r) * D + d, lt != 0.f ? y * (a.v_scale / lt) : 0.f);
                } else {
                    a.ws_acc[(part_row + r) * D + d] = y;
                    if (d == 0) {
                        a.ws_m[part_row + r] = mx;
                        a.ws_l[part_row + r] = lt;
                    }
                }
            }
        }
        if (!kWhole && thread == 0 && begun) {  // a whole segment has no list and no workspace
            int4 cut = make_int4(-1, 0, 0, 0);
            if (!done) {
                const int n = tl.n + kPartCost;
                cut = make_int4(part.b, part.hz, place, sh.shares.place_of(part.u - part.rem % n + n - 1));
            }
            if (a.by_segment)
                a.cut[part.b * (a.Hkv * a.Z) + part.hz] = cut;
            else if (!done)
                a.cut[place] = cut;
        }
        team_sync();  // the part and the sums are read
        if (thread == 0) next_part<W>(sh.parts[turn], sh.parts[turn ^ 1], a, sh.end);
        team_sync();
    }
}

// Joins the parts of the segment cut[blockIdx.x]: the part in its first place's second slot and those in the first
// slots of the places behind it. The W warps take a row each, or share a row's parts where there are fewer rows,
// kJoinBatch at a time; kRow: the block takes row blockIdx.y alone. What bounds this kernel is its launch and the chain
// of loads (cut, then parts), so a block is as small as the number of parts lets it be. When this was chosen, a decode of
// 64 segments in 7 parts each took 18.2 us with 16 warps and all rows a block and 17.3 with 4 warps a row; of 8 segments
// in 57 parts 38.8 and, with 8 warps a row, 35.9; of 512 mostly in one part 122.4 and, with 4 warps a block, 118.3.
constexpr int kJoinBatch = 8;

template <typename T, int D, int W, bool kRow>
__global__ void __launch_bounds__(32 * W) kv4_join_kernel(DecodeArgs a) {
    __shared__ float sm_m[W], sm_l[W];
    __shared__ float4 sm_y[W][D / 4];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 cut = a.cut[blockIdx.x];
    if (cut.x < 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r0 = (cut.y % a.Z) * ROWS, rows = min(ROWS, a.G * a.M - r0);
    if (kRow && (int)blockIdx.y >= rows) return;
    const int most = kRow || rows <= 1 ? W : rows <= 2 ? W / 2 : rows <= 4 ? W / 4 : W / 8;
    const int team = most > 1 ? most : 1;  // warps of a row
    const int share = warp % team;
    const int parts = cut.w - cut.z + 1;
    const bool has = lane < D / 4;
    for (int r = kRow ? (int)blockIdx.y : warp / team; r < ROWS; r += W / team) {  // one turn unless rows exceed warps
        float mx = -FLT_MAX, l = 0.f;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int x0 = share; r < rows && x0 < parts; x0 += kJoinBatch * team) {
            float m[kJoinBatch], s[kJoinBatch];
            float4 v[kJoinBatch];
#pragma unroll
            for (int e = 0; e < kJoinBatch; ++e) {
                const int x = x0 + e * team;
                m[e] = -FLT_MAX;
                s[e] = 0.f;
                v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (x < parts) {
                    const size_t row = ((size_t)(cut.z + x) * 2 + (x == 0)) * ROWS + r;
                    m[e] = a.ws_m[row];
                    s[e] = a.ws_l[row];
                    if (has) v[e] = reinterpret_cast<const float4*>(a.ws_acc + row * D)[lane];
                }
            }
            float top = mx;
#pragma unroll
            for (int e = 0; e < kJoinBatch; ++e) top = fmaxf(top, m[e]);
            const float f0 = ptx::ex2(mx - top);
            l *= f0;
            y = make_float4(y.x * f0, y.y * f0, y.z * f0, y.w * f0);
            mx = top;
#pragma unroll
            for (int e = 0; e < kJoinBatch; ++e) {
                const float f = ptx::ex2(m[e] - top);
                l = fmaf(f, s[e], l);
                y = make_float4(fmaf(f, v[e].x, y.x), fmaf(f, v[e].y, y.y), fmaf(f, v[e].z, y.z), fmaf(f, v[e].w, y.w));
            }
        }
        if (team > 1) {
            if (lane == 0) {
                sm_m[warp] = mx;
                sm_l[warp] = l;
            }
            if (has) sm_y[warp][lane] = y;
            __syncthreads();
            if (share != 0 || r >= rows || !has) return;
            float top = mx;
            for (int w = warp + 1; w < warp + team; ++w) top = fmaxf(top, sm_m[w]);
            l = 0.f;
            y = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int w = warp; w < warp + team; ++w) {
                const float f = ptx::ex2(sm_m[w] - top);
                const float4 v = sm_y[w][lane];
                l = fmaf(f, sm_l[w], l);
                y = make_float4(fmaf(f, v.x, y.x), fmaf(f, v.y, y.y), fmaf(f, v.z, y.z), fmaf(f, v.w, y.w));
            }
        }
        if (r < rows && has) {
            const size_t at = (((size_t)cut.x * a.Hq + cut.y / a.Z * a.G) * a.M + r0 + r) * D + 4 * lane;
            const float f = l != 0.f ? a.v_scale / l : 0.f;
            put<T>(a.o, at, y.x * f);
            put<T>(a.o, at + 1, y.y * f);
            put<T>(a.o, at + 2, y.z * f);
            put<T>(a.o, at + 3, y.w * f);
        }
        if (team > 1) return;
    }
}

struct Kv4Call {
    Problem p;
    Kv4Cache c;
    int max_pages, max_len, sinks;
    float k_descale, v_descale;
};

int sm_count() {
    const int n = device_sm_count();
    return n > 0 ? n : 148;
}

int row_blocks(const Problem& p) { return (int)(((long long)p.G * p.M + ROWS - 1) / ROWS); }

// Few short segments are left whole, one to a team of four warps: no sums of costs, no second kernel. Microseconds whole
// and cut, 2 KV heads of one sequence, D = 64, FP16: 300 keys (5 tiles) 5.4 and 7.8, 1000 (16 tiles) 8.9 and 8.1, 2000
// 13.9 and 8.2; 64 KV heads (8 sequences), D = 128: 6.8 and 10.5, 11.0 and 11.3, 16.6 and 13.2; 456 of 900 keys 17.1 and
// 23.0.
// Otherwise a team is one warp where a segment is cut into kManyParts parts or less on average, and four warps (a
// quarter of the parts) where there are fewer segments. With one and with four, D = 128: 8 segments of 131072 keys 38.7
// and 35.0; 16 of 4096 11.3 and 11.0; 32 of 32768 35.5 and 36.0; 64 of 2048 13.5 and 14.0; 128 of up to 8192 24.3
// and 24.2; 512 of up to 16384 112.2 and 114.3; at D = 64 30.4 and 26.3 (8), 27.2 and 26.4 (32), 11.5 and 11.1 (64), 18.9
// and 18.6 (128), 20.9 and 24.8 (1024 of up to 1000).
struct Plan {
    int blocks, warps;  // warps of a team
    bool whole;
};
constexpr int kWholeTiles = 16;  // of 64 keys
constexpr int kManyParts = 32;

long long segments_of(const Problem& p) { return (long long)p.B * p.Hkv * row_blocks(p); }

// The most segments of this and of any smaller call (at most B, Hq, Hkv and M of p): fewer KV heads may make more of
// them, 18 query heads on 2 KV heads 4 (9 rows each), on 3 KV heads 3.
long long most_segments(const Problem& p) {
    long long most = 0;
    for (int h = 1; h <= p.Hkv && h <= p.Hq; ++h) {
        const long long n = h * (((long long)(p.Hq / h) * p.M + ROWS - 1) / ROWS);
        if (n > most) most = n;
    }
    return p.B * most;
}

// One block for every SM, fewer while the longest lengths could not give one team of each kMinTiles tiles. What a plan
// needs of workspace does not fall as the segments or the longest length rise.
Plan plan_blocks(const Kv4Call& c, long long segments) {
    const Problem& p = c.p;
    const long long sms = sm_count();
    const auto tiles_at = [&](int kTile) {
        long long tiles = ((long long)c.max_len + kTile - 1) / kTile;
        if (p.window > 0) {
            const long long span = (long long)p.window + p.M - 1 + (kTile - 1);
            const long long wt = (span + kTile - 1) / kTile + ((long long)c.sinks + kTile - 1) / kTile;
            if (wt < tiles) tiles = wt;
        }
        return tiles < 1 ? 1 : tiles;
    };
    if (tiles_at(tile_of(4)) <= kWholeTiles && segments <= sms * teams_of(4))
        return Plan{(int)(segments < sms ? segments : sms), 4, true};
    const int W = segments * kManyParts >= sms * teams_of(1) ? 1 : 4;
    const long long want = ((tiles_at(tile_of(W)) + kPartCost) * segments + kMinTiles - 1) / kMinTiles;
    return Plan{(int)(want < sms ? want : sms), W, false};
}

template <typename T, int D, int W, bool kWhole>
cudaError_t launch_t(const DecodeArgs& a, int blocks, cudaStream_t s) {
    constexpr int kTeams = teams_of(W), kSmem = kTeams * kTeamBytes<D, W>;
    static PerDeviceOnce once;
    const cudaError_t e = once_per_device(once, [] {
        return cudaFuncSetAttribute(kv4_decode_kernel<T, D, W, kWhole>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kSmem);
    });
    if (e != cudaSuccess) return e;
    const cudaError_t r =
        launch_programmatic(kv4_decode_kernel<T, D, W, kWhole>, dim3((unsigned)blocks), kThreads, s, a, kSmem);
    if (r != cudaSuccess || kWhole) return r;
    const unsigned entries = (unsigned)(a.by_segment ? a.B * a.Hkv * a.Z : blocks * kTeams);
    const unsigned rows = (unsigned)(a.G * a.M < ROWS ? a.G * a.M : ROWS);
    const unsigned parts = (unsigned)(blocks * kTeams) / entries;  // of a segment, about
    if (parts >= 16) return launch_programmatic(kv4_join_kernel<T, D, 8, true>, dim3(entries, rows), 32 * 8, s, a);
    if (parts >= 3) return launch_programmatic(kv4_join_kernel<T, D, 4, true>, dim3(entries, rows), 32 * 4, s, a);
    return launch_programmatic(kv4_join_kernel<T, D, 4, false>, dim3(entries), 32 * 4, s, a);
}

template <typename T, int D>
cudaError_t launch_w(const DecodeArgs& a, const Plan& plan, cudaStream_t s) {
    if (plan.whole) return launch_t<T, D, 4, true>(a, plan.blocks, s);
    return plan.warps == 4 ? launch_t<T, D, 4, false>(a, plan.blocks, s) : launch_t<T, D, 1, false>(a, plan.blocks, s);
}

template <typename T>
cudaError_t launch_d(const DecodeArgs& a, int D, const Plan& plan, cudaStream_t s) {
    switch (D) {
        case 32: return launch_w<T, 32>(a, plan, s);
        case 64: return launch_w<T, 64>(a, plan, s);
        default: return launch_w<T, 128>(a, plan, s);
    }
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
    const int64_t nq = elements({B, Hq, M, D}), ntab = elements({B, max_pages});
    const int64_t cover = (int64_t)max_pages * cache.page_size;
    const int64_t longest = cover < max_seq_len ? cover : max_seq_len;
    if (nq > kI32Max || ntab > kI32Max || (int64_t)B * Hkv > 65535 || ((int64_t)G * M + ROWS - 1) / ROWS > 65535 ||
        longest > kI32Max - tile_of(4) || (int64_t)cache.num_pages * (cache.page_size / 16) * Hkv > kI32Max)
        return ATTN_ERR_OVERFLOW;
    if (!kv4_descale(k_descale) || !kv4_descale(v_descale)) return ATTN_ERR_SCALE;
    if ((nq > 0 && (!q || !o)) || (ntab > 0 && !table) || (B > 0 && !lens)) return ATTN_ERR_NULL;
    if (!aligned(q, 16) || !aligned(o, 16) || !aligned(table, 4) || !aligned(lens, 4)) return ATTN_ERR_ALIGN;
    const int max_len = (int)longest;
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

// Cut segments and their parts, two per team: [places] int4, then m, l and acc.
int places_of(const Plan& plan) { return plan.blocks * teams_of(plan.warps); }
size_t workspace_bytes(const Plan& plan, int D) {
    return plan.whole ? 0 : (size_t)places_of(plan) * (sizeof(int4) + (size_t)2 * ROWS * (2 + D) * sizeof(float));
}

int run(const Kv4Call& c, const void* q, const int* table, const int* lens, void* o, void* ws, size_t ws_bytes,
        const Plan& plan, cudaStream_t s) {
    const Problem& p = c.p;
    const int places = places_of(plan);
    if (!plan.whole) {  // (the cut segments' list has an entry per place, and is by segment only where it has room)
        if (!ws || ws_bytes < workspace_bytes(plan, p.D)) return ATTN_ERR_WORKSPACE;
        if (!aligned(ws, 16)) return ATTN_ERR_ALIGN;
    }
    const size_t n = (size_t)places * 2 * ROWS;
    int4* cut = static_cast<int4*>(ws);
    float* wm = plan.whole ? nullptr : reinterpret_cast<float*>(cut + places);
    const int by_segment = segments_of(p) <= places;
    const DecodeArgs a{q, c.c, table, lens, o, wm, wm + n, wm + 2 * n, cut, by_segment, p.B, p.Hq, p.Hkv, p.M, p.G, row_blocks(p),
                       c.max_pages, c.max_len, p.causal, p.window, c.sinks, p.scale_log2, c.v_descale};
    const cudaError_t e =
        p.dtype == ATTN_BF16 ? launch_d<__nv_bfloat16>(a, p.D, plan, s) : launch_d<__half>(a, p.D, plan, s);
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
    if (elements({B, Hq, M}) == 0 || nothing_to_attend(c)) return 0;
    return workspace_bytes(plan_blocks(c, most_segments(c.p)), D);
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
    if (elements({B, Hq, M}) == 0) return ATTN_OK;
    if (nothing_to_attend(c))  // no sequence can hold a key: every row outputs 0
        return cudaMemsetAsync(o, 0, (size_t)B * Hq * M * D * 2, s) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
    const Plan plan = plan_blocks(c, segments_of(c.p));
    const size_t bytes = workspace_bytes(plan, D);
    if (workspace || bytes == 0) return run(c, q, block_table, seq_lens, o, workspace, ws_bytes, plan, s);
    void* ws = nullptr;
    if (cudaMallocAsync(&ws, bytes, s) != cudaSuccess) return ATTN_ERR_CUDA;
    rc = run(c, q, block_table, seq_lens, o, ws, bytes, plan, s);
    if (cudaFreeAsync(ws, s) != cudaSuccess && rc == ATTN_OK) rc = ATTN_ERR_CUDA;
    return rc;
}

}  // extern "C"
