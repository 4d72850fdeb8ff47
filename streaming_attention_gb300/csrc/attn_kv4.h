// The 4-bit paged KV cache: its format and what its kernels share.
//
// A row is one key or value of one KV head: D elements (D = 32, 64 or 128) in
// NG = D / 32 groups. A group is 32 codes of 4 bits and one E4M3 scale s, and an
// element stands for descale * s * (code - 8); s * (code - 8) has at most 4 + 4
// significant bits, so it is exact in FP16 and in BF16.
//
// Order of the codes in a row (D / 2 bytes, lower nibble first): a group's units
// of consecutive elements are dealt over the row, unit u of group i at position
// u * NG + i; a unit is 8 elements (one 32-bit word) in a key row and 4 (16 bits)
// in a value row. This is the order in which the matrix instructions of the
// decode kernel take a row: thread c of a quad holds unit c of every group of a
// key (one load of 4 * NG bytes), and thread group g holds unit g of every group
// of a value (one load of 2 * NG bytes).
#pragma once

#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "attn_internal.h"

namespace attn {

constexpr int kKv4Group = 32;  // elements that share a scale

struct Kv4Cache {
    uint8_t* k_codes;   // [num_pages][Hkv][page_size][D / 2]
    uint8_t* k_scales;  // [num_pages][Hkv][page_size][D / 32], E4M3
    uint8_t* v_codes;
    uint8_t* v_scales;
    int num_pages, page_size;
};

inline bool kv4_head_dim(int D) { return D == 32 || D == 64 || D == 128; }
inline bool kv4_page_size(int ps) { return ps == 16 || ps == 32 || ps == 64 || (ps > 0 && ps % 128 == 0); }

// A power of two from 2^-64 to 2^64: scaling by it is exact, and what the kernels make of it (its product with a scale,
// its reciprocal over a scale, its quotient by a row sum) stays in the normal range of FP32.
inline bool kv4_descale(float x) {
    union {
        float f;
        uint32_t u;
    } b;
    b.f = x;
    const uint32_t e = b.u >> 23;
    return (b.u & 0x007FFFFFu) == 0 && e >= 127 - 64 && e <= 127 + 64;
}

// A load of what kernels in front of this one may have written. Not a non-coherent one: those want data that nothing
// writes from the kernel's start on, and this one may have started before the kernel in front had ended.
template <class T>
__device__ __forceinline__ T load_global(const T* p) {
    return *p;
}

// Launches a kernel that may start while the one in front of it in the stream runs, and waits for its end itself
// (griddepcontrol.wait) before it touches memory.
template <class Args>
inline cudaError_t launch_programmatic(void (*kernel)(Args), dim3 grid, int threads, cudaStream_t stream, const Args& args,
                                       size_t smem = 0) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args);
}

// Pools, table and lengths of a call; every pointer may be null only with nothing behind it.
int kv4_validate_cache(const Kv4Cache& c, int Hkv, int D);

}  // namespace attn
