// attn_common.hpp -- argument blocks and launchers of the softmax-attention
// kernels (rotary positions, tree attention over a paged cache, append, page
// bookkeeping), internal to the library.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "gdn_attn.h"
#include "gdn_common.hpp"

namespace gdn {

// Rows of heads, strides in elements (gdn_attn_rows).
struct Rows {
    char* p;
    int64_t row, head;
};

// One layer of one pool (keys or values), strides in elements.
struct Pool {
    char* p;
    int64_t page, row, head;
};

// Quotient and remainder by a divisor that the host knows: n / d = (n m) >> 32 >> s for
// 0 <= n < 2^31, with m = ceil(2^(32+s) / d), 2^s >= d > 2^(s-1), less 2^32 (the
// multiplier has 33 bits; its top bit is the addition of n).
struct FastDiv {
    uint32_t d, m, s;
};
inline FastDiv fast_div(uint32_t d) {
    uint32_t s = 0;
    while ((1ull << s) < d) ++s;
    const uint64_t m = (((1ull << s) - d) << 32) / d + 1;
    return FastDiv{d, (uint32_t)m, s};
}
__device__ __forceinline__ uint32_t quot(FastDiv f, uint32_t n) {
    return (uint32_t)(((uint64_t)__umulhi(n, f.m) + n) >> f.s);
}

// Launch a kernel; the status is this launch's own (an earlier call's error stays where it is).
template <class... P>
inline hipError_t launch(void (*kernel)(P...), dim3 grid, dim3 block, size_t lds, hipStream_t stream, P... args) {
    if (lds > 0) {                           // with the static part it may pass the default limit of 64 KiB
        hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    void* ptrs[] = {(void*)&args...};
    return hipLaunchKernel((const void*)kernel, grid, block, ptrs, lds, stream);
}

struct RopeArgs {
    int B, N, Hq, Hk, d, rot, layout;
    double amp;
    int64_t rows;
    const int32_t* offsets;
    Rows q, k, q_out, k_out;
    const double* freq;
    const int32_t* ctx;
    const int32_t* depth;
};
hipError_t launch_rope(const RopeArgs& a, int io, hipStream_t stream);

struct AppendArgs {
    int B, N, Hk, d, n_pages, width;
    FastDiv page;
    const int32_t* offsets;
    Pool kp, vp;
    Rows k, v;
    const int32_t* table;
    const int32_t* ctx;
    const int32_t* path;
    const int32_t* path_len;
    int32_t* new_len;
};
hipError_t launch_append(const AppendArgs& a, int io, hipStream_t stream);

struct CopyArgs {
    int n, n_pages, n_layers, page_rows, Hk, d;
    Pool kp, vp;
    int64_t k_layer, v_layer;
    const int32_t* src;
    const int32_t* dst;
    const int32_t* count;
};
hipError_t launch_pages_copy(const CopyArgs& a, int io, hipStream_t stream);

struct PageArgs {
    int n_pages, page_rows, n_slots, width;
    int32_t* ref;
    int32_t* table;
    int32_t* held;
    int32_t* length;
};
hipError_t launch_pages_fork(const PageArgs& a, int n, const int32_t* src_seq, const int32_t* dst_seq,
                             int32_t* status, hipStream_t stream);
hipError_t launch_pages_reserve(const PageArgs& a, const int32_t* need, int32_t* src, int32_t* dst,
                                int32_t* count, int32_t* status, hipStream_t stream);
hipError_t launch_pages_free(const PageArgs& a, const int32_t* drop, hipStream_t stream);
hipError_t launch_pages_compact(const PageArgs& a, int n, int32_t* src, int32_t* dst, int32_t* count,
                                int32_t* remap, hipStream_t stream);

struct AttnArgs {
    int B, N, Hq, Hk, group, d, n_pages, width, words;
    float scale;
    FastDiv page, group_div;
    const int32_t* offsets;
    Pool kp, vp;                             // page and row in pieces of 16 bytes, head in bytes
    Rows q, k, v, o;                         // strides in bytes
    const int32_t* table;
    const int32_t* ctx;
    const uint32_t* anc;
    const int32_t* status;
    char* ws;
};
size_t attn_workspace(int B, int N, int Hq, int Hk, int d, int io);
hipError_t launch_attn(const AttnArgs& a, int io, hipStream_t stream);

}  // namespace gdn
