// arf_attn.cuh: what the attention operators' translation units share:
// host checks of their tensors, fast division by a launch constant, and the
// PDL launch helper.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "arf_internal.h"

namespace arf {

// Extents (rows x stride) stay below this many elements, so that no index
// computation overflows.
constexpr int64_t kMaxExtent = (int64_t)1 << 40;

inline bool is_io_dtype(int d) { return d == ARF_BF16 || d == ARF_FP16; }
inline bool is_aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1u)) == 0; }
inline int elem_bytes(arf_dtype_t d) { return d == ARF_E4M3 ? 1 : 2; }

// A [rows, heads, D] tensor: INVALID_ARG for what no tensor can be,
// UNSUPPORTED for an extent or address beyond the kernels.
inline arf_status_t check_heads(const arf_heads_t* t, int64_t rows) {
    if (!t || t->heads < 1 || t->token_stride < 0 || t->head_stride < 0) return ARF_ERR_INVALID_ARG;
    if (rows == 0) return ARF_OK;
    if (!t->data) return ARF_ERR_INVALID_ARG;
    if (!is_aligned(t->data, 2)) return ARF_ERR_UNSUPPORTED;
    if (t->token_stride > kMaxExtent / rows || t->head_stride > kMaxExtent / t->heads) return ARF_ERR_UNSUPPORTED;
    return ARF_OK;
}

// A written tensor: rows and heads must not overlap one another.
inline bool disjoint_heads(const arf_heads_t* t, int64_t rows, int64_t D) {
    const int64_t in = t->heads > 1 ? t->head_stride : D;
    const int64_t out = rows > 1 ? t->token_stride : t->heads * in + D;
    if (in < D && t->heads > 1) return false;
    // heads inside a token, or tokens inside a head
    return rows <= 1 || out >= (int64_t)(t->heads - 1) * in + D || (out >= D && in >= (rows - 1) * out + D);
}

inline arf_status_t check_cache(const arf_kv_cache_t* c) {
    if (!c || c->num_pages < 0 || c->page_size < 1 || c->kv_heads < 1 || c->head_dim < 1) return ARF_ERR_INVALID_ARG;
    if (c->dtype != ARF_BF16 && c->dtype != ARF_FP16 && c->dtype != ARF_E4M3) return ARF_ERR_INVALID_ARG;
    if (c->page_stride < 0 || c->token_stride < 0 || c->head_stride < 0) return ARF_ERR_INVALID_ARG;
    for (const float x : {c->k_scale, c->v_scale})
        if (!(x > 0.0f) || !isfinite(x) || !isfinite(1.0f / x)) return ARF_ERR_INVALID_ARG;
    if (c->dtype != ARF_E4M3 && (c->k_scale != 1.0f || c->v_scale != 1.0f)) return ARF_ERR_INVALID_ARG;
    if (c->num_pages > 0) {
        if (!c->k || !c->v) return ARF_ERR_INVALID_ARG;
        if (c->page_stride > kMaxExtent / c->num_pages || c->token_stride > kMaxExtent / c->page_size ||
            c->head_stride > kMaxExtent / c->kv_heads)
            return ARF_ERR_UNSUPPORTED;
        if (c->dtype != ARF_E4M3 && (!is_aligned(c->k, 2) || !is_aligned(c->v, 2))) return ARF_ERR_UNSUPPORTED;
    }
    return ARF_OK;
}

// A written cache: no two rows (page, token, head) may overlap. Dimensions by
// ascending stride, each step beyond everything inside it (sufficient, and
// true of any slice of a contiguous tensor).
inline bool disjoint_cache(const arf_kv_cache_t* c) {
    int64_t stride[3] = {c->page_stride, c->token_stride, c->head_stride};
    int64_t size[3] = {c->num_pages, c->page_size, c->kv_heads};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (stride[j] < stride[i] || (stride[j] == stride[i] && size[j] < size[i])) {
                const int64_t s = stride[i], n = size[i];
                stride[i] = stride[j], size[i] = size[j];
                stride[j] = s, size[j] = n;
            }
    int64_t inside = c->head_dim;  // extent of what is inside a step
    for (int i = 0; i < 3; ++i) {
        if (size[i] <= 1) continue;
        if (stride[i] < inside) return false;
        inside += (size[i] - 1) * stride[i];
    }
    return true;
}

// n / d for 0 <= n < 2^31 by one multiplication (Granlund and Montgomery
// 1994): with s = ceil(log2 d), m = floor(2^32 (2^s - d) / d) + 1,
// n / d = (hi32(n m) + n) >> s.
struct FastDiv {
    uint32_t d, m, s;
    FastDiv() = default;
    explicit FastDiv(uint32_t div) : d(div), m(0), s(0) {
        while (((uint64_t)1 << s) < d) ++s;
        m = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << s) - d)) / d + 1);
    }
    __device__ __forceinline__ uint32_t div(uint32_t n) const { return (uint32_t)(((uint64_t)__umulhi(n, m) + n) >> s); }
};

// Launch, as a programmatic dependent if `pdl`: the kernel may then begin
// while the stream's previous one drains, and waits for it itself.
template <typename P>
cudaError_t launch_kernel(void (*fn)(P), const P& p, dim3 grid, int threads, size_t smem, cudaStream_t s, bool pdl,
                          int cluster = 1) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    if (pdl) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = (unsigned)cluster;
        attr[cfg.numAttrs].val.clusterDim.y = 1;
        attr[cfg.numAttrs++].val.clusterDim.z = 1;
    }
    return cudaLaunchKernelEx(&cfg, fn, p);
}

// The L2 policy of data that is read once: it leaves the cache first.
__device__ __forceinline__ uint64_t evict_first() {
    uint64_t policy;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    return policy;
}
__device__ __forceinline__ uint4 ld_hint(const uint4* p, uint64_t policy) {
    uint4 v;
    asm volatile("ld.global.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p), "l"(policy)
                 : "memory");
    return v;
}

// 16 bytes that are not read again. Coherent, and kept in program order: a
// programmatic dependent is resident while the launch before it may still be
// writing what it will read, so such data takes no .nc load (which asks for
// memory that is read-only for the kernel's whole life, and which the compiler
// may move above the wait of dependent_start).
__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// Start of every kernel launched by launch_kernel: let the next kernel begin
// launching, then wait until everything before this one has completed. What
// comes after is read by plain loads or those above, never by __ldg.
__device__ __forceinline__ void dependent_start() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace arf
