// arf_decode.cu: the entry points of the decode attention (arf_decode.cuh).
#include <algorithm>
#include <climits>

#include "arf_decode.cuh"

namespace arf {
namespace {

bool kernels_for(arf_dtype_t dtype, int head_dim, bool e4m3, int nt, DecodeKernels* out) {
    return dtype == ARF_BF16 ? decode_kernels_bf16(head_dim, e4m3, nt, out)
                             : decode_kernels_fp16(head_dim, e4m3, nt, out);
}

// Groups of 8 query heads per item: two where a key head has more than 8 and
// their accumulators fit in registers (head_dim 256 takes one group, and
// reads its keys once per 8 heads).
int groups_of(int head_dim, int group) { return group > 8 && head_dim <= 128 ? 2 : 1; }

// CTAs of one launch: what shared memory lets every SM hold. The kernel's
// CTAs do not wait for one another, so this is a choice, not a limit.
int decode_grid(const arf_device_caps_t& caps, size_t smem) {
    const int per_sm = (int)(((size_t)caps.max_smem_per_block + 1024) / (smem + 1024));
    return caps.num_sms * (per_sm < 1 ? 1 : (per_sm > 4 ? 4 : per_sm));
}

// The form of a call: CTAs per item for short caches, or one of kForm....
// `bound` is the most tiles, `runs` the most warp's runs of tokens, that a
// sequence of the call can have.
//
// Clusters: a candidate is the most CTAs (up to 16, and not more than tiles)
// that run all at once; clusters of 8 and 16 leave a part of each group of SMs
// unused (15 and 7 of them fit on 152 SMs with one CTA per SM). It
// is taken where its time, about 3.3 us + 0.75 us per tile of a CTA, is below
// the dealt form's, about 6.2 us + 0.9 us per tile of a CTA of the device-full
// grid; beyond 12 tiles a CTA's share follows the lengths too unevenly.
// Measured with the cache's pages out of L2 (head_dim 128, bf16, 4 heads, us,
// cluster / dealt): 1 item of 64 tokens 4.9 / 7.0, of 1024 5.9 / 8.4, of 2048
// 6.7 / 8.5, of 4096 (clusters of 8) 12.7 / 8.8; 4 items of 4096 9.8 / 10.8
// (clusters of 8 13.6); 64 items of up to 512 tokens 8.2 / 10.8, of up to 2048 15.4 /
// 16.3, of up to 4096 24.4 / 23.1; 256 items of 64 tokens 6.9 / 9.5, of up to
// 512 14.5 / 15.6, of up to 1024 23.4 / 21.3.
//
// A warp per item: the dealt form's ends of items cost it where there are many
// (a warp per item / dealt): 400 items of up to 64 tokens 9.1 / 11.0, of up to
// 256 20.5 / 14.6; 1024 of up to 64 10.3 / 15.7, of 256 28.6 / 31.8; 1024 of
// up to 128 with 16 heads, pages in L2, 16.9 / 28.1.
int decode_form(arf_workspace_t ws, const DecodeKernels& k, int64_t items, int64_t bound, int64_t runs) {
    const arf_device_caps_t& caps = workspace_caps(ws);
    const int64_t grid = decode_grid(caps, k.smem);
    for (int c = workspace_decode_cluster(ws); c >= 1; c /= 2) {
        if (c > 1 && c / 2 >= bound) continue;
        const int64_t per_sm = ((int64_t)caps.max_smem_per_block + 1024) / (int64_t)(k.smem + (c - 1) * k.sent + kDecStaticSmem + 1024);
        const int64_t room = caps.num_sms * per_sm;
        if (items * c > (c >= 8 ? room * 3 / 4 : room)) continue;
        if (bound <= 12 * c && 4 * grid * bound <= c * (16 * grid + 5 * items * bound)) return c;
        break;
    }
    return runs <= 16 && runs * grid <= 4 * items ? kFormWarps : kFormDealt;
}
int64_t tile_bound(int64_t cap_tokens, int window, int tile) {
    const int64_t n = window > 0 && window < cap_tokens ? (int64_t)window + tile - 1 : cap_tokens;
    return (n + tile - 1) / tile;
}
int token_cap(int32_t table_width, int32_t page_size) {
    // a tile may reach past the last token: token numbers stay below 2^31
    const int64_t cap = (int64_t)table_width * page_size;
    return (int)(cap < INT_MAX - 4096 ? cap : INT_MAX - 4096);
}

struct Scratch {
    size_t stat, cut, total;  // the parts come first
};
Scratch scratch_layout(int grid, int heads, int head_dim) {
    const auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
    Scratch s = {};
    s.stat = up((size_t)2 * grid * heads * head_dim * sizeof(float));
    s.cut = s.stat + up((size_t)2 * grid * heads * sizeof(float2));
    s.total = s.cut + up((size_t)grid * sizeof(int2));
    return s;
}

}  // namespace

cudaError_t configure_decode(bool clusters, int max_smem, int* max_cluster) {
    int most = clusters ? kDecMaxCluster : 1;
    for (const arf_dtype_t dt : {ARF_BF16, ARF_FP16})
        for (const int d : {64, 128, 256})
            for (int nt = 1; nt <= 2; ++nt)
                for (const bool e4m3 : {false, true}) {
                    DecodeKernels k;
                    if (!kernels_for(dt, d, e4m3, nt, &k)) continue;
                    const void* fn = reinterpret_cast<const void*>(k.main);
                    const int room = max_smem - kDecStaticSmem;
                    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                         std::min((int)(k.smem + (kDecMaxCluster - 1) * k.sent), room));
                    if (e == cudaSuccess && clusters)
                        e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
                    if (e != cudaSuccess) return e;
                    // The largest cluster that can be resident, of every
                    // instance: a size whose shared memory an instance has no
                    // room for is not launched for it, and says nothing here.
                    for (; most > 1; most /= 2) {
                        const size_t smem = k.smem + (most - 1) * k.sent;
                        if (smem > (size_t)room) break;
                        cudaLaunchConfig_t cfg = {};
                        cudaLaunchAttribute attr[1];
                        cfg.gridDim = dim3((unsigned)most);
                        cfg.blockDim = dim3(kDecThreads);
                        cfg.dynamicSmemBytes = smem;
                        attr[0].id = cudaLaunchAttributeClusterDimension;
                        attr[0].val.clusterDim.x = (unsigned)most;
                        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
                        cfg.attrs = attr;
                        cfg.numAttrs = 1;
                        int n = 0;
                        if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) == cudaSuccess && n > 0) break;
                        (void)cudaGetLastError();
                    }
                }
    *max_cluster = most;
    return cudaSuccess;
}

}  // namespace arf

extern "C" arf_status_t arf_paged_decode_scratch_bytes(arf_workspace_t ws, const arf_kv_cache_t* cache, int64_t B,
                                                       int heads, int32_t table_width, int32_t window, size_t* bytes) {
    using namespace arf;
    if (!ws || !bytes || B < 0 || heads < 1 || table_width < 0 || window < 0) return ARF_ERR_INVALID_ARG;
    const arf_status_t st = check_cache(cache);
    if (st != ARF_OK) return st;
    if (heads % cache->kv_heads != 0) return ARF_ERR_INVALID_ARG;
    const arf_status_t ready = workspace_check_decode(ws);
    if (ready != ARF_OK) return ready;
    const int group = heads / cache->kv_heads;
    const int nt = groups_of(cache->head_dim, group);
    DecodeKernels k;
    // the tile and shared memory do not depend on the 16-bit type
    if (!kernels_for(ARF_BF16, cache->head_dim, cache->dtype == ARF_E4M3, nt, &k)) return ARF_ERR_UNSUPPORTED;
    const int64_t per_seq = (int64_t)cache->kv_heads * ((group + 8 * nt - 1) / (8 * nt));
    if (B > kMaxItems / per_seq) return ARF_ERR_UNSUPPORTED;
    const arf_device_caps_t& caps = workspace_caps(ws);
    const int64_t bound = tile_bound(token_cap(table_width, cache->page_size), window, k.tile);
    *bytes = 0;
    const int64_t runs = tile_bound(token_cap(table_width, cache->page_size), window, k.tile / kDecWarps);
    if (B > 0 && decode_form(ws, k, B * per_seq, bound, runs) == kFormDealt)
        *bytes = scratch_layout(decode_grid(caps, k.smem), 8 * nt, cache->head_dim).total;
    return ARF_OK;
}

extern "C" arf_status_t arf_paged_decode(arf_workspace_t ws, const arf_kv_cache_t* cache, int64_t B,
                                         arf_dtype_t dtype, const arf_heads_t* q, const int32_t* block_table,
                                         int64_t table_stride, int32_t table_width, const int32_t* lens,
                                         float softmax_scale, float softcap, int32_t window, const arf_heads_t* out,
                                         float* lse, void* scratch, size_t scratch_bytes, void* stream_v) {
    using namespace arf;
    if (!ws || B < 0 || !is_io_dtype(dtype)) return ARF_ERR_INVALID_ARG;
    arf_status_t st = check_cache(cache);
    if (st == ARF_OK) st = check_heads(q, B);
    if (st == ARF_OK) st = check_heads(out, B);
    if (st != ARF_OK) return st;
    const int D = cache->head_dim;
    if (q->heads != out->heads || q->heads % cache->kv_heads != 0) return ARF_ERR_INVALID_ARG;
    if (!disjoint_heads(out, B, D)) return ARF_ERR_INVALID_ARG;
    if (!isfinite(softmax_scale) || !isfinite(softcap) || softcap < 0.0f || window < 0) return ARF_ERR_INVALID_ARG;
    // the factors that the kernel works with have to be numbers too
    const double score = (double)softmax_scale * cache->k_scale * (softcap > 0.0f ? 1.0 : 1.4426950408889634);
    if (!isfinite((float)score) ||
        (softcap > 0.0f && (!isfinite(softcap * 1.4426950408889634f) || !isfinite(1.0f / softcap))))
        return ARF_ERR_INVALID_ARG;
    if (table_width < 0 || (B > 1 && table_stride < 0)) return ARF_ERR_INVALID_ARG;
    if (cache->dtype != dtype && cache->dtype != ARF_E4M3) return ARF_ERR_UNSUPPORTED;
    const bool e4m3 = cache->dtype == ARF_E4M3;
    const int group = q->heads / cache->kv_heads, nt = groups_of(D, group);
    DecodeKernels k;
    if (!kernels_for(dtype, D, e4m3, nt, &k)) return ARF_ERR_UNSUPPORTED;
    if (B > 0 && (!lens || (table_width > 0 && !block_table))) return ARF_ERR_INVALID_ARG;
    const int es = elem_bytes(cache->dtype);
    const int64_t unit = 16 / es;
    if (cache->page_stride % unit || cache->token_stride % unit || cache->head_stride % unit ||
        !is_aligned(cache->k, 16) || !is_aligned(cache->v, 16))
        return ARF_ERR_UNSUPPORTED;
    for (const arf_heads_t* t : {q, out})
        if (t->token_stride % 8 || t->head_stride % 8 || !is_aligned(t->data, 16)) return ARF_ERR_UNSUPPORTED;
    if (!is_aligned(block_table, 4) || !is_aligned(lens, 4) || !is_aligned(lse, 4) || !is_aligned(scratch, 256))
        return ARF_ERR_UNSUPPORTED;
    const int per_kv = (group + 8 * nt - 1) / (8 * nt);
    const int64_t per_seq = (int64_t)cache->kv_heads * per_kv;
    if (B > kMaxItems / per_seq || B > INT_MAX / q->heads) return ARF_ERR_UNSUPPORTED;
    if (B > 1 && table_stride > kMaxExtent / B) return ARF_ERR_UNSUPPORTED;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_v);
    st = workspace_check_device(ws, stream);
    if (st == ARF_OK) st = workspace_check_decode(ws);
    if (st != ARF_OK || B == 0) return st;
    const int cap_tokens = token_cap(table_width, cache->page_size);
    // units of a sequence, and of a CTA, are 32-bit numbers
    const int64_t units = per_seq * (cap_tokens / k.tile + 2);
    if (units > INT_MAX || units * B / decode_grid(workspace_caps(ws), k.smem) >= INT_MAX) return ARF_ERR_UNSUPPORTED;
    const int64_t items = B * per_seq;
    const int form = decode_form(ws, k, items, tile_bound(cap_tokens, window, k.tile),
                                 tile_bound(cap_tokens, window, k.tile / kDecWarps));
    const int grid = form > 0                ? (int)(items * form)
                     : form == kFormWarps ? (int)((items + kDecWarps - 1) / kDecWarps)
                                             : decode_grid(workspace_caps(ws), k.smem);
    const Scratch sc = form == kFormDealt ? scratch_layout(grid, 8 * nt, D) : Scratch{};
    if (sc.total > 0 && (!scratch || scratch_bytes < sc.total)) return ARF_ERR_INVALID_ARG;

    DecodeParams p = {};
    p.q = q->data;
    p.qts = q->token_stride, p.qhs = q->head_stride;
    p.k = static_cast<const char*>(cache->k);
    p.v = static_cast<const char*>(cache->v);
    p.cps = cache->page_stride * es, p.cts = cache->token_stride * es, p.chs = cache->head_stride * es;
    p.table = block_table;
    p.table_stride = table_stride;
    p.lens = lens;
    p.out = out->data;
    p.ots = out->token_stride, p.ohs = out->head_stride;
    p.lse = lse;
    p.form = form;
    p.grid = grid;
    if (form == kFormDealt) {
        char* base = static_cast<char*>(scratch);
        p.part = reinterpret_cast<float*>(base);
        p.stat = reinterpret_cast<float2*>(base + sc.stat);
        p.cut = reinterpret_cast<int2*>(base + sc.cut);
    }
    p.bad = workspace_bad_counter(ws);
    p.timeouts = workspace_timeout_counter(ws);
    p.B = (int)B;
    p.heads = q->heads;
    p.group = group;
    p.num_pages = cache->num_pages;
    p.per_kv = per_kv;
    p.per_seq = (int)per_seq;
    p.cap_tokens = cap_tokens;
    p.window = window;
    p.page = FastDiv((uint32_t)cache->page_size);
    p.d_kv = FastDiv((uint32_t)per_kv);
    p.score = (float)score;
    if (softcap > 0.0f) {
        p.cap2 = softcap * 1.4426950408889634f;
        p.inv_cap = 1.0f / softcap;
    }
    p.vscale = cache->v_scale;
    cudaError_t e = launch_kernel(k.main, p, dim3((unsigned)grid), kDecThreads,
                                  k.smem + (form > 1 ? (form - 1) * k.sent : 0), stream, true, form > 1 ? form : 1);
    if (e == cudaSuccess && form == kFormDealt)
        e = launch_kernel(k.join, p, dim3((unsigned)(grid + ((grid + kFewPieces - 1) / kFewPieces) * std::min(group, 8 * nt))), kJoinThreads, 0, stream, true);
    if (e != cudaSuccess) {
        note_cuda_error(ws, e);
        return ARF_ERR_CUDA;
    }
    return ARF_OK;
}
