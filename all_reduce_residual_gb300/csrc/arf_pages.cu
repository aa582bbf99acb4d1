// arf_pages.cu: copying pages of paged caches, and the host's page pool.
//
// The copy moves whole pages of keys and values of all layers in one launch:
// nothing is computed, so HBM bounds it (each byte read and written once).
// A block moves kPieceChunks 16-byte chunks of one page, all of a thread's
// loads issued before its first store; page pairs and cache pointers travel
// in the launch parameters, so the host has checked them and no device array
// has to stay alive. Measured in a graph: 141 us for 901 pages of 32 KiB, keys
// and values of 8 layers (6.7 TB/s, the copy rate); 3.9 us for 7 pages of 16
// KiB in 32 layers.
#include <algorithm>
#include <climits>
#include <mutex>
#include <new>
#include <queue>
#include <unordered_map>
#include <vector>

#include "arf_attn.cuh"

namespace arf {
namespace {

constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;
constexpr int kPieceChunks = kCopyThreads * kCopyUnroll;

// Pairs and pointers of one launch: a small and a large set of parameters
// (a launch's cost grows with their bytes).
constexpr int kCopyPtrs = 128;

template <int PAIRS>
struct CopyParams {
    int2 pair[PAIRS];
    char* base[kCopyPtrs];
    int64_t page_stride;        // bytes
    int64_t outer_stride, inner_stride;
    int chunks;                 // 16-byte chunks per page
    // blocks per page, pointers, chunks per contiguous run, runs per outer step
    FastDiv d_piece, d_ptr, d_run, d_inner;
};

template <int PAIRS>
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyParams<PAIRS> p) {
    dependent_start();
    // block -> (pair, pointer, piece of the page)
    const uint32_t x = p.d_piece.div(blockIdx.x);
    const int piece = (int)(blockIdx.x - x * p.d_piece.d);
    const uint32_t pr = p.d_ptr.div(x);
    const int2 pair = p.pair[pr];
    char* base = p.base[x - pr * p.d_ptr.d];
    const char* src = base + (int64_t)pair.x * p.page_stride;
    char* dst = base + (int64_t)pair.y * p.page_stride;
    uint4 v[kCopyUnroll];
    int64_t at[kCopyUnroll];
#pragma unroll
    for (int i = 0; i < kCopyUnroll; ++i) {
        const int c = piece * kPieceChunks + i * kCopyThreads + (int)threadIdx.x;
        at[i] = -1;
        if (c < p.chunks) {
            const uint32_t run = p.d_run.div((uint32_t)c);
            const uint32_t outer = p.d_inner.div(run);
            at[i] = (int64_t)outer * p.outer_stride + (int64_t)(run - outer * p.d_inner.d) * p.inner_stride +
                    (int64_t)(c - (int)(run * p.d_run.d)) * 16;
            v[i] = ld_stream(reinterpret_cast<const uint4*>(src + at[i]));
        }
    }
#pragma unroll
    for (int i = 0; i < kCopyUnroll; ++i)
        if (at[i] >= 0) *reinterpret_cast<uint4*>(dst + at[i]) = v[i];
}

template <int PAIRS>
cudaError_t launch_copies(const std::vector<int2>& pairs, const std::vector<char*>& bases, CopyParams<PAIRS>& p,
                          cudaStream_t stream) {
    const int pieces = (p.chunks + kPieceChunks - 1) / kPieceChunks;
    p.d_piece = FastDiv((uint32_t)pieces);
    for (size_t b0 = 0; b0 < bases.size(); b0 += kCopyPtrs) {
        const int np = (int)std::min<size_t>(kCopyPtrs, bases.size() - b0);
        std::copy(bases.begin() + b0, bases.begin() + b0 + np, p.base);
        p.d_ptr = FastDiv((uint32_t)np);
        // a launch's blocks stay below 2^31
        const int64_t most = std::max<int64_t>(1, std::min<int64_t>(PAIRS, INT_MAX / ((int64_t)np * pieces)));
        for (size_t i = 0; i < pairs.size(); i += (size_t)most) {
            const int n = (int)std::min<size_t>((size_t)most, pairs.size() - i);
            std::copy(pairs.begin() + i, pairs.begin() + i + n, p.pair);
            const cudaError_t e = launch_kernel(copy_pages_kernel<PAIRS>, p, dim3((unsigned)((int64_t)n * np * pieces)),
                                                kCopyThreads, 0, stream, true);
            if (e != cudaSuccess) return e;
        }
    }
    return cudaSuccess;
}

// Validated pairs without those that copy nothing. Throws bad_alloc.
arf_status_t check_pairs(const int32_t* src, const int32_t* dst, int n, int32_t num_pages, std::vector<int2>* out) {
    std::vector<int32_t> s, d;
    s.reserve(n), d.reserve(n), out->reserve(n);
    for (int i = 0; i < n; ++i) {
        if (src[i] < 0 || src[i] >= num_pages || dst[i] < 0 || dst[i] >= num_pages) return ARF_ERR_INVALID_ARG;
        d.push_back(dst[i]);
        if (src[i] != dst[i]) s.push_back(src[i]), out->push_back(make_int2(src[i], dst[i]));
    }
    std::sort(d.begin(), d.end());
    if (std::adjacent_find(d.begin(), d.end()) != d.end()) return ARF_ERR_INVALID_ARG;
    for (const int32_t x : s)
        if (std::binary_search(d.begin(), d.end(), x)) return ARF_ERR_INVALID_ARG;
    return ARF_OK;
}

arf_status_t copy_pages(arf_workspace_t ws, const arf_kv_cache_t* caches, int n_caches, const int32_t* src,
                        const int32_t* dst, int n, cudaStream_t stream) {
    const arf_kv_cache_t& c = caches[0];
    std::vector<char*> bases;
    bases.reserve(2 * (size_t)n_caches);
    for (int i = 0; i < n_caches; ++i) {
        const arf_kv_cache_t& x = caches[i];
        const arf_status_t st = check_cache(&x);
        if (st != ARF_OK) return st;
        if (x.num_pages != c.num_pages || x.page_size != c.page_size || x.kv_heads != c.kv_heads ||
            x.head_dim != c.head_dim || x.page_stride != c.page_stride || x.token_stride != c.token_stride ||
            x.head_stride != c.head_stride || x.dtype != c.dtype)
            return ARF_ERR_INVALID_ARG;
        bases.push_back(static_cast<char*>(x.k));
        bases.push_back(static_cast<char*>(x.v));
    }
    if (!disjoint_cache(&c)) return ARF_ERR_INVALID_ARG;
    std::vector<int2> pairs;
    const arf_status_t pst = check_pairs(src, dst, n, c.num_pages, &pairs);
    if (pst != ARF_OK) return pst;
    const int64_t es = elem_bytes(c.dtype);
    const int64_t row = c.head_dim * es, ts = c.token_stride * es, hs = c.head_stride * es;
    for (const int64_t x : {row, ts, hs, c.page_stride * es})
        if (x % 16 != 0) return ARF_ERR_UNSUPPORTED;
    for (const char* b : bases)
        if (!is_aligned(b, 16)) return ARF_ERR_UNSUPPORTED;
    const int64_t bytes = row * c.page_size * c.kv_heads;
    if (bytes / 16 > INT_MAX / 2) return ARF_ERR_UNSUPPORTED;
    const arf_status_t dst_ = workspace_check_device(ws, stream);
    if (dst_ != ARF_OK) return dst_;
    if (pairs.empty()) return ARF_OK;
    // the page as outer x inner runs of contiguous bytes, the smaller stride
    // inside, runs that touch merged
    int64_t outer_n = c.page_size, inner_n = c.kv_heads, outer_s = ts, inner_s = hs, run = row;
    if (hs > ts) std::swap(outer_n, inner_n), std::swap(outer_s, inner_s);
    if (inner_s == run || inner_n == 1) {
        run *= inner_n;
        inner_n = outer_n, inner_s = outer_s;
        outer_n = 1, outer_s = 0;
        if (inner_s == run || inner_n == 1) run *= inner_n, inner_n = 1, inner_s = 0;
    }
    const auto fill = [&](auto& p) {
        p.page_stride = c.page_stride * es;
        p.outer_stride = outer_s, p.inner_stride = inner_s;
        p.chunks = (int)(bytes / 16);
        p.d_run = FastDiv((uint32_t)(run / 16));
        p.d_inner = FastDiv((uint32_t)inner_n);
    };
    cudaError_t e;
    if (pairs.size() <= 64) {
        CopyParams<64> p = {};
        fill(p);
        e = launch_copies(pairs, bases, p, stream);
    } else {
        CopyParams<1024> p = {};
        fill(p);
        e = launch_copies(pairs, bases, p, stream);
    }
    if (e != cudaSuccess) {
        note_cuda_error(ws, e);
        return ARF_ERR_CUDA;
    }
    return ARF_OK;
}

}  // namespace
}  // namespace arf

extern "C" arf_status_t arf_copy_pages(arf_workspace_t ws, const arf_kv_cache_t* caches, int n_caches,
                                       const int32_t* src, const int32_t* dst, int n, void* stream) {
    if (!ws || !caches || n_caches < 1 || n_caches > (1 << 20) || n < 0 || (n > 0 && (!src || !dst)))
        return ARF_ERR_INVALID_ARG;
    try {
        return arf::copy_pages(ws, caches, n_caches, src, dst, n, static_cast<cudaStream_t>(stream));
    } catch (...) {  // host memory
        return ARF_ERR_CUDA;
    }
}

// ---------------------------------------------------------------------------
// the pool
// ---------------------------------------------------------------------------

struct arf_pages {
    struct Sequence {
        std::vector<int32_t> pages;
        int64_t tokens = 0;
    };
    std::mutex mu;
    int32_t page_size = 1;
    std::vector<int32_t> refs;  // holders of each page
    // free pages, the lowest on top
    std::priority_queue<int32_t, std::vector<int32_t>, std::greater<int32_t>> free;
    std::unordered_map<int32_t, Sequence> seqs;
    int32_t next_seq = 0;

    int32_t take() {
        const int32_t page = free.top();
        free.pop();
        refs[page] = 1;
        return page;
    }
    void drop(int32_t page) {
        if (--refs[page] == 0) free.push(page);  // its room was reserved by the constructor
    }
    int64_t pages_for(int64_t tokens) const { return tokens / page_size + (tokens % page_size != 0); }
    // A number no open sequence has.
    int32_t fresh() {
        while (seqs.count(next_seq)) next_seq = next_seq == INT_MAX ? 0 : next_seq + 1;
        const int32_t s = next_seq;
        next_seq = next_seq == INT_MAX ? 0 : next_seq + 1;
        return s;
    }
};

namespace {

// Run f under the pool's lock; host memory exhausted -> CUDA.
template <typename F>
arf_status_t with_pool(arf_pages_t pool, F f) {
    if (!pool) return ARF_ERR_INVALID_ARG;
    try {
        std::lock_guard<std::mutex> lock(pool->mu);
        return f(*pool);
    } catch (...) {
        return ARF_ERR_CUDA;
    }
}

}  // namespace

extern "C" arf_status_t arf_pages_create(int32_t num_pages, int32_t page_size, arf_pages_t* pool_out) {
    if (!pool_out) return ARF_ERR_INVALID_ARG;
    *pool_out = nullptr;
    if (num_pages < 0 || page_size < 1) return ARF_ERR_INVALID_ARG;
    arf_pages* pool = nullptr;
    try {
        pool = new arf_pages();
        pool->page_size = page_size;
        pool->refs.assign(num_pages, 0);
        std::vector<int32_t> all(num_pages);  // ascending numbers are a heap
        for (int32_t i = 0; i < num_pages; ++i) all[i] = i;
        pool->free = decltype(pool->free)(std::greater<int32_t>(), std::move(all));
    } catch (...) {
        delete pool;
        return ARF_ERR_CUDA;
    }
    *pool_out = pool;
    return ARF_OK;
}

extern "C" arf_status_t arf_pages_destroy(arf_pages_t pool) {
    delete pool;
    return ARF_OK;
}

extern "C" arf_status_t arf_pages_open(arf_pages_t pool, int64_t tokens, int32_t* seq) {
    if (!seq || tokens < 0) return ARF_ERR_INVALID_ARG;
    return with_pool(pool, [&](arf_pages& p) {
        const int64_t need = p.pages_for(tokens);
        if (need > (int64_t)p.free.size()) return ARF_ERR_NO_PAGES;
        arf_pages::Sequence s;
        s.pages.reserve((size_t)need);
        s.tokens = tokens;
        const int32_t id = p.fresh();
        auto& kept = p.seqs.emplace(id, std::move(s)).first->second;
        for (int64_t i = 0; i < need; ++i) kept.pages.push_back(p.take());
        *seq = id;
        return ARF_OK;
    });
}

extern "C" arf_status_t arf_pages_extend(arf_pages_t pool, int32_t seq, int64_t tokens, int32_t* copy_src,
                                         int32_t* copy_dst) {
    if (!copy_src || !copy_dst || tokens < 0) return ARF_ERR_INVALID_ARG;
    return with_pool(pool, [&](arf_pages& p) {
        const auto it = p.seqs.find(seq);
        if (it == p.seqs.end()) return ARF_ERR_INVALID_ARG;
        arf_pages::Sequence& s = it->second;
        if (tokens > INT64_MAX - s.tokens) return ARF_ERR_INVALID_ARG;
        const bool partial = s.tokens % p.page_size != 0;
        const bool copy = tokens > 0 && partial && p.refs[s.pages.back()] > 1;
        const int64_t more = p.pages_for(s.tokens + tokens) - (int64_t)s.pages.size();
        if (more + (copy ? 1 : 0) > (int64_t)p.free.size()) return ARF_ERR_NO_PAGES;
        s.pages.reserve(s.pages.size() + (size_t)more);
        *copy_src = *copy_dst = -1;
        if (copy) {
            *copy_src = s.pages.back();
            s.pages.back() = *copy_dst = p.take();
            p.drop(*copy_src);
        }
        for (int64_t i = 0; i < more; ++i) s.pages.push_back(p.take());
        s.tokens += tokens;
        return ARF_OK;
    });
}

extern "C" arf_status_t arf_pages_fork(arf_pages_t pool, int32_t seq, int32_t* child) {
    if (!child) return ARF_ERR_INVALID_ARG;
    return with_pool(pool, [&](arf_pages& p) {
        const auto it = p.seqs.find(seq);
        if (it == p.seqs.end()) return ARF_ERR_INVALID_ARG;
        arf_pages::Sequence s = it->second;
        const int32_t id = p.fresh();
        const auto& kept = p.seqs.emplace(id, std::move(s)).first->second;
        for (const int32_t page : kept.pages) ++p.refs[page];
        *child = id;
        return ARF_OK;
    });
}

extern "C" arf_status_t arf_pages_close(arf_pages_t pool, int32_t seq) {
    return with_pool(pool, [&](arf_pages& p) {
        const auto it = p.seqs.find(seq);
        if (it == p.seqs.end()) return ARF_ERR_INVALID_ARG;
        for (const int32_t page : it->second.pages) p.drop(page);
        p.seqs.erase(it);
        return ARF_OK;
    });
}

extern "C" arf_status_t arf_pages_compact(arf_pages_t pool, int32_t* src, int32_t* dst, int32_t cap, int32_t* n) {
    if (!n || cap < 0 || (cap > 0 && (!src || !dst))) return ARF_ERR_INVALID_ARG;
    return with_pool(pool, [&](arf_pages& p) {
        const int32_t total = (int32_t)p.refs.size(), used = total - (int32_t)p.free.size();
        std::vector<int32_t> from, to, place(total);
        for (int32_t i = 0; i < total; ++i) {
            place[i] = i;
            if (i < used && p.refs[i] == 0) to.push_back(i);
            if (i >= used && p.refs[i] > 0) from.push_back(i);
        }
        *n = (int32_t)from.size();
        if (*n > cap) return ARF_ERR_INVALID_ARG;
        std::vector<int32_t> rest;
        rest.reserve((size_t)total);  // room for every page to be freed later
        for (int32_t i = used; i < total; ++i) rest.push_back(i);
        decltype(p.free) free(std::greater<int32_t>(), std::move(rest));
        for (int32_t i = 0; i < *n; ++i) {
            src[i] = from[i];
            dst[i] = place[from[i]] = to[i];
            std::swap(p.refs[from[i]], p.refs[to[i]]);
        }
        for (auto& s : p.seqs)
            for (int32_t& page : s.second.pages) page = place[page];
        p.free = std::move(free);
        return ARF_OK;
    });
}

extern "C" arf_status_t arf_pages_table(arf_pages_t pool, int32_t seq, int32_t* table, int32_t cap, int32_t* n,
                                        int64_t* tokens) {
    if (!n || !tokens || cap < 0 || (cap > 0 && !table)) return ARF_ERR_INVALID_ARG;
    return with_pool(pool, [&](arf_pages& p) {
        const auto it = p.seqs.find(seq);
        if (it == p.seqs.end()) return ARF_ERR_INVALID_ARG;
        const auto& pages = it->second.pages;
        *n = (int32_t)pages.size();
        *tokens = it->second.tokens;
        std::copy(pages.begin(), pages.begin() + std::min<size_t>(pages.size(), (size_t)cap), table);
        return ARF_OK;
    });
}

extern "C" arf_status_t arf_pages_free(arf_pages_t pool, int32_t* n) {
    if (!n) return ARF_ERR_INVALID_ARG;
    return with_pool(pool, [&](arf_pages& p) {
        *n = (int32_t)p.free.size();
        return ARF_OK;
    });
}
