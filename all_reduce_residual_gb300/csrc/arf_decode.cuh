// arf_decode.cuh: attention of one new token per sequence over a paged
// key-value cache (arf_paged_decode).
//
// Mathematics. For one sequence and one key head with its G query heads, in
// tiles of tokens: S^T = K Q^T, the running maximum m and sum l of a softmax
// kept per query head in binary32 (in units of log2), O^T += V^T P^T with
// O^T rescaled when m grows. Two runs over parts of a sequence are joined by
// weights 2^(m_i - m).
//
// What bounds it. 4 G flops per key-value element of 1 or 2 bytes: HBM, as
// long as the products run on the matrix pipe (mma.sync reaches a multiple
// of what these few heads need; a 128-row tcgen05 tile would be empty but
// for G rows). Tokens are the rows of both products, so the 8 columns hold
// the query heads of one key head and no padding rows are read.
//
// Split, for long caches. The linear list of all work (sequence, block of
// query heads, tile) is dealt out evenly to the CTAs, whatever the lengths:
// CTA c of g takes units [total c / g, total (c + 1) / g). An item has a unit
// per tile and one more for its end, the joining of the warps (about 0.9 us;
// a tile takes a CTA about 1.5 us). Every CTA finds its range from the
// lengths on the device. What is cut goes to the scratch buffer as (O, m, l)
// and decode_join_kernel adds it up in the order of the CTAs.
//
// Split, for short caches (the table's width bounds the lengths). An item's
// tiles go to the CTAs of one thread-block cluster, which send (O, m, l) to
// its first CTA by asynchronous stores into distributed shared memory: one
// launch and no scratch. Latency counts there, not balance.
//
// Split, for many short caches. A warp per item, and nothing to join: where
// there are more items than CTAs fit on the device, their ends would cost more
// than their tokens. The choice is made in decode_form.
//
// Within a CTA the warps are independent: warp w takes every kDecWarps-th run
// of 16 (or, of short rows, 32) tokens, through its own ring of cp.async stages in shared memory
// (rows rotated by XOR so that ldmatrix reads are free of bank conflicts).
// They meet only at the end of a sequence's range.
//
// Measured, in a graph: 83 us for 128 sequences of up to 4096 tokens, 16 / 4
// heads of 128, bf16 (507 MB, 6.1 TB/s; a read-only pass takes 69 us, the SMs
// end about 73 to 79 us after the start, the join and the launches take 5); 65
// us for 48 of up to 30011 tokens, 16 / 2 heads, e4m3 (371 MB, 5.7 TB/s); 41.5
// us for two of 262001, 8 / 1 heads, fp16 (217 MB); 56.5 us for 24 with a window
// of 4096, 8 / 4 heads of 256 (318 MB); 4.8 us for one of 517.
#pragma once

#include <type_traits>

#include "arf_attn.cuh"
#include "arf_bulk.cuh"

namespace arf {

constexpr int kDecWarps = 4;
constexpr int kDecThreads = 32 * kDecWarps;
constexpr int64_t kMaxItems = (1 << 29) - 1;  // an item's number leaves three bits of flags
constexpr int kFormDealt = 0;      // units dealt out over the device, cut items joined by a second kernel
constexpr int kFormWarps = -1;     // a warp per item
constexpr int kDecMaxCluster = 16;  // CTAs of a cluster (8 is the portable limit)

struct DecodeParams {
    const void* q;
    int64_t qts, qhs;
    const char* k;
    const char* v;
    int64_t cps, cts, chs;  // cache strides, bytes
    const int32_t* table;
    int64_t table_stride;
    const int32_t* lens;
    void* out;
    int64_t ots, ohs;
    float* lse;
    int form;               // CTAs per item (a cluster), or one of kForm...
    int grid;               // CTAs then
    float* part;            // [2 * grid][heads per item][D] partial O
    float2* stat;           // [2 * grid][heads per item] (m, l)
    int2* cut;              // [grid] the item that begins in a CTA and ends in a later one, and that CTA
    unsigned int* bad;
    unsigned int* timeouts; // waits that gave up (arf_workspace_wait_timeouts)
    int B, heads, group, num_pages;
    int per_kv, per_seq;    // items (blocks of query heads) per key head and per sequence
    int cap_tokens;         // table_width * page_size
    int window;
    FastDiv page;
    FastDiv d_kv;           // by per_kv
    float score;            // softmax scale * k_scale (times log2 e without a cap)
    float cap2, inv_cap;    // cap * log2 e, 1 / cap (0: no cap)
    float vscale;
};

// Sizes of an instance: ES cache element bytes.
template <int D, int ES, int NT>
struct DecodeShape {
    static constexpr int row = D * ES;                            // bytes of a token's key
    static constexpr int tok = row >= 256 ? 16 : 32;              // tokens of a warp's stage
    static constexpr int tile = tok * kDecWarps;
    static constexpr int stage = 2 * tok * row;                   // keys and values
    static constexpr int heads = 8 * NT;
    // ring depth: one stage being read, one on its way. A third measured the
    // same, and would leave no room for the joining kernel's blocks to wait
    // on the SM for this kernel's end.
    static constexpr int stages = 2;
    static constexpr int ld = D + 4;                              // row of the joining buffer, floats
    static constexpr size_t ring = (size_t)kDecWarps * stages * stage;
    static constexpr size_t smem = ring + (size_t)kDecWarps * (8 * ld + 16) * sizeof(float);
    // what a CTA of a cluster sends to the first: O and (m, l) of its heads
    static constexpr int sent = heads * (D * 4 + 8);
};

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 16 bytes (or, of `bytes`, 0: zeros) to shared memory. Keys and values are
// read once and leave L2 first: 83.2 us for 85.3 on 507 MB (128 sequences of
// up to 4096 tokens), 40.8 for 42.8 on 217 MB.
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "l"(evict_first())
                 : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
    uint32_t b;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(b) : "r"(a));
    return b;
}
// Two e4m3 values as two fp16 values (exact).
__device__ __forceinline__ uint32_t e4m3_to_half2(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)two));
    return h;
}

// The matrix instruction's 16-bit type: the cache's own, fp16 for e4m3.
template <typename T>
struct MmaType;
template <>
struct MmaType<__nv_bfloat16> {
    static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<uint32_t*>(&h);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t w) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
};
template <>
struct MmaType<__half> {
    static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<uint32_t*>(&h);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t w) {
        return __half22float2(*reinterpret_cast<__half2*>(&w));
    }
};

// The address of a shared variable in CTA `rank` of the cluster, and stores
// there that complete on that CTA's barrier by their bytes.
__device__ __forceinline__ uint32_t peer(const void* local, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(a)
                 : "r"((uint32_t)__cvta_generic_to_shared(local)), "r"(rank));
    return a;
}
__device__ __forceinline__ void send4(uint32_t at, const float4& v, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(at),
                 "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void send2(uint32_t at, const float2& v, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(at),
                 "f"(v.x), "f"(v.y), "r"(bar)
                 : "memory");
}

// Wait for phase 0 of this CTA's barrier that other CTAs' stores complete on;
// false once `limit` SM cycles have passed. Those stores release at cluster
// scope, so the wait acquires there (without a scope it would be the CTA's).
__device__ __forceinline__ bool cluster_wait_bounded(uint32_t bar, long long limit) {
    const auto arrived = [&]() {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], 0;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(bar)
            : "memory");
        return done != 0;
    };
    const long long t0 = clock64();
    while (!arrived())
        if (clock64() - t0 > limit) return false;
    return true;
}

// tanh(z) = 1 - 2 / (1 + e^2z), off by 2^-22 or so; below 1/4, where that
// would be much of the value, its series to z^9 (the term left out is below
// 2^-26 of the value).
__device__ __forceinline__ float tanh_of(float z) {
    const float e = exp2_fast(z * 2.885390082f);
    const float far = 1.0f - __fdividef(2.0f, 1.0f + e);
    const float y = __fmul_rn(z, z);
    float c = fmaf(y, 0.021869489f, -0.053968254f);  // 62/2835, -17/315
    c = fmaf(y, c, 0.13333333f);                     // 2/15
    c = fmaf(y, c, -0.33333333f);
    return fabsf(z) < 0.25f ? fmaf(__fmul_rn(z, y), c, z) : far;
}

// The weight of a part with reference m in a sum with reference `top`. A part
// without a finite score adds nothing, but its NaN.
__device__ __forceinline__ float join_factor(float m, float top) {
    return m == -INFINITY ? (top == -INFINITY ? 1.0f : 0.0f) : exp2_fast(m - top);
}

// A sum of parts (O, m, l), four elements of a head.
struct JoinSum {
    float m = -INFINITY, l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    // Adds N parts.
    template <int N>
    __device__ __forceinline__ void add(const float2 (&ml)[N], const float4 (&v)[N]) {
        float top = m;
#pragma unroll
        for (int i = 0; i < N; ++i) top = fmaxf(top, ml[i].x);
        const float f0 = join_factor(m, top);
        m = top;
        l *= f0;
        o.x *= f0, o.y *= f0, o.z *= f0, o.w *= f0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float f = join_factor(ml[i].x, top);
            l = fmaf(ml[i].y, f, l);
            o.x = fmaf(v[i].x, f, o.x), o.y = fmaf(v[i].y, f, o.y);
            o.z = fmaf(v[i].z, f, o.z), o.w = fmaf(v[i].w, f, o.w);
        }
    }
};

// Four elements of a head's result, and its lse beside the first.
template <typename T>
__device__ __forceinline__ void write_out(const DecodeParams& p, int b, int head, int d, const float4& o, float m,
                                          float l) {
    const float inv = l == 0.0f ? 0.0f : p.vscale / l;
    uint2 w;
    w.x = MmaType<T>::pack(o.x * inv, o.y * inv);
    w.y = MmaType<T>::pack(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + b * p.ots + head * p.ohs + d) = w;
    if (d == 0 && p.lse) p.lse[(int64_t)b * p.heads + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471806f;
}

// A sequence's range of tokens: [lo, n).
__device__ __forceinline__ int2 token_range(const DecodeParams& p, int len) {
    int n = len < 0 ? 0 : len;
    n = n > p.cap_tokens ? p.cap_tokens : n;
    const int lo = p.window > 0 && n > p.window ? n - p.window : 0;
    return make_int2(lo, n);
}
// Its tiles (a run of TOK tokens for each of the CTA's warps, or for the one
// warp) start at lo rounded down to a run, so that 16 tokens of a run never
// cross a page whose size is a multiple of 16.
template <int TOK>
__device__ __forceinline__ int tiles_of(const DecodeParams& p, int2 range) {
    const int n = range.y - (range.x & ~(TOK - 1));
    return p.form == kFormWarps ? (n + TOK - 1) / TOK : (n + TOK * kDecWarps - 1) / (TOK * kDecWarps);
}
template <int TOK>
__device__ __forceinline__ int tiles_of(const DecodeParams& p, int len) {
    return tiles_of<TOK>(p, token_range(p, len));
}

// T: type of q and out. C: matrix type (T, or __half for an e4m3 cache).
// ES: bytes of a cache element. NT: groups of 8 query heads per item.
template <typename T, typename C, int ES, int D, int NT>
__global__ void __launch_bounds__(kDecThreads) decode_kernel(const __grid_constant__ DecodeParams p) {
    using S = DecodeShape<D, ES, NT>;
    constexpr int TOK = S::tok, TILE = S::tile, MT = TOK / 16;
    constexpr int KS = D / 16;           // k-steps of the scores, and row blocks of O^T
    constexpr int CPR = S::row / 16;     // 16-byte chunks per row
    constexpr int NS = S::stages;
    extern __shared__ __align__(128) char s_mem[];
    __shared__ long long s_scan[kDecWarps];
    __shared__ int s_begin[2];
    __shared__ __align__(8) uint64_t s_bar;  // what the cluster's other CTAs send has arrived
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    dependent_start();

    // ---- this CTA's range of tiles, and the sequence it starts in --------
    const int cta = (int)blockIdx.x;
    int grid = 0;
    long long total = 0, t_begin = 0, t_end = 0;
    // Sequences without tokens have no tile; CTA c answers for sequences c, c
    // + grid, ... and counts lengths out of range.
    const auto answer_empty = [&]() {
        for (int e = cta; e < p.B; e += (int)gridDim.x) {
            const int len = p.lens[e];
            const int2 r = token_range(p, len);
            if (threadIdx.x == 0 && (len < 0 || len > p.cap_tokens)) atomicAdd(p.bad, 1u);
            if (r.y > r.x) continue;
            for (int64_t x = threadIdx.x; x < (int64_t)p.heads * (D / 4); x += kDecThreads)
                write_out<T>(p, e, (int)(x / (D / 4)), (int)(x % (D / 4)) * 4, make_float4(0.0f, 0.0f, 0.0f, 0.0f), 0.0f, 0.0f);
        }
    };
    int first_b, first_off;  // first sequence, and the units of its items before ours
    int rank = 0, used = 0;  // place in the cluster, CTAs of it that have tiles
    if (p.form > 0) {
        // one item per cluster; units count from its first
        const int item = cta / p.form;
        rank = cta - item * p.form;
        first_b = item / p.per_seq;
        const int in_seq = item - first_b * p.per_seq;
        const int len = p.lens[first_b];
        const int n = tiles_of<TOK>(p, len);
        const int each = (n + p.form - 1) / p.form;
        used = each > 0 ? (n + each - 1) / each : 0;
        t_begin = min(rank * each, n), t_end = min(rank * each + each, n);
        first_off = in_seq * (n + 1) + (int)t_begin;
        if (rank == 0) {
            if (in_seq == 0 && threadIdx.x == 0 && (len < 0 || len > p.cap_tokens)) atomicAdd(p.bad, 1u);
            if (used == 0) {  // no tokens: zeros
                const int kv = (int)p.d_kv.div((uint32_t)in_seq), h0 = (in_seq - kv * p.per_kv) * S::heads;
                for (int x = threadIdx.x; x < min(p.group - h0, S::heads) * (D / 4); x += kDecThreads)
                    write_out<T>(p, first_b, kv * p.group + h0 + x / (D / 4), x % (D / 4) * 4,
                                 make_float4(0.0f, 0.0f, 0.0f, 0.0f), 0.0f, 0.0f);
            }
        }
        if (rank >= used) return;
        if (used > 1) {
            // the barrier that counts what arrives must be set up before
            // anything is sent: all arrive here, the senders wait later
            if (rank == 0 && threadIdx.x == 0) {
                const uint32_t bar = (uint32_t)__cvta_generic_to_shared(&s_bar);
                mbar_init(bar, 1);
                asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
                const int live = min(p.group - (in_seq - (int)p.d_kv.div((uint32_t)in_seq) * p.per_kv) * S::heads, S::heads);
                mbar_arrive_expect_tx(bar, (uint32_t)((used - 1) * live * (D * 4 + 8)));
            }
            __syncwarp();
            asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        }
    } else if (p.form == kFormWarps) {
        const int item = cta * kDecWarps + warp;
        if (item >= p.B * p.per_seq) return;
        first_b = item / p.per_seq;
        const int in_seq = item - first_b * p.per_seq;
        const int len = p.lens[first_b];
        const int n = tiles_of<TOK>(p, len);
        if (in_seq == 0 && lane == 0 && (len < 0 || len > p.cap_tokens)) atomicAdd(p.bad, 1u);
        if (n == 0) {
            const int kv = (int)p.d_kv.div((uint32_t)in_seq), h0 = (in_seq - kv * p.per_kv) * S::heads;
            for (int x = lane; x < min(p.group - h0, S::heads) * (D / 4); x += 32)
                write_out<T>(p, first_b, kv * p.group + h0 + x / (D / 4), x % (D / 4) * 4,
                             make_float4(0.0f, 0.0f, 0.0f, 0.0f), 0.0f, 0.0f);
            return;
        }
        t_end = n;
        first_off = in_seq * (n + 1);
    } else {
        // Units before each sequence: every thread adds up a run of
        // sequences, one scan over the threads, and the thread in whose run
        // this CTA's place is walks it.
        const auto count = [&](int b) {
            const int tiles = tiles_of<TOK>(p, p.lens[b]);
            return tiles > 0 ? (long long)(tiles + 1) * p.per_seq : 0ll;
        };
        const int run = (p.B + kDecThreads - 1) / kDecThreads;
        const int b_lo = min((int)threadIdx.x * run, p.B), b_hi = min(b_lo + run, p.B);
        long long n = 0;
#pragma unroll 4
        for (int b = b_lo; b < b_hi; ++b) n += count(b);
        long long x = n;  // inclusive scan
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(~0u, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) s_scan[warp] = x;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) {
            if (w < warp) x += s_scan[w];
            total += s_scan[w];
        }
        // not more CTAs than units, so that none in between is without one
        grid = (int)(total < (long long)gridDim.x ? total : (long long)gridDim.x);
        if (threadIdx.x == 0) p.cut[cta] = make_int2(-1, -1);
        if (cta >= grid) {
            answer_empty();
            return;
        }
        t_begin = total * cta / grid, t_end = total * (cta + 1) / grid;
        if (x - n <= t_begin && t_begin < x) {
            long long before = x - n;
            int b = b_lo;
            for (long long m; before + (m = count(b)) <= t_begin; ++b) before += m;
            s_begin[0] = b;
            s_begin[1] = (int)(t_begin - before);
        }
        __syncthreads();
        first_b = s_begin[0], first_off = s_begin[1];
    }

    // ---- the producer: walks the tiles NS stages ahead ------------------
    int p_left = (int)(t_end - t_begin);  // units
    int pb = first_b, p_item, p_tile, p_tiles, p_lo, p_n;
    // On to the first tile of the next item; units are left, so one follows.
    auto next_item = [&]() {
        p_tile = 0;
        if (++p_item < p.per_seq) return;
        p_item = 0;
        int2 r;
        do {
            ++pb;
            r = token_range(p, p.lens[pb]);
        } while (r.y <= r.x);
        p_lo = r.x, p_n = r.y;
        p_tiles = tiles_of<TOK>(p, r);
    };
    {
        const int2 r = token_range(p, p.lens[pb]);
        p_lo = r.x, p_n = r.y;
        p_tiles = tiles_of<TOK>(p, r);
        p_item = first_off / (p_tiles + 1);
        p_tile = first_off - p_item * (p_tiles + 1);
        if (p_tile == p_tiles) {  // the end of an item that another CTA works on
            ++t_begin;
            if (--p_left > 0) next_item();
        }
    }
    // A stage's item, with flags: the last tile of the item in this CTA, the
    // item's last, the item's first. None: -1.
    constexpr int kEnds = (int)0x80000000, kLast = 0x40000000, kFirst = 0x20000000, kItem = 0x1fffffff;
    // whether every 16 tokens of a warp's run lie in one page: then their rows
    // are one base address and a stride (lanes 0 and 16 look the pages up),
    // else every lane below TOK looks up its own token
    const bool one_page = p.page.d % 16 == 0;
    // the next stage to issue: page (already loaded), row, item, valid rows
    int n_page = -1, n_row = 0, n_item = -1, n_kv = 0;
    uint32_t n_mask = 0;
    // Fetch the page numbers of the next tile.
    auto fetch = [&]() {
        n_item = -1;
        n_mask = 0;
        if (p_left <= 0) return;
        const int tok0 = (p_lo & ~(TOK - 1)) + (p.form == kFormWarps ? p_tile * TOK : p_tile * TILE + warp * TOK);
        const int cnt = p_n - tok0, front = p_lo - tok0;
        n_mask = cnt >= 32 ? ~0u : (cnt > 0 ? (1u << cnt) - 1u : 0u);
        if (TOK < 32) n_mask &= (1u << (TOK & 31)) - 1u;
        if (front > 0) n_mask = front >= 32 ? 0u : n_mask & (~0u << front);
        n_kv = (int)p.d_kv.div((uint32_t)p_item);
        if (n_mask != 0) {
            const int tok = tok0 + (one_page ? lane & (TOK - 16) : lane);
            if (one_page ? (n_mask & (0xffffu << (lane & (TOK - 16)))) != 0 : ((n_mask >> lane) & 1u) != 0) {
                const uint32_t page = p.page.div((uint32_t)tok);
                n_row = tok - (int)(page * p.page.d);
                n_page = p.table[(int64_t)pb * p.table_stride + page];
            }
        }
        n_item = pb * p.per_seq + p_item;
        if (p_tile == 0) n_item |= kFirst;
        if (p_left == 1) n_item |= kEnds;
        --p_left;
        if (++p_tile == p_tiles) {
            n_item |= kEnds | kLast;
            if (p_left > 0 && --p_left > 0) next_item();
        }
    };
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(s_mem) + warp * (NS * S::stage);
    auto swizzle = [](int r, int c) {
        return CPR >= 8 ? r * S::row + ((c ^ (r & 7)) << 4) : r * S::row + ((c ^ ((r >> 1) & 3)) << 4);
    };
    constexpr int RPI = 32 / CPR;                  // rows per copy instruction
    constexpr uint32_t FULL = TOK == 32 ? ~0u : (1u << (TOK & 31)) - 1u;
    const int c_row = lane / CPR, c_chunk = lane % CPR;  // the lane's row within an instruction, and its chunk
    const int64_t c_off = (int64_t)c_row * p.cts + c_chunk * 16;
    const int64_t c_step = (int64_t)RPI * p.cts;
    const int64_t v_minus_k = p.v - p.k;
    // Issue the fetched stage into ring slot `slot`; returns the mask of its
    // tokens that count. Rows that do not count are filled with zeros: a
    // masked NaN or infinity must not reach the products.
    auto issue = [&](int slot) -> uint32_t {
        uint32_t mask = n_mask;
        const uint32_t base = ring + slot * S::stage;
        if (mask != 0) {
            if (one_page) {
                // a half whose page is out of range does not count
                const bool half = (mask & (0xffffu << (lane & (TOK - 16)))) != 0;
                const bool bad = half && (uint32_t)n_page >= (uint32_t)p.num_pages;
                if (bad && (lane & 15) == 0 && lane < TOK) atomicAdd(p.bad, 1u);
                const uint32_t fine = __ballot_sync(~0u, !bad);
                mask &= TOK == 32 ? fine : fine & FULL;
                const int64_t off = half && !bad ? (int64_t)n_page * p.cps + (int64_t)n_row * p.cts : 0;
                const char* base_k = p.k + ((int64_t)n_kv * p.chs + c_off);
#pragma unroll
                for (int r = 0; r < TOK / 16; ++r) {
                    const char* src = base_k + __shfl_sync(~0u, off, r * 16);
                    if (((mask >> (r * 16)) & 0xffffu) == 0xffffu) {
#pragma unroll
                        for (int i = 0; i < 16 / RPI; ++i) {
                            const uint32_t dst = base + swizzle(r * 16 + i * RPI + c_row, c_chunk);
                            cp16(dst, src);
                            cp16(dst + TOK * S::row, src + v_minus_k);
                            src += c_step;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 16 / RPI; ++i) {
                            const uint32_t dst = base + swizzle(r * 16 + i * RPI + c_row, c_chunk);
                            const bool in = (mask >> (r * 16 + i * RPI + c_row)) & 1u;
                            cp16(dst, in ? src : p.k, in ? 16u : 0u);
                            cp16(dst + TOK * S::row, in ? src + v_minus_k : p.v, in ? 16u : 0u);
                            src += c_step;
                        }
                    }
                }
            } else {
                int64_t off = -1;
                if ((mask >> lane) & 1u) {
                    if ((uint32_t)n_page < (uint32_t)p.num_pages)
                        off = (int64_t)n_page * p.cps + (int64_t)n_row * p.cts + (int64_t)n_kv * p.chs;
                    else
                        atomicAdd(p.bad, 1u);
                }
                mask = __ballot_sync(~0u, off >= 0);
#pragma unroll 4
                for (int i = 0; i < TOK / RPI; ++i) {
                    const int64_t o = __shfl_sync(~0u, off, i * RPI + c_row);
                    const uint32_t dst = base + swizzle(i * RPI + c_row, c_chunk), bytes = o >= 0 ? 16u : 0u;
                    const char* src = p.k + (o >= 0 ? o + c_chunk * 16 : 0);
                    cp16(dst, src, bytes);
                    cp16(dst + TOK * S::row, src + v_minus_k, bytes);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        return mask;
    };

    // The consumer's item and its queries, loaded as soon as the item is
    // known: for the first one here, for later ones before the joining of the
    // warps of the item before.
    uint32_t qf[NT][KS][2];
    int b = 0, kv = 0, h0 = 0, hn = 0;  // sequence, key head, first head in its group, heads
    int tiles = 0;                      // tiles of the sequence
    auto load_item = [&](int item) {
        b = item / p.per_seq;
        const int in_seq = item - b * p.per_seq;
        kv = (int)p.d_kv.div((uint32_t)in_seq);
        h0 = (in_seq - kv * p.per_kv) * S::heads;
        hn = p.group - h0 < S::heads ? p.group - h0 : S::heads;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const bool live = n * 8 + g < hn;
            const T* q = static_cast<const T*>(p.q) + (int64_t)b * p.qts +
                         (int64_t)(kv * p.group + h0 + n * 8 + g) * p.qhs;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                if constexpr (ES == 2) {
                    qf[n][ks][0] = live ? *reinterpret_cast<const uint32_t*>(q + ks * 16 + 2 * t) : 0u;
                    qf[n][ks][1] = live ? *reinterpret_cast<const uint32_t*>(q + ks * 16 + 8 + 2 * t) : 0u;
                } else {
                    const uint2 w = live ? *reinterpret_cast<const uint2*>(q + ks * 16 + 4 * t) : make_uint2(0u, 0u);
                    qf[n][ks][0] = w.x, qf[n][ks][1] = w.y;
                }
            }
        }
        tiles = tiles_of<TOK>(p, p.lens[b]);
    };
    if (p_left > 0) load_item(pb * p.per_seq + p_item);

    // stages in flight, oldest first
    int f_item[NS];
    uint32_t f_mask[NS];
    fetch();
#pragma unroll
    for (int i = 0; i < NS - 1; ++i) {
        f_item[i] = n_item;
        f_mask[i] = issue(i);
        fetch();
    }
    f_item[NS - 1] = -1;
    f_mask[NS - 1] = 0;

    // ---- the consumer ----------------------------------------------------
    float qs[NT][2];       // score factor of the lane's two heads (columns)
    // O^T from the upper and from the lower half of P: apart for 16-bit
    // caches, whose values can be infinite (a lower half of either sign or 0
    // would turn an infinite sum into NaN); e4m3 has no infinity
    constexpr int LO = ES == 2 ? 1 : 0;
    // P as the sum of two 16-bit values (2^-16 of it, or 2^-22 in fp16): one
    // alone would be as large an error as the rounding of out for values of
    // the cache's type, and an eighth of it for bf16 out of an fp16 product
    // (where the second costs 1.7 us of the 64.6 of the e4m3 batch above).
    float o[1 + LO][NT][KS][4];
    // The softmax's reference, in units of log2, per head: kRoom below the
    // maximum when it was last set. It is set anew only when a score exceeds
    // it by more than `over` (kRoom + kSlack; -inf until the first score that
    // counts), so that most steps need no exchange between lanes. P stays
    // below 2^(kRoom + kSlack): in fp16 the room keeps what is far below the
    // maximum out of the subnormal numbers.
    constexpr float kSlack = 8.0f, kRoom = std::is_same<C, __half>::value ? 7.0f : 0.0f;
    float m[NT][2], over[NT][2], l[NT][2];
    bool fresh = true;
    int slot = 0;
    long long at = t_begin;   // unit of the current step
    long long seg_begin = at;
    bool first_here = false;  // whether the item begins in this CTA
    float* s_join = reinterpret_cast<float*>(s_mem + S::ring);
    float* s_stat = s_join + kDecWarps * 8 * S::ld;  // [warp][8] (m, l)
    // What the first CTA of a cluster is sent: per sender O [heads][D], then
    // (m, l) [heads]. Its own part waits in the ring, which it no longer needs.
    char* s_sent = s_mem + S::smem;
    float4* s_own = reinterpret_cast<float4*>(s_mem);
    float2* s_own_ml = reinterpret_cast<float2*>(s_mem + S::heads * D * 4);

    // The warp's result for head group n, to its rows of the joining buffer.
    auto keep = [&](int n) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) l[n][j] += __shfl_xor_sync(~0u, l[n][j], w);
        float* row = s_join + warp * 8 * S::ld;
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int d = ES == 2 ? i * 16 + g + (e >> 1) * 8 : i * 16 + 2 * g + (e >> 1);
                float x = o[0][n][i][e];
                if (LO && fabsf(x) < INFINITY) x += o[LO][n][i][e];
                row[(2 * t + (e & 1)) * S::ld + d] = x;
            }
        if (g == 0) {
            float* st = s_stat + (warp * 8 + 2 * t) * 2;
            st[0] = over[n][0] > 0.0f ? m[n][0] : -INFINITY, st[1] = l[n][0];
            st[2] = over[n][1] > 0.0f ? m[n][1] : -INFINITY, st[3] = l[n][1];
        }
    };

    for (; f_item[0] != -1; ++at) {
        asm volatile("cp.async.wait_group %0;" ::"n"(NS - 2) : "memory");
        __syncwarp();
        {
            int issue_slot = slot + NS - 1;
            if (issue_slot >= NS) issue_slot -= NS;
            f_item[NS - 1] = n_item;
            f_mask[NS - 1] = issue(issue_slot);
            fetch();
        }
        const bool ends = (f_item[0] & kEnds) != 0;
        const uint32_t mask = f_mask[0];

        if (fresh) {
            fresh = false;
            seg_begin = at;
            first_here = (f_item[0] & kFirst) != 0;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                qs[n][0] = qs[n][1] = p.score;
                if constexpr (ES == 1) {
                    // q enters an fp16 product: times a power of two that
                    // brings the head's largest finite value to [2^13, 2^14),
                    // which is exact for what is within 2^-28 of it (beside an
                    // infinity too: one that a large value became would meet
                    // it with either sign)
                    const auto size = [](float x) { return fabsf(x) < INFINITY ? fabsf(x) : 0.0f; };
                    float big = 0.0f;
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        const float2 x = MmaType<T>::unpack(qf[n][ks][0]), y = MmaType<T>::unpack(qf[n][ks][1]);
                        big = fmaxf(big, fmaxf(fmaxf(size(x.x), size(x.y)), fmaxf(size(y.x), size(y.y))));
                    }
                    big = fmaxf(big, __shfl_xor_sync(~0u, big, 1));
                    big = fmaxf(big, __shfl_xor_sync(~0u, big, 2));
                    int e = (int)(__float_as_uint(big) >> 23) - 127 - 13;  // floor(log2) - 13
                    if (big == 0.0f) e = 0;
                    // 2^-e in two factors: each is a normal number
                    const float f0 = __uint_as_float((uint32_t)(127 - e / 2) << 23);
                    const float f1 = __uint_as_float((uint32_t)(127 - (e - e / 2)) << 23);
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        const float2 x = MmaType<T>::unpack(qf[n][ks][0]), y = MmaType<T>::unpack(qf[n][ks][1]);
                        qf[n][ks][0] = MmaType<C>::pack(x.x * f0 * f1, x.y * f0 * f1);
                        qf[n][ks][1] = MmaType<C>::pack(y.x * f0 * f1, y.y * f0 * f1);
                    }
                    // the lane's columns are heads 2t and 2t + 1: their
                    // factors are with the lanes whose g is that head
                    const int e0 = __shfl_sync(~0u, e, (2 * t) * 4), e1 = __shfl_sync(~0u, e, (2 * t + 1) * 4);
                    qs[n][0] = ldexpf(p.score, e0);
                    qs[n][1] = ldexpf(p.score, e1);
                }
                m[n][0] = m[n][1] = 0.0f;
                over[n][0] = over[n][1] = -INFINITY;
                l[n][0] = l[n][1] = 0.0f;
#pragma unroll
                for (int u = 0; u <= LO; ++u)
#pragma unroll
                    for (int i = 0; i < KS; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[u][n][i][e] = 0.0f;
            }
        }

        if (mask != 0) {  // the same for the whole warp
            const uint32_t sk = ring + slot * S::stage, sv = sk + TOK * S::row;
            float s[NT][MT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[n][i][e] = 0.0f;
            // S^T = K Q^T
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int r = i * 16 + (lane & 15);
#pragma unroll
                for (int c = 0; c < CPR; c += 2) {
                    uint32_t a[4];
                    ldsm4(a, sk + swizzle(r, c + (lane >> 4)));
                    if constexpr (ES == 2) {
#pragma unroll
                        for (int n = 0; n < NT; ++n) MmaType<C>::mma(s[n][i], a, qf[n][c / 2][0], qf[n][c / 2][1]);
                    } else {
                        // chunk = 16 elements; a lane's word is d = 4t..4t+3
                        // of its row, the order qf was loaded in
                        uint32_t x[4] = {e4m3_to_half2(a[0]), e4m3_to_half2(a[1]), e4m3_to_half2(a[0] >> 16),
                                         e4m3_to_half2(a[1] >> 16)};
                        uint32_t y[4] = {e4m3_to_half2(a[2]), e4m3_to_half2(a[3]), e4m3_to_half2(a[2] >> 16),
                                         e4m3_to_half2(a[3] >> 16)};
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            MmaType<C>::mma(s[n][i], x, qf[n][c][0], qf[n][c][1]);
                            MmaType<C>::mma(s[n][i], y, qf[n][c + 1][0], qf[n][c + 1][1]);
                        }
                    }
                }
            }
            // scores against the reference
            bool rises = false;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (p.inv_cap != 0.0f) {
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            s[n][i][e] = fmaf(p.cap2, tanh_of(s[n][i][e] * qs[n][e & 1] * p.inv_cap), -m[n][e & 1]);
                        }
                } else {
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[n][i][e] = fmaf(s[n][i][e], qs[n][e & 1], -m[n][e & 1]);
                }
                if (mask != FULL) {
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (!((mask >> (i * 16 + g + (e >> 1) * 8)) & 1u)) s[n][i][e] = -INFINITY;
                }
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) rises |= s[n][i][e] > over[n][e & 1];
            }
            if (__any_sync(~0u, rises)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float top = -INFINITY;
#pragma unroll
                        for (int i = 0; i < MT; ++i) top = fmaxf(top, fmaxf(s[n][i][j], s[n][i][j + 2]));
#pragma unroll
                        for (int w = 4; w < 32; w <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, w));
                        if (top > over[n][j]) {
                            top -= kRoom;
                            const float f = over[n][j] == -INFINITY ? 1.0f : exp2_fast(-top);
                            m[n][j] += top;
                            over[n][j] = kRoom + kSlack;
                            l[n][j] *= f;
#pragma unroll
                            for (int i = 0; i < MT; ++i) s[n][i][j] -= top, s[n][i][j + 2] -= top;
#pragma unroll
                            for (int u = 0; u <= LO; ++u)
#pragma unroll
                                for (int i = 0; i < KS; ++i) o[u][n][i][j] *= f, o[u][n][i][j + 2] *= f;
                        }
                    }
            }
            uint32_t ph[NT][MT][2], pl[NT][MT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const float p0 = exp2_fast(s[n][i][0]), p1 = exp2_fast(s[n][i][1]);
                    const float p2 = exp2_fast(s[n][i][2]), p3 = exp2_fast(s[n][i][3]);
                    l[n][0] += p0 + p2;
                    l[n][1] += p1 + p3;
                    const uint32_t h0 = MmaType<C>::pack(p0, p1), h1 = MmaType<C>::pack(p2, p3);
                    ph[n][i][0] = transpose8(h0);
                    ph[n][i][1] = transpose8(h1);
                    const float2 u0 = MmaType<C>::unpack(h0), u1 = MmaType<C>::unpack(h1);
                    pl[n][i][0] = transpose8(MmaType<C>::pack(p0 - u0.x, p1 - u0.y));
                    pl[n][i][1] = transpose8(MmaType<C>::pack(p2 - u1.x, p3 - u1.y));
                }
            // O^T += V^T P^T
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                // matrices of ldmatrix: (tokens 0-7, first chunk), (tokens
                // 0-7, second), (tokens 8-15, first), (tokens 8-15, second)
                const int r = i * 16 + (lane >> 4) * 8 + (lane & 7);
#pragma unroll
                for (int c = 0; c < CPR; c += 2) {
                    uint32_t a[4];
                    ldsm4t(a, sv + swizzle(r, c + ((lane >> 3) & 1)));
                    if constexpr (ES == 2) {
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            MmaType<C>::mma(o[0][n][c / 2], a, ph[n][i][0], ph[n][i][1]);
                            MmaType<C>::mma(o[LO][n][c / 2], a, pl[n][i][0], pl[n][i][1]);
                        }
                    } else {
                        // a word holds d = 2g, 2g + 1 of two tokens: row g of
                        // the product is d = 2g, row g + 8 is d = 2g + 1
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const uint32_t lo = __byte_perm(a[half], 0, 0x3120), hi = __byte_perm(a[half + 2], 0, 0x3120);
                            uint32_t x[4] = {e4m3_to_half2(lo), e4m3_to_half2(lo >> 16), e4m3_to_half2(hi),
                                             e4m3_to_half2(hi >> 16)};
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                MmaType<C>::mma(o[0][n][c + half], x, ph[n][i][0], ph[n][i][1]);
                                MmaType<C>::mma(o[0][n][c + half], x, pl[n][i][0], pl[n][i][1]);
                            }
                        }
                    }
                }
            }
        }

        if (ends && p.form == kFormWarps) {  // the warp's one item is done
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                keep(n);
                __syncwarp();
                for (int x = lane; x < 8 * (D / 4); x += 32) {
                    const int h = x / (D / 4), d = (x - h * (D / 4)) * 4;
                    if (n * 8 + h < hn)
                        write_out<T>(p, b, kv * p.group + h0 + n * 8 + h, d,
                                     *reinterpret_cast<const float4*>(s_join + (warp * 8 + h) * S::ld + d),
                                     s_stat[(warp * 8 + h) * 2], s_stat[(warp * 8 + h) * 2 + 1]);
                }
                __syncwarp();
            }
            return;
        }
        if (ends) {  // the same for the whole CTA: join the warps
            fresh = true;
            // what the join needs of this item, before the next one's loads
            const int item = f_item[0] & kItem, it_tiles = tiles, it_b = b, it_hn = hn;
            const int it_head = kv * p.group + h0;
            const bool whole = first_here && (f_item[0] & kLast) != 0;
            if (f_item[0] & kLast) ++at;
            if (f_item[1] != -1) load_item(f_item[1] & kItem);
            if (rank > 0) {  // rank 0 is set up
                __syncwarp();
                asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
            }
            const int piece = 2 * cta + (first_here ? 1 : 0);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                __syncthreads();  // the buffer's last readers are done
                keep(n);
                __syncthreads();
                for (int x = threadIdx.x; x < 8 * (D / 4); x += kDecThreads) {
                    const int h = x / (D / 4), d = (x - h * (D / 4)) * 4;
                    if (n * 8 + h >= it_hn) continue;
                    float big = -INFINITY, sum = 0.0f;
#pragma unroll
                    for (int w = 0; w < kDecWarps; ++w) big = fmaxf(big, s_stat[(w * 8 + h) * 2]);
                    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                    for (int w = 0; w < kDecWarps; ++w) {
                        const float mw = s_stat[(w * 8 + h) * 2];
                        const float f = join_factor(mw, big);
                        const float4 v = *reinterpret_cast<const float4*>(s_join + (w * 8 + h) * S::ld + d);
                        acc.x = fmaf(v.x, f, acc.x), acc.y = fmaf(v.y, f, acc.y);
                        acc.z = fmaf(v.z, f, acc.z), acc.w = fmaf(v.w, f, acc.w);
                        sum = fmaf(s_stat[(w * 8 + h) * 2 + 1], f, sum);
                    }
                    const int slot_h = n * 8 + h;
                    if (rank > 0) {
                        const uint32_t at = peer(s_sent + (rank - 1) * S::sent, 0), bar = peer(&s_bar, 0);
                        send4(at + (slot_h * D + d) * 4, acc, bar);
                        if (d == 0) send2(at + S::heads * D * 4 + slot_h * 8, make_float2(big, sum), bar);
                    } else if (used > 1) {
                        s_own[(slot_h * D + d) / 4] = acc;
                        if (d == 0) s_own_ml[slot_h] = make_float2(big, sum);
                    } else if (whole) {
                        write_out<T>(p, it_b, it_head + n * 8 + h, d, acc, big, sum);
                    } else {
                        const int64_t at_head = (int64_t)piece * S::heads + n * 8 + h;
                        *reinterpret_cast<float4*>(p.part + at_head * D + d) = acc;
                        if (d == 0) p.stat[at_head] = make_float2(big, sum);
                    }
                }
            }
            if (p.form == kFormDealt && first_here && !whole && threadIdx.x == 0) {
                // the CTA that holds the item's last tile: the largest c with
                // total c / grid <= that unit
                const long long last = seg_begin + it_tiles - 1;
                const int c1 = (int)(((last + 1) * grid - 1) / total);
                p.cut[cta] = make_int2(item, c1);
            }
        }

        // the next stage becomes the oldest
#pragma unroll
        for (int i = 0; i + 1 < NS; ++i) f_item[i] = f_item[i + 1], f_mask[i] = f_mask[i + 1];
        if (++slot == NS) slot = 0;
        __syncwarp();
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (p.form == kFormDealt) answer_empty();
    if (rank > 0 || used <= 1) return;

    // ---- the first CTA of a cluster joins what the others have sent -------
    __syncthreads();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    const uint32_t bar = (uint32_t)__cvta_generic_to_shared(&s_bar);
    if (!cluster_wait_bounded(bar, kBulkSpinLimit)) {
        // never seen: count it, give what is on its way as long again, and
        // leave without an answer
        (void)cluster_wait_bounded(bar, kBulkSpinLimit);
        if (threadIdx.x == 0) atomicAdd(p.timeouts, 1u);
        return;
    }
    for (int x = threadIdx.x; x < hn * (D / 4); x += kDecThreads) {
        const int h = x / (D / 4), d = (x - h * (D / 4)) * 4;
        JoinSum s;
        s.m = s_own_ml[h].x, s.l = s_own_ml[h].y, s.o = s_own[(h * D + d) / 4];
        for (int r0 = 1; r0 < used; r0 += 4) {
            float2 ml[4];
            float4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const char* part = s_sent + (r0 + i - 1) * S::sent;
                const bool in = r0 + i < used;
                ml[i] = in ? reinterpret_cast<const float2*>(part + S::heads * D * 4)[h] : make_float2(-INFINITY, 0.0f);
                v[i] = in ? *reinterpret_cast<const float4*>(part + (h * D + d) * 4) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
            s.add(ml, v);
        }
        write_out<T>(p, first_b, kv * p.group + h0 + h, d, s.o, s.m, s.l);
    }
}

// Adds up the pieces of the items that were cut; what it costs is latency.
// Items in up to kFewPieces pieces: block c takes the one that begins in CTA
// c, a thread per four elements of a head. Items in more: a block per query
// head, whose threads are GROUPS groups of D / 4, each taking every GROUPS-th
// piece, four loads at a time. At most one of those begins in any kFewPieces
// CTAs in a row, so grid / kFewPieces blocks per head are enough.
constexpr int kJoinThreads = 512;
constexpr int kFewPieces = 8;

// Adds pieces c, c + step, ... up to `last` of the item that begins in CTA
// `first`; element d of head h.
template <int D, int HEADS>
__device__ __forceinline__ void gather(const DecodeParams& p, JoinSum& sum, int first, int c, int last, int step, int h,
                                       int d) {
    for (; c <= last; c += 4 * step) {
        float2 ml[4];
        float4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at_c = c + i * step;
            ml[i] = make_float2(-INFINITY, 0.0f);
            v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (at_c <= last) {
                const int64_t at = (int64_t)(2 * at_c + (at_c == first ? 1 : 0)) * HEADS + h;
                ml[i] = p.stat[at];
                v[i] = *reinterpret_cast<const float4*>(p.part + at * D + d);
            }
        }
        sum.add(ml, v);
    }
}

template <typename T, int D, int HEADS>
__global__ void __launch_bounds__(kJoinThreads) decode_join_kernel(const __grid_constant__ DecodeParams p) {
    constexpr int LANES = D / 4, GROUPS = kJoinThreads / LANES;
    __shared__ float4 s_o[GROUPS][LANES];
    __shared__ float2 s_ml[GROUPS];
    dependent_start();
    const int group = threadIdx.x / LANES, d = (threadIdx.x - group * LANES) * 4;
    int first = (int)blockIdx.x, one_head = -1;
    int2 cut;
    if (first < p.grid) {
        cut = p.cut[first];
        if (cut.x < 0 || cut.y - first >= kFewPieces) return;
    } else {
        const int heads = p.group < HEADS ? p.group : HEADS;
        const int j = (first - p.grid) / heads;
        one_head = first - p.grid - j * heads;
        first = -1;
#pragma unroll
        for (int i = 0; i < kFewPieces; ++i) {
            const int c = j * kFewPieces + i;
            if (c < p.grid) {
                const int2 x = p.cut[c];
                if (x.x >= 0 && x.y - c >= kFewPieces) first = c, cut = x;
            }
        }
        if (first < 0) return;
    }
    const int b = cut.x / p.per_seq, in_seq = cut.x - b * p.per_seq;
    const int kv = in_seq / p.per_kv, h0 = (in_seq - kv * p.per_kv) * HEADS;
    const int live = p.group - h0 < HEADS ? p.group - h0 : HEADS;
    if (one_head < 0) {
        for (int h = group; h < live; h += GROUPS) {
            JoinSum s;
            gather<D, HEADS>(p, s, first, first, cut.y, 1, h, d);
            write_out<T>(p, b, kv * p.group + h0 + h, d, s.o, s.m, s.l);
        }
        return;
    }
    if (one_head >= live) return;
    JoinSum s;
    gather<D, HEADS>(p, s, first, first + group, cut.y, GROUPS, one_head, d);
    s_o[group][d / 4] = s.o;
    if (d == 0) s_ml[group] = make_float2(s.m, s.l);
    __syncthreads();
    if (group != 0) return;
    float2 ml[GROUPS];
    float4 v[GROUPS];
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) ml[i] = s_ml[i], v[i] = s_o[i][d / 4];
    JoinSum all;
    all.add(ml, v);
    write_out<T>(p, b, kv * p.group + h0 + one_head, d, all.o, all.m, all.l);
}

// ---------------------------------------------------------------------------

constexpr int kDecStaticSmem = 256;  // upper bound of the kernel's __shared__ variables

struct DecodeKernels {
    void (*main)(DecodeParams);
    void (*join)(DecodeParams);
    int tile;
    size_t smem, sent;  // shared memory, and what each sender of a cluster adds to it
};

template <typename T, typename C, int ES, int D, int NT>
DecodeKernels decode_kernels_of() {
    using S = DecodeShape<D, ES, NT>;
    return {decode_kernel<T, C, ES, D, NT>, decode_join_kernel<T, D, 8 * NT>, S::tile, S::smem, S::sent};
}

template <typename T>
bool decode_kernels_t(int head_dim, bool e4m3, int nt, DecodeKernels* out) {
#define ARF_DECODE(D_, NT_)                                                   \
    if (head_dim == D_ && nt == NT_) {                                        \
        *out = e4m3 ? decode_kernels_of<T, __half, 1, D_, NT_>() : decode_kernels_of<T, T, 2, D_, NT_>(); \
        return true;                                                          \
    }
    ARF_DECODE(64, 1)
    ARF_DECODE(64, 2)
    ARF_DECODE(128, 1)
    ARF_DECODE(128, 2)
    ARF_DECODE(256, 1)
#undef ARF_DECODE
    return false;
}

bool decode_kernels_bf16(int head_dim, bool e4m3, int nt, DecodeKernels* out);
bool decode_kernels_fp16(int head_dim, bool e4m3, int nt, DecodeKernels* out);

}  // namespace arf
