// arf_rotary.cu: rotary positions, alone and fused with the append of keys
// and values to the paged cache.
//
// Mathematics. Pair i of a head at position p is the complex number
// (a + ib) times m exp(2 pi i f_i p), f_i turns per position. f_i is a 64-bit
// fixed-point fraction of a turn, so f_i * p modulo 2^64 is one integer
// multiplication that drops whole turns exactly. Its upper 32 bits give the
// nearest quarter turn and a rest of at most an eighth, whose sine and cosine
// are short Taylor polynomials. No 64-bit float instruction is needed at any
// position, and what a far one's angle is off by is the table's own error, the
// frequencies' in binary64 (2^-53 of the angle, or a few of those).
//
// What bounds it. About 1 flop per byte: HBM for prompts, launch latency for
// decode steps. Split: a lane of a block owns one unit of a token's heads
// (the two 16-byte chunks of a head that hold 8 pairs, or two chunks that are
// only copied), the block's warps own groups of HPT heads of q, of k or of v.
// A thread issues all its loads; while they are under way each warp takes two
// of the 8 cosines and sines of every lane's unit, and the four warps share
// them through shared memory. HPT is kManyHeads for many tokens and 1 where
// that would leave SMs without threads. Measured, in a graph: 26.1 us for 8191
// tokens of 32 + 8 heads of 128, half rotated, fp16 (6.4 TB/s; with every
// thread taking its own 8 sines and four heads 28.3, a block per token with a
// table of sines 37.2); 11.3 us for the append of 5851 tokens of 16 + 2 x 4
// heads (6.3 TB/s), 11.2 to e4m3 pages (5.9 TB/s); 1.9 us for 128 tokens of 16 + 4.
#include <algorithm>
#include <climits>

#include "arf_attn.cuh"
#include "arf_kernels.cuh"

namespace arf {
namespace {

constexpr int kRotWarps = 4;  // 8 / kRotWarps pairs of a unit per warp
constexpr int kRotThreads = 32 * kRotWarps;
constexpr int kManyHeads = 2;  // heads per thread for many tokens

struct RotSegment {  // q or k: [T, heads, D] read and written
    const unsigned short* in;
    unsigned short* out;
    int64_t its, ihs, ots, ohs;
};

struct RotParams {
    const uint64_t* turns;
    const int32_t* pos;
    const int64_t* slots;  // null without a cache
    float mag;
    int64_t T;
    int D, rot, interleaved;
    int q_heads, k_heads;
    bool q_in_place, k_in_place;
    RotSegment q, k;
    const unsigned short* v;
    int64_t vts, vhs;
    char* ck;         // cache
    char* cv;
    int64_t cps, cts, chs;
    int64_t num_slots;
    float kinv, vinv;
    unsigned int* bad;
    int rot_units;              // units of a head that rotate
    int q_groups, k_groups;     // groups of HPT heads; v has as many as k
    int groups;                 // of all of q, k and v
    FastDiv units;              // units per head
    FastDiv page;
};

template <typename T>
struct Io;
template <>
struct Io<__nv_bfloat16> {
    static __device__ __forceinline__ float get(unsigned short h) { return __uint_as_float((uint32_t)h << 16); }
    static __device__ __forceinline__ unsigned short put(float f) {
        return __bfloat16_as_ushort(__float2bfloat16_rn(f));
    }
};
template <>
struct Io<__half> {
    static __device__ __forceinline__ float get(unsigned short h) { return __half2float(__ushort_as_half(h)); }
    static __device__ __forceinline__ unsigned short put(float f) { return __half_as_ushort(__float2half_rn(f)); }
};

// Round to e4m3, saturating at 448; NaN stays NaN.
__device__ __forceinline__ unsigned char e4m3(float f) {
    return (unsigned char)__nv_cvt_float_to_fp8(f, __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint2 e4m3x8(const float f[8], float inv) {
    uint32_t w[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(f[4 * j], inv), __fmul_rn(f[4 * j + 1], inv)),
                                                     __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(
            make_float2(__fmul_rn(f[4 * j + 2], inv), __fmul_rn(f[4 * j + 3], inv)), __NV_SATFINITE, __NV_E4M3);
        w[j] = lo | (hi << 16);
    }
    return make_uint2(w[0], w[1]);
}

// Sine and cosine of a 2^-32 turns. With q quarter turns taken off, |x| <= pi
// / 4: the first terms left out of the Taylor series are x^11 / 11! < 2^-29
// and x^10 / 10! < 2^-25, and x is off by 2^-24 of itself twice. Measured
// against sincospif on the whole angle when every thread took 8 of them (T =
// 8191, 40 heads of 128, half rotated, fp16): 28.5 us for 29.5, and closer to
// the exact angle.
__device__ __forceinline__ void sincos_turns(uint32_t a, float* sn, float* cs) {
    const uint32_t q = (a + 0x20000000u) >> 30;
    const float x = __fmul_rn((float)(int32_t)(a - (q << 30)), 1.4629180792671596e-09f);  // 2 pi / 2^32
    const float z = __fmul_rn(x, x);
    float s = fmaf(z, 2.7557319e-06f, -1.9841270e-04f);  // 1/9!, -1/7!
    s = fmaf(z, s, 8.3333333e-03f);                      // 1/5!
    s = fmaf(z, s, -1.6666667e-01f);                     // -1/3!
    s = fmaf(__fmul_rn(x, z), s, x);
    float c = fmaf(z, 2.4801587e-05f, -1.3888889e-03f);  // 1/8!, -1/6!
    c = fmaf(z, c, 4.1666667e-02f);                      // 1/4!
    c = fmaf(z, c, -0.5f);
    c = fmaf(z, c, 1.0f);
    // quarter turns: (s, c), (c, -s), (-s, -c), (-c, s)
    const float u = q & 1u ? c : s, v = q & 1u ? s : c;
    *sn = __uint_as_float(__float_as_uint(u) ^ ((q & 2u) << 30));
    *cs = __uint_as_float(__float_as_uint(v) ^ (((q + 1u) & 2u) << 30));
}

// One unit of one head: two pieces of E elements.
template <int E>
struct Pieces;
template <>
struct Pieces<8> {
    uint4 a, b;
    // ONCE: what is read is not read again and leaves L2 first
    template <bool ONCE>
    static __device__ __forceinline__ uint4 get(const unsigned short* p) {
        if constexpr (ONCE) return ld_hint(reinterpret_cast<const uint4*>(p), evict_first());
        return *reinterpret_cast<const uint4*>(p);
    }
    template <bool ONCE>
    __device__ __forceinline__ void load(const unsigned short* p, int e0, int e1, bool second) {
        a = get<ONCE>(p + e0);
        if (second) b = get<ONCE>(p + e1);
    }
    template <typename T>
    __device__ __forceinline__ void widen(float x[8], float y[8]) const {
        Pack8<T>::widen(a, x);
        Pack8<T>::widen(b, y);
    }
    template <typename T>
    static __device__ __forceinline__ void store(char* p, const float x[8]) {
        *reinterpret_cast<uint4*>(p) = Pack8<T>::narrow(x);
    }
    static __device__ __forceinline__ void store8(char* p, const float x[8], float inv) {
        *reinterpret_cast<uint2*>(p) = e4m3x8(x, inv);
    }
    static __device__ __forceinline__ void copy(char* p, const uint4& v) { *reinterpret_cast<uint4*>(p) = v; }
};
template <>
struct Pieces<1> {
    unsigned short a, b;
    template <bool ONCE>
    __device__ __forceinline__ void load(const unsigned short* p, int e0, int e1, bool second) {
        a = p[e0];
        b = second ? p[e1] : (unsigned short)0;
    }
    template <typename T>
    __device__ __forceinline__ void widen(float x[1], float y[1]) const {
        x[0] = Io<T>::get(a);
        y[0] = Io<T>::get(b);
    }
    template <typename T>
    static __device__ __forceinline__ void store(char* p, const float x[1]) {
        *reinterpret_cast<unsigned short*>(p) = Io<T>::put(x[0]);
    }
    static __device__ __forceinline__ void store8(char* p, const float x[1], float inv) {
        *reinterpret_cast<unsigned char*>(p) = e4m3(__fmul_rn(x[0], inv));
    }
    static __device__ __forceinline__ void copy(char* p, unsigned short v) {
        *reinterpret_cast<unsigned short*>(p) = v;
    }
};

// T: I/O type. E: elements per piece, 8 (16-byte vectors) or 1. HPT: heads
// per thread. APPEND: keys and values go to the cache, whose elements are CB
// bytes.
template <typename T, int E, int HPT, bool APPEND, int CB>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const __grid_constant__ RotParams p) {
    dependent_start();
    // lane -> (token, unit); warp -> group of heads
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t first = (int64_t)blockIdx.x * 32;
    const int64_t t_first = first < (1ll << 31) ? (int64_t)p.units.div((uint32_t)first) : first / p.units.d;
    const uint32_t x_unit = (uint32_t)(first - t_first * p.units.d) + (uint32_t)lane;
    const uint32_t dt = p.units.div(x_unit), u = x_unit - dt * p.units.d;
    const int64_t t = t_first + dt;
    int group = (int)blockIdx.y * kRotWarps + warp;
    const bool live = t < p.T && group < p.groups;

    // the group's heads: where they are read and written
    const unsigned short* in = nullptr;
    char* out = nullptr;
    int64_t ihs = 0, ohs = 0;
    int n = 0;
    bool in_cache = false, rotates = (int)u < p.rot_units, copies = true;
    float inv = 1.0f;
    if (!live) {
        copies = rotates = false;
    } else if (group < p.q_groups) {
        const int h = group * HPT;
        n = p.q_heads - h;
        in = p.q.in + t * p.q.its + h * p.q.ihs;
        ihs = p.q.ihs;
        out = reinterpret_cast<char*>(p.q.out + t * p.q.ots + h * p.q.ohs);
        ohs = p.q.ohs * 2;
        copies = !p.q_in_place;
    } else {
        group -= p.q_groups;
        const bool is_v = group >= p.k_groups;
        if (is_v) group -= p.k_groups;
        const int h = group * HPT;
        n = p.k_heads - h;
        if (is_v) {
            in = p.v + t * p.vts + h * p.vhs;
            ihs = p.vhs;
        } else {
            in = p.k.in + t * p.k.its + h * p.k.ihs;
            ihs = p.k.ihs;
        }
        if constexpr (APPEND) {
            int64_t slot = p.slots[t];
            if (slot >= p.num_slots) {
                if (!is_v && group == 0 && u == 0) atomicAdd(p.bad, 1u);
                slot = -1;
            }
            if (slot < 0) n = 0;  // nothing to write
            const int64_t page = slot < 0 ? 0 : (slot < (1ll << 31) ? (int64_t)p.page.div((uint32_t)slot) : slot / p.page.d);
            const int64_t at = slot < 0 ? 0 : page * p.cps + (slot - page * p.page.d) * p.cts + h * p.chs;
            out = (is_v ? p.cv : p.ck) + at * CB;
            ohs = p.chs * CB;
            inv = is_v ? p.vinv : p.kinv;
            in_cache = true;
            rotates = rotates && !is_v;
        } else {
            out = reinterpret_cast<char*>(p.k.out + t * p.k.ots + h * p.k.ohs);
            ohs = p.k.ohs * 2;
            copies = !p.k_in_place;
        }
    }
    if (!rotates && !copies) n = 0;
    if (n > HPT) n = HPT;
    const int pair = (int)u * E;
    int e0, e1;
    bool second = true;
    if (rotates) {
        e0 = p.interleaved ? 2 * pair : pair;
        e1 = p.interleaved ? e0 + E : pair + p.rot / 2;
    } else {
        // units of a head tile it in order where nothing rotates
        e0 = 2 * pair;
        e1 = e0 + E;
        second = e1 < p.D;
    }
    // An append's inputs have served when it is done (11.3 us for 11.7 at the
    // 5851 tokens above); queries and keys on their own may be read again.
    Pieces<E> w[HPT];
#pragma unroll
    for (int i = 0; i < HPT; ++i)
        if (i < n) w[i].template load<APPEND>(in + i * ihs, e0, e1, second);

    // the unit's cosines and sines
    float cs[E], sn[E];
    const bool turns = t < p.T && (int)u < p.rot_units;  // the same in every warp
    const auto one = [&](int i, float* c, float* s) {
        const uint64_t a = p.turns[pair + i] * (uint64_t)(int64_t)p.pos[t];
        sincos_turns((uint32_t)(a >> 32), s, c);
        *c = __fmul_rn(*c, p.mag);
        *s = __fmul_rn(*s, p.mag);
    };
    if constexpr (E == 1) {
        if (turns) one(0, &cs[0], &sn[0]);
    } else {
        __shared__ float4 s_cs[kRotWarps][32];  // (cosine, sine) of two pairs
        static_assert(E == 2 * kRotWarps, "two pairs per warp");
        if (turns) {
            float4 v;
            one(2 * warp, &v.x, &v.y);
            one(2 * warp + 1, &v.z, &v.w);
            s_cs[warp][lane] = v;
        }
        __syncthreads();
        if (turns) {
#pragma unroll
            for (int i = 0; i < kRotWarps; ++i) {
                const float4 v = s_cs[i][lane];
                cs[2 * i] = v.x, sn[2 * i] = v.y, cs[2 * i + 1] = v.z, sn[2 * i + 1] = v.w;
            }
        }
    }

    if (rotates) {
#pragma unroll
        for (int i = 0; i < HPT; ++i) {
            if (i >= n) break;
            float x[E], y[E];
            w[i].template widen<T>(x, y);
            if (E > 1 && p.interleaved) {
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    float* z = 2 * j < E ? x + 2 * j : y + (2 * j - E);
                    const float re = z[0], im = z[1 % E];
                    z[0] = fmaf(re, cs[j], -__fmul_rn(im, sn[j]));
                    z[1 % E] = fmaf(re, sn[j], __fmul_rn(im, cs[j]));
                }
            } else {
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    const float re = x[j], im = y[j];
                    x[j] = fmaf(re, cs[j], -__fmul_rn(im, sn[j]));
                    y[j] = fmaf(re, sn[j], __fmul_rn(im, cs[j]));
                }
            }
            char* o = out + i * ohs;
            if (APPEND && CB == 1 && in_cache) {
                Pieces<E>::store8(o + e0, x, inv);
                Pieces<E>::store8(o + e1, y, inv);
            } else {
                Pieces<E>::template store<T>(o + e0 * 2, x);
                Pieces<E>::template store<T>(o + e1 * 2, y);
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < HPT; ++i) {
        if (i >= n) break;
        char* o = out + i * ohs;
        if (APPEND && CB == 1 && in_cache) {
            float x[E], y[E];
            w[i].template widen<T>(x, y);
            Pieces<E>::store8(o + e0, x, inv);
            if (second) Pieces<E>::store8(o + e1, y, inv);
        } else {  // a copied 16-bit value keeps its bits (NaN payloads too)
            Pieces<E>::copy(o + e0 * 2, w[i].a);
            if (second) Pieces<E>::copy(o + e1 * 2, w[i].b);
        }
    }
}

using RotFn = void (*)(RotParams);

template <typename T, int E, int HPT>
RotFn rot_fn_of(bool append, int cb) {
    if (!append) return rotary_kernel<T, E, HPT, false, 2>;
    return cb == 1 ? rotary_kernel<T, E, HPT, true, 1> : rotary_kernel<T, E, HPT, true, 2>;
}
template <typename T>
RotFn rot_fn(bool vec, bool many, bool append, int cb) {
    if (!vec) return rot_fn_of<T, 1, 1>(append, cb);
    return many ? rot_fn_of<T, 8, kManyHeads>(append, cb) : rot_fn_of<T, 8, 1>(append, cb);
}

bool vec_heads(const arf_heads_t* t) {
    return t->token_stride % 8 == 0 && t->head_stride % 8 == 0 && is_aligned(t->data, 16);
}
RotSegment segment(const arf_heads_t* in, const arf_heads_t* out) {
    RotSegment s = {};
    s.in = static_cast<const unsigned short*>(in->data);
    s.its = in->token_stride, s.ihs = in->head_stride;
    if (out) {
        s.out = static_cast<unsigned short*>(out->data);
        s.ots = out->token_stride, s.ohs = out->head_stride;
    }
    return s;
}

arf_status_t check_pair(const arf_heads_t* in, const arf_heads_t* out, int64_t T, int D) {
    arf_status_t st = check_heads(in, T);
    if (st == ARF_OK) st = check_heads(out, T);
    if (st != ARF_OK) return st;
    if (in->heads != out->heads) return ARF_ERR_INVALID_ARG;
    if (T > 0 && in->data == out->data &&
        ((T > 1 && in->token_stride != out->token_stride) || (in->heads > 1 && in->head_stride != out->head_stride)))
        return ARF_ERR_INVALID_ARG;
    if (!disjoint_heads(out, T, D)) return ARF_ERR_INVALID_ARG;
    return ARF_OK;
}

arf_status_t check_rotary(const arf_rotary_t* rot, const int32_t* positions, int64_t T, int D) {
    if (!rot || rot->rot_dim < 2 || rot->rot_dim % 2 != 0 || rot->rot_dim > D) return ARF_ERR_INVALID_ARG;
    if (!isfinite(rot->magnitude)) return ARF_ERR_INVALID_ARG;
    if (T > 0 && (!rot->turns || !positions)) return ARF_ERR_INVALID_ARG;
    if (!is_aligned(rot->turns, 8) || !is_aligned(positions, 4)) return ARF_ERR_UNSUPPORTED;
    return ARF_OK;
}

arf_status_t run_rotary(arf_workspace_t ws, const arf_rotary_t* rot, const int32_t* positions, const int64_t* slots,
                        int64_t T, int D, arf_dtype_t dtype, const arf_heads_t* q, const arf_heads_t* q_out,
                        const arf_heads_t* k, const arf_heads_t* k_out, const arf_heads_t* v,
                        const arf_kv_cache_t* cache, void* stream_v) {
    cudaStream_t stream = static_cast<cudaStream_t>(stream_v);
    const arf_status_t st = workspace_check_device(ws, stream);
    if (st != ARF_OK) return st;
    if (T == 0) return ARF_OK;
    RotParams p = {};
    p.T = T;
    p.D = D;
    p.pos = positions;
    if (rot) {
        p.turns = rot->turns;
        p.rot = rot->rot_dim;
        p.interleaved = rot->interleaved != 0;
        p.mag = rot->magnitude;
    }
    bool vec = D % 8 == 0 && p.rot % 16 == 0;
    if (q) {
        p.q = segment(q, q_out);
        p.q_heads = q->heads;
        vec = vec && vec_heads(q) && vec_heads(q_out);
    }
    if (k) {
        p.k = segment(k, k_out);
        p.k_heads = k->heads;
        vec = vec && vec_heads(k) && (!k_out || vec_heads(k_out));
    }
    if (cache) {
        p.v = static_cast<const unsigned short*>(v->data);
        p.vts = v->token_stride, p.vhs = v->head_stride;
        p.slots = slots;
        p.ck = static_cast<char*>(cache->k);
        p.cv = static_cast<char*>(cache->v);
        p.cps = cache->page_stride, p.cts = cache->token_stride, p.chs = cache->head_stride;
        p.num_slots = (int64_t)cache->num_pages * cache->page_size;
        p.page = FastDiv((uint32_t)cache->page_size);
        p.kinv = 1.0f / cache->k_scale;
        p.vinv = 1.0f / cache->v_scale;
        p.bad = workspace_bad_counter(ws);
        vec = vec && vec_heads(v) && p.cps % 8 == 0 && p.cts % 8 == 0 && p.chs % 8 == 0 && is_aligned(p.ck, 16) &&
              is_aligned(p.cv, 16);
    }
    const int e = vec ? 8 : 1;
    p.rot_units = p.rot / (2 * e);
    const uint32_t units = (uint32_t)((D + 2 * e - 1) / (2 * e));
    p.q_in_place = q && q->data == q_out->data;
    p.k_in_place = k && k_out && k->data == k_out->data;
    // Two heads per thread once that still gives every SM 512 threads. At 8191
    // tokens of 40 heads of 128, half rotated, 1, 2 and 4 heads per thread
    // took 29.4, 26.2 and 26.6 us; the append of 5851 tokens 13.2, 11.7, 11.6.
    const auto groups = [&](int hpt) {
        return (int64_t)(p.q_heads + hpt - 1) / hpt + (int64_t)(p.k_heads + hpt - 1) / hpt * (cache ? 2 : 1);
    };
    const int64_t device_full = (int64_t)workspace_caps(ws).num_sms * 512;
    const bool many = vec && T * units >= device_full / groups(kManyHeads);
    const int hpt = many ? kManyHeads : 1;
    p.q_groups = (p.q_heads + hpt - 1) / hpt;
    p.k_groups = (p.k_heads + hpt - 1) / hpt;
    p.groups = (int)std::min<int64_t>(groups(hpt), INT_MAX);
    p.units = FastDiv(units);
    const int64_t blocks = T > kMaxExtent / units ? INT64_MAX : (T * units + 31) / 32;
    const int64_t rows = (groups(hpt) + kRotWarps - 1) / kRotWarps;
    if (blocks > 0x7fffffff || rows > 65535) return ARF_ERR_UNSUPPORTED;
    const int cb = cache ? elem_bytes(cache->dtype) : 2;
    RotFn fn = dtype == ARF_BF16 ? rot_fn<__nv_bfloat16>(vec, many, cache != nullptr, cb)
                                 : rot_fn<__half>(vec, many, cache != nullptr, cb);
    const cudaError_t ce = launch_kernel(fn, p, dim3((unsigned)blocks, (unsigned)rows), kRotThreads, 0, stream, true);
    if (ce != cudaSuccess) {
        note_cuda_error(ws, ce);
        return ARF_ERR_CUDA;
    }
    return ARF_OK;
}

}  // namespace
}  // namespace arf

extern "C" arf_status_t arf_rotary_turns(int rot_dim, double base, arf_rope_scaling_t scaling, double factor,
                                         double original_length, double beta_fast, double beta_slow,
                                         uint64_t* turns_out, float* magnitude_out) {
    if (!turns_out || !magnitude_out || rot_dim < 2 || rot_dim % 2 != 0) return ARF_ERR_INVALID_ARG;
    if (!(base > 1.0) || !std::isfinite(base) || !(factor >= 1.0) || !std::isfinite(factor))
        return ARF_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586476925286766559;
    double mag = 1.0;
    switch (scaling) {
        case ARF_ROPE_NONE:
        case ARF_ROPE_LINEAR: break;
        case ARF_ROPE_NTK:
            if (rot_dim < 4) return ARF_ERR_INVALID_ARG;
            base *= std::pow(factor, rot_dim / (rot_dim - 2.0));
            if (!std::isfinite(base)) return ARF_ERR_INVALID_ARG;
            break;
        case ARF_ROPE_YARN:
            if (!(original_length >= 1.0) || !std::isfinite(original_length) || !std::isfinite(beta_fast) ||
                !std::isfinite(beta_slow) || !(beta_fast > beta_slow))
                return ARF_ERR_INVALID_ARG;
            mag = 0.1 * std::log(factor) + 1.0;
            break;
        default: return ARF_ERR_INVALID_ARG;
    }
    for (int i = 0; i < rot_dim / 2; ++i) {
        double w = std::pow(base, -2.0 * i / rot_dim);
        if (scaling == ARF_ROPE_LINEAR) w /= factor;
        if (scaling == ARF_ROPE_YARN) {
            const double turns = original_length * w / two_pi;
            double keep = (turns - beta_slow) / (beta_fast - beta_slow);
            keep = keep < 0.0 ? 0.0 : (keep > 1.0 ? 1.0 : keep);
            w *= keep + (1.0 - keep) / factor;
        }
        turns_out[i] = (uint64_t)std::nearbyint(w / two_pi * 0x1p64);  // w <= 1: below 2^62
    }
    *magnitude_out = (float)mag;
    return ARF_OK;
}

extern "C" arf_status_t arf_rotary(arf_workspace_t ws, const arf_rotary_t* rot, const int32_t* positions, int64_t T,
                                   int D, arf_dtype_t dtype, const arf_heads_t* q, const arf_heads_t* q_out,
                                   const arf_heads_t* k, const arf_heads_t* k_out, void* stream) {
    using namespace arf;
    if (!ws || T < 0 || D < 1 || !is_io_dtype(dtype)) return ARF_ERR_INVALID_ARG;
    if (T > kMaxExtent || D > (1 << 20)) return ARF_ERR_UNSUPPORTED;
    arf_status_t st = check_rotary(rot, positions, T, D);
    if (st == ARF_OK) st = check_pair(q, q_out, T, D);
    if (st != ARF_OK) return st;
    if (!k != !k_out) return ARF_ERR_INVALID_ARG;
    if (k) st = check_pair(k, k_out, T, D);
    if (st != ARF_OK) return st;
    return run_rotary(ws, rot, positions, nullptr, T, D, dtype, q, q_out, k, k_out, nullptr, nullptr, stream);
}

extern "C" arf_status_t arf_rotary_append(arf_workspace_t ws, const arf_rotary_t* rot, const int32_t* positions,
                                          const int64_t* slots, int64_t T, arf_dtype_t dtype, const arf_heads_t* q,
                                          const arf_heads_t* q_out, const arf_heads_t* k, const arf_heads_t* v,
                                          const arf_kv_cache_t* cache, void* stream) {
    using namespace arf;
    if (!ws || T < 0 || !is_io_dtype(dtype)) return ARF_ERR_INVALID_ARG;
    if (T > kMaxExtent) return ARF_ERR_UNSUPPORTED;
    arf_status_t st = check_cache(cache);
    if (st != ARF_OK) return st;
    const int D = cache->head_dim;
    if (D > (1 << 20)) return ARF_ERR_UNSUPPORTED;
    if (!disjoint_cache(cache)) return ARF_ERR_INVALID_ARG;
    if (cache->dtype != dtype && cache->dtype != ARF_E4M3) return ARF_ERR_UNSUPPORTED;
    if (T > 0 && !slots) return ARF_ERR_INVALID_ARG;
    if (!is_aligned(slots, 8)) return ARF_ERR_UNSUPPORTED;
    if (!q != !q_out || (!rot && q)) return ARF_ERR_INVALID_ARG;
    if (rot) st = check_rotary(rot, positions, T, D);
    if (st == ARF_OK && q) st = check_pair(q, q_out, T, D);
    if (st == ARF_OK) st = check_heads(k, T);
    if (st == ARF_OK) st = check_heads(v, T);
    if (st != ARF_OK) return st;
    if (k->heads != cache->kv_heads || v->heads != cache->kv_heads) return ARF_ERR_INVALID_ARG;
    return run_rotary(ws, rot, positions, slots, T, D, dtype, q, q_out, k, nullptr, v, cache, stream);
}
