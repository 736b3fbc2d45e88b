// Shared by the paged-cache kernels: the append (cache.hip) and the attention
// kernels (attention_rows.hpp, attention_prompt.hpp).
//
// Cache layout: K and V each [pages][kv_heads][page][D] in the activations'
// 16-bit type, `page_stride` elements from page to page. The keys of one head
// in one page are contiguous rows of D values (page * D * 2 bytes: 4 KiB at
// page 16, D 128), so a tile of 16 keys, the unit the matrix instructions
// take, never crosses a page (pages are powers of two from 16 on) and costs
// one page lookup.
#pragma once

#include <math.h>

#include "w4a16_internal.hpp"

namespace w4a16 {

typedef _Float16 attn_h8_t __attribute__((ext_vector_type(8)));
typedef __bf16 attn_b8_t __attribute__((ext_vector_type(8)));
typedef uint32_t attn_u4_t __attribute__((ext_vector_type(4)));
typedef uint32_t attn_u2_t __attribute__((ext_vector_type(2)));
typedef float attn_f4_t __attribute__((ext_vector_type(4)));
typedef float attn_f16_t __attribute__((ext_vector_type(16)));

// v_mfma_f32_16x16x32: A lane (r, g) = row r, k 8g..8g+7; B lane (c, g) =
// column c, k 8g..8g+7; C lane (c, g) element i = column c, row 4g + i.
template <bool BF>
__device__ inline attn_f4_t attn_mfma16(const uint4 &a, const uint4 &b, attn_f4_t c) {
    if constexpr (BF)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(attn_b8_t, a),
                                                       __builtin_bit_cast(attn_b8_t, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(attn_h8_t, a),
                                                      __builtin_bit_cast(attn_h8_t, b), c, 0, 0, 0);
}

template <bool BF>
__device__ inline float attn_to_f32(uint16_t b) {
    if constexpr (BF)
        return __builtin_bit_cast(float, (uint32_t)b << 16);
    else
        return (float)__builtin_bit_cast(_Float16, b);
}
template <bool BF>
__device__ inline uint16_t attn_to_16(float v) {
    return BF ? f32_to_bf16_bits(v) : f32_to_f16_bits(v);
}
template <bool BF>
__device__ inline uint32_t attn_pack2(float lo, float hi) {
    if constexpr (BF) {
        bf162_t v = {(__bf16)lo, (__bf16)hi};
        return __builtin_bit_cast(uint32_t, v);
    } else {
        half2_t v = {(_Float16)lo, (_Float16)hi};
        return __builtin_bit_cast(uint32_t, v);
    }
}
__device__ inline float attn_exp2(float x) { return __builtin_amdgcn_exp2f(x); }

// What a tile's scores, `x` the largest, are held against (exp2 units): weights are exp2(s * scale - m). fp16 holds
// nothing below 2^-25, and many small weights are much: 131068 keys exp(-17.5) below four others are 0.08 % of the sum,
// and would be none of the product. So fp16 weights are carried 2^lift times larger, m smaller, to the top of the type's range;
// sums are carried alike, and lse = m + log2(l) holds as it stands. m is rounded up by a step, so that a weight of scores
// whose steps are larger than one cannot pass the range (the products s * scale are not rounded beside m). Weights 2^-29
// of a part's largest (few rows, many rows 2^-21) keep their relative precision, smaller ones an absolute 2^-40 (2^-32).
template <bool BF>
__device__ __forceinline__ float attn_against(float x, float scale, float lift) {
    if constexpr (BF) return x * scale;
    const float m = fmaf(x, scale, -lift);
    return fmaf(fabsf(m), 0x1.008p-24f, m);   // (-inf turns into NaN, which no maximum takes)
}

// ln of a row's sum: l weights of exp2(s - m). A row that sees nothing: l 0, -inf. One whose scores are NaN: l is NaN (m may
// be any value, as no maximum takes a NaN).
__device__ inline float attn_lse(float m, float l) { return (m + __log2f(l)) * 0.693147180559945309f; }

// v, which the compiler no longer knows: what seldom-run code derives from it is computed there, not kept in registers
// over the main loop (which has none to spare; a spill's reload would wait for the loads under way).
__device__ __forceinline__ int attn_opaque(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

// A value that every lane holds, in scalar registers.
__device__ __forceinline__ int64_t attn_uniform(int64_t v) {
    return (int64_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32 | (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
}

// The arguments of one attention launch (kernel argument, passed by value).
struct AttnArgs {
    const uint16_t *q, *kc, *vc;
    const int *table, *kv_lens, *q_starts;   // q_starts NULL: token b is sequence b's
    uint16_t *out;
    float *lse;                              // NULL: not written
    int64_t q_stride, out_stride;            // elements from token to token
    int64_t page_stride;                     // elements from page to page
    int tokens, batch, heads, kv_heads, share;   // share = heads / kv_heads
    int page_log2, pages, table_stride;
    int max_q, max_kv;
    float scale_log2;                        // softmax scale * log2(e)
    int window, sinks;                       // window 0: none (sinks then 0)
    int row_tiles;                           // row tiles per sequence and KV head
    int whole;                               // few rows: a workgroup for each row tile and KV head
    int least;                               // few rows: key tiles of a workgroup at least
    int splits, split_tiles;                 // many rows: key splits per row tile at most, key tiles per split
    int slices, slice_tiles;                 // many rows: XCDs that a unit's row tiles are dealt to, row tiles of each
    int group;                               // many rows: units of an XCD that run side by side
    float *part;                             // partial results of the splits, by slot
    unsigned long long *flags;               // their arrival flags
    unsigned long long token;                // this launch's token
    unsigned int *err;                       // process error word
};

// Tells the host of an index outside its range that the kernel met in device
// memory (a page number, a length): the next compute call returns
// W4A16_ERR_HIP.
__device__ inline void attn_raise(unsigned int *err) {
    if (err) __hip_atomic_store(err, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
}

// One sequence's new tokens [q0, q0 + nq) and its length with them, held to
// the ranges the launch was planned for (`tell`: the lanes that report one outside).
struct AttnSeq {
    int q0, nq, len;
};
__device__ inline AttnSeq attn_seq(const AttnArgs &a, int b, bool tell) {
    AttnSeq s;
    bool bad = false;
    if (a.q_starts) {
        const int q0 = a.q_starts[b], q1 = a.q_starts[b + 1];
        s.q0 = min(max(q0, 0), a.tokens);
        const int e = min(max(q1, s.q0), a.tokens);
        s.nq = min(e - s.q0, a.max_q);
        bad = s.q0 != q0 || s.q0 + s.nq != q1;
    } else {
        s.q0 = b;
        s.nq = 1;
    }
    const int len = a.kv_lens[b];
    s.len = min(max(len, 0), a.max_kv);
    bad = bad || s.len != len;
    if (bad && tell) attn_raise(a.err);
    return s;
}

// The key tiles (TK keys, TK-aligned) that a tile of rows reads: the tiles of
// the first visible keys, then those from the lowest row's window up to the
// highest row's position. Tile t of `total` starts at key(t).
template <int TK>
struct AttnTiles {
    int lo, hi;         // keys [lo, hi) are the window's; keys below `sinks` are visible too
    int lo_tile, first;   // first: tiles of first keys below lo_tile
    int total;
    __device__ AttnTiles(int p_lo, int p_hi, int len, int window, int sinks) {
        hi = max(0, min(len, p_hi + 1));
        lo = window > 0 ? min(max(0, p_lo - window + 1), hi) : 0;
        lo_tile = lo / TK;
        first = min((min(sinks, hi) + TK - 1) / TK, lo_tile);
        total = first + ((hi + TK - 1) / TK - lo_tile);
    }
    __device__ int key(int t) const { return (t < first ? t : lo_tile + t - first) * TK; }
};

__device__ inline bool attn_visible(int j, int p, int window, int sinks) {
    return j <= p && (window == 0 || j > p - window || j < sinks);
}

// Whether a packed pair of 16-bit values holds an infinity or a NaN (1 or 0, without branches).
template <bool BF>
__device__ inline int attn_nonfinite(uint32_t w) {
    constexpr uint32_t e = BF ? 0x7F80u : 0x7C00u;
    return (int)((w & e) == e) | (int)((w & (e << 16)) == (e << 16));
}
template <bool BF, typename V>
__device__ inline int attn_nonfinite4(const V &v) {
    return attn_nonfinite<BF>(v.x) | attn_nonfinite<BF>(v.y) | attn_nonfinite<BF>(v.z) | attn_nonfinite<BF>(v.w);
}
// Bits 15 and 31: whether the pair's low and high value are an infinity or a NaN (other bits are anything).
template <bool BF>
__device__ inline uint32_t attn_exponents(uint32_t w) {
    return BF ? (w & 0x7F807F80u) + 0x00800080u : (w & 0x7C007C00u) + 0x04000400u;
}
// The pair with infinities and NaN replaced by zero.
template <bool BF>
__device__ inline uint32_t attn_finite(uint32_t w) {
    constexpr uint32_t e = BF ? 0x7F80u : 0x7C00u;
    return ((w & e) == e ? 0 : w & 0xFFFFu) | ((w & (e << 16)) == (e << 16) ? 0 : w & 0xFFFF0000u);
}

// Splits of one row tile: `n` of them, split i in slot slot(i) of the flags and partials.
struct AttnSplits {
    int n, first, odd;   // slot 2 (first + i), the first split's one further where odd
    __device__ int slot(int i) const { return 2 * (first + i) + (i == 0 ? odd : 0); }
};
// Arrival of split `mine`: true for the last of them, and for any other that finds all of them there (they then join
// the same partials in the same order into the same bits). The caller's partials were written with agent-scope stores
// (they reach memory that every XCD sees without writing caches back); each wave waits for its stores before the
// barrier, the flag is written after it and has arrived before the others are read. A flag is the launch's 64-bit
// token, so flags need no clearing before; who joins clears them, so that a replay starts anew. (A counter would make
// n workgroups that end together take turns: 128 of them cost 300 us.)
__device__ inline bool attn_arrive(const AttnArgs &a, const AttnSplits &sp, int mine) {
    __shared__ int all;
    __builtin_amdgcn_s_waitcnt(0x0F70);
    if (threadIdx.x == 0) all = 1;
    __syncthreads();
    if (threadIdx.x < 64) {
        if (threadIdx.x == 0) __hip_atomic_store(a.flags + sp.slot(mine), a.token, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __builtin_amdgcn_s_waitcnt(0x0F70);
        for (int i = threadIdx.x; i < sp.n; i += 64)
            if (__hip_atomic_load(a.flags + sp.slot(i), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != a.token) all = 0;
    }
    __syncthreads();
    return all != 0;
}
// After the join: every thread of the workgroup.
__device__ inline void attn_clear_flags(const AttnArgs &a, const AttnSplits &sp) {
    for (int i = threadIdx.x; i < sp.n; i += blockDim.x)
        __hip_atomic_store(a.flags + sp.slot(i), 0ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ inline void attn_store2(float *p, float x, float y) {
    const unsigned long long v =
        (unsigned long long)__builtin_bit_cast(uint32_t, y) << 32 | __builtin_bit_cast(uint32_t, x);
    __hip_atomic_store(reinterpret_cast<unsigned long long *>(p), v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ inline float2 attn_load2(const float *p) {
    const unsigned long long v = __hip_atomic_load(reinterpret_cast<const unsigned long long *>(p), __ATOMIC_RELAXED,
                                                   __HIP_MEMORY_SCOPE_AGENT);
    return make_float2(__builtin_bit_cast(float, (uint32_t)v), __builtin_bit_cast(float, (uint32_t)(v >> 32)));
}

// Host side. The plan of one attention call.
struct AttnPlan {
    int kind;          // 0: few rows (attention_rows.hpp), 1: many rows (attention_prompt.hpp)
    int tile_rows;     // rows of a workgroup
    int row_tiles;     // row tiles per sequence and KV head
    int alone;         // kind 0: a wave a workgroup
    int wgs, whole, least;   // kind 0: workgroups, one for each unit?, key tiles of each at least
    int splits, split_tiles;   // kind 1
    int once;          // kind 1: keys and values are read once, and are more than the last-level cache keeps
    int64_t slots;     // partials (0: no row tile is split)
};
// A split's partial result: sums [rows][dim], then (m, l) [rows].
__host__ __device__ inline int64_t attn_part_floats(int rows, int dim) { return (int64_t)rows * (dim + 2); }
size_t attn_workspace(const AttnPlan &p, int32_t dim);
AttnPlan attn_plan(int64_t batch, int32_t kv_heads, int32_t share, int32_t dim, int64_t max_q, int64_t max_kv,
                   int32_t window, int32_t sinks);
hipError_t launch_attention(AttnArgs a, bool bf16, int dim, const AttnPlan &plan, void *workspace,
                            hipStream_t stream);
template <int D, bool BF>
hipError_t launch_attention_rows(const AttnArgs &a, const AttnPlan &plan, hipStream_t stream);
template <int D, bool BF>
hipError_t launch_attention_prompt(const AttnArgs &a, const AttnPlan &plan, hipStream_t stream);

struct AppendArgs {
    const uint16_t *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;   // elements from token to token
    int tokens, heads, kv_heads, dim;       // heads 0: no queries
    const int64_t *slots;
    const int *positions;
    const float *cos_sin;
    int positions_max, rot;                 // rot 0: no rotation
    int interleaved;
    const uint16_t *q_weight, *k_weight;    // NULL: no norm
    float eps;
    uint16_t *q_out;
    int64_t q_out_stride;
    uint16_t *kc, *vc;
    int64_t page_stride;
    int pages, page_log2;
    unsigned int *err;
};
hipError_t launch_kv_append(const AppendArgs &a, bool bf16, hipStream_t stream);

}  // namespace w4a16
