// Attention of few rows over the paged cache: one new token a sequence, or a
// few drafted ones, times the heads that share a key/value head.
//
//   o = sum_j exp(c s_j - m) v_j / l,  s_j = q . k_j,  m = max_j c s_j,  l = sum_j exp(c s_j - m)
// in one pass over the keys: a tile of 32 keys at a time, with the running m
// and l (fp32) and the sum rescaled when m grows.
//
// Every visible key and value is read once and used for a few rows only, so
// the kernel is bound by the cache's bytes and its work is to keep loads in
// flight. A wave holds one tile of 32 keys (K and V, 64 D bytes each) in
// registers while the next ones are on their way; nothing passes through LDS
// until the waves of a workgroup meet at the end.
// * S^T = K Q^T on v_mfma_f32_16x16x32: keys are the A rows (a lane's operand
//   is 16 consecutive bytes of a key), the rows of q the 16 columns. A lane
//   then holds, of its column, keys 4g..4g+3 of both 16-key halves: its
//   softmax weights, which are already the B operand (k = those 8 keys) of
// * O^T = V^T P^T. The k order of a product is free, so each lane loads the
//   rows of its own 8 keys, 16 bytes of each, and pairs values of two keys
//   with v_perm (D / 4 of them per 32 keys and lane: hidden under the loads).
// * The 16 columns are (token, head) pairs of one sequence and KV head, heads fastest. (32 rows, a second column tile
//   of the same keys, were slower than the kernel for many rows at all but short lengths of narrow heads: 15
//   sequences of up to 5000 keys, 32 rows of 8 heads of 128: 57 us against 51; 2000 keys of one: 25 against 15.)
// * Shared work: the key tiles of all units (a sequence and KV head), one after the other, are cut into equal shares,
//   one for each workgroup, so that a batch of unequal lengths (or one long sequence) ends everywhere at once. A
//   workgroup finds its share from the lengths, and takes each unit's part of it in turn: its waves take key tiles in
//   turn, meet in LDS, and write the result, or, where the unit's keys are shared with other workgroups, a partial
//   (m, l, sum) that the last of them to arrive joins in key order.
// Measured: one token over 131072 keys, 64 heads on 8 of 128: 88.5 us, 6.07 TB/s,
// where a plain read of the same bytes reaches 7.0; 48 of them over 2048 .. 8192
// keys 167 us, 6.1 TB/s; bytes fetched are those of the keys and values within
// 1 %. Short calls are a chain of loads that wait for each other, 5.5 us for one
// tile a unit, and 5 more for a join.
#pragma once

#include <type_traits>

#include "attention_common.hpp"

namespace w4a16 {

constexpr int kRowsRT = 16;        // rows of a sequence and KV head at most
constexpr int kRowsWaves = 4;
constexpr int kRowsTK = 32;        // keys of a tile
constexpr int kRowsUnit = 6;       // key tiles that the start and end of a row tile's part cost (4 us; a tile 0.6)
constexpr float kRowsLift = 15.0f;   // fp16 weights are up to 2^15 (attn_against)
constexpr int kRowsMaxSplits = 58;   // workgroups that share a row tile at most

// Keys and values are read once: past the caches' retention (262 MB: 293 -> 264 us).
__device__ __forceinline__ uint4 attn_stream16(const char *p) {
    return __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const attn_u4_t *>(p)));
}
__device__ __forceinline__ uint2 attn_stream8(const char *p) {
    return __builtin_bit_cast(uint2, __builtin_nontemporal_load(reinterpret_cast<const attn_u2_t *>(p)));
}

// Sequence b: its rows and key tiles. A sequence that sees no key counts as one tile (its result has to be written), one
// without rows as none.
struct AttnRows {
    AttnSeq sq;
    int rows, pos0, p_hi;
    __device__ AttnRows(const AttnArgs &a, int b) : sq(attn_seq(a, b, true)) {
        rows = sq.nq * a.share;
        pos0 = sq.len - sq.nq;
        p_hi = sq.len - 1;
    }
    __device__ AttnTiles<kRowsTK> tiles(const AttnArgs &a) const {
        return AttnTiles<kRowsTK>(pos0, p_hi, sq.len, a.window, a.sinks);
    }
    __device__ int count(const AttnArgs &a) const { return rows == 0 ? 0 : max(1, tiles(a).total); }
};

// ALONE: a wave a workgroup, which takes one unit whole.
template <int D, bool BF, bool ALONE>
__global__ __launch_bounds__(ALONE ? 64 : 64 * kRowsWaves, D == 64 ? 4 : D == 128 ? 2 : 1) void attn_rows_kernel(const AttnArgs a) {
    constexpr int W = ALONE ? 1 : kRowsWaves;
    constexpr int KS = D / 32;                  // k steps of S
    constexpr int VW = D >= 128 ? 8 : 4;        // dims of a value row per lane and load
    constexpr int VH = D / (16 * VW);           // loads per value row
    constexpr int RT = kRowsRT;
    constexpr int TK = kRowsTK;
    constexpr int LD = D + 4;                   // LDS row of a sum (padded)
    constexpr int REDS = ALONE || W * 16 * LD > 2 * kRowsMaxSplits * RT ? W * 16 * LD : 2 * kRowsMaxSplits * RT;
    __shared__ __align__(16) float red[REDS];
    __shared__ float ml[2][W][RT];

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    // This workgroup's share [begin, end) of the work. Entries are the sequences; an entry's key tiles and
    // kRowsUnit more for its start and end count once for each KV head, one head after the other, and all of them are
    // cut evenly (a share that ends in those first kRowsUnit has no part of the unit). Where no entry is a quarter longer
    // than the mean and the workgroups are (nearly) a multiple of the units (entries times heads), every unit is cut
    // into the same number of pieces instead, and a workgroup has one: a second part costs some 8 us, its loads starting
    // from nothing and its sums left and joined. Every wave counts for itself. a.whole: a workgroup for each unit.
    const int entries = a.batch;
    auto tiles_of = [&](int e) { return e < entries ? AttnRows(a, e).count(a) : 0; };
    int per_wg, begin, end, base = 0, e = 0;   // base: weights before entry e, all heads
    int pieces = 1;   // of each unit; 0: cut evenly
    if (ALONE || a.whole) {
        e = __builtin_amdgcn_readfirstlane(blockIdx.x / a.kv_heads);
        base = e * a.kv_heads;
        per_wg = 1, begin = blockIdx.x, end = begin + 1;
        if (tiles_of(e) == 0) return;
    } else {
        const int lane = attn_opaque(threadIdx.x & 63);
        int total = 0, units = 0, longest = 0;
        for (int i = lane; i < entries; i += 64) {
            const int n = tiles_of(i);
            total += n;
            units += n > 0;
            longest = max(longest, n);
        }
        if (entries > 1) {
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) {
                total += __shfl_xor(total, o);
                units += __shfl_xor(units, o);
                longest = max(longest, __shfl_xor(longest, o));
            }
        }
        total = __builtin_amdgcn_readfirstlane(total) * a.kv_heads;
        units = __builtin_amdgcn_readfirstlane(units) * a.kv_heads;
        longest = __builtin_amdgcn_readfirstlane(longest);
        pieces = min((int)gridDim.x / max(units, 1), kRowsMaxSplits - 2);
        if (4 * (int64_t)longest * units > 5 * (int64_t)total || 4 * units * pieces < 3 * (int)gridDim.x) pieces = 0;
        total += units * kRowsUnit;
        per_wg = pieces ? 1 : max((total + (int)gridDim.x - 1) / (int)gridDim.x, a.least + kRowsUnit);
        begin = per_wg * blockIdx.x, end = min(pieces ? units * pieces : total, begin + per_wg);
        if (begin >= end) return;
        for (int e0 = 0; entries > 1; e0 += 64) {
            const int n = tiles_of(e0 + lane), w = n == 0 ? 0 : pieces ? pieces : n + kRowsUnit;
            int sum = w;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int y = __shfl_up(sum, o);
                sum += lane >= o ? y : 0;
            }
            const uint64_t past = __ballot(base + sum * a.kv_heads > begin);
            if (past) {
                const int at = __builtin_ctzll(past);
                e = e0 + at;
                base += __builtin_amdgcn_readlane(sum - w, at) * a.kv_heads;
                break;
            }
            base += __builtin_amdgcn_readlane(sum, 63) * a.kv_heads;
        }
    }

    for (int x = begin; x < end;) {
    const int b = __builtin_amdgcn_readfirstlane(e);
    const AttnRows seq(a, b);
    const int n_tiles = seq.count(a);
    if (n_tiles == 0) {
        ++e;
        continue;
    }
    const AttnTiles<TK> tiles = seq.tiles(a);
    const AttnSeq sq = seq.sq;
    const int rows = seq.rows, p_lo = seq.pos0, p_hi = seq.p_hi;
    const int skip = pieces ? 0 : kRowsUnit, weight = pieces ? pieces : n_tiles + kRowsUnit;
    const int kvh = __builtin_amdgcn_readfirstlane((x - base) / weight);
    const int unit0 = base + kvh * weight;
    const int piece = x - unit0;
    if (end - unit0 <= skip) return;
    const int t0 = __builtin_amdgcn_readfirstlane(pieces ? (unsigned)tiles.total * piece / pieces : max(0, piece - skip));
    const int t1 = __builtin_amdgcn_readfirstlane(pieces ? (unsigned)tiles.total * (piece + 1) / pieces : min(tiles.total, end - unit0 - skip));
    const int first_wg = __builtin_amdgcn_readfirstlane((unit0 + skip) / per_wg);
    const AttnSplits sp{__builtin_amdgcn_readfirstlane((unit0 + weight - 1) / per_wg) - first_wg + 1, first_wg,
                        unit0 + skip != first_wg * per_wg};
    x = min(unit0 + weight, end);
    if (kvh == a.kv_heads - 1 && x == unit0 + weight) {
        base = x;
        ++e;
    }
    __syncthreads();   // (the last part's LDS is free)
    const int lane = attn_opaque(threadIdx.x & 63), col = lane & 15, g = lane >> 4;

    // rows of q: columns of the products (absent rows are zero)
    uint4 qf[KS];
    const int row = min(col, rows - 1), pos = p_lo + row / a.share;
    const uint16_t *qp = a.q + (int64_t)(sq.q0 + row / a.share) * a.q_stride + (int64_t)(kvh * a.share + row % a.share) * D + 8 * g;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        qf[s] = *reinterpret_cast<const uint4 *>(qp + 32 * s);
        if (col >= rows) qf[s] = make_uint4(0, 0, 0, 0);
    }

    attn_f4_t acc[VH][VW];
    float m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int h = 0; h < VH; ++h)
#pragma unroll
        for (int c = 0; c < VW; ++c) acc[h][c] = attn_f4_t{0.0f, 0.0f, 0.0f, 0.0f};

    const int count = t1 - t0 > wave ? (t1 - t0 - wave + W - 1) / W : 0;   // tiles of this wave
    // page numbers of this wave's next 32 tiles, two halves each: lane 2n + half
    auto lookup = [&](int n0) -> int {
        const int n = n0 + (lane >> 1);
        int id = -1;
        if (n < count) {
            const int j = tiles.key(t0 + wave + W * n) + 16 * (lane & 1);
            if (j < tiles.hi) {
                id = a.table[(int64_t)b * a.table_stride + (j >> a.page_log2)];
                if ((unsigned)id >= (unsigned)a.pages) {   // no such page: its keys stay hidden
                    id = -1;
                    attn_raise(a.err);
                }
            }
        }
        return id;
    };
    const int page_mask = (1 << a.page_log2) - 1;
    // element offset of a 16-key half's first row (page 0 where there is none: in bounds, hidden below)
    auto half_at = [&](int id, int j) -> int64_t {
        return (int64_t)max(id, 0) * a.page_stride + (((int64_t)kvh << a.page_log2) + (j & page_mask)) * D;
    };
    uint4 kf[2][KS];
    uint4 vf[8][VH];   // (VW == 4: the low two words)
    // (uniform base and 32-bit offset: the bases stay in scalar registers)
    const uint32_t k_off = (col * D + 8 * g) * 2, v_off = (4 * g * D + col * VW) * 2;
    auto load_k = [&](int id0, int id1, int j) __attribute__((always_inline)) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const char *p = reinterpret_cast<const char *>(a.kc) + attn_uniform(2 * half_at(hf ? id1 : id0, j + 16 * hf));
#pragma unroll
            for (int s = 0; s < KS; ++s) kf[hf][s] = attn_stream16(p + k_off + 64 * s);
        }
    };
    auto load_v = [&](int id0, int id1, int j) __attribute__((always_inline)) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const char *p = reinterpret_cast<const char *>(a.vc) + attn_uniform(2 * half_at(hf ? id1 : id0, j + 16 * hf));
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int h = 0; h < VH; ++h) {
                    const char *q = p + v_off + i * 2 * D + h * 32 * VW;
                    if constexpr (VW == 8) {
                        vf[4 * hf + i][h] = attn_stream16(q);
                    } else {
                        const uint2 v = attn_stream8(q);
                        vf[4 * hf + i][h] = make_uint4(v.x, v.y, 0, 0);
                    }
                }
        }
    };

    int ids = lookup(0);
    // Tile n of this wave; `more`: another one follows (the last is apart, so that no register holds what may be loaded).
    auto key_tile = [&](int n, auto more) __attribute__((always_inline)) {
        const int j0 = tiles.key(t0 + wave + W * n);
        const int id0 = __builtin_amdgcn_readlane(ids, 2 * (n & 31)), id1 = __builtin_amdgcn_readlane(ids, 2 * (n & 31) + 1);
        // S^T of the tile
        attn_f4_t st[2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            attn_f4_t s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < KS; ++k) s = attn_mfma16<BF>(kf[hf][k], qf[k], s);
            st[hf] = s;
        }
        // the next tile's keys, in the registers just read
        int nid0 = 0, nid1 = 0, nj = 0;
        if constexpr (decltype(more)::value) {
            if (((n + 1) & 31) == 0) ids = lookup(n + 1);
            nid0 = __builtin_amdgcn_readlane(ids, 2 * ((n + 1) & 31));
            nid1 = __builtin_amdgcn_readlane(ids, 2 * ((n + 1) & 31) + 1);
            nj = tiles.key(t0 + wave + W * (n + 1));
            load_k(nid0, nid1, nj);
        }
        // a tile that some row sees in part only
        const bool masked = j0 + TK > p_lo + 1 || (a.window > 0 && j0 <= p_hi - a.window && j0 + TK > a.sinks) ||
                            id0 < 0 || id1 < 0;
        int poison = 0;   // an infinity or a NaN among values that not every row sees
        if (masked) {
            const int at = attn_opaque(j0 + 4 * g);   // key of element 0; element i is 16 (i / 4) + i % 4 behind it
            const int hi = tiles.hi - at, lo = tiles.lo - at, first = a.sinks - at;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int j = 16 * (i / 4) + i % 4;
                const int page = (i < 4 ? id0 : id1) >= 0;
                const int last = pos - at, from = a.window > 0 ? last - a.window + 1 : -at;
                const int see = page & (int)(j <= last) & ((int)(j >= from) | (int)(j < first));
                st[i >> 2][i & 3] = see ? st[i >> 2][i & 3] : -INFINITY;
                // a value that no row sees must not reach the product (0 x NaN)
                const int some = page & (int)(j < hi) & ((int)(j >= lo) | (int)(j < first));
#pragma unroll
                for (int h = 0; h < VH; ++h) {
                    vf[i][h] = make_uint4(some ? vf[i][h].x : 0, some ? vf[i][h].y : 0, some ? vf[i][h].z : 0, some ? vf[i][h].w : 0);
                    if (p_lo != p_hi)
                        poison |= attn_nonfinite4<BF>(vf[i][h]);
                }
            }
            poison = __any(poison);
        }
        // running softmax; pf: the weights as the B operand of the second product
        float mx = st[0][0];
#pragma unroll
        for (int i = 1; i < 8; ++i) mx = fmaxf(mx, st[i >> 2][i & 3]);
        mx = fmaxf(mx, __shfl_xor(mx, 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        const float mn = fmaxf(m, attn_against<BF>(mx, a.scale_log2, kRowsLift));
        const float ms = mn == -INFINITY ? 0.0f : mn;   // no key so far: every weight is exp2(-inf) = 0
        if (__any(mn > m)) {
            const float f = attn_exp2(m - ms);
            l *= f;
#pragma unroll
            for (int h = 0; h < VH; ++h)
#pragma unroll
                for (int c = 0; c < VW; ++c) acc[h][c] *= f;
            m = mn;
        }
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            w[i] = attn_exp2(fmaf(st[i >> 2][i & 3], a.scale_log2, -ms));
            l += w[i];
        }
        // weights are rounded to the values' type for the product (l keeps them whole): a relative error of 2^-8 (bf16)
        // or 2^-11 (f16, down to the type's normal range) at most each, where they differ of random sign, as the
        // output's own rounding
        const uint4 pf = make_uint4(attn_pack2<BF>(w[0], w[1]), attn_pack2<BF>(w[2], w[3]), attn_pack2<BF>(w[4], w[5]),
                                    attn_pack2<BF>(w[6], w[7]));
        if (poison) {
            // What infinities and NaN add, key by key and to the rows that see them only (0 x NaN would spoil the others),
            // through this wave's part of the LDS array, 16 keys at a time; then they are cleared for the product.
            const int lane = attn_opaque(threadIdx.x & 63), col = lane & 15, g = lane >> 4;
            float *pb = red + wave * 16 * LD;
            uint16_t *vb = reinterpret_cast<uint16_t *>(pb + 256);
            static_assert(1024 + 32 * D <= 64 * LD, "weights and values of 16 keys fit");
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t word = hf == 0 ? (i < 2 ? pf.x : pf.y) : (i < 2 ? pf.z : pf.w);
                    pb[(4 * g + i) * 16 + col] = attn_to_f32<BF>((uint16_t)(i % 2 ? word >> 16 : word));
#pragma unroll
                    for (int h = 0; h < VH; ++h) {
                        uint4 &v = vf[4 * hf + i][h];
                        uint16_t *p = vb + (4 * g + i) * D + h * 16 * VW + col * VW;
                        if constexpr (VW == 8)
                            *reinterpret_cast<uint4 *>(p) = v;
                        else
                            *reinterpret_cast<uint2 *>(p) = make_uint2(v.x, v.y);
                        v = make_uint4(attn_finite<BF>(v.x), attn_finite<BF>(v.y), attn_finite<BF>(v.z), attn_finite<BF>(v.w));
                    }
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
#pragma unroll 1
                for (int k = 0; k < 16; ++k) {
                    const int j = j0 + 16 * hf + k;
                    const bool see = (hf ? id1 : id0) >= 0 && attn_visible(j, pos, a.window, a.sinks);
                    const float p = pb[k * 16 + col];
#pragma unroll
                    for (int h = 0; h < VH; ++h)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
#pragma unroll
                            for (int c = 0; c < VW; ++c) {
                                const uint16_t v = vb[k * D + h * 16 * VW + (4 * g + e) * VW + c];
                                acc[h][c][e] += ((int)see & attn_nonfinite<BF>(v)) ? p * attn_to_f32<BF>(v) : 0.0f;
                            }
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
            }
        }
        // O^T += V^T P^T
#pragma unroll
        for (int h = 0; h < VH; ++h)
#pragma unroll
            for (int c = 0; c < VW; ++c) {
                const uint32_t sel = (c & 1) ? 0x07060302u : 0x05040100u;
                auto word = [&](int i) -> uint32_t {
                    const uint4 &v = vf[i][h];
                    return c / 2 == 0 ? v.x : c / 2 == 1 ? v.y : c / 2 == 2 ? v.z : v.w;
                };
                const uint4 vt = make_uint4(__builtin_amdgcn_perm(word(1), word(0), sel),
                                            __builtin_amdgcn_perm(word(3), word(2), sel),
                                            __builtin_amdgcn_perm(word(5), word(4), sel),
                                            __builtin_amdgcn_perm(word(7), word(6), sel));
                acc[h][c] = attn_mfma16<BF>(vt, pf, acc[h][c]);
                if (c % 2 == 1) __builtin_amdgcn_sched_barrier(0);   // (two operands' words at a time)
            }
        if constexpr (decltype(more)::value) load_v(nid0, nid1, nj);
    };
    if (count > 0) {
        const int id0 = __builtin_amdgcn_readlane(ids, 0), id1 = __builtin_amdgcn_readlane(ids, 1);
        const int j = tiles.key(t0 + wave);
        load_k(id0, id1, j);
        load_v(id0, id1, j);
        for (int n = 0; n < count - 1; ++n) key_tile(n, std::true_type{});
        key_tile(count - 1, std::false_type{});
    }

    // The waves meet: each scales its sums to the common maximum and leaves
    // them in LDS, 16 rows at a time.
    {
    const int tid = attn_opaque(threadIdx.x), lane = tid & 63, col = lane & 15, g = lane >> 4;
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (g == 0) {
        ml[0][wave][col] = m;
        ml[1][wave][col] = l;
    }
    const bool whole = ALONE || sp.n <= 1;
    const int mine = (int)blockIdx.x - sp.first;
    const int64_t pf_floats = attn_part_floats(RT, D);
    float *part = whole ? nullptr : a.part + sp.slot(mine) * pf_floats;
    __syncthreads();
    float mt = ml[0][0][col];
    for (int v = 1; v < W; ++v) mt = fmaxf(mt, ml[0][v][col]);
    const float f = mt == -INFINITY ? 0.0f : attn_exp2(ml[0][wave][col] - mt);
    float *dst = red + (wave * 16 + col) * LD;
#pragma unroll
    for (int h = 0; h < VH; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int c = 0; c < VW; c += 4) {
                const float4 v = make_float4(acc[h][c][e] * f, acc[h][c + 1][e] * f,
                                             acc[h][c + 2][e] * f, acc[h][c + 3][e] * f);
                *reinterpret_cast<float4 *>(dst + h * 16 * VW + (4 * g + e) * VW + c) = v;
            }
    __syncthreads();
    for (int e = tid; e < 16 * D / 4; e += 64 * W) {
        const int rr = e / (D / 4), d = e % (D / 4) * 4;
        if (rr >= rows) break;
        float4 o = make_float4(0, 0, 0, 0);
        float mr = ml[0][0][rr];
#pragma unroll
        for (int v = 0; v < W; ++v) {
            const float4 x = *reinterpret_cast<const float4 *>(red + (v * 16 + rr) * LD + d);
            o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
            mr = fmaxf(mr, ml[0][v][rr]);
        }
        float lr = 0.0f;
#pragma unroll
        for (int v = 0; v < W; ++v)
            lr += ml[1][v][rr] * (mr == -INFINITY ? 0.0f : attn_exp2(ml[0][v][rr] - mr));
        if (whole) {
            const int tok = sq.q0 + rr / a.share, h = kvh * a.share + rr % a.share;
            const float inv = mr == -INFINITY ? 0.0f : 1.0f / lr;
            const uint2 v = make_uint2(attn_pack2<BF>(o.x * inv, o.y * inv), attn_pack2<BF>(o.z * inv, o.w * inv));
            *reinterpret_cast<uint2 *>(a.out + (int64_t)tok * a.out_stride + (int64_t)h * D + d) = v;
            if (d == 0 && a.lse)
                a.lse[(int64_t)tok * a.heads + h] = attn_lse(mr, lr);
        } else {
            float *p = part + rr * D + d;
            attn_store2(p, o.x, o.y);
            attn_store2(p + 2, o.z, o.w);
            if (d == 0) attn_store2(part + RT * D + 2 * rr, mr, lr);
        }
    }
    // (at once, not when the whole share is done: the workgroups end together, and would all join then)
    if constexpr (!ALONE) {
    if (whole || !attn_arrive(a, sp, mine)) continue;

    // The last split joins them all in split order. red: (m, l) [split][row], then the splits' weights exp2(m_s - m) in
    // m's place; ml: each row's m and l. What matters here is how few times one load waits for another (a partial comes
    // from beyond the L2, 2 us away): all (m, l) and the first 16 float4 of sums a thread at once.
    const int live = rows;
    static_assert(2 * kRowsMaxSplits * RT <= REDS || ALONE, "(m, l) of every split fit the LDS array");
    float2 *rm = reinterpret_cast<float2 *>(red);
    auto join = [&](auto per_thread) __attribute__((always_inline)) {
        constexpr int E = decltype(per_thread)::value, U = 16 / E;
        const int all = live * D / 4;
        float2 v[U][E][2];
        auto load = [&](int s0) __attribute__((always_inline)) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float *p = a.part + sp.slot(min(s0 + u, sp.n - 1)) * pf_floats;
#pragma unroll
                for (int k = 0; k < E; ++k) {
                    const int i = 4 * min(tid + 64 * W * k, all - 1);
                    v[u][k][0] = attn_load2(p + i);
                    v[u][k][1] = attn_load2(p + i + 2);
                }
            }
        };
        load(0);
        for (int i = tid; i < sp.n * live; i += 64 * W)
            rm[i] = attn_load2(a.part + sp.slot(i / live) * pf_floats + RT * D + 2 * (i % live));
        __syncthreads();
        for (int rr = wave; rr < live; rr += W) {
            float mr = -INFINITY;
            for (int s = lane; s < sp.n; s += 64) mr = fmaxf(mr, rm[s * live + rr].x);
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) mr = fmaxf(mr, __shfl_xor(mr, o));
            float lr = 0.0f;
            for (int s = lane; s < sp.n; s += 64) {
                const float2 x = rm[s * live + rr];
                const float f = mr == -INFINITY ? 0.0f : attn_exp2(x.x - mr);
                rm[s * live + rr].x = f;
                lr += x.y * f;
            }
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) lr += __shfl_xor(lr, o);
            if (lane == 0) {
                ml[0][0][rr] = mr;
                ml[1][0][rr] = lr;
            }
        }
        __syncthreads();
        float4 o[E];
#pragma unroll
        for (int k = 0; k < E; ++k) o[k] = make_float4(0, 0, 0, 0);
        for (int s0 = 0;;) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (s0 + u < sp.n) {
#pragma unroll
                    for (int k = 0; k < E; ++k) {
                        const float f = rm[(s0 + u) * live + min(tid + 64 * W * k, all - 1) / (D / 4)].x;
                        o[k].x += v[u][k][0].x * f, o[k].y += v[u][k][0].y * f, o[k].z += v[u][k][1].x * f, o[k].w += v[u][k][1].y * f;
                    }
                }
            s0 += U;
            if (s0 >= sp.n) break;
            load(s0);
        }
#pragma unroll
        for (int k = 0; k < E; ++k) {
            const int i = tid + 64 * W * k, rr = i / (D / 4), d = i % (D / 4) * 4;
            if (i >= all) break;
            const float mr = ml[0][0][rr], lr = ml[1][0][rr];
            const int tok = sq.q0 + rr / a.share, h = kvh * a.share + rr % a.share;
            const float inv = mr == -INFINITY ? 0.0f : 1.0f / lr;
            const uint2 w = make_uint2(attn_pack2<BF>(o[k].x * inv, o[k].y * inv), attn_pack2<BF>(o[k].z * inv, o[k].w * inv));
            *reinterpret_cast<uint2 *>(a.out + (int64_t)tok * a.out_stride + (int64_t)h * D + d) = w;
            if (d == 0 && a.lse)
                a.lse[(int64_t)tok * a.heads + h] = attn_lse(mr, lr);
        }
    };
    if (live * D / 4 <= 64 * W) {
        join(std::integral_constant<int, 1>{});
    } else if constexpr (D >= 128) {   // (16 rows of 64 values are one float4 a thread)
        if (D == 128 || live * D / 4 <= 128 * W)
            join(std::integral_constant<int, 2>{});
        else
            join(std::integral_constant<int, D / 64>{});
    }
    attn_clear_flags(a, sp);
    }
    }
    }
}

template <int D, bool BF>
hipError_t launch_attention_rows(const AttnArgs &a, const AttnPlan &plan, hipStream_t stream) {
    if (plan.alone)
        attn_rows_kernel<D, BF, true><<<dim3((unsigned)plan.wgs), dim3(64), 0, stream>>>(a);
    else
        attn_rows_kernel<D, BF, false><<<dim3((unsigned)plan.wgs), dim3(64 * kRowsWaves), 0, stream>>>(a);
    return hipGetLastError();
}

#define W4A16_EXTERN_ROWS(D)                                                                                  \
    extern template hipError_t launch_attention_rows<D, false>(const AttnArgs &, const AttnPlan &, hipStream_t); \
    extern template hipError_t launch_attention_rows<D, true>(const AttnArgs &, const AttnPlan &, hipStream_t);
W4A16_EXTERN_ROWS(64)
W4A16_EXTERN_ROWS(128)
W4A16_EXTERN_ROWS(256)
#undef W4A16_EXTERN_ROWS

}  // namespace w4a16
