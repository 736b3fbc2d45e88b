// Attention of many rows over the paged cache: prompts, and pieces of prompts
// behind cached keys.
//
// The sums are those of attention_rows.hpp, in tiles of BM rows ((token, head)
// pairs of one sequence and KV head, heads fastest) by TK keys, 4 D
// multiply-adds a pair: bound by the matrix cores once the tiles are in LDS.
// * Each wave holds 32 rows: their q as B operands, the sums O^T.
//   S^T = K Q^T and O^T = V^T P^T run on v_mfma_f32_32x32x16, whose C layout
//   (column = row of q, element i = key 8 (i/4) + 4 half + i%4) is, rounded,
//   the B operand of the second product in the key order 4 half + {0..3, 8..11}.
//   So P never leaves its lane, and a row's maximum costs one exchange between
//   the two halves of the wave.
// * K and V tiles go from global memory into LDS without passing registers
//   (global_load_lds, 16 bytes a lane), three buffers each: two tiles are on
//   their way while one is read. Tiles of 32 keys, so that three workgroups of
//   128 rows (53 KB of LDS, 168 registers a lane) share a compute unit: one
//   wave's products run under another's exponentials. (64-key tiles with two
//   waves a SIMD: 547 us where this takes 508; 64 rows a wave, half the LDS
//   reads but one wave a SIMD, were no faster.) LDS rows are not padded (the
//   load writes lanes in order); instead the 16-byte pieces of a row are permuted
//   on the way (the lanes load from permuted places): piece c of row r sits at
//   c ^ fk(r), so that the b128 reads of K (a lane a row) and the transposing
//   b64 reads of V (4 rows by 16 values, one operand quarter) touch every bank
//   once.
// * The running maximum is raised only when a row's new one exceeds it by more
//   than 2^8 (in exp2 units 8): the weights then stay below 256 (fp16: 2^15,
//   carried 2^7 times larger), which the 16-bit types hold as precisely, and
//   the sums are rarely rescaled.
// * Step t of a wave is the product with V of tile t, and beside its matrix
//   instructions the score maxima of tile t + 1; before it S of tile t + 1, and
//   beside that the weights of tile t: vector work fills the issue slots that a
//   matrix instruction leaves (front, back).
// Measured: 8192 tokens, a window of 2048, 64 heads on 8 of 128, bf16: 500 us,
// 963 TFLOP/s; ragged prompts of up to 1900 tokens behind 1500 keys, f16: 673 us,
// 921; a library product of 8192 x 8192 x 8192 reaches 1313 (bf16) and 1250 (f16).
// The matrix cores are busy 51 % of the time at the 1.8 GHz that the power limit
// leaves, the vector units 59 %, LDS 30 %. Dim 64 fills the vector units first (62 %
// beside 32 %: 4096 tokens of 40 heads 118 us, 728 TFLOP/s); dim 256 has one wave a
// SIMD, whose waits nothing fills (25 % and 21 %: 16 heads on 4 213 us, 645).
#pragma once

#include "attention_common.hpp"

namespace w4a16 {

template <bool BF>
__device__ inline attn_f16_t attn_mfma32(const uint4 &a, const uint4 &b, attn_f16_t c) {
    if constexpr (BF)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(attn_b8_t, a),
                                                       __builtin_bit_cast(attn_b8_t, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(attn_h8_t, a),
                                                      __builtin_bit_cast(attn_h8_t, b), c, 0, 0, 0);
}

typedef short attn_s4_t __attribute__((ext_vector_type(4)));

// Where piece c (16 bytes) of row r sits in its row of D values.
template <int D>
__device__ inline int attn_swz_k(int r) {
    return D == 64 ? (r >> 1) & 7 : r & 15;
}
template <int D>
__device__ inline int attn_swz_v(int r) {
    return D == 64 ? ((r >> 1) & 1) << 2 : (r & 3) << 2;
}

// 16 bytes a lane from global memory (`from` + `offset` bytes of the lane) straight into LDS at `to` + 16 lane; `from`
// and `to` are uniform over the wave. Written as asm because the builtin makes the compiler wait for all such loads
// before any LDS read that it cannot prove apart; no register but m0 is written (which is reserved: the compiler keeps
// nothing in it, takes it in no clobber list, and uses it nowhere here), and the kernel itself waits (vmcnt)
// before the barrier behind which the tile is read.
// ONCE: read by this workgroup alone, past the caches' retention.
template <bool ONCE>
__device__ __forceinline__ void attn_load_lds(const uint16_t *from, uint32_t offset, uint32_t to) {
    if constexpr (ONCE)
        asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1 nt"
                     :: "v"(offset), "s"(from), "s"(__builtin_amdgcn_readfirstlane(to)) : "memory");
    else
        asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                     :: "v"(offset), "s"(from), "s"(__builtin_amdgcn_readfirstlane(to)) : "memory");
}

// The larger of a lane's value and that of its partner in the other half.
__device__ inline float attn_max_halves(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
    return fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}
__device__ inline float attn_sum_halves(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
    return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}

constexpr int kPromptTK = 32;   // keys of a tile
constexpr int kPromptRows = 128;   // rows of a workgroup
constexpr int kPromptMaxSplits = 64;   // workgroups that share a row tile's keys at most
constexpr float kPromptLift = 7.0f;   // fp16 weights are up to 2^8, by the running maximum's lag, times 2^7 (attn_against)
constexpr float kNone = -3e38f;   // a running maximum below every score: weights of hidden keys are exp2(-inf) = 0 beside it

// What a lane keeps of its place, in LDS: read where a step needs it, before the step's barrier. (Kept in registers
// they were the few too many: an operand of q then went through scratch memory, whose loads wait for those of the next
// tiles: 85 us instead of 69 for 2048 tokens of 40 heads.)
struct __align__(16) AttnLane {
    uint32_t kv_at;      // byte offsets of the lane's first K operand (low half) and V operand in a tile
    uint32_t ko, vo;     // byte offsets of its piece of K and of V in the group that its first load takes
    int pos;             // position of its row of q
};
__device__ __forceinline__ int attn_lane() { return __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0)); }

template <int D, bool BF, int NW>
struct AttnPrompt {
    static constexpr int TK = kPromptTK;
    static constexpr int KS = D / 16;             // k steps of S, an MFMA each
    static constexpr int DB = D / 32;             // 32-value blocks of O, two MFMAs each
    static constexpr int CH = D / 8;              // 16-byte pieces of a row
    static constexpr int RPI = 64 / CH;           // rows of one wave-wide load
    static constexpr int NI = TK / RPI / NW;      // loads per wave and matrix
    static constexpr int BM = 32 * NW;
    // operands read ahead of the MFMAs: as many as the registers of three waves a SIMD allow (D 256: one wave)
    static constexpr int RING = D == 256 ? 4 : 2;
    static constexpr int BUFS = 3;                // LDS buffers of K and of V

    const AttnArgs &a;
    int wave;
    const __attribute__((address_space(3))) AttnLane *mine;   // the lane's constants
    uint4 qf[KS];
    attn_f16_t acc[DB];
    float m, l0, l1;             // the running maximum (kNone: none yet) and sum, the sum in two parts

    __device__ AttnPrompt(const AttnArgs &args) : a(args) {}

    // K operand k of a tile: piece 2 k + half of row col (the steps differ in bits that only the permutation
    // touches). base: the lane's first operand in the buffer.
    __device__ __forceinline__ uint4 keys(uint32_t base, int k) const {
        return __builtin_bit_cast(uint4, *(const __attribute__((address_space(3))) attn_u4_t *)(uintptr_t)(base ^ (k * 32)));
    }
    // V^T operand n: values 32 (n % DB) .. of keys 16 (n / DB) ..
    __device__ __forceinline__ uint4 values(uint32_t base, int n) const {
        const uint32_t at = (base ^ (n % DB * 64)) + n / DB * 32 * D;
        const attn_s4_t v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) attn_s4_t *)(uintptr_t)at);
        const attn_s4_t v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) attn_s4_t *)(uintptr_t)(at + 16 * D));
        const uint2 lo = __builtin_bit_cast(uint2, v0), hi = __builtin_bit_cast(uint2, v1);
        return make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
    // One step's first half: S^T of the next tile (QK), and beside its MFMAs the weights of this one (W). A wave issues
    // in order, and an MFMA keeps the matrix core for 32 clocks but the issue port for 4: the fences hold the mix in
    // which vector work fills the rest. Operands are read RING MFMAs ahead (an LDS read takes longer than an MFMA).
    // The weights (B operands of the second product) are rounded to the values' type; l keeps them whole (as in
    // attention_rows.hpp; in fp16 those from 2^-21 of a row's largest on to 2^-11 of themselves).
    template <bool QK, bool W>
    __device__ __forceinline__ void front(uint32_t kb, attn_f16_t &nx, const attn_f16_t &cu, uint32_t vb, uint4 (&vf)[RING],
                                          uint4 (&p)[2]) {
        uint4 kf[RING];
        uint32_t w[8];
        if (QK) {
#pragma unroll
            for (int i = 0; i < RING; ++i) kf[i] = keys(kb, i);
#pragma unroll
            for (int e = 0; e < 16; ++e) nx[e] = 0.0f;
        }
#pragma unroll
        for (int n = 0; n < KS; ++n) {
            if (QK) {
                nx = attn_mfma32<BF>(kf[n % RING], qf[n], nx);
                if (n + RING < KS) kf[n % RING] = keys(kb, n + RING);
            }
            if (W) {
#pragma unroll
                for (int q = n * 8 / KS; q < (n + 1) * 8 / KS; ++q) {
                    const float w0 = attn_exp2(fmaf(cu[2 * q], a.scale_log2, -m));
                    const float w1 = attn_exp2(fmaf(cu[2 * q + 1], a.scale_log2, -m));
                    l0 += w0;
                    l1 += w1;
                    w[q] = attn_pack2<BF>(w0, w1);
                    asm volatile("" : "+v"(w[q]), "+v"(l0), "+v"(l1));   // (here, not where they are used)
                }
                if (n >= KS - RING) vf[n - (KS - RING)] = values(vb, n - (KS - RING));
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if (W) {
            p[0] = make_uint4(w[0], w[1], w[2], w[3]);
            p[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
    }

    // The second half: O^T += V^T P^T of this tile, and beside it the lane's largest score of the next.
    __device__ __forceinline__ float back(const attn_f16_t &nx, uint32_t vb, uint4 (&vf)[RING], const uint4 (&p)[2]) {
        constexpr int N = 2 * DB;
        float x = -INFINITY;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            acc[n % DB] = attn_mfma32<BF>(vf[n % RING], p[n / DB], acc[n % DB]);
            if (n + RING < N) vf[n % RING] = values(vb, n + RING);
#pragma unroll
            for (int q = n * 8 / N; q < (n + 1) * 8 / N; ++q) x = fmaxf(fmaxf(x, nx[2 * q]), nx[2 * q + 1]);
            asm volatile("" : "+v"(x));
            __builtin_amdgcn_sched_barrier(0);
        }
        return x;
    }

    // Whether the V tile holds an infinity or a NaN (every wave reads all of it, as for its product).
    __device__ __forceinline__ bool spoiled(uint32_t vb) const {
        uint32_t bad = 0;
        vb = attn_opaque(vb);
#pragma unroll 1
        for (int n = 0; n < 2 * DB; ++n) {
            const uint4 x = values(vb, n);
            bad |= attn_exponents<BF>(x.x) | attn_exponents<BF>(x.y) | attn_exponents<BF>(x.z) | attn_exponents<BF>(x.w);
        }
        return __any((bad & 0x80008000u) != 0);
    }

    // What infinities and NaN among the values of key tile `tile` add to the rows that see them, key by key: in the product they
    // would reach the others too (a weight of 0 times NaN). A weight is positive: they add themselves. From memory once
    // more, past the main loop, which has no registers for it.
    __device__ __forceinline__ void apart(const AttnTiles<TK> &tiles, int tile, int b, int kvh) {
        const int lane = attn_lane(), pos = mine->pos;
#pragma unroll 1
        for (int r = 0; r < TK; r += RPI) {
            const int j = tiles.key(tile) + r + lane / CH;
            int64_t at = 0;
            int bad = 0;
            if (j < tiles.hi) {
                const int id = a.table[(int64_t)b * a.table_stride + (j >> a.page_log2)];
                if ((unsigned)id < (unsigned)a.pages) {
                    at = (int64_t)id * a.page_stride + (((int64_t)kvh << a.page_log2) + (j & ((1 << a.page_log2) - 1))) * D;
                    bad = attn_nonfinite4<BF>(*reinterpret_cast<const attn_u4_t *>(a.vc + at + 8 * (lane % CH)));
                }
            }
#pragma unroll 1
            for (uint64_t left = __ballot(bad); left != 0;) {
                const int first = __builtin_ctzll(left), k = first / CH;
                left &= ~((CH == 64 ? ~0ull : (1ull << CH) - 1) << (k * CH));
                const int64_t row = (int64_t)__builtin_amdgcn_readlane((int)(at >> 32), first) << 32 |
                                    (uint32_t)__builtin_amdgcn_readlane((int)at, first);
                const int see = (int)attn_visible(tiles.key(tile) + r + k, pos, a.window, a.sinks);
#pragma unroll
                for (int q = 0; q < 4 * DB; ++q) {   // the lane's values 8 q + 4 half ..
                    const attn_u2_t y = *reinterpret_cast<const attn_u2_t *>(a.vc + row + 8 * q + 4 * (lane >> 5));
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint16_t z = (uint16_t)((e < 2 ? y.x : y.y) >> 16 * (e % 2));
                        acc[q / 4][4 * (q % 4) + e] += see & attn_nonfinite<BF>(z) ? attn_to_f32<BF>(z) : 0.0f;
                    }
                }
            }
        }
    }

    // Hides what the lane's row does not see: the tile's 32 keys as bits. gone: the 16-key groups that no row sees, as bits.
    __device__ __forceinline__ void hide(attn_f16_t &st, int j0, unsigned gone) {
        static_assert(TK == 32, "a tile's keys as bits of a word");
        const int last = min(mine->pos - j0, 31);   // keys up to this one
        uint32_t bits = last < 0 ? 0u : ~0u >> (31 - last);
        if (a.window > 0) {
            const int from = max(mine->pos - a.window + 1 - j0, 0), first = min(max(a.sinks - j0, 0), 32);
            bits &= (from > 31 ? 0u : ~0u << from) | (first > 31 ? ~0u : (1u << first) - 1u);
        }
        bits &= ~((gone & 1 ? 0xFFFFu : 0u) | (gone & 2 ? 0xFFFF0000u : 0u));
        bits = attn_opaque((int)(bits >> (4 * (attn_lane() >> 5))));   // element i is key 8 (i / 4) + 4 half + i % 4
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t see = (uint32_t)((int)(bits << (31 - (8 * (i / 4) + i % 4))) >> 31);   // all ones, or none
            const float x = st[i];
            st[i] = __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, x) & see) | (0xFF800000u & ~see));
        }
    }

    // Raises the running maximum where a tile's, the larger of the halves' x, is more than 8 above it.
    __device__ __forceinline__ void maximum(float x) {
        const float mn = attn_against<BF>(attn_max_halves(x), a.scale_log2, kPromptLift);
        if (__any(mn > m + 8.0f)) {
            const float n = fmaxf(m, mn), f = attn_exp2(m - n);
            m = n;
            l0 *= f;
            l1 *= f;
#pragma unroll
            for (int d = 0; d < DB; ++d) acc[d] *= f;
        }
    }
};

template <int D, bool BF, int NW, bool ONCE>
__global__ __launch_bounds__(64 * NW, D == 64 ? 4 : D == 128 ? 3 : 1) void attn_prompt_kernel(const AttnArgs a) {
    using P = AttnPrompt<D, BF, NW>;
    constexpr int TK = P::TK, CH = P::CH, BM = P::BM;
    __shared__ __align__(16) uint16_t lds[2][P::BUFS][TK * D];   // [K, V][buffer]
    __shared__ AttnLane lanes[64 * NW];
    __shared__ int apart;   // 1: infinities or NaN in a tile that not every row sees whole, 2: in one that lacks a page

    // Workgroups go to the 8 XCDs in turn; a unit (sequence, KV head, split; splits slowest) stays on one, where its
    // row tiles find its keys in the L2, or, where units are few, its row tiles are dealt to a.slices of them, each with a
    // unit of its own from here on. On each XCD units come in groups of a.group, a group's row tiles from the
    // last (the longest, under the causal order) to the first, all units of the group side by side. a.group is odd:
    // an XCD hands workgroups to its 4 shader engines in turn, and 4 sequences of unequal lengths side by side left
    // one engine the longest all along (984 us against 710).
    // Every second 32 workgroups of an XCD (one for each of its compute units) go backwards: where all of them start at
    // once, a unit's share is then long ones and short ones (2048 tokens of 40 heads: 70.4 -> 69.4 us).
    const int count = gridDim.x / 8, at32 = blockIdx.x / 8 / 32 * 32, off32 = blockIdx.x / 8 % 32;
    const int idx = at32 + (at32 / 32 % 2 ? min(32, count - at32) - 1 - off32 : off32);
    const int grp = idx / (a.group * a.slice_tiles), in = idx % (a.group * a.slice_tiles);
    const int dealt = (grp * a.group + in % a.group) * 8 + blockIdx.x % 8, unit = dealt / a.slices;
    const int rt = (a.slice_tiles - 1 - in / a.group) * a.slices + dealt % a.slices;
    const int pairs = a.batch * a.kv_heads;
    if (unit >= pairs * a.splits || rt >= a.row_tiles) return;
    // (uniform, but divided on the vector unit: back to scalar registers)
    const int split = __builtin_amdgcn_readfirstlane(unit / pairs);
    const int b = __builtin_amdgcn_readfirstlane((unit % pairs) / a.kv_heads);
    const int kvh = __builtin_amdgcn_readfirstlane((unit % pairs) % a.kv_heads);

    const AttnSeq sq = attn_seq(a, b, threadIdx.x == 0);
    const int rows = sq.nq * a.share;
    const int r0 = rt * BM;
    if (r0 >= rows) return;
    const int pos0 = sq.len - sq.nq;
    const int p_lo = pos0 + r0 / a.share, p_hi = pos0 + (min(r0 + BM, rows) - 1) / a.share;
    const AttnTiles<TK> tiles(p_lo, p_hi, sq.len, a.window, a.sinks);
    const int n_split = (tiles.total + a.split_tiles - 1) / a.split_tiles;
    if (split >= max(n_split, 1)) return;
    const int t0 = split * a.split_tiles, t1 = min(tiles.total, t0 + a.split_tiles);

    P s(a);
    s.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // The wave's rows. Which of the four waves (one on each SIMD) has the first ones changes from workgroup to workgroup,
    // and a wave without rows loads with the others but computes nothing: row tiles of few rows side by side do not all
    // compute on the same SIMD (16 sequences of up to 5000 keys, 32 rows of 8 heads of 128: 52.6 -> 50.2 us).
    const int wr0 = r0 + 32 * ((s.wave + blockIdx.x / 8 + blockIdx.x / 256) % NW);
    const bool live = wr0 < rows;
    // A wave's share of a tile's loads: instruction i covers rows RPI (i NW + wave) .., all of one 16-key group.
    constexpr int STEP = P::RPI * NW % 16;   // rows between two instructions' places in their groups: 0, or 8 (D 256)
    static_assert(STEP == 0 || STEP == 8, "rows of a wave's loads");
    {
        const int lane = attn_lane(), col = lane & 31, half = lane >> 5;
        AttnLane c;
        // V: row 4 half + .., value 16 (lane / 16 % 2) + 4 (lane % 4) of the block (the layout of the transposing read)
        const int vr = 4 * half + ((lane & 15) >> 2);
        c.kv_at = col * 2 * D + ((half ^ attn_swz_k<D>(col)) << 4) |
                  (vr * 2 * D + (((2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) ^ attn_swz_v<D>(vr)) << 4) + (lane & 1) * 8) << 16;
        const int r = (P::RPI * s.wave + lane / CH) & 15, piece = lane % CH;
        c.ko = r * 2 * D + ((piece ^ attn_swz_k<D>(r)) << 4);
        c.vo = r * 2 * D + ((piece ^ attn_swz_v<D>(r)) << 4);
        const int row = min(wr0 + col, rows - 1);   // (absent rows compute what the last one does, and write nothing)
        const int tok = sq.q0 + row / a.share, head = kvh * a.share + row % a.share;
        c.pos = pos0 + row / a.share;
        lanes[threadIdx.x] = c;
        if (threadIdx.x == 0) apart = 0;
        s.mine = (const __attribute__((address_space(3))) AttnLane *)&lanes[threadIdx.x];
        const uint16_t *qp = a.q + (int64_t)tok * a.q_stride + (int64_t)head * D + 8 * half;
#pragma unroll
        for (int k = 0; k < P::KS; ++k) s.qf[k] = *reinterpret_cast<const uint4 *>(qp + 16 * k);
    }
    s.m = kNone;
    s.l0 = s.l1 = 0.0f;
#pragma unroll
    for (int d = 0; d < P::DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) s.acc[d][i] = 0.0f;

    // Where the next 32 tiles' 16-key groups start in the caches (elements), one group a lane, and as bits the groups
    // behind the last key or without a page: those read page 0 (in bounds) and stay hidden.
    uint32_t at_lo = 0, at_hi = 0;
    uint64_t missing = 0;
    auto lookup = [&](int t) {
        const int lane = attn_opaque(attn_lane()), tt = t + lane / 2;
        int id = -1, j = 0;
        if (tt < t1) {
            j = tiles.key(tt) + 16 * (lane % 2);
            if (j < tiles.hi) {
                id = a.table[(int64_t)b * a.table_stride + (j >> a.page_log2)];
                if ((unsigned)id >= (unsigned)a.pages) {
                    id = -1;
                    attn_raise(a.err);
                }
            }
        }
        const int64_t at = (int64_t)max(id, 0) * a.page_stride +
                           (((int64_t)kvh << a.page_log2) + (j & ((1 << a.page_log2) - 1))) * D;
        at_lo = (uint32_t)at;
        at_hi = (uint32_t)(at >> 32);
        missing = __ballot(id < 0);
    };
    // A tile's V is loaded one step after its K, from the same places.
    constexpr uint32_t MAT = TK * D * 2;   // bytes of a buffer
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint16_t *)&lds[0][0][0];
    int64_t at[P::NI];
    unsigned gone = 0;   // two bits a tile: the current one's lowest, then the next three's
    auto find = [&](int t, int place) __attribute__((always_inline)) {
        const int n = (t - t0) % 32;
        if (n == 0) lookup(t);
#pragma unroll
        for (int i = 0; i < P::NI; ++i) {
            const int g = 2 * n + P::RPI * (i * NW + s.wave) / 16;
            at[i] = (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane(at_hi, g) << 32 |
                              (uint32_t)__builtin_amdgcn_readlane(at_lo, g));
        }
        gone |= ((unsigned)(missing >> (2 * n)) & 3u) << (2 * place);
    };
    auto load = [&](const uint16_t *cache, uint32_t off, uint32_t odd, uint32_t buffer) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < P::NI; ++i)
            attn_load_lds<ONCE>(cache + at[i], i % 2 && STEP ? off ^ odd : off, buffer + P::RPI * (i * NW + s.wave) * 2 * D);
    };
    auto load_k = [&](uint32_t off, uint32_t buffer) __attribute__((always_inline)) { load(a.kc, off, STEP * (2 * D + 16), buffer); };
    auto load_v = [&](uint32_t off, uint32_t buffer) __attribute__((always_inline)) { load(a.vc, off, STEP * 2 * D, buffer); };

    // Tiles [plain0, plain0 + plains) are seen whole by every row of the workgroup.
    const int plain0 = tiles.first + (a.window > 0 ? max(0, (max(0, p_hi - a.window + 1) + TK - 1) / TK - tiles.lo_tile) : 0);
    const int plains = max(0, tiles.first + max(0, p_lo + 1) / TK - tiles.lo_tile - plain0);
    auto plain = [&](int t, unsigned g) { return (unsigned)(t - plain0) < (unsigned)plains && (g & 3) == 0; };
    // V of a tile that is not plain: what no row of the workgroup sees is cleared (a weight of 0 times NaN is NaN);
    // true where an infinity or a NaN is left that some rows may see and others not. Every wave looks for itself, and at
    // the same values: no barrier where nothing is cleared, as in the causal order's tiles of the row tile's own tokens.
    auto spoils = [&](int j0, unsigned g, uint32_t buffer, uint32_t vb) -> bool {
        if (j0 + TK > tiles.hi || max(j0, a.sinks) < min(tiles.lo, j0 + TK) || (g & 3) != 0) {
            const uint32_t zero = attn_opaque(0);   // (no zeros in registers over the loop)
#pragma unroll 1
            for (int e = 64 * s.wave + attn_opaque(attn_lane()); e < TK * CH; e += 64 * NW) {
                const int r = e / CH, j = j0 + r;
                if (j >= tiles.hi || (j < tiles.lo && j >= a.sinks) || ((g >> (r / 16)) & 1))
                    *(__attribute__((address_space(3))) attn_u4_t *)(uintptr_t)(buffer + e * 16) = attn_u4_t{zero, zero, zero, zero};
            }
            __syncthreads();
        }
        return s.spoiled(vb);
    };
    // Such a tile: they are cleared for the product, and added to the rows that see them after the last tile.
    auto clear = [&](unsigned g, uint32_t buffer) {
        const int tid = 64 * s.wave + attn_opaque(attn_lane());
        if (tid == 0) (&apart)[attn_opaque(0)] |= (g & 3) != 0 ? 3 : 1;
        __syncthreads();
#pragma unroll 1
        for (int e = tid; e < TK * CH; e += 64 * NW) {
            const auto p = (__attribute__((address_space(3))) attn_u4_t *)(uintptr_t)(buffer + e * 16);
            const attn_u4_t x = *p;
            *p = attn_u4_t{attn_finite<BF>(x.x), attn_finite<BF>(x.y), attn_finite<BF>(x.z), attn_finite<BF>(x.w)};
        }
        __syncthreads();
    };

    // Buffers go round: K of tile t + 1 and V of tile t are in LDS when step t starts, the next two of each on their
    // way. kb0: K of t + 1, then t + 2 and t + 3 (whose place K of t has left); vb0: V of t, then t + 1 and t + 2.
    uint32_t kb0 = lds0 + MAT, kb1 = lds0 + 2 * MAT, kb2 = lds0;
    uint32_t vb0 = lds0 + 3 * MAT, vb1 = lds0 + 4 * MAT, vb2 = lds0 + 5 * MAT;
    // Step t: the weights of tile t beside S of tile t + 1, then the product of tile t beside the maxima of t + 1.
    auto step = [&](int t, attn_f16_t &cu, attn_f16_t &nx) __attribute__((always_inline)) {
        const uint32_t kv = s.mine->kv_at, ko = s.mine->ko, vo = s.mine->vo;
        // the loads of the step before last have landed: only the last step's may be under way
        if (t + 2 < t1)
            __builtin_amdgcn_s_waitcnt(0x0F70 | (2 * P::NI));
        else
            __builtin_amdgcn_s_waitcnt(0x0F70);
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
        if (t + 2 < t1) load_v(vo, vb2);
        if (t + 3 < t1) {
            find(t + 3, 3);
            load_k(ko, kb2);
        }
        if (!plain(t, gone) && spoils(tiles.key(t), gone, vb0, vb0 + (kv >> 16))) clear(gone, vb0);
        gone >>= 2;
        const uint32_t kb = kb0 + (kv & 0xFFFF), vb = vb0 + (kv >> 16);
        if (live) {
            uint4 vf[P::RING], p[2];
            s.template front<true, true>(kb, nx, cu, vb, vf, p);
            if (!plain(t + 1, gone)) s.hide(nx, tiles.key(t + 1), gone);
            s.maximum(s.back(nx, vb, vf, p));
        }
        const uint32_t k = kb0, v = vb0;
        kb0 = kb1, kb1 = kb2, kb2 = k;
        vb0 = vb1, vb1 = vb2, vb2 = v;
    };
    if (t0 < t1) {
        attn_f16_t sa, sb;
        uint4 vf[P::RING], p[2];
        const uint32_t kv = s.mine->kv_at, ko = s.mine->ko, vo = s.mine->vo;
        find(t0, 0);
        load_k(ko, kb2);
        load_v(vo, vb0);
        if (t0 + 1 < t1) {
            find(t0 + 1, 1);
            load_k(ko, kb0);
            load_v(vo, vb1);
        }
        if (t0 + 2 < t1) {
            find(t0 + 2, 2);
            load_k(ko, kb1);
        }
        __builtin_amdgcn_s_waitcnt(0x0F70);
        __syncthreads();
        s.template front<true, false>(kb2 + (kv & 0xFFFF), sa, sa, 0, vf, p);
        if (!plain(t0, gone)) s.hide(sa, tiles.key(t0), gone);
        float x = sa[0];
#pragma unroll
        for (int q = 1; q < 16; ++q) x = fmaxf(x, sa[q]);
        s.maximum(x);
        int t = t0;
        while (t + 1 < t1) {
            step(t, sa, sb);
            ++t;
            if (t + 1 >= t1) {
                sa = sb;
                break;
            }
            step(t, sb, sa);
            ++t;
        }
        __builtin_amdgcn_s_waitcnt(0x0F70);
        __syncthreads();
        // the last tile
        const uint32_t vb = vb0 + (s.mine->kv_at >> 16);
        if (!plain(t, gone) && spoils(tiles.key(t), gone, vb0, vb)) clear(gone, vb0);
        s.template front<false, true>(0, sa, sa, vb, vf, p);
        s.back(sa, vb, vf, p);
        const int left = __builtin_amdgcn_readfirstlane(apart);
        if (live && left != 0) {
#pragma unroll 1
            for (t = t0; t < t1; ++t)
                if ((left & 2) != 0 || (unsigned)(t - plain0) >= (unsigned)plains) s.apart(tiles, t, b, kvh);
        }
    }

    const int lane = attn_opaque(attn_lane()), col = lane & 31, half = lane >> 5;
    const int pair_rt = (b * a.kv_heads + kvh) * a.row_tiles + rt;
    float *part = n_split > 1 ? a.part + ((int64_t)pair_rt * a.splits + split) * attn_part_floats(BM, D) : nullptr;
    {
        const float lt = attn_sum_halves(s.l0 + s.l1);
        const int mine = wr0 + col, row = min(mine, rows - 1);
        const int tok = sq.q0 + row / a.share, head = kvh * a.share + row % a.share;
        const bool live = mine < rows;
        if (n_split <= 1) {
            const bool none = s.m == kNone;
            const float inv = none ? 0.0f : 1.0f / lt;
            uint16_t *o = a.out + (int64_t)tok * a.out_stride + (int64_t)head * D + 8 * half;
#pragma unroll
            for (int d = 0; d < P::DB; ++d)
#pragma unroll
                for (int i = 0; i < 16; i += 8) {
                    // elements i..i+3 are values 8 (i/4) + 4 half .. of the block: the halves trade, 16 bytes a lane
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = attn_pack2<BF>(s.acc[d][i + 2 * e] * inv, s.acc[d][i + 2 * e + 1] * inv);
                    const auto x = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
                    const auto y = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
                    if (live)
                        *reinterpret_cast<uint4 *>(o + 32 * d + 2 * i) =
                            make_uint4((uint32_t)x[0], (uint32_t)y[0], (uint32_t)x[1], (uint32_t)y[1]);
                }
            if (live && half == 0 && a.lse)
                a.lse[(int64_t)tok * a.heads + head] = attn_lse(s.m, lt);
        } else if (live) {
            const int lr = mine - r0;
#pragma unroll
            for (int d = 0; d < P::DB; ++d)
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                    *reinterpret_cast<float4 *>(part + lr * D + 32 * d + 2 * i + 4 * half) =
                        make_float4(s.acc[d][i], s.acc[d][i + 1], s.acc[d][i + 2], s.acc[d][i + 3]);
            if (half == 0) *reinterpret_cast<float2 *>(part + BM * D + 2 * lr) = make_float2(s.m == kNone ? -INFINITY : s.m, lt);
        }
    }
}

// Joins the splits of a row tile, 16 rows a workgroup: first each row's m and l, 16 lanes a row, and in LDS the splits'
// weights exp2(m_s - m) / l; then the sums. A kernel of its own: one workgroup of the last to arrive, which took all of
// a row tile's partials (64 KB each at D 128) through one compute unit at some 70 GB/s, was slower from a few splits on
// (41 tokens behind 4643 keys, 32 heads on 8 of 128, 16 splits: 43.5 us, so 24).
template <int D, bool BF>
__global__ __launch_bounds__(256) void attn_join_kernel(const AttnArgs a) {
    constexpr int BM = kPromptRows, ROWS = 16, E = ROWS * D / 4 / 256, U = 16 / E;   // E float4 a thread, of U splits at once
    __shared__ float weight[kPromptMaxSplits][ROWS];
    const int slice = blockIdx.x % (BM / ROWS), pair_rt = blockIdx.x / (BM / ROWS);
    const int rt = pair_rt % a.row_tiles, kvh = pair_rt / a.row_tiles % a.kv_heads, b = pair_rt / a.row_tiles / a.kv_heads;
    const AttnSeq sq = attn_seq(a, b, false);
    const int rows = sq.nq * a.share, r0 = rt * BM + slice * ROWS, pos0 = sq.len - sq.nq;
    if (r0 >= rows) return;
    const AttnTiles<kPromptTK> tiles(pos0 + rt * BM / a.share, pos0 + (min(rt * BM + BM, rows) - 1) / a.share, sq.len, a.window, a.sinks);
    const int n = (tiles.total + a.split_tiles - 1) / a.split_tiles;
    if (n <= 1) return;
    const int64_t pf_floats = attn_part_floats(BM, D);
    const float *part = a.part + (int64_t)pair_rt * a.splits * pf_floats;
    float4 v[U][E];
    auto load = [&](int q) __attribute__((always_inline)) {
        const float *p = part + slice * ROWS * D + 4 * threadIdx.x;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < E; ++e) v[u][e] = *reinterpret_cast<const float4 *>(p + min(q + u, n - 1) * pf_floats + 1024 * e);
    };
    load(0);   // (beside the loads of m and l)
    {
        constexpr int M = kPromptMaxSplits / 16;
        const int row = threadIdx.x / 16, sub = threadIdx.x % 16;
        float2 x[M];
        float m = -INFINITY, l = 0.0f;
#pragma unroll
        for (int k = 0; k < M; ++k) {
            x[k] = *reinterpret_cast<const float2 *>(part + min(sub + 16 * k, n - 1) * pf_floats + BM * D + 2 * (slice * ROWS + row));
            m = fmaxf(m, x[k].x);
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
#pragma unroll
        for (int k = 0; k < M; ++k) {
            x[k].x = m == -INFINITY ? 0.0f : attn_exp2(x[k].x - m);
            l += sub + 16 * k < n ? x[k].y * x[k].x : 0.0f;
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) l += __shfl_xor(l, o);
        const float inv = m == -INFINITY ? 0.0f : 1.0f / l;
#pragma unroll
        for (int k = 0; k < M; ++k)
            if (sub + 16 * k < n) weight[sub + 16 * k][row] = x[k].x * inv;
        if (sub == 0 && a.lse && r0 + row < rows) {
            const int tok = sq.q0 + (r0 + row) / a.share, h = kvh * a.share + (r0 + row) % a.share;
            a.lse[(int64_t)tok * a.heads + h] = attn_lse(m, l);
        }
    }
    __syncthreads();
    float4 o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = make_float4(0, 0, 0, 0);
    for (int q = 0;;) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (q + u < n) {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float f = weight[q + u][(threadIdx.x + 256 * e) / (D / 4)];
                    o[e].x += v[u][e].x * f, o[e].y += v[u][e].y * f, o[e].z += v[u][e].z * f, o[e].w += v[u][e].w * f;
                }
            }
        q += U;
        if (q >= n) break;
        load(q);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int i = threadIdx.x + 256 * e, row = r0 + i / (D / 4), d = i % (D / 4) * 4;
        if (row >= rows) break;
        const int tok = sq.q0 + row / a.share, h = kvh * a.share + row % a.share;
        *reinterpret_cast<uint2 *>(a.out + (int64_t)tok * a.out_stride + (int64_t)h * D + d) =
            make_uint2(attn_pack2<BF>(o[e].x, o[e].y), attn_pack2<BF>(o[e].z, o[e].w));
    }
}

template <int D, bool BF>
hipError_t launch_attention_prompt(const AttnArgs &a, const AttnPlan &plan, hipStream_t stream) {
    const int64_t upx = ceil_div((int64_t)a.batch * a.kv_heads * a.splits * a.slices, 8);   // units of an XCD
    const dim3 grid((unsigned)(ceil_div(upx, a.group) * a.group * 8 * a.slice_tiles));
    if (plan.once)
        attn_prompt_kernel<D, BF, kPromptRows / 32, true><<<grid, dim3(2 * kPromptRows), 0, stream>>>(a);
    else
        attn_prompt_kernel<D, BF, kPromptRows / 32, false><<<grid, dim3(2 * kPromptRows), 0, stream>>>(a);
    if (a.splits > 1) {
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        attn_join_kernel<D, BF><<<dim3((unsigned)(a.batch * a.kv_heads * a.row_tiles * (kPromptRows / 16))), dim3(256), 0, stream>>>(a);
    }
    return hipGetLastError();
}

#define W4A16_EXTERN_PROMPT(D)                                                                                  \
    extern template hipError_t launch_attention_prompt<D, false>(const AttnArgs &, const AttnPlan &, hipStream_t); \
    extern template hipError_t launch_attention_prompt<D, true>(const AttnArgs &, const AttnPlan &, hipStream_t);
W4A16_EXTERN_PROMPT(64)
W4A16_EXTERN_PROMPT(128)
W4A16_EXTERN_PROMPT(256)
#undef W4A16_EXTERN_PROMPT

}  // namespace w4a16
