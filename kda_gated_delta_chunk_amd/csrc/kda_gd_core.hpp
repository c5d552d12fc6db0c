// The gated delta rule with one decay per head: operands, and the pass over the states that the forward call and both
// directions of the backward call share.
//
// With b_t the sum of a chunk's log-decays up to token t, E_ri = e^{b_r - b_i} and S the state before the chunk, the
// recurrence  S <- e^g S;  z = v - S^T k;  S <- S + beta k z^T;  o = scale S^T q  is, over a chunk of C tokens,
//   z_r = v_r - e^{b_r} S^T k_r - sum_{i<r} E_ri (k_r.k_i) beta_i z_i,        so  z = (1 + A)^-1 (v - e^b K S)
//   o_r = scale ( e^{b_r} S^T q_r + sum_{i<=r} E_ri (q_r.k_i) beta_i z_i )
//   S  <- e^{b_C} S + sum_i e^{b_C - b_i} beta_i k_i z_i^T
// with A strictly lower. (1 + A)^-1 = 1 + N does not depend on the state: a first kernel forms N and the weights of the
// pairs for every chunk at once, and what follows chunk by chunk is products with the state. Backward, with G the
// gradient behind the chunk and D, y those of what is written (beta z) and of z:
//   D_i = e^{b_C - b_i} G^T k_i + scale sum_{r>=i} E_ri (q_r.k_i) do_r,   dw = (1 + N')^T D,   y = beta dw = dv
//   G  <- e^{b_C} G + scale sum_r e^{b_r} q_r do_r^T - sum_r e^{b_r} k_r y_r^T
// where 1 + N' = (1 + A')^-1 with A'_ri = beta_r E_ri k_r.k_i (no division by beta, which may be 0). Its shape is the
// forward's: a product with the state, a triangular one, an update. All differences of b that are used are at most 0.
#pragma once

#include "kda_gd.hpp"
#include "kda_hd_core.hpp"

namespace kda {
namespace gd {

using hd::lane_value;
using hd::u32x2;
using hd::u32x4;

// ------------------------------------------------------------------ operands
// What rounding a pair left of its first (second) value: x - hi, exact, in one instruction. Where the pair's other value
// is not finite the result is NaN: only for pairs that are summed over, or of finite values. (-1 comes in a register: as
// an inline constant the instruction takes it for the upper half's.)
__device__ __forceinline__ float rest_lo(float x, uint32_t hi) {
    uint32_t one = 0x0000bf80u;
    asm("" : "+s"(one));
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, hi), __builtin_bit_cast(bf16x2, one), x, false);
}
__device__ __forceinline__ float rest_hi(float x, uint32_t hi) {
    uint32_t one = 0xbf800000u;
    asm("" : "+s"(one));
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, hi), __builtin_bit_cast(bf16x2, one), x, false);
}
// An operand in N bf16 parts (fp32 I/O: as it is): one for inputs, two hold a computed value to 2^-17 of it, three all
// its 24 bits. Products leave out the parts' products that are too small to show beside the smallest part.
template <bool BF, int N> struct Multi { Frag8<BF> p[BF ? N : 1]; };
template <bool BF> using Exact = Multi<BF, 1>;
template <bool BF> using Pair = Multi<BF, 2>;
template <int N>
__device__ __forceinline__ void set_multi(Multi<true, N> &m, const float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a = x[2 * i], b = x[2 * i + 1];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            m.p[n].p[i] = pack_bf16(a, b);
            if (n + 1 < N) {
                const float ra = rest_lo(a, m.p[n].p[i]), rb = rest_hi(b, m.p[n].p[i]);
                a = ra;
                b = rb;
            }
        }
    }
}
template <int N>
__device__ __forceinline__ void set_multi(Multi<false, N> &m, const float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m.p[0].f[i] = x[i];
}
template <bool BF, int N>
__device__ __forceinline__ Multi<BF, N> multi_of(const f32x4 &u, const f32x4 &w) {
    const float x[8] = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w};
    Multi<BF, N> m;
    set_multi(m, x);
    return m;
}
// c[i] += a[i] b[i] for M products at a time, their steps in turn: a matrix instruction waits for the one before it on its
// accumulator. A single a or b serves all.
template <bool BF, int M, int MA, int MB, int NA, int NB>
__device__ __forceinline__ void mmx(f32x4 (&c)[M], const Multi<BF, NA> (&a)[MA], const Multi<BF, NB> (&b)[MB]) {
    constexpr int PA = BF ? NA : 1, PB = BF ? NB : 1, MOST = PA > PB ? PA : PB;
#pragma unroll
    for (int s = 0; s < MOST; ++s)
#pragma unroll
        for (int i = 0; i <= s; ++i)
            if (i < PA && s - i < PB)
#pragma unroll
                for (int m = 0; m < M; ++m) c[m] = mma32(c[m], a[MA == 1 ? 0 : m].p[i], b[MB == 1 ? 0 : m].p[s - i]);
}
template <bool BF, int NA, int NB>
__device__ __forceinline__ f32x4 mmx(f32x4 c, const Multi<BF, NA> &a, const Multi<BF, NB> &b) {
    constexpr int PA = BF ? NA : 1, PB = BF ? NB : 1, MOST = PA > PB ? PA : PB;
#pragma unroll
    for (int s = 0; s < MOST; ++s)
#pragma unroll
        for (int i = 0; i <= s; ++i)
            if (i < PA && s - i < PB) c = mma32(c, a.p[i], b.p[s - i]);
    return c;
}

__device__ __forceinline__ void widen(const Frag8<true> &f, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf_lo(f.p[i]);
        x[2 * i + 1] = bf_hi(f.p[i]);
    }
}
__device__ __forceinline__ void widen(const Frag8<false> &f, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = f.f[i];
}

// The compiler would sink loads to where they are used.
#define KDA_ORDER __builtin_amdgcn_sched_barrier(0)

// ------------------------------------------------------------------ tokens
// An accumulator of 32 tokens is two tiles of 16; slot 4 tt + i of lane group g is row 4g + i of tile tt, token 16 tt + 4g
// + i. So the two tiles are, as they are, an operand whose slots are the chunk's tokens.
__device__ __forceinline__ int token_of(int tt, int g) { return 16 * tt + 4 * g; }
__device__ __forceinline__ int slot_token(int g, int j) { return token_of(j >> 2, g) + (j & 3); }

// ------------------------------------------------------------------ rows in LDS
// NCOL elements a row. bf16: the 16-byte slots of a row are permuted by an exclusive or with bits of its index. The LDS
// serves a 16-byte read in four steps of sixteen lanes, and the steps that matter take lanes 0-3, 12-15 and 20-27 and
// lanes 4-11, 16-19 and 28-31: eight rows at one slot and the other eight at the slot beside it, which the row's bits 2 and
// 3 keep on different banks (counting the lanes in order instead had every read of rows take 8 cycles, not 4). An 8-byte
// transposing read takes 32 lanes a step: 8 rows at two adjacent slots.
// fp32: rows padded by 16 bytes to the same end. Channels: slots 0-7 of a 32-deep product are channels 32c + 8g + j (bf16,
// one 16-byte read) or 4g + i and 16 + 4g + i (fp32), and a state's tile kt has its rows in the same order.
template <bool BF, int NCOL> struct Rw;
template <int NCOL> struct Rw<true, NCOL> {
    static constexpr int NS = NCOL / 8, RB = NCOL * 2;
    static constexpr int bytes(int rows) { return rows * RB; }
    static __device__ __forceinline__ int swz(int row) {
        const int high = NCOL == 128 ? (row & 3) << 2 : NCOL == 64 ? (row & 2) << 1 : 0;
        return high | (((row >> 1) ^ row) & 4) >> 1 | ((row >> 3) & 1);
    }
    static __device__ __forceinline__ int slot(int row, int s) { return row * RB + ((s ^ swz(row)) << 4); }
    static __device__ __forceinline__ int state_row(int kt, int g) { return 32 * (kt >> 1) + 8 * g + 4 * (kt & 1); }
    // channels 32c .. 32c + 31 of row l % 16 (+ what is added to t)
    static __device__ __forceinline__ int row_at(int lane) { return slot(lane & 15, lane >> 4); }
    static __device__ __forceinline__ Frag8<true> row_frag(const char *t, int at, int c) {
        const u32x4 u = *reinterpret_cast<const u32x4 *>(t + (at ^ (c << 6)));
        return Frag8<true>{{u.x, u.y, u.z, u.w}};
    }
    // The transposing read gives lane i of sixteen column i of a 4 x 16 block, of which its lane j holds the four elements
    // j % 4 of row j / 4. Rows 4g .. and, from `next` bytes on, the second four.
    static __device__ __forceinline__ Frag8<true> tr_frag(const char *t, int next) {
        typedef __attribute__((address_space(3))) s16x4 *lds4;
        const uint2 a = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(t)));
        const uint2 b = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(t + next)));
        return Frag8<true>{{a.x, a.y, b.x, b.y}};
    }
    // the chunk's tokens at column 16w + l % 16
    static __device__ __forceinline__ int col_at(int lane, int w) {
        return slot(4 * (lane >> 4) + ((lane >> 2) & 3), 2 * w + ((lane >> 1) & 1)) + (lane & 1) * 8;
    }
    static __device__ __forceinline__ Frag8<true> col_frag(const char *t, int at) { return tr_frag(t + at, 16 * RB); }
    // the chunk's tokens at the channels of a state's tile kt
    static __device__ __forceinline__ int tile_at(int lane) {
        return slot(4 * (lane >> 4) + ((lane >> 2) & 3), lane & 3);
    }
    static __device__ __forceinline__ Frag8<true> tile_frag(const char *t, int at, int kt) {
        return tr_frag(t + (at ^ (kt >> 1 << 6)) + 8 * (kt & 1), 16 * RB);
    }
    static __device__ __forceinline__ int quad(int row, int col) { return slot(row, col >> 3) + ((col & 4) << 1); }
    static __device__ __forceinline__ void load_quad(const char *t, int row, int col, float (&x)[4]) {
        const uint2 u = *reinterpret_cast<const uint2 *>(t + quad(row, col));
        x[0] = bf_lo(u.x); x[1] = bf_hi(u.x); x[2] = bf_lo(u.y); x[3] = bf_hi(u.y);
    }
};
template <int NCOL> struct Rw<false, NCOL> {
    static constexpr int NS = NCOL / 4, RB = (NCOL + 4) * 4;
    static constexpr int bytes(int rows) { return rows * RB; }
    static __device__ __forceinline__ int slot(int row, int s) { return row * RB + (s << 4); }
    static __device__ __forceinline__ int state_row(int kt, int g) { return 16 * kt + 4 * g; }
    static __device__ __forceinline__ int row_at(int lane) { return slot(lane & 15, lane >> 4); }
    static __device__ __forceinline__ Frag8<false> row_frag(const char *t, int at, int c) {
        const f32x4 u = *reinterpret_cast<const f32x4 *>(t + at + 128 * c);
        const f32x4 w = *reinterpret_cast<const f32x4 *>(t + at + 128 * c + 64);
        return Frag8<false>{{u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w}};
    }
    static __device__ __forceinline__ int col_at(int lane, int w) {
        return 4 * (lane >> 4) * RB + (16 * w + (lane & 15)) * 4;
    }
    static __device__ __forceinline__ Frag8<false> col_frag(const char *t, int at) {
        Frag8<false> f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f.f[j] = *reinterpret_cast<const float *>(t + at + j * RB);
            f.f[4 + j] = *reinterpret_cast<const float *>(t + at + (16 + j) * RB);
        }
        return f;
    }
    static __device__ __forceinline__ int tile_at(int lane) { return col_at(lane, 0); }
    static __device__ __forceinline__ Frag8<false> tile_frag(const char *t, int at, int kt) { return col_frag(t + 64 * kt, at); }
    static __device__ __forceinline__ int quad(int row, int col) { return row * RB + col * 4; }
    static __device__ __forceinline__ void load_quad(const char *t, int row, int col, float (&x)[4]) {
        const f32x4 u = *reinterpret_cast<const f32x4 *>(t + quad(row, col));
        x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
    }
    static __device__ __forceinline__ float load_one(const char *t, int row, int col) {
        return *reinterpret_cast<const float *>(t + quad(row, col));
    }
};

// C rows on their way to LDS, `pitch` bytes apart: a lane's offsets are made once, a chunk's place goes into the buffer's
// descriptor, and rows behind the last of `n` come as zeros (past the buffer's end). take() issues the loads, put() waits
// for them: a chunk's rows travel while the one before it is worked on.
template <bool BF, int NCOL, int C, int NT>
struct RowsIn {
    static constexpr int NS = Rw<BF, NCOL>::NS, RL = NT / NS;  // rows per round of loads
    static constexpr int NL = C > RL ? C / RL : 1, SIZE = NCOL * (BF ? 2 : 4);
    static_assert(NT % NS == 0 && C % (RL < C ? RL : C) == 0, "whole rounds of whole rows");
    uint32_t from[NL], pitch;
    int to[NL];
    u32x4 w[NL];
    __device__ __forceinline__ void init(int tid, uint32_t bytes) {
        pitch = bytes;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            int row = tid / NS + i * RL;
            if (RL > C) row &= C - 1;  // lanes left over bring a row once more
            from[i] = row * pitch + (tid % NS) * 16;
            to[i] = Rw<BF, NCOL>::slot(row, tid % NS);
        }
    }
    __device__ __forceinline__ void take(const char *p, int n) {
        const auto rows = __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(p), 0, (n - 1) * pitch + SIZE, 0x00027000);
#pragma unroll
        for (int i = 0; i < NL; ++i) w[i] = __builtin_amdgcn_raw_buffer_load_b128(rows, from[i], 0, 0);
    }
    __device__ __forceinline__ void put(char *t) const {
#pragma unroll
        for (int i = 0; i < NL; ++i) *reinterpret_cast<u32x4 *>(t + to[i]) = w[i];
    }
};
// The same for consecutive bytes.
template <int BYTES, int NT>
struct BytesIn {
    static constexpr int NL = (BYTES / 16 + NT - 1) / NT;
    static_assert(BYTES % 16 == 0, "16 bytes a load");
    uint32_t at[NL];
    u32x4 w[NL];
    __device__ __forceinline__ void init(int tid) {
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            at[i] = (i * NT + tid) * 16;
            if (at[i] >= BYTES) at[i] = BYTES - 16;  // lanes left over bring the last bytes once more
        }
    }
    __device__ __forceinline__ void take(const char *p) {
        const auto b = __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(p), 0, BYTES, 0x00027000);
#pragma unroll
        for (int i = 0; i < NL; ++i) w[i] = __builtin_amdgcn_raw_buffer_load_b128(b, at[i], 0, 0);
    }
    __device__ __forceinline__ void put(char *t) const {
#pragma unroll
        for (int i = 0; i < NL; ++i) *reinterpret_cast<u32x4 *>(t + at[i]) = w[i];
    }
};

// ------------------------------------------------------------------ records
// A tile of a record's matrix as an operand, and one of its entries: row m of the tile, source slot j of lane group g (bf16: of
// two parts; a third is too small to matter beside values that are not finite, and the tokens before them keep 2^-17).
template <bool BF>
__device__ __forceinline__ Pair<BF> load_mat(const char *m, int tt, int lane) {
    Pair<BF> p;
    const u32x4 u = *reinterpret_cast<const u32x4 *>(m + ((2 * tt) * 64 + lane) * 16);
    const u32x4 w = *reinterpret_cast<const u32x4 *>(m + ((2 * tt + 1) * 64 + lane) * 16);
    __builtin_memcpy(&p, &u, 16);
    __builtin_memcpy(reinterpret_cast<char *>(&p) + 16, &w, 16);
    return p;
}
template <bool BF>
__device__ __forceinline__ void store_mat(char *m, int tt, int lane, const Pair<BF> &p) {
    u32x4 u, w;
    __builtin_memcpy(&u, &p, 16);
    __builtin_memcpy(&w, reinterpret_cast<const char *>(&p) + 16, 16);
    *reinterpret_cast<u32x4 *>(m + ((2 * tt) * 64 + lane) * 16) = u;
    *reinterpret_cast<u32x4 *>(m + ((2 * tt + 1) * 64 + lane) * 16) = w;
}
template <bool BF>
__device__ __forceinline__ float mat_entry(const char *mat, int tt, int m, int g, int j) {
    if constexpr (BF) {
        const uint16_t *hi = reinterpret_cast<const uint16_t *>(mat + ((2 * tt) * 64 + 16 * g + m) * 16);
        return bf2f(hi[j]) + bf2f(hi[j + 512]);
    } else {
        return reinterpret_cast<const float *>(mat + ((2 * tt + (j >> 2)) * 64 + 16 * g + m) * 16)[j & 3];
    }
}

// Whether all of a wavefront's values are finite. A masked weight is 0, and 0 times an infinity is NaN, which a token
// must not take from one that it does not depend on: where a source is not finite, the products below go source by
// source, for the tokens that depend on it.
__device__ __forceinline__ bool all_finite(const float (&x)[8]) {
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) z = fmaf(x[i], 0.f, z);
    return __builtin_amdgcn_ballot_w64(z != 0.f) == 0;
}
// (Of a pair that rounds to an infinity the values count as such.)
__device__ __forceinline__ bool finite(const Pair<true> &p) {
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        z = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, p.p[0].p[i]), __builtin_bit_cast(bf16x2, 0u), z, false);
    return __builtin_amdgcn_ballot_w64(z != 0.f) == 0;
}
__device__ __forceinline__ bool finite(const Pair<false> &p) { return all_finite(p.p[0].f); }
// acc[token][column] += sum over sources j of M[token][j] x_j[column], x in the lanes of their columns. REV: sources from
// the token on, else up to it.
template <bool BF, bool REV>
__device__ __forceinline__ void mix_rows(f32x4 (&acc)[2], const float (&x)[8], const char *mat, int lane) {
    const int g = lane >> 4, li = lane & 15;
#pragma unroll 1
    for (int gs = 0; gs < 4; ++gs)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float xs = __shfl(x[j], 16 * gs + li);
            const int src = slot_token(gs, j);
#pragma unroll
            for (int tt = 0; tt < 2; ++tt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = token_of(tt, g) + i;
                    const float w = mat_entry<BF>(mat, tt, 4 * g + i, gs, j);
                    if (REV ? src >= t : src <= t) acc[tt][i] = fmaf(w, xs, acc[tt][i]);
                }
        }
}
// The same for accumulators of [column 4g + i][token 16 tt + l % 16].
template <bool BF>
__device__ __forceinline__ void mix_cols(f32x4 (&acc)[2], const float (&x)[8], const char *mat, int lane) {
    const int g = lane >> 4, li = lane & 15;
#pragma unroll 1
    for (int gs = 0; gs < 4; ++gs)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int src = slot_token(gs, j);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float xs = __shfl(x[j], 16 * gs + 4 * g + i);
#pragma unroll
                for (int tt = 0; tt < 2; ++tt) {
                    const float w = mat_entry<BF>(mat, tt, li, gs, j);
                    if (src <= 16 * tt + li) acc[tt][i] = fmaf(w, xs, acc[tt][i]);
                }
            }
        }
}

// ------------------------------------------------------------------ the pass over the states
template <bool BF, int K, int VT, int MODE>
struct StateLds {
    static constexpr int C = kChunkTokens, NB = BF ? 2 : 1;
    static constexpr int K_ = Rw<BF, K>::bytes(C), V_ = Rw<BF, VT>::bytes(C), R_ = rec_bytes(MODE != kForward);
    static constexpr int k = 0, q = k + NB * K_, v = q + (MODE == kErrors ? 0 : NB * K_), rec = v + NB * V_;
    static constexpr int bytes = rec + NB * R_;
};

// One (sequence, head), columns vt * VT .. of the state, a wavefront 16 of them: all K rows as fp32 accumulators, which
// are at once operands of the products with the state, so it never leaves the registers. A third of the wavefronts bring
// the rows, a chunk ahead in LDS and another on its way: done by the rest beside their products it took 700 cycles a chunk.
// bf16: products of inputs are exact, the state and computed operands go in as two bf16 parts, what is added to the state
// as three (the state after 4096 tokens is off by 5e-7 of its size, an output by what its own rounding gives: with three parts
// in the forward pass neighbouring bf16 values would still flip with the order of the sums). NP = 3, the gradients beside fp32
// gates: all of them three (4100 tokens of 32 heads: 177 us for 157).
//
// Bound by one wavefront's way through a chunk, whose steps wait for one another: forward 68 matrix instructions (1088
// cycles), about 230 vector ones (1100), 40 reads of an LDS that three others read as well (870): 3300 cycles, 170 us for
// 4096 tokens of one head, 195 for 96 (410 + 100 MB, 2.6 TB/s; matrix instructions run in 32% of the cycles of the units in
// use, LDS in 29%). Other orders of the products, the next chunk's first operands read ahead of the barrier, the state's parts
// formed between the update's products: all within 3%. Backward, both passes of 96 heads 411 us (1.4 GB, 3.4 TB/s).
template <bool BF, int K, int VT, int MODE, int NP>
__device__ __forceinline__ void state_pass(const StateArgs &A, int V, int64_t blk, char *smem) {
    using L = StateLds<BF, K, VT, MODE>;
    using RK = Rw<BF, K>;
    using RV = Rw<BF, VT>;
    constexpr int NW = VT / 16, NT = NW * 64, NS = NT / 2, KT = K / 16, KC = K / 32, C = kChunkTokens, NB = L::NB;
    constexpr int EB = BF ? 2 : 4;
    constexpr bool REV = MODE == kReverse;

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4,
              li = lane & 15;
    // the tiles of a head 8 workgroups apart: the same XCD, whose L2 then holds the rows they share
    const int64_t grp = blk / (8 * A.tiles);
    const int in = (int)(blk - grp * 8 * A.tiles), vt = in >> 3;
    const int64_t item = grp * 8 + (in & 7), nth = item / A.c.H;
    const int h = (int)(item - nth * A.c.H), group = A.c.H / A.c.Hk;
    if (nth >= A.c.N) return;
    const int64_t n = A.c.order ? A.c.order[nth] : nth;
    const Seq sq = seq_of(A.c, n);
    const int len = (int)(sq.t1 - sq.t0);  // under 2^31
    const int nch = (int)(((int64_t)len + C - 1) / C);
    const int col = vt * VT + wave * 16;  // this wavefront's first column

    // ---- the last third of the wavefronts: rows on their way to LDS
    if (wave >= NW) {
        const uint32_t lk = (uint32_t)A.c.Hk * (K * EB), lv = (uint32_t)A.c.H * (uint32_t)(V * EB);
        constexpr int RECB = L::R_;
        RowsIn<BF, K, C, NS> rk, rq;
        RowsIn<BF, VT, C, NS> rv;
        BytesIn<RECB, NS> rr;
        rk.init(tid - NT, lk);
        rq.init(tid - NT, lk);
        rv.init(tid - NT, lv);
        rr.init(tid - NT);
        // the next chunk to be asked for, and where it lies
        const int64_t c_first = REV ? nch - 1 : 0, step = REV ? -1 : 1;
        const char *pk = reinterpret_cast<const char *>(A.k) + ((sq.t0 + c_first * C) * A.c.Hk + h / group) * (K * EB);
        const char *pq = reinterpret_cast<const char *>(A.q) + ((sq.t0 + c_first * C) * A.c.Hk + h / group) * (K * EB);
        const char *pv = reinterpret_cast<const char *>(A.v) + (((sq.t0 + c_first * C) * A.c.H + h) * V + vt * VT) * EB;
        const char *prec = A.c.rec + ((sq.first + c_first) * A.c.H + h) * RECB;
        const int64_t step_k = step * C * lk, step_v = step * C * lv, step_r = step * A.c.H * RECB;
        auto take = [&](int i) __attribute__((always_inline)) {
            const int c = REV ? nch - 1 - i : i, m = len - c * C < C ? len - c * C : C;
            rk.take(pk, m);
            if constexpr (MODE != kErrors) rq.take(pq, m);
            rv.take(pv, m);
            rr.take(prec);
            pk += step_k;
            if constexpr (MODE != kErrors) pq += step_k;
            pv += step_v;
            prec += step_r;
        };
        auto put = [&](int b) __attribute__((always_inline)) {
            rk.put(smem + L::k + b * L::K_);
            if constexpr (MODE != kErrors) rq.put(smem + L::q + b * L::K_);
            rv.put(smem + L::v + b * L::V_);
            rr.put(smem + L::rec + b * L::R_);
        };
        if (nch > 0) {
            take(0);
            if constexpr (NB == 2) {
                put(0);
                if (nch > 1) take(1);
            }
        }
        for (int cc = 0; cc < nch; ++cc) {
            __syncthreads();
            if constexpr (NB == 1) {
                put(0);
                if (cc + 1 < nch) take(cc + 1);
                __syncthreads();
            } else if (cc + 1 < nch) {
                put((cc + 1) & 1);
                if (cc + 2 < nch) take(cc + 2);
            }
        }
        return;
    }

    // ---- the state at its start
    f32x4 st[KT];
    const int64_t sstate = (int64_t)K * V, nh = n * A.c.H + h;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
        st[kt] = zero4();
        if (A.s_init) {
            const float *p = A.s_init + nh * sstate + (int64_t)RK::state_row(kt, g) * V + col + li;
#pragma unroll
            for (int i = 0; i < 4; ++i) st[kt][i] = p[i * V];
        }
    }
    auto put_state = [&](float *s) __attribute__((always_inline)) {
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
            float *p = s + (int64_t)RK::state_row(kt, g) * V + col + li;
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i * V] = st[kt][i];
        }
    };

    hd::mfma_fence_state(reinterpret_cast<f32x4(&)[1][KT]>(st));  // the loads end here: no waits for them in the loop

    const uint32_t lv = (uint32_t)A.c.H * (uint32_t)(V * EB);
    const int64_t step_v = (REV ? -1 : 1) * (int64_t)C * lv;
    char *po = reinterpret_cast<char *>(A.o) + ((sq.t0 + (REV ? nch - 1 : 0) * (int64_t)C) * A.c.H + h) * V * EB;
    auto tokens_of = [&](int c) __attribute__((always_inline)) { return len - c * C < C ? len - c * C : C; };
    const int row0 = RK::row_at(lane), tile0 = RK::tile_at(lane), col0 = RV::col_at(lane, wave);
    Multi<BF, NP> sf[KC][1];  // the state as an operand
#pragma unroll
    for (int kc = 0; kc < KC; ++kc) sf[kc][0] = multi_of<BF, NP>(st[2 * kc], st[2 * kc + 1]);
    Frag8<BF> next[REV ? 2 : 1][2];  // the next chunk's third parts of P's transpose and N's, or of N
    auto thirds = [&](int c) __attribute__((always_inline)) {
        if constexpr (BF && NP == 3)
#pragma unroll
            for (int n = 0; n < (REV ? 2 : 1); ++n)
#pragma unroll
                for (int tt = 0; tt < 2; ++tt)
                    __builtin_memcpy(&next[n][tt],
                                     A.c.third + (((sq.first + c) * A.c.H + h) * 3 + (REV ? kMatPT - n : kMatN)) * kThirdBytes +
                                         tt * (kThirdBytes / 2) + lane * 16, 16);
    };
    if (nch > 0) thirds(REV ? nch - 1 : 0);
    for (int cc = 0; cc < nch; ++cc) {
        const int c = REV ? nch - 1 - cc : cc, b = cc & (NB - 1);
        __syncthreads();  // nobody reads the last chunk's rows any more (NB = 2: and this one's are there)
        if constexpr (NB == 1) __syncthreads();
        const char *sk = smem + L::k + b * L::K_, *sv = smem + L::v + b * L::V_, *sr = smem + L::rec + b * L::R_;
        const char *sq_ = smem + L::q + b * L::K_;
        (void)sq_;
        const float *wt = reinterpret_cast<const float *>(sr + rec_weights(MODE != kForward));
        auto weights = [&](int which, float (&w)[8]) __attribute__((always_inline)) {  // of the tokens in a lane's slots
            *reinterpret_cast<f32x4 *>(w) = *reinterpret_cast<const f32x4 *>(wt + which * C + token_of(0, g));
            *reinterpret_cast<f32x4 *>(w + 4) = *reinterpret_cast<const f32x4 *>(wt + which * C + token_of(1, g));
        };
        if (MODE == kErrors && c > 0 && (c & (A.c.seg - 1)) == 0)
            put_state(A.seed + ((sq.border + c / A.c.seg - 1) * A.c.H + h) * sstate);
        if (MODE == kReverse && c + 1 < nch && ((c + 1) & (A.c.seg - 1)) == 0)
            put_state(A.seed + ((sq.border + c / A.c.seg) * A.c.H + h) * sstate);

        Frag8<BF> third[REV ? 2 : 1][2];
        if constexpr (BF && NP == 3) {
#pragma unroll
            for (int n = 0; n < (REV ? 2 : 1); ++n)
#pragma unroll
                for (int tt = 0; tt < 2; ++tt) third[n][tt] = next[n][tt];
            if (cc + 1 < nch) thirds(REV ? c - 1 : c + 1);
        }
        auto mat_of = [&](Multi<BF, NP> &m, int which, int tt) __attribute__((always_inline)) {
            const Pair<BF> p = load_mat<BF>(sr + which * kMatBytes, tt, lane);
            __builtin_memcpy(&m, &p, sizeof(p));
            if constexpr (BF && NP == 3) m.p[2] = third[REV && which == kMatNT][tt];
        };

        // ---- products with the state: K S, and S^T q. The operands are asked for ahead of the products.
        f32x4 x[2] = {zero4(), zero4()}, y[2] = {zero4(), zero4()};
        Exact<BF> kf[KC][2], qf[KC][2];
        Multi<BF, NP> mat[2];
        float vx[8], r[8], z[8], w[8];
#pragma unroll
        for (int kc = 0; kc < KC; ++kc)
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) kf[kc][tt].p[0] = RK::row_frag(sk + 16 * tt * RK::RB, row0, kc);
        const Frag8<BF> vf = RV::col_frag(sv, col0);
        weights(REV ? kLeave : kEnter, w);
        KDA_ORDER;
#pragma unroll
        for (int kc = 0; kc < KC; ++kc) mmx(x, kf[kc], sf[kc]);
        KDA_ORDER;
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) mat_of(mat[tt], REV ? kMatPT : kMatN, tt);
        if constexpr (MODE == kForward)
#pragma unroll
            for (int kc = 0; kc < KC; ++kc)
#pragma unroll
                for (int tt = 0; tt < 2; ++tt) qf[kc][tt].p[0] = RK::row_frag(sq_ + 16 * tt * RK::RB, row0, kc);
        KDA_ORDER;
        widen(vf, vx);
        mfma_fence(x[0], x[1]);
        if constexpr (!REV) {
            // ---- z = r + N r,  r = v - e^b K S
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i >> 2][i & 3] = r[i] = fmaf(-w[i], x[i >> 2][i & 3], vx[i]);
        } else {
            // ---- D = e^{b_C - b} K G + P^T do, then dw = D + N'^T D
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i >> 2][i & 3] *= w[i];
            const bool fine = all_finite(vx);
            if (fine) {
                const Exact<BF> f[1] = {{{vf}}};
                mmx(x, mat, f);
            } else {
                mix_rows<BF, true>(x, vx, sr + kMatPT * kMatBytes, lane);
            }
            mfma_fence(x[0], x[1]);
#pragma unroll
            for (int i = 0; i < 8; ++i) r[i] = x[i >> 2][i & 3];
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) mat_of(mat[tt], kMatNT, tt);
        }
        {
            Multi<BF, NP> rp[1];
            set_multi(rp[0], r);
            mmx(x, mat, rp);
        }
        if constexpr (MODE == kForward)
#pragma unroll
            for (int kc = 0; kc < KC; ++kc) mmx(y, sf[kc], qf[kc]);
        KDA_ORDER;
        // the update's operands, while those products run
        Frag8<BF> kt_f[KT];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) kt_f[kt] = RK::tile_frag(sk, tile0, kt);
        const float total = wt[kTotal * C];
        if constexpr (!REV) weights(kLeaveBeta, w);
        if constexpr (MODE == kForward) {
            // ---- o^T = scale e^b S^T q + P z
            mfma_fence(y[0], y[1]);
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
                y[tt] *= wt[kEnterScaled * C + 16 * tt + li];
                mat_of(mat[tt], kMatP, tt);
            }
        }
        KDA_ORDER;
        mfma_fence(x[0], x[1]);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = x[i >> 2][i & 3];
        Pair<BF> zp[1];
        set_multi(zp[0], z);
        const bool fine_z = finite(zp[0]);
        if (!fine_z) {  // a source that is not shows in its own row
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i >> 2][i & 3] = r[i];
            mix_rows<BF, REV>(x, r, sr + (REV ? kMatNT : kMatN) * kMatBytes, lane);
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] = x[i >> 2][i & 3];
            if constexpr (MODE == kForward) {
                mix_cols<BF>(y, z, sr + kMatP * kMatBytes, lane);
                zp[0] = Pair<BF>{};
#pragma unroll
                for (int tt = 0; tt < 2; ++tt) mat[tt] = Multi<BF, NP>{};
            } else if constexpr (BF) {
#pragma unroll
                for (int i = 0; i < 4; ++i) split_bf16(z[2 * i], z[2 * i + 1], zp[0].p[0].p[i], zp[0].p[1].p[i]);
            }
        }
        if constexpr (MODE == kForward) {
            mmx(y, zp, mat);
        } else {
            // ---- z or dw by columns: [V][32], the parts one after the other
            char *rows = A.rows + ((sq.first + c) * A.c.H + h) * (int64_t)V * (C * (BF ? 2 * A.parts : 4));
            if constexpr (BF) {
                char *p = rows + (col + li) * (C * 2) + 16 * g;
#pragma unroll
                for (int n = 0; n < 2; ++n) __builtin_memcpy(p + n * V * (C * 2), &zp[0].p[n], 16);
                if (A.parts == 3) {
                    Multi<true, 3> all;
                    if (fine_z) {
                        set_multi(all, z);
                    } else {  // a token's parts by themselves: the gradients read them token by token
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t hi = zp[0].p[0].p[i], lo = zp[0].p[1].p[i];
                            all.p[2].p[i] = pack_bf16(z[2 * i] - bf_lo(hi) - bf_lo(lo), z[2 * i + 1] - bf_hi(hi) - bf_hi(lo));
                        }
                    }
                    __builtin_memcpy(p + 2 * V * (C * 2), &all.p[2], 16);
                }
            } else {
                char *p = rows + (col + li) * (C * 4) + 16 * g;
                *reinterpret_cast<f32x4 *>(p) = f32x4{z[0], z[1], z[2], z[3]};
                *reinterpret_cast<f32x4 *>(p + 64) = f32x4{z[4], z[5], z[6], z[7]};
            }
        }
        // ---- the state's update
        if constexpr (!REV) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] *= z[i];
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) st[kt] *= total;
            Multi<BF, 3> f;
            set_multi(f, w);
            constexpr int KG = KT < 4 ? KT : 4;  // products of different tiles follow each other
#pragma unroll
            for (int k0 = 0; k0 < KT; k0 += KG)
#pragma unroll
                for (int p = 0; p < (BF ? 3 : 1); ++p)
#pragma unroll
                    for (int j = 0; j < KG; ++j) st[k0 + j] = mma32(st[k0 + j], kt_f[k0 + j], f.p[p]);
        } else {
            float wq[8], be[8];
            weights(kEnterScaled, wq);
            weights(kBeta, be);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                z[i] *= be[i];  // dL/dz, which is dL/dv
                wq[i] *= vx[i];
            }
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) st[kt] *= total;
            Multi<BF, 3> f;
            set_multi(f, wq);
            constexpr int KG = KT < 4 ? KT : 4;
#pragma unroll
            for (int k0 = 0; k0 < KT; k0 += KG) {
                Frag8<BF> a[KG];
#pragma unroll
                for (int j = 0; j < KG; ++j) a[j] = RK::tile_frag(sq_, tile0, k0 + j);
#pragma unroll
                for (int p = 0; p < (BF ? 3 : 1); ++p)
#pragma unroll
                    for (int j = 0; j < KG; ++j) st[k0 + j] = mma32(st[k0 + j], a[j], f.p[p]);
            }
            KDA_ORDER;
            weights(kEnter, wq);
#pragma unroll
            for (int i = 0; i < 8; ++i) wq[i] *= -z[i];
            set_multi(f, wq);
#pragma unroll
            for (int k0 = 0; k0 < KT; k0 += KG)
#pragma unroll
                for (int p = 0; p < (BF ? 3 : 1); ++p)
#pragma unroll
                    for (int j = 0; j < KG; ++j) st[k0 + j] = mma32(st[k0 + j], kt_f[k0 + j], f.p[p]);
            const auto out = __builtin_amdgcn_make_buffer_rsrc(po, 0, (tokens_of(c) - 1) * lv + V * EB, 0x00027000);
            po += step_v;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t at = (uint32_t)slot_token(g, i) * lv + (uint32_t)(col + li) * EB;
                if constexpr (BF) __builtin_amdgcn_raw_buffer_store_b16((uint16_t)pack_bf16(z[i], 0.f), out, at, 0, 0);
                else __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, z[i]), out, at, 0, 0);
            }
        }
        if constexpr (MODE == kForward) {
            mfma_fence(y[0], y[1]);
            // the hardware drops the stores behind the chunk's last row (past the buffer's end)
            const auto out = __builtin_amdgcn_make_buffer_rsrc(po, 0, (tokens_of(c) - 1) * lv + V * EB, 0x00027000);
            po += step_v;
            const uint32_t at = li * lv + (uint32_t)(col + 4 * g) * EB;
#pragma unroll
            for (int tt = 0; tt < 2; ++tt)
                if constexpr (BF)
                    __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack_bf16(y[tt].x, y[tt].y), pack_bf16(y[tt].z, y[tt].w)},
                                                          out, at + 16 * tt * lv, 0, 0);
                else
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, y[tt]), out, at + 16 * tt * lv, 0, 0);
        }
        hd::mfma_fence_state(reinterpret_cast<f32x4(&)[1][KT]>(st));
#pragma unroll
        for (int kc = 0; kc < KC; ++kc) sf[kc][0] = multi_of<BF, NP>(st[2 * kc], st[2 * kc + 1]);
    }
    if (A.s_end) put_state(A.s_end + nh * sstate);
}

template <bool BF, int K, int VT>
__global__ __launch_bounds__(VT * 6, (VT == 128 ? 3 : 2)) void kda_gd_state_kernel(const StateArgs A, int V) {
    __shared__ __align__(16) char smem[StateLds<BF, K, VT, kForward>::bytes];
    state_pass<BF, K, VT, kForward, 2>(A, V, blockIdx.x + (int64_t)blockIdx.y * gridDim.x, smem);
}
// The backward call's two passes wait for nothing of each other's: one launch, the longer one's workgroups first.
template <bool BF, int K, int VT, int NP>
__global__ __launch_bounds__(VT * 6, (VT == 128 ? 3 : 2)) void kda_gd_states_kernel(const StateArgs R,
                                                                                          const StateArgs E, int V,
                                                                                          int64_t blocks) {
    __shared__ __align__(16) char smem[StateLds<BF, K, VT, kReverse>::bytes];
    const int64_t blk = blockIdx.x + (int64_t)blockIdx.y * gridDim.x;
    if (blk < blocks) state_pass<BF, K, VT, kReverse, NP>(R, V, blk, smem);
    else state_pass<BF, K, VT, kErrors, NP>(E, V, blk - blocks, smem);
}

}  // namespace gd
}  // namespace kda
