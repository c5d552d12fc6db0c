// Linear attention with one decay per head: the chunk kernel that its forward pass and every gradient share.
//
// With b_t the sum of the log-decays up to token t, the forward pass is
//   o_t = scale ( sum_{s<=t} e^{b_t - b_s} (q_t.k_s) v_s + e^{b_t} S_0^T q_t ),   S = sum e^{b_T - b_s} k_s v_s^T + e^{b_T} S_0
// and its gradients have the same form, with the roles of the tensors exchanged and, for dk and dv, time reversed:
//   dq: rows do against v, summing k;   dv: rows k against q, summing do;   dk: rows v against do, summing q.
// So one kernel computes, for rows a, b (KD channels) and c (VD channels) of a head,
//   y_t = s_intra sum_s D_ts (a_t.b_s) c_s + s_inter win_t St^T a_t,    St <- e^{b_C} St + s_up sum_s wup_s b_s c_s^T
// chunk by chunk: forward in time (s <= t, win = e^{b_t}, wup = e^{b_C - b_s}) or backward (REV: s >= t,
// win = e^{b_C - b_t}, wup = e^{b_s}). The differences of b are at most 0 wherever they are used, so no weight
// overflows however strong the decay; b is kept (base 2) as a multiple of 2^-8, whose sums and differences are exact, and
// a rest, so a token that decays everything (down to -inf, held at e^-104 = 0) does not cost its neighbours precision.
//
// Layout (16x16 matrix-core tiles, see kda_common.hpp). A workgroup owns one (segment of a sequence, head, tile of VT
// columns); each wavefront owns CT 16-column tiles of the state, all KD rows, as fp32 accumulators. An accumulator
// tile St[4g+i][l%16] is at once the left operand of St^T a, so the state never leaves the registers; y comes out
// transposed (four adjacent columns of one token per lane: one 8-byte store). The rows lie in LDS as loaded; operands
// that run along tokens come through the transposing LDS read (bf16) or element reads (fp32). The chunk's weighted
// products D (a.b) go through LDS once, shared by all wavefronts.
//
// Precision (bf16 I/O). Products of inputs are exact in the matrix cores' fp32 sums. Three operands are computed
// values. The weighted products D (a.b) and the state as an operand go in as two bf16 parts each, which hold a value to
// 2^-16: the error of a bf16 result against fp64 is then its own rounding's, 0.0017 of its size (with the weighted
// products in one part 1.4 times that, with the state in one part 1.1 to 1.2 times; the state's second part takes the
// forward pass of 4096 tokens of 96 heads from 151 to 161 us). wup c, which everything later in the sequence is summed
// from, goes in as three parts, all 24 bits of it, so the fp32 state carries no rounding of its operands.
//
// What bounds it. Per token and head of K = V = 128 in bf16 the forward pass moves 1 KB and multiplies 0.27 MFLOP in its
// two passes, of which 0.18 MFLOP are the three parts of wup c: at the card's rates the bytes take longer, but a chunk's
// steps (weighted products, one barrier, the state's products) follow each other, so what bounds it is their latency and
// the vector instructions that convert, scale and address, with two workgroups of 8 wavefronts a CU to hide behind one
// another: of the forward kernel's cycles 58% issue a vector instruction and 32% a matrix one. 4096 tokens of 96 heads:
// 110 us in the forward kernel, 48 us in the increments; 369 us in the gradients' kernel (the fastest of 20 dispatches).
// What brought the forward call there from 427 us of simple kernels: rows one chunk ahead (271), fewer exponentials (249),
// chunks of 32 tokens on 128 columns (198), zero weights in place of cleared rows (180), 8 wavefronts and addresses made
// anew (174), decays made 16 chunks at a time (162), stores without branches and 16-byte operand reads (156), segments'
// states formed by the workgroups that start from them (150); the state's second part took it to 161.
#pragma once

#include "kda_common.hpp"
#include "kda_hd.hpp"

namespace kda {
namespace hd {

typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;

constexpr int kChunk = 32;  // tokens per chunk

// ------------------------------------------------------------------ rows in LDS
// NCOL elements a row. bf16: the 16-byte slots of a row are permuted by an exclusive or with bits of the row's index,
// chosen so that 8 rows at one slot (a row read's eight lanes) and 4 rows at two adjacent slots (a transposing read's
// sixteen) fall on different banks. fp32: rows padded by 16 bytes to the same end.
//
// Which index an operand's slot or a state tile's row stands for is free as long as both operands of a product agree:
//   bf16: channel slots 0-7 of a 32-deep product <-> channels 32c + 8g + j (one 16-byte read of a row), so row 4g + i of
//         the state's tile kt is channel 32 (kt / 2) + 8g + 4 (kt % 2) + i; token slots <-> tokens 8g + j;
//   fp32: slots 0-3 <-> 4g + i, slots 4-7 <-> 16 + 4g + i, tile rows in order.
template <bool BF, int NCOL> struct Rows;
template <int NCOL> struct Rows<true, NCOL> {
    static constexpr int NS = NCOL / 8, RB = NCOL * 2;
    static constexpr int bytes(int rows) { return rows * RB; }
    static __device__ __forceinline__ int swz(int row) {
        if (NCOL == 32) return (row & 2) | ((row >> 2) & 1);
        return ((row & 3) << 1) | ((row >> 2) & 1) | (NCOL == 128 ? row & 8 : 0);
    }
    static __device__ __forceinline__ int slot(int row, int s) { return row * RB + ((s ^ swz(row)) << 4); }
    static __device__ __forceinline__ int quad(int row, int col) { return slot(row, col >> 3) + ((col & 4) << 1); }
    static __device__ __forceinline__ void put16(char *t, int row, int s, u32x4 w) {
        *reinterpret_cast<u32x4 *>(t + slot(row, s)) = w;
    }
    static __device__ __forceinline__ int state_row(int kt, int g) { return 32 * (kt >> 1) + 8 * g + 4 * (kt & 1); }
    static __device__ __forceinline__ int token(int half, int g) { return 8 * g + 4 * half; }  // of slots 4 half + i
    // Channels 32c .. 32c+31 of row l%16 (+ what is added to t). at: row_at(lane), the lane's address for c = 0; the
    // others differ from it in the bits of c alone.
    static __device__ __forceinline__ int row_at(int lane) { return slot(lane & 15, lane >> 4); }
    static __device__ __forceinline__ Frag8<true> row_frag(const char *t, int at, int c) {
        const u32x4 u = *reinterpret_cast<const u32x4 *>(t + (at ^ (c << 6)));
        Frag8<true> f;
        f.p[0] = u.x; f.p[1] = u.y; f.p[2] = u.z; f.p[3] = u.w;
        return f;
    }
    // 32 tokens at the column of lane l%16. The transposing read gives lane i of sixteen column i of a 4 x 16 block, of
    // which its lane j holds the four elements j % 4 of row j / 4. ats: the addresses for the first and second four
    // tokens of the lanes' groups (the row's bit 2 moves its slots by one).
    static __device__ __forceinline__ Frag8<true> tr_frag(const char *t, int at, int at4) {
        typedef __attribute__((address_space(3))) s16x4 *lds4;
        const s16x4 u = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(t + at));
        const s16x4 w = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(t + at4));
        const uint2 a = __builtin_bit_cast(uint2, u), b = __builtin_bit_cast(uint2, w);
        Frag8<true> f;
        f.p[0] = a.x; f.p[1] = a.y; f.p[2] = b.x; f.p[3] = b.y;
        return f;
    }
    static __device__ __forceinline__ int col_row(int lane) { return 8 * (lane >> 4) + ((lane >> 2) & 3); }
    // plain columns 16c + l%16
    static __device__ __forceinline__ int col_at(int lane) { return slot(col_row(lane), (lane >> 1) & 1) + (lane & 1) * 8; }
    static __device__ __forceinline__ Frag8<true> col_frag(const char *t, int at, int c) {
        const int x = at ^ (c << 5);
        return tr_frag(t, x, (x ^ 16) + 4 * RB);
    }
    // the channels of the state tile kt
    static __device__ __forceinline__ int tile_at(int lane) { return slot(col_row(lane), lane & 3); }
    static __device__ __forceinline__ Frag8<true> tile_frag(const char *t, int at, int kt) {
        const int x = at ^ (kt >> 1 << 6);
        return tr_frag(t, x + 8 * (kt & 1), (x ^ 16) + 4 * RB + 8 * (kt & 1));
    }
    static __device__ __forceinline__ void store_quad(char *t, int row, int col, float a, float b, float c, float d) {
        *reinterpret_cast<uint2 *>(t + quad(row, col)) = make_uint2(pack_bf16(a, b), pack_bf16(c, d));
    }
    static __device__ __forceinline__ float load_one(const char *t, int row, int col) {
        return bf2f(*reinterpret_cast<const uint16_t *>(t + quad(row, col) + 2 * (col & 3)));
    }
    static __device__ __forceinline__ void load_quad(const char *t, int row, int col, float (&x)[4]) {
        const uint2 u = *reinterpret_cast<const uint2 *>(t + quad(row, col));
        x[0] = bf_lo(u.x); x[1] = bf_hi(u.x); x[2] = bf_lo(u.y); x[3] = bf_hi(u.y);
    }
};
template <int NCOL> struct Rows<false, NCOL> {
    static constexpr int NS = NCOL / 4, RB = (NCOL + 4) * 4;
    static constexpr int bytes(int rows) { return rows * RB; }
    static __device__ __forceinline__ int quad(int row, int col) { return row * RB + col * 4; }
    static __device__ __forceinline__ void put16(char *t, int row, int s, u32x4 w) {
        *reinterpret_cast<u32x4 *>(t + row * RB + (s << 4)) = w;
    }
    static __device__ __forceinline__ int state_row(int kt, int g) { return 16 * kt + 4 * g; }
    static __device__ __forceinline__ int token(int half, int g) { return 16 * half + 4 * g; }
    static __device__ __forceinline__ int row_at(int lane) { return quad(lane & 15, 4 * (lane >> 4)); }
    static __device__ __forceinline__ Frag8<false> row_frag(const char *t, int at, int c) {
        const f32x4 u = *reinterpret_cast<const f32x4 *>(t + at + 128 * c);
        const f32x4 w = *reinterpret_cast<const f32x4 *>(t + at + 128 * c + 64);
        return Frag8<false>{{u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w}};
    }
    static __device__ __forceinline__ int col_at(int lane) { return quad(4 * (lane >> 4), lane & 15); }
    static __device__ __forceinline__ Frag8<false> col_frag(const char *t, int at, int c) {
        Frag8<false> f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f.f[j] = *reinterpret_cast<const float *>(t + at + 64 * c + j * RB);
            f.f[4 + j] = *reinterpret_cast<const float *>(t + at + 64 * c + (16 + j) * RB);
        }
        return f;
    }
    static __device__ __forceinline__ int tile_at(int lane) { return col_at(lane); }
    static __device__ __forceinline__ Frag8<false> tile_frag(const char *t, int at, int kt) { return col_frag(t, at, kt); }
    static __device__ __forceinline__ void store_quad(char *t, int row, int col, float a, float b, float c, float d) {
        *reinterpret_cast<float4 *>(t + quad(row, col)) = make_float4(a, b, c, d);
    }
    static __device__ __forceinline__ float load_one(const char *t, int row, int col) {
        return *reinterpret_cast<const float *>(t + quad(row, col));
    }
    static __device__ __forceinline__ void load_quad(const char *t, int row, int col, float (&x)[4]) {
        const float4 u = *reinterpret_cast<const float4 *>(t + quad(row, col));
        x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
    }
};

// C rows of a chunk on their way to LDS: from p, `pitch` bytes apart; rows behind the last of `n` repeat it (their
// weights are zero). take() issues the loads, put() waits for them: a chunk's rows travel while the one before it is
// worked on. A lane's offsets (32 rows: under 2^31) grow with the row, so holding them to the last row's is a minimum;
// the base is the same for all lanes.
template <bool BF, int NCOL, int C, int NT>
struct Stage {
    static constexpr int NS = Rows<BF, NCOL>::NS, RL = NT / NS;  // rows per round of loads
    static constexpr int NL = C > RL ? C / RL : 1;
    static_assert(NT % NS == 0 && C % (RL < C ? RL : C) == 0, "whole rounds of whole rows");
    u32x4 w[NL];
    __device__ __forceinline__ void take(int tid, const char *p, uint32_t pitch, int n) {
        const uint32_t col = ((uint32_t)tid % NS) * 16u, off = ((uint32_t)tid / NS) * pitch + col;
        const uint32_t last = (uint32_t)(n - 1) * pitch + col;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const uint32_t at = off + (uint32_t)i * RL * pitch;
            w[i] = *reinterpret_cast<const u32x4 *>(p + (at < last ? at : last));
        }
    }
    __device__ __forceinline__ void put(int tid, char *t) const {
        const int row = (uint32_t)tid / NS, s = (uint32_t)tid % NS;
        if (RL > C && row >= C) return;
#pragma unroll
        for (int i = 0; i < NL; ++i) Rows<BF, NCOL>::put16(t, row + i * RL, s, w[i]);
    }
};

// A log-decay in base 2: a multiple of 2^-8 (a chunk's sum is at most 32 * 151 in size: 21 bits, exact in fp32) and a
// rest of at most 2^-9 (2^-4 in a chunk's sum).
struct Decay { float hi, lo; };
__device__ __forceinline__ Decay decay_base2(float g) {
    g = g < -104.f ? -104.f : g;  // e^-104 is 0 in fp32; NaN stays
    constexpr float L2E = 1.4426950408889634f, L2E_LO = 1.9259629911266175e-8f;  // log2(e) in two parts
    const float x = g * L2E, rest = fmaf(g, L2E, -x) + g * L2E_LO;
    const float hi = rintf(x * 256.f) * 0.00390625f;
    return Decay{hi, (x - hi) + rest};
}
__device__ __forceinline__ float lane_value(float x, int lane) {  // the same for all lanes
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), lane));
}

// The pair as it was packed: the compiler would convert each half again to take it from its value.
__device__ __forceinline__ uint32_t seen(uint32_t x) {
    asm("" : "+v"(x));
    return x;
}
// Two fp32 tiles of the state (rows 32c .. 32c+31, one column tile) as a left operand, and the rest of its rounding.
__device__ __forceinline__ void state_frag(const f32x4 &u, const f32x4 &w, Frag8<true> &hi, Frag8<true> &lo) {
    const float x[8] = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        hi.p[i] = seen(pack_bf16(x[2 * i], x[2 * i + 1]));
        lo.p[i] = pack_bf16(x[2 * i] - bf_lo(hi.p[i]), x[2 * i + 1] - bf_hi(hi.p[i]));
    }
}
__device__ __forceinline__ void state_frag(const f32x4 &u, const f32x4 &w, Frag8<false> &hi, Frag8<false> &lo) {
    hi = Frag8<false>{{u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w}};
    lo = hi;
}
// w c as three bf16 operands whose sum has all 24 bits (fp32: as it is)
__device__ __forceinline__ void scaled_frags(const Frag8<true> &c, const float (&w)[8], Frag8<true> (&f)[3]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float x = bf_lo(c.p[i]) * w[2 * i], y = bf_hi(c.p[i]) * w[2 * i + 1];
        f[0].p[i] = seen(pack_bf16(x, y));
        const float x1 = x - bf_lo(f[0].p[i]), y1 = y - bf_hi(f[0].p[i]);
        f[1].p[i] = seen(pack_bf16(x1, y1));
        f[2].p[i] = pack_bf16(x1 - bf_lo(f[1].p[i]), y1 - bf_hi(f[1].p[i]));
    }
}
__device__ __forceinline__ void scaled_frags(const Frag8<false> &c, const float (&w)[8], Frag8<false> (&f)[1]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[0].f[i] = c.f[i] * w[i];
}

// Whether all entries of an operand in the wavefront are finite: 0 times them is 0.
__device__ __forceinline__ bool all_finite(const Frag8<true> &f) {
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        z = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, f.p[i]), __builtin_bit_cast(bf16x2, 0u), z, false);
    return __builtin_amdgcn_ballot_w64(z != 0.f) == 0;
}
__device__ __forceinline__ bool all_finite(const Frag8<false> &f) {
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) z = fmaf(f.f[i], 0.f, z);
    return __builtin_amdgcn_ballot_w64(z != 0.f) == 0;
}

// One wait for a whole register tile of products (see mfma_fence).
template <int M, int N>
__device__ __forceinline__ void mfma_fence_state(f32x4 (&x)[M][N]) {
    if constexpr (M * N <= 4) {
        f32x4 *f = &x[0][0];
        if constexpr (M * N == 2) mfma_fence(f[0], f[1]);
        else mfma_fence(f[0], f[1], f[2], f[3]);
    } else {
        f32x4 *f = &x[0][0];
#pragma unroll
        for (int i = 0; i < M * N; i += 8)
            asm volatile("s_nop 7\n\ts_nop 7"
                         : "+v"(f[i]), "+v"(f[i + 1]), "+v"(f[i + 2]), "+v"(f[i + 3]), "+v"(f[i + 4]), "+v"(f[i + 5]),
                           "+v"(f[i + 6]), "+v"(f[i + 7]));
    }
}

// Where a pass keeps what in LDS. bf16 holds rows twice, the next chunk's arrive while this one's are read (fp32's would
// leave one workgroup per CU).
template <bool BF, int KD, int VT, int NW, bool INC, bool DG>
struct Lds {
    static constexpr int C = kChunk, NB = BF ? 2 : 1, DB = 2 * NW;  // DB: chunks whose decays are made at a time
    static constexpr int K = Rows<BF, KD>::bytes(C), V = Rows<BF, VT>::bytes(C), P = Rows<BF, C>::bytes(C);
    static constexpr int b = 0, c = b + NB * K, a = c + NB * V, x = a + (INC ? 0 : NB * K), p = x + (DG ? NB * V : 0);
    static constexpr int pl = p + (INC ? 0 : P), wup = pl + (BF && !INC ? P : 0), win = wup + DB * C * 4;
    static constexpr int bh = win + (INC ? 0 : DB * C * 4), bl = bh + (INC ? 0 : DB * C * 4);
    static constexpr int f = bl + (INC ? 0 : DB * C * 4), ec = f + (INC ? 0 : DB * C * 4), u = ec + DB * 4;
    static constexpr int red = u + (DG ? NW * C * 4 : 0), bytes = red + NW * 4;
};

// One (segment, head), column tile vt; NW * 64 threads, Lds::bytes of LDS. TS: states are stored by columns (KD adjacent
// rows), else by rows (VD adjacent columns).
template <bool BF, int KD, int VT, int NW, bool REV, bool INC, bool DG, bool YF, bool TS>
__device__ __forceinline__ void chunk_pass(const CoreArgs &A, int64_t item, int vt, char *smem) {
    using L = Lds<BF, KD, VT, NW, INC, DG>;
    constexpr int NT = NW * 64, CT = VT / (16 * NW), KT = KD / 16, KC = KD / 32;
    constexpr int C = kChunk, TT = C / 16, SC = C / 32;  // token tiles; 32-token steps
    constexpr int DB = L::DB, NB = L::NB;
    constexpr int NPART = BF ? 3 : 1;
    static_assert(CT >= 1 && CT * 16 * NW == VT, "column tiles per wavefront");
    using E = typename IO<BF>::T;
    using RK = Rows<BF, KD>;
    using RV = Rows<BF, VT>;
    using RP = Rows<BF, C>;
    constexpr int SZ_K = L::K, SZ_V = L::V, SZ_P = L::P;
    char *const s_a = smem + L::a, *const s_b = smem + L::b, *const s_c = smem + L::c, *const s_x = smem + L::x;
    char *const s_p = smem + L::p, *const s_pl = smem + L::pl;
    float(*const s_wup2)[C] = reinterpret_cast<float(*)[C]>(smem + L::wup);
    float(*const s_win2)[C] = reinterpret_cast<float(*)[C]>(smem + L::win);
    float(*const s_bh2)[C] = reinterpret_cast<float(*)[C]>(smem + L::bh);
    float(*const s_bl2)[C] = reinterpret_cast<float(*)[C]>(smem + L::bl);
    float(*const s_f2)[C] = reinterpret_cast<float(*)[C]>(smem + L::f);
    float(*const s_u)[C] = reinterpret_cast<float(*)[C]>(smem + L::u);
    float *const s_ec2 = reinterpret_cast<float *>(smem + L::ec), *const s_red = reinterpret_cast<float *>(smem + L::red);
    (void)s_a; (void)s_x; (void)s_p; (void)s_pl; (void)s_u; (void)s_red;

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4,
              li = lane & 15;
    const int64_t slot = item / A.H;
    const int h = (int)(item - slot * A.H);
    const Segment sg = segment_of(A, slot);
    if (sg.seq < 0) return;
    if (INC && (REV ? sg.j == 0 : sg.j == sg.nseg - 1)) return;  // no segment needs what it would add

    const int64_t nh = (int64_t)sg.seq * A.H + h;
    const int64_t sstate = (int64_t)KD * A.VD;
    const int col0 = vt * VT + wave * CT * 16;  // this wavefront's first column
    const int len = (int)(sg.t1 - sg.t0), nch = (len + C - 1) / C;

    // ---- the state at the segment's start (REV: at its end)
    f32x4 st[KT][CT];
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) st[kt][ct] = zero4();
    // where a lane's first entry of a state tile lies in a state, in bytes, and its four entries
    const uint32_t vd4 = 4 * (uint32_t)A.VD;
    auto state_at = [&](int lane, int kt, int ct) __attribute__((always_inline)) {
        const uint32_t r = RK::state_row(kt, lane >> 4), c = col0 + 16 * ct + (lane & 15);
        return TS ? (c * KD + r) * 4u : r * vd4 + c * 4u;
    };
    auto get_state = [&](const float *state, int lane, int kt, int ct) __attribute__((always_inline)) -> f32x4 {
        const char *p = reinterpret_cast<const char *>(state);
        const uint32_t at = state_at(lane, kt, ct);
        if constexpr (TS) return *reinterpret_cast<const f32x4 *>(p + at);
        f32x4 x;
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float *>(p + (at + i * vd4));
        return x;
    };
    if constexpr (!INC) {
        auto add_state = [&](float d, const float *p) __attribute__((always_inline)) {  // st <- d st + the state at p
            int at = lane;
            asm volatile("" : "+v"(at));  // no addresses kept over the loop below
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    const f32x4 x = get_state(p, at, kt, ct);
#pragma unroll
                    for (int i = 0; i < 4; ++i) st[kt][ct][i] = fmaf(st[kt][ct][i], d, x[i]);
                }
        };
        const bool first = REV ? sg.j == sg.nseg - 1 : sg.j == 0;
        const bool fold = !REV && sg.nseg <= A.fold;
        if (!first && !fold) add_state(0.f, A.s_seg + (slot * A.H + h) * sstate);
        else if (A.s_init) add_state(0.f, A.s_init + nh * sstate);
        if (fold)
            for (int64_t at = (slot - sg.j) * A.H + h; at < slot * A.H; at += A.H)
                add_state(__builtin_amdgcn_exp2f(A.seg_decay[at]), A.s_seg + at * sstate);
    }
    mfma_fence_state(st);  // the loads end here: a wait for them inside the loop would hold up the rows under way
    // ---- what the border behind the segment passes on to its log-decays: <state gradient, state> there. (Behind the
    // last one the state is not known yet: the last kernel adds its part.)
    if constexpr (DG && REV) {
        float dot = 0.f;
        if (sg.j < sg.nseg - 1) {
            const float *se = A.s_seg_fwd + ((slot + 1) * A.H + h) * sstate;
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    const f32x4 x = get_state(se, lane, kt, ct);
#pragma unroll
                    for (int i = 0; i < 4; ++i) dot += st[kt][ct][i] * x[i];
                }
        }
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) dot += __shfl_xor(dot, d);
        if (lane == 0) s_red[wave] = dot;
        __syncthreads();
        if (threadIdx.x == 0) {
#pragma unroll
            for (int w = 1; w < NW; ++w) dot += s_red[w];
            A.border[((int64_t)vt * A.slots + slot) * A.H + h] = dot;
        }
    }

    // the head's rows and the bytes from one token's to the next
    constexpr int EB = BF ? 2 : 4;
    const uint32_t la = (uint32_t)(A.H / A.ga) * (KD * EB), lb = (uint32_t)(A.H / A.gb) * (KD * EB);
    const uint32_t lc = (uint32_t)(A.H / A.gc) * (uint32_t)(A.VD * EB), lx = (uint32_t)(A.H / A.gx) * (uint32_t)(A.VD * EB);
    const char *pa = reinterpret_cast<const char *>(A.a) + (int64_t)(h / A.ga) * (KD * EB);
    const char *pb = reinterpret_cast<const char *>(A.b) + (int64_t)(h / A.gb) * (KD * EB);
    const char *pc = reinterpret_cast<const char *>(A.c) + ((int64_t)(h / A.gc) * A.VD + vt * VT) * EB;
    const char *px = reinterpret_cast<const char *>(A.x) + ((int64_t)(h / A.gx) * A.VD + vt * VT) * EB;

    if constexpr (!INC) {  // tiles across the diagonal that are read but never computed
        for (int i = threadIdx.x; i < SZ_P / 16; i += NT) {
            reinterpret_cast<uint4 *>(s_p)[i] = make_uint4(0, 0, 0, 0);
            if constexpr (BF) reinterpret_cast<uint4 *>(s_pl)[i] = make_uint4(0, 0, 0, 0);
        }
    }
    float btot = 0.f;
    const int lane0 = lane, rowk0 = RK::row_at(lane), tilek0 = RK::tile_at(lane), rowv0 = RV::row_at(lane);
    const int rowp0 = RP::row_at(lane);
    const int colv0 = BF ? RV::col_at(lane) ^ (wave * CT << 5) : RV::col_at(lane) + 64 * wave * CT;
    auto chunk_at = [&](int i, int64_t &tc, int &n) __attribute__((always_inline)) {  // its first token and how many
        tc = sg.t0 + (int64_t)(REV ? nch - 1 - i : i) * C;
        n = (int)(sg.t1 - tc < C ? sg.t1 - tc : C);
    };
    // The decays of DB chunks are made at a time, two by each wavefront (a token per lane), from log-decays that were
    // loaded while the DB chunks before were worked on.
    static_assert(C == 32, "two chunks of two tiles per wavefront");
    auto take_decay = [&](int lane, int first) __attribute__((always_inline)) -> float {
        const int i = first + 2 * wave + (lane >> 5), t = lane & 31;
        int64_t tc;
        int n;
        chunk_at(i, tc, n);
        if (i >= nch || t >= n) return 0.f;
        return A.g_head ? reinterpret_cast<const float *>(A.g)[h]
                        : IO<BF>::ld(reinterpret_cast<const E *>(A.g), (tc + t) * A.H + h);
    };
    auto put_decay = [&](int lane, float gv, int first) __attribute__((always_inline)) {
        const int i = first + 2 * wave + (lane >> 5), t = lane & 31, at = 2 * wave + (lane >> 5);
        int64_t tc;
        int n;
        chunk_at(i, tc, n);
        const bool live = i < nch && t < n;  // the others carry no weight, into the state, out of it or to each other
        Decay d = decay_base2(gv);
        d.hi = row_scan16(d.hi);
        d.lo = row_scan16(d.lo);
        // a source's weight up to its tile's edge on the output's side
        const float f = REV ? __builtin_amdgcn_exp2f(d.hi + d.lo)
                            : __builtin_amdgcn_exp2f((row_last(d.hi) - d.hi) + (row_last(d.lo) - d.lo));
        const float h0 = lane < 32 ? lane_value(d.hi, 15) : lane_value(d.hi, 47);
        const float l0 = lane < 32 ? lane_value(d.lo, 15) : lane_value(d.lo, 47);
        d.hi += lane & 16 ? h0 : 0.f;
        d.lo += lane & 16 ? l0 : 0.f;
        const float h31 = lane_value(d.hi, 31), l31 = lane_value(d.lo, 31);
        const float h63 = lane_value(d.hi, 63), l63 = lane_value(d.lo, 63);
        // Of a pair of chunks that decays mildly the first leaves the state undecayed (what it adds is scaled up
        // instead, by less than 2^24) and the second decays it for both.
        const bool both = first + 2 * wave + 1 < nch && h31 + l31 > -24.f;
        const float hc = lane < 32 ? h31 : h63, lc2 = lane < 32 ? l31 : l63;
        const float uh = both && lane < 32 ? h31 : 0.f, ul = both && lane < 32 ? l31 : 0.f;    // added to the state
        const float rh = both && lane >= 32 ? h31 : 0.f, rl = both && lane >= 32 ? l31 : 0.f;  // read from it
        const float dh = REV ? d.hi : hc - d.hi, dl = REV ? d.lo : lc2 - d.lo;  // from a token to the state behind it
        const float eh = REV ? hc - d.hi : d.hi, el = REV ? lc2 - d.lo : d.lo;  // from the state before it to a token
        const float wup = __builtin_amdgcn_exp2f((dh - uh) + (dl - ul)), win = __builtin_amdgcn_exp2f((eh + rh) + (el + rl));
        s_wup2[at][t] = live ? wup * A.s_up : 0.f;
        if constexpr (!INC) {
            s_bh2[at][t] = d.hi;
            s_bl2[at][t] = d.lo;
            s_f2[at][t] = live ? f * A.s_intra : 0.f;
            s_win2[at][t] = live ? win * A.s_inter : 0.f;
        }
        if (t == 0) s_ec2[at] = __builtin_amdgcn_exp2f(((hc - uh) + rh) + ((lc2 - ul) + rl));
        if constexpr (INC) btot += hc + lc2;  // lanes 0 and 32: this wavefront's chunks
    };
    Stage<BF, KD, C, NT> ra, rb;
    Stage<BF, VT, C, NT> rc, rx;
    auto take_rows = [&](int tid, int i) __attribute__((always_inline)) {
        int64_t tc;
        int n;
        chunk_at(i, tc, n);
        if constexpr (!INC) ra.take(tid, pa + tc * la, la, n);
        rb.take(tid, pb + tc * lb, lb, n);
        rc.take(tid, pc + tc * lc, lc, n);
        if constexpr (DG) rx.take(tid, px + tc * lx, lx, n);
    };
    auto put_rows = [&](int tid, int i) __attribute__((always_inline)) {
        const int j = i & (NB - 1);
        if constexpr (!INC) ra.put(tid, s_a + j * SZ_K);
        rb.put(tid, s_b + j * SZ_K);
        rc.put(tid, s_c + j * SZ_V);
        if constexpr (DG) rx.put(tid, s_x + j * SZ_V);
    };
    float gnext = 0.f;
    if (nch > 0) {
        take_rows(threadIdx.x, 0);
        gnext = take_decay(lane, 0);
        if constexpr (NB == 2) {
            put_rows(threadIdx.x, 0);
            if (nch > 1) take_rows(threadIdx.x, 1);
        }
    }
    if constexpr (!INC) {
        // As many stores as a chunk ends with, into a buffer of no bytes (nothing is written): rows are waited for by
        // how many memory operations came after them, and the loop's first chunk has to look like the others, or all of
        // them would wait for the last chunk's stores as well.
        const auto none = __builtin_amdgcn_make_buffer_rsrc(A.y, 0, 0, 0x00027000);
#pragma unroll
        for (int i = 0; i < CT * TT; ++i) __builtin_amdgcn_raw_buffer_store_b64(u32x2{0, 0}, none, 16 * i, 0, 0);
    }

    for (int cc = 0; cc < nch; ++cc) {
        int64_t tc;
        int n;
        chunk_at(cc, tc, n);
        const int buf = cc & (DB - 1), rbuf = cc & (NB - 1);
        const float *s_wup = s_wup2[buf], *s_win = s_win2[INC ? 0 : buf], *s_bh = s_bh2[INC ? 0 : buf],
                    *s_bl = s_bl2[INC ? 0 : buf], *s_f = s_f2[INC ? 0 : buf];
        // The rows' buffer enters the lanes' addresses (its size is above all their bits). What is derived from them is
        // made anew each chunk, from values that the compiler cannot see through: kept over the loop, the some forty
        // addresses would take the registers the products need.
        int rowk = rowk0 + rbuf * SZ_K, tilek = tilek0 + rbuf * SZ_K, rowv = rowv0 + rbuf * SZ_V;
        int colv = colv0 + rbuf * SZ_V, rowp = rowp0, lane = lane0;
        asm volatile("" : "+v"(rowk), "+v"(tilek), "+v"(rowv), "+v"(colv), "+v"(rowp), "+v"(lane));
        const int g = lane >> 4, li = lane & 15;
        (void)rowk; (void)rowv; (void)rowp; (void)s_a; (void)s_x; (void)s_win; (void)s_bh; (void)s_bl; (void)s_f;
        __syncthreads();  // nobody reads the last chunk's rows any more (NB = 2: and this one's are there)
        if (buf == 0) {
            put_decay(lane, gnext, cc);
            if (cc + DB < nch) gnext = take_decay(lane, cc + DB);
        }
        if constexpr (NB == 1) {
            put_rows(threadIdx.x, cc);
            if (cc + 1 < nch) take_rows(threadIdx.x, cc + 1);
        }
        if (NB == 1 || buf == 0) __syncthreads();
        if (NB == 2 && cc + 1 < nch) {
            put_rows(threadIdx.x, cc + 1);
            if (cc + 2 < nch) take_rows(threadIdx.x, cc + 2);
        }

        // ---- weighted products D (a.b), tile by tile, transposed: lane holds sources 16ts+4g+i of token 16tt+l%16
        if constexpr (!INC) {
            if constexpr (DG && REV)
                if (lane < C) s_u[wave][lane] = 0.f;
            constexpr int NTILE = TT * (TT + 1) / 2;
            for (int p = wave; p < NTILE; p += NW) {
                int x = 0, y = p;
                while (y > x) { y -= x + 1; ++x; }  // p-th pair (x, y <= x)
                const int tt = REV ? y : x, ts = REV ? x : y;
                f32x4 acc = zero4(), acd = zero4();
                Frag8<BF> fb[KC], fa[KC];
#pragma unroll
                for (int c = 0; c < KC; ++c) {
                    fb[c] = RK::row_frag(s_b + 16 * ts * RK::RB, rowk, c);
                    fa[c] = RK::row_frag(s_a + 16 * tt * RK::RB, rowk, c);
                }
#pragma unroll
                for (int c = 0; c < KC; ++c) acc = mma32(acc, fb[c], fa[c]);
                if constexpr (DG && REV) {
#pragma unroll
                    for (int c = 0; c < VT / 32; ++c)
                        acd = mma32(acd, RV::row_frag(s_c + 16 * ts * RV::RB, rowv, c), RV::row_frag(s_x + 16 * tt * RV::RB, rowv, c));
                }
                const int t = 16 * tt + li;
                const float th = s_bh[t], tl = s_bl[t];
                f32x4 w;
                if (tt == ts) {
                    const f32x4 sh = *reinterpret_cast<const f32x4 *>(s_bh + 16 * ts + 4 * g);
                    const f32x4 sl = *reinterpret_cast<const f32x4 *>(s_bl + 16 * ts + 4 * g);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w[i] = __builtin_amdgcn_exp2f(REV ? (sh[i] - th) + (sl[i] - tl) : (th - sh[i]) + (tl - sl[i])) *
                               A.s_intra;
                    mfma_fence(acc, acd);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int s = 16 * ts + 4 * g + i;
                        const bool in_past = REV ? s >= t && s < n : s <= t;
                        w[i] = in_past ? acc[i] * w[i] : 0.f;
                        if constexpr (DG && REV) acd[i] = in_past ? acd[i] : 0.f;
                    }
                } else {
                    // over the edge between the tiles: the source's weight up to it, the output's from there
                    const int e = REV ? 16 * ts - 1 : 16 * ts + 15;
                    w = *reinterpret_cast<const f32x4 *>(s_f + 16 * ts + 4 * g) *
                        __builtin_amdgcn_exp2f(REV ? (s_bh[e] - th) + (s_bl[e] - tl) : (th - s_bh[e]) + (tl - s_bl[e]));
                    mfma_fence(acc, acd);
                    w *= acc;
                }
                if constexpr (DG && REV) {
                    // pairs (row s, column t) of the log-decays' gradient: + at the row, - at the column
                    float csum = 0.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float X = w[i] * acd[i];
                        csum += X;
                        const float r = row_scan16(X);  // the row's sum, in its last lane
                        if (li == 15) s_u[wave][16 * ts + 4 * g + i] += r;
                    }
                    csum += __shfl_xor(csum, 16);
                    csum += __shfl_xor(csum, 32);
                    __builtin_amdgcn_wave_barrier();
                    if (g == 0) s_u[wave][t] -= csum;
                    __builtin_amdgcn_wave_barrier();
                }
                if constexpr (BF) {
                    uint2 hi, lo;
                    split_bf16(w[0], w[1], hi.x, lo.x);
                    split_bf16(w[2], w[3], hi.y, lo.y);
                    const int at = RP::quad(t, 16 * ts + 4 * g);
                    *reinterpret_cast<uint2 *>(s_p + at) = hi;
                    *reinterpret_cast<uint2 *>(s_pl + at) = lo;
                } else {
                    RP::store_quad(s_p, t, 16 * ts + 4 * g, w[0], w[1], w[2], w[3]);
                }
            }
        }
        // ---- what the state gives: y^T = win (St^T a)
        f32x4 y[CT][TT];
        if constexpr (!INC) {
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                for (int tt = 0; tt < TT; ++tt) y[ct][tt] = zero4();
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                Frag8<BF> hi[CT], lo[CT];
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) state_frag(st[2 * c][ct], st[2 * c + 1][ct], hi[ct], lo[ct]);
#pragma unroll
                for (int tt = 0; tt < TT; ++tt) {
                    const Frag8<BF> f = RK::row_frag(s_a + 16 * tt * RK::RB, rowk, c);
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) {
                        y[ct][tt] = mma32(y[ct][tt], hi[ct], f);
                        if constexpr (BF) y[ct][tt] = mma32(y[ct][tt], lo[ct], f);
                    }
                }
            }
            mfma_fence_all(y);
#pragma unroll
            for (int tt = 0; tt < TT; ++tt) {
                const float w = s_win[16 * tt + li];
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) y[ct][tt] *= w;
            }
            if constexpr (DG) {
                // the state's share of a token in its log-decay: x_t . y_t over this workgroup's columns
#pragma unroll
                for (int tt = 0; tt < TT; ++tt) {
                    const int t = 16 * tt + li;
                    float d = 0.f;
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) {
                        float x[4];
                        RV::load_quad(s_x + rbuf * SZ_V, t, wave * CT * 16 + 16 * ct + 4 * g, x);
#pragma unroll
                        for (int i = 0; i < 4; ++i) d = fmaf(x[i], y[ct][tt][i], d);
                    }
                    d += __shfl_xor(d, 16);
                    d += __shfl_xor(d, 32);
                    if (g == 0) {
                        if constexpr (REV) s_u[wave][t] -= d;
                        else s_u[wave][t] = d;
                    }
                }
            }
        }
        if constexpr (!INC) __syncthreads();  // the weighted products (and the shares) of every wavefront are there

        if constexpr (DG) {
            if (wave == 0) {  // a token's part of the log-decays' gradient; stores as for y below
                float u = 0.f;
#pragma unroll
                for (int w = 0; w < NW; ++w) u += s_u[w][lane & (C - 1)];
                const auto out = __builtin_amdgcn_make_buffer_rsrc(
                    A.part + ((int64_t)vt * A.H + h) * A.ntok + tc, 0, n * 4, 0x00027000);
                __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, u), out, lane * 4, 0, 0);
            }
        }
        // ---- the chunk's own products, and the state's update
        const float ec = lane_value(s_ec2[buf], 0);
        if (ec != 1.f)
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) st[kt][ct] *= ec;
#pragma unroll
        for (int s = 0; s < SC; ++s) {
            Frag8<BF> cw[CT][NPART];
            float w[8];
            *reinterpret_cast<float4 *>(w) = *reinterpret_cast<const float4 *>(s_wup + 32 * s + RV::token(0, g));
            *reinterpret_cast<float4 *>(w + 4) = *reinterpret_cast<const float4 *>(s_wup + 32 * s + RV::token(1, g));
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                const Frag8<BF> cf = RV::col_frag(s_c + 32 * s * RV::RB, colv, ct);
                if constexpr (!INC) {
                    if (all_finite(cf)) {
#pragma unroll
                        for (int tt = 0; tt < TT; ++tt) {
                            if (REV ? 2 * s + 1 < tt : 2 * s > tt) continue;
                            y[ct][tt] = mma32(y[ct][tt], cf, RP::row_frag(s_p + 16 * tt * RP::RB, rowp, s));
                            if constexpr (BF)
                                y[ct][tt] = mma32(y[ct][tt], cf, RP::row_frag(s_pl + 16 * tt * RP::RB, rowp, s));
                        }
                    } else {
                        // A masked weight is 0, and 0 times infinity is NaN, which a token must not take from one that
                        // it does not see: source by source, for those that see it. (The check that it takes to get
                        // here costs up to 1.5%.)
#pragma unroll 1
                        for (int j = 32 * s; j < 32 * s + 32; ++j) {
                            float x[4];
                            RV::load_quad(s_c + rbuf * SZ_V, j, wave * CT * 16 + 16 * ct + 4 * g, x);
#pragma unroll
                            for (int tt = 0; tt < TT; ++tt) {
                                const int t = 16 * tt + li;
                                float p = RP::load_one(s_p, t, j);
                                if constexpr (BF) p += RP::load_one(s_pl, t, j);
                                if (REV ? j >= t && j < n : j <= t)
#pragma unroll
                                    for (int i = 0; i < 4; ++i) y[ct][tt][i] = fmaf(p, x[i], y[ct][tt][i]);
                            }
                        }
                    }
                }
                scaled_frags(cf, w, cw[ct]);
            }
            constexpr int KG = KT < 4 ? KT : 4;  // products of different tiles follow each other
#pragma unroll
            for (int k0 = 0; k0 < KT; k0 += KG) {
                Frag8<BF> bf[KG];
#pragma unroll
                for (int j = 0; j < KG; ++j) bf[j] = RK::tile_frag(s_b + 32 * s * RK::RB, tilek, k0 + j);
#pragma unroll
                for (int q = 0; q < NPART; ++q)
#pragma unroll
                    for (int j = 0; j < KG; ++j)
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) st[k0 + j][ct] = mma32(st[k0 + j][ct], bf[j], cw[ct][q]);
            }
        }
        if constexpr (!INC) {
            mfma_fence_all(y);
            // Stores of all lanes, the hardware drops those behind the chunk's last row (past the buffer's end): a branch
            // around them would make the next chunk's rows, which were asked for before, wait for them too. (The whole
            // offset is in the lane's part: the scalar part is not held against the buffer's end.)
            constexpr int eb = BF && !YF ? 2 : 4;
            const uint32_t pitch = (uint32_t)A.H * (uint32_t)(A.VD * eb);  // 32 rows: under 2^31
            const auto out = __builtin_amdgcn_make_buffer_rsrc(
                reinterpret_cast<char *>(A.y) + ((int64_t)tc * A.H + h) * A.VD * eb, 0, (n - 1) * pitch + A.VD * eb,
                0x00027000);
            const uint32_t lane_off = li * pitch + (uint32_t)(col0 + 4 * g) * eb;
            if constexpr (eb == 2) {
#pragma unroll
                for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct)
                        __builtin_amdgcn_raw_buffer_store_b64(
                            u32x2{pack_bf16(y[ct][tt].x, y[ct][tt].y), pack_bf16(y[ct][tt].z, y[ct][tt].w)}, out,
                            lane_off + 16 * tt * pitch + 32 * ct, 0, 0);
            } else {
#pragma unroll
                for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct)
                        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, y[ct][tt]), out,
                                                               lane_off + 16 * tt * pitch + 64 * ct, 0, 0);
            }
        }
        mfma_fence_state(st);
    }
    // ---- the state at the other end
    float *so = nullptr;
    if (INC) so = A.s_inc + (slot * A.H + h) * sstate;
    else if (REV ? sg.j == 0 : sg.j == sg.nseg - 1) so = A.s_out ? A.s_out + nh * sstate : nullptr;
    if (so) {
        int lane = lane0;
        asm volatile("" : "+v"(lane));  // no address of the loop's other end is kept over it
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                char *p = reinterpret_cast<char *>(so);
                const uint32_t at = state_at(lane, kt, ct);
                if constexpr (TS)
                    *reinterpret_cast<f32x4 *>(p + at) = st[kt][ct];
                else
#pragma unroll
                    for (uint32_t i = 0; i < 4; ++i) *reinterpret_cast<float *>(p + (at + i * vd4)) = st[kt][ct][i];
            }
    }
    if constexpr (INC) {  // the segment's whole decay: the wavefronts' sums
        btot = lane_value(btot, 0) + lane_value(btot, 32);
        if (lane == 0) s_red[wave] = btot;
        __syncthreads();
        if (threadIdx.x == 0 && vt == 0) {
#pragma unroll
            for (int w = 1; w < NW; ++w) btot += s_red[w];
            A.seg_decay[slot * A.H + h] = btot;
        }
    }
}

// Workgroups of one (segment, head) sit 8 apart: the same XCD, whose L2 then holds the rows they share. So do those of
// the heads that share rows of q and k (A.share).
__device__ __forceinline__ bool item_of(const CoreArgs &A, int per_item, int64_t &item, int &r) {
    const int64_t blk = blockIdx.x + (int64_t)blockIdx.y * gridDim.x, grp = blk / (8 * per_item * A.share);
    const int in = (int)(blk - grp * 8 * per_item * A.share), head = (in >> 3) / per_item;
    r = (in >> 3) - head * per_item;
    item = (grp * 8 + (in & 7)) * A.share + head;
    return item < A.slots * A.H;
}
template <int NW> constexpr int kWavesPerSimd = NW == 8 ? 4 : 2;  // two workgroups of 8 or 4 wavefronts per CU

template <bool BF, int KD, int VT>
__global__ __launch_bounds__(VT * 4, kWavesPerSimd<VT / 16>) void kda_hd_fwd_kernel(const CoreArgs A) {
    __shared__ __align__(16) char smem[Lds<BF, KD, VT, VT / 16, false, false>::bytes];
    int64_t item;
    int r;
    if (!item_of(A, A.tiles, item, r)) return;
    chunk_pass<BF, KD, VT, VT / 16, false, false, false, false, false>(A, item, r, smem);
}
// The increments of the states (and, from workgroup tiles on, of their gradients).
template <bool BF, int KD, int VT>
__global__ __launch_bounds__(VT * 4, kWavesPerSimd<VT / 16>) void kda_hd_inc_kernel(const CoreArgs F, const CoreArgs R, int both) {
    __shared__ __align__(16) char smem[Lds<BF, KD, VT, VT / 16, true, false>::bytes];
    int64_t item;
    int r;
    if (!item_of(F, both ? 2 * F.tiles : F.tiles, item, r)) return;
    if (r < F.tiles)
        chunk_pass<BF, KD, VT, VT / 16, false, true, false, false, false>(F, item, r, smem);
    else
        chunk_pass<BF, KD, VT, VT / 16, true, true, false, false, false>(R, item, r - F.tiles, smem);
}
// The three gradients of a (segment, head) as workgroups of one launch: dv and dk walk back through the same rows side
// by side (what one fetches the other finds in L2), dq walks forward.
template <bool BF, int K, int V, int VT, bool DG, bool YF>
__global__ __launch_bounds__(VT * 4, kWavesPerSimd<VT / 16>) void kda_hd_grad_kernel(const GradArgs G) {
    constexpr int NW = VT / 16;
    constexpr int L1 = Lds<BF, V, VT, NW, false, DG>::bytes, L2 = Lds<BF, K, VT, NW, false, DG>::bytes;
    __shared__ __align__(16) char smem[L1 > L2 ? L1 : L2];
    int64_t item;
    int r;
    if (!item_of(G.dv, G.dv.tiles + 2 * G.dk.tiles, item, r)) return;
    if (r < G.dv.tiles) {
        chunk_pass<BF, K, VT, NW, true, false, DG, false, false>(G.dv, item, r, smem);
        return;
    }
    r -= G.dv.tiles;
    if (r < G.dk.tiles)
        chunk_pass<BF, V, VT, NW, true, false, false, YF, true>(G.dk, item, r, smem);
    else
        chunk_pass<BF, V, VT, NW, false, false, DG, YF, true>(G.dq, item, r - G.dk.tiles, smem);
}

inline dim3 grid_of(const CoreArgs &a, int64_t per_item) {
    return wide_grid((a.slots * (a.H / a.share) + 7) / 8 * 8 * a.share * per_item);
}

}  // namespace hd
}  // namespace kda
