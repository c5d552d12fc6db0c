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
using hd::Rows;
using hd::Stage;
using hd::u32x2;
using hd::u32x4;

// ------------------------------------------------------------------ operands
// A computed operand: bf16 I/O holds it as two bf16 parts (2^-18 of a value), fp32 I/O as it is.
template <bool BF> struct Pair;
template <> struct Pair<true> { Frag8<true> hi, lo; };
template <> struct Pair<false> { Frag8<false> f; };

__device__ __forceinline__ void set_pair(Pair<true> &p, const float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        p.hi.p[i] = hd::seen(pack_bf16(x[2 * i], x[2 * i + 1]));
        p.lo.p[i] = pack_bf16(x[2 * i] - bf_lo(p.hi.p[i]), x[2 * i + 1] - bf_hi(p.hi.p[i]));
    }
}
__device__ __forceinline__ void set_pair(Pair<false> &p, const float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) p.f.f[i] = x[i];
}
template <bool BF>
__device__ __forceinline__ Pair<BF> pair_of(const f32x4 &u, const f32x4 &w) {
    const float x[8] = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w};
    Pair<BF> p;
    set_pair(p, x);
    return p;
}
// The parts of a computed operand that the fp32 state is summed from: three bf16 parts are all 24 bits.
template <bool BF> constexpr int kParts = BF ? 3 : 1;
__device__ __forceinline__ void set_parts(Frag8<true> (&f)[3], const float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[0].p[i] = hd::seen(pack_bf16(x[2 * i], x[2 * i + 1]));
        const float a = x[2 * i] - bf_lo(f[0].p[i]), b = x[2 * i + 1] - bf_hi(f[0].p[i]);
        f[1].p[i] = hd::seen(pack_bf16(a, b));
        f[2].p[i] = pack_bf16(a - bf_lo(f[1].p[i]), b - bf_hi(f[1].p[i]));
    }
}
__device__ __forceinline__ void set_parts(Frag8<false> (&f)[1], const float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[0].f[i] = x[i];
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

// Products of pairs (the two small parts' own product is left out) and of pairs with exact operands.
__device__ __forceinline__ f32x4 mm(f32x4 c, const Pair<true> &a, const Pair<true> &b) {
    c = mma32(c, a.hi, b.hi);
    c = mma32(c, a.hi, b.lo);
    return mma32(c, a.lo, b.hi);
}
__device__ __forceinline__ f32x4 mm(f32x4 c, const Pair<false> &a, const Pair<false> &b) { return mma32(c, a.f, b.f); }
__device__ __forceinline__ f32x4 mm(f32x4 c, const Frag8<true> &a, const Pair<true> &b) {
    c = mma32(c, a, b.hi);
    return mma32(c, a, b.lo);
}
__device__ __forceinline__ f32x4 mm(f32x4 c, const Frag8<false> &a, const Pair<false> &b) { return mma32(c, a, b.f); }
__device__ __forceinline__ f32x4 mm(f32x4 c, const Pair<true> &a, const Frag8<true> &b) {
    c = mma32(c, a.hi, b);
    return mma32(c, a.lo, b);
}
__device__ __forceinline__ f32x4 mm(f32x4 c, const Pair<false> &a, const Frag8<false> &b) { return mma32(c, a.f, b); }

// ------------------------------------------------------------------ tokens
// An accumulator of 32 tokens is two tiles of 16 rows; row m of tile tt is the token that slot 4 tt + m % 4 of lane group
// m / 4 stands for, so the two tiles are, as they are, an operand whose slots are the chunk's tokens.
template <bool BF> __device__ __forceinline__ int token_of(int tt, int g) {  // of row 4g (the next three follow)
    return BF ? 8 * g + 4 * tt : 16 * tt + 4 * g;
}
template <bool BF> __device__ __forceinline__ int token_row(int tt, int m) {
    return token_of<BF>(tt, m >> 2) + (m & 3);
}
template <bool BF> __device__ __forceinline__ int slot_token(int g, int j) { return token_of<BF>(j >> 2, g) + (j & 3); }

// A tile of a record's matrix as an operand, and one of its entries: row m of the tile, source slot j of lane group g.
__device__ __forceinline__ void load_mat(const char *m, int tt, int lane, Pair<true> &p) {
    const u32x4 u = *reinterpret_cast<const u32x4 *>(m + ((2 * tt) * 64 + lane) * 16);
    const u32x4 w = *reinterpret_cast<const u32x4 *>(m + ((2 * tt + 1) * 64 + lane) * 16);
    p.hi.p[0] = u.x; p.hi.p[1] = u.y; p.hi.p[2] = u.z; p.hi.p[3] = u.w;
    p.lo.p[0] = w.x; p.lo.p[1] = w.y; p.lo.p[2] = w.z; p.lo.p[3] = w.w;
}
__device__ __forceinline__ void load_mat(const char *m, int tt, int lane, Pair<false> &p) {
    const f32x4 u = *reinterpret_cast<const f32x4 *>(m + ((2 * tt) * 64 + lane) * 16);
    const f32x4 w = *reinterpret_cast<const f32x4 *>(m + ((2 * tt + 1) * 64 + lane) * 16);
    p.f = Frag8<false>{{u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w}};
}
__device__ __forceinline__ void store_mat(char *m, int tt, int lane, const Pair<true> &p) {
    *reinterpret_cast<u32x4 *>(m + ((2 * tt) * 64 + lane) * 16) = u32x4{p.hi.p[0], p.hi.p[1], p.hi.p[2], p.hi.p[3]};
    *reinterpret_cast<u32x4 *>(m + ((2 * tt + 1) * 64 + lane) * 16) = u32x4{p.lo.p[0], p.lo.p[1], p.lo.p[2], p.lo.p[3]};
}
__device__ __forceinline__ void store_mat(char *m, int tt, int lane, const Pair<false> &p) {
    *reinterpret_cast<f32x4 *>(m + ((2 * tt) * 64 + lane) * 16) = f32x4{p.f.f[0], p.f.f[1], p.f.f[2], p.f.f[3]};
    *reinterpret_cast<f32x4 *>(m + ((2 * tt + 1) * 64 + lane) * 16) = f32x4{p.f.f[4], p.f.f[5], p.f.f[6], p.f.f[7]};
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
            const int src = slot_token<BF>(gs, j);
#pragma unroll
            for (int tt = 0; tt < 2; ++tt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = token_of<BF>(tt, g) + i;
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
            const int src = slot_token<BF>(gs, j);
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

// Consecutive bytes on their way to LDS.
template <int BYTES, int NT>
struct Copy {
    static constexpr int NL = (BYTES / 16 + NT - 1) / NT;
    static_assert(BYTES % 16 == 0, "16 bytes a load");
    u32x4 w[NL];
    __device__ __forceinline__ void take(int tid, const char *p) {
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int at = (i * NT + tid) * 16;
            w[i] = *reinterpret_cast<const u32x4 *>(p + (at < BYTES ? at : BYTES - 16));
        }
    }
    __device__ __forceinline__ void put(int tid, char *t) const {
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int at = (i * NT + tid) * 16;
            if (at < BYTES) *reinterpret_cast<u32x4 *>(t + at) = w[i];
        }
    }
};

// ------------------------------------------------------------------ the pass over the states
// Rows 16-row tiles read at the tokens of token_row: the lane's address for tile 0, and how tile 1's differs from it.
template <bool BF, int NCOL> __device__ __forceinline__ int tok_row_at(int lane) {
    if constexpr (BF) return Rows<true, NCOL>::slot(token_row<true>(0, lane & 15), lane >> 4);
    else return Rows<false, NCOL>::row_at(lane);
}
template <bool BF, int NCOL>
__device__ __forceinline__ Frag8<BF> tok_row_frag(const char *t, int at, int tt, int c) {
    using R = Rows<BF, NCOL>;
    if constexpr (BF) return R::row_frag(t + (tt ? 4 * R::RB : 0), tt ? at ^ 16 : at, c);
    else return R::row_frag(t + 16 * tt * R::RB, at, c);
}

template <bool BF, int K, int VT, int MODE>
struct StateLds {
    static constexpr int C = kChunkTokens, NB = BF ? 2 : 1;
    static constexpr int K_ = Rows<BF, K>::bytes(C), V_ = Rows<BF, VT>::bytes(C), R_ = rec_bytes(MODE != kForward);
    static constexpr int k = 0, q = k + NB * K_, v = q + (MODE == kErrors ? 0 : NB * K_), rec = v + NB * V_;
    static constexpr int bytes = rec + NB * R_;
};

// One (sequence, head), columns vt * VT .. of the state, a wavefront 16 of them: all K rows as fp32 accumulators, which
// are at once operands of the products with the state, so it never leaves the registers.
template <bool BF, int K, int VT, int MODE>
__global__ __launch_bounds__(VT * 4, 2) void kda_gd_state_kernel(const StateArgs A, int V) {
    using L = StateLds<BF, K, VT, MODE>;
    using RK = Rows<BF, K>;
    using RV = Rows<BF, VT>;
    constexpr int NW = VT / 16, NT = NW * 64, KT = K / 16, KC = K / 32, C = kChunkTokens, NB = L::NB;
    constexpr int EB = BF ? 2 : 4;
    constexpr bool REV = MODE == kReverse;
    __shared__ __align__(16) char smem[L::bytes];

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4,
              li = lane & 15;
    const int64_t blk = blockIdx.x + (int64_t)blockIdx.y * gridDim.x;
    // the tiles of a head 8 workgroups apart: the same XCD, whose L2 then holds the rows they share
    const int64_t grp = blk / (8 * A.tiles);
    const int in = (int)(blk - grp * 8 * A.tiles), vt = in >> 3;
    const int64_t item = grp * 8 + (in & 7), n = item / A.c.H;
    const int h = (int)(item - n * A.c.H), group = A.c.H / A.c.Hk;
    if (n >= A.c.N) return;
    const Seq sq = seq_of(A.c, n);
    const int64_t len = sq.t1 - sq.t0;
    const int nch = (int)((len + C - 1) / C);
    const int col = vt * VT + wave * 16;  // this wavefront's first column

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

    const uint32_t lk = (uint32_t)A.c.Hk * (K * EB), lv = (uint32_t)A.c.H * (uint32_t)(V * EB);
    const char *pk = reinterpret_cast<const char *>(A.k) + (sq.t0 * A.c.Hk + h / group) * (K * EB);
    const char *pq = reinterpret_cast<const char *>(A.q) + (sq.t0 * A.c.Hk + h / group) * (K * EB);
    const char *pv = reinterpret_cast<const char *>(A.v) + ((sq.t0 * A.c.H + h) * V + vt * VT) * EB;
    constexpr int RECB = L::R_;
    const char *prec = A.c.rec + (sq.first * A.c.H + h) * RECB;
    const int64_t rec_step = (int64_t)A.c.H * RECB;

    Stage<BF, K, C, NT> rk, rq;
    Stage<BF, VT, C, NT> rv;
    Copy<RECB, NT> rr;
    auto chunk_of = [&](int i) __attribute__((always_inline)) { return REV ? nch - 1 - i : i; };
    auto take = [&](int i) __attribute__((always_inline)) {
        const int64_t c = chunk_of(i), t = c * C;
        const int m = (int)(len - t < C ? len - t : C);
        rk.take(tid, pk + t * lk, lk, m);
        if constexpr (MODE != kErrors) rq.take(tid, pq + t * lk, lk, m);
        rv.take(tid, pv + t * lv, lv, m);
        rr.take(tid, prec + c * rec_step);
    };
    auto put = [&](int b) __attribute__((always_inline)) {
        rk.put(tid, smem + L::k + b * L::K_);
        if constexpr (MODE != kErrors) rq.put(tid, smem + L::q + b * L::K_);
        rv.put(tid, smem + L::v + b * L::V_);
        rr.put(tid, smem + L::rec + b * L::R_);
    };
    if (nch > 0) {
        take(0);
        if constexpr (NB == 2) {
            put(0);
            if (nch > 1) take(1);
        }
    }
    const int tok0 = tok_row_at<BF, K>(lane), row0 = RK::row_at(lane), tile0 = RK::tile_at(lane);
    const int col0 = BF ? RV::col_at(lane) ^ (wave << 5) : RV::col_at(lane) + 64 * wave;

    for (int cc = 0; cc < nch; ++cc) {
        const int c = chunk_of(cc), b = cc & (NB - 1);
        __syncthreads();  // nobody reads the last chunk's rows any more (NB = 2: and this one's are there)
        if constexpr (NB == 1) {
            put(0);
            if (cc + 1 < nch) take(cc + 1);
            __syncthreads();
        } else if (cc + 1 < nch) {
            put(b ^ 1);
            if (cc + 2 < nch) take(cc + 2);
        }
        const char *sk = smem + L::k + b * L::K_, *sv = smem + L::v + b * L::V_, *sr = smem + L::rec + b * L::R_;
        const char *sq_ = smem + L::q + b * L::K_;
        (void)sq_;
        const float *wt = reinterpret_cast<const float *>(sr + rec_weights(MODE != kForward));
        auto weights = [&](int which, float (&w)[8]) __attribute__((always_inline)) {  // of the tokens in a lane's slots
            *reinterpret_cast<f32x4 *>(w) = *reinterpret_cast<const f32x4 *>(wt + which * C + token_of<BF>(0, g));
            *reinterpret_cast<f32x4 *>(w + 4) = *reinterpret_cast<const f32x4 *>(wt + which * C + token_of<BF>(1, g));
        };
        if (MODE == kErrors && c > 0 && c % kSegmentChunks == 0)
            put_state(A.seed + ((sq.seg + c / kSegmentChunks) * A.c.H + h) * sstate);
        if (MODE == kReverse && c + 1 < nch && (c + 1) % kSegmentChunks == 0)
            put_state(A.seed + ((sq.seg + c / kSegmentChunks) * A.c.H + h) * sstate);

        // ---- products with the state: K S, and S^T q
        f32x4 x[2] = {zero4(), zero4()}, y[2] = {zero4(), zero4()};
#pragma unroll
        for (int kc = 0; kc < KC; ++kc) {
            const Pair<BF> s = pair_of<BF>(st[2 * kc], st[2 * kc + 1]);
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) x[tt] = mm(x[tt], tok_row_frag<BF, K>(sk, tok0, tt, kc), s);
            if constexpr (MODE == kForward)
#pragma unroll
                for (int tt = 0; tt < 2; ++tt) y[tt] = mm(y[tt], s, RK::row_frag(sq_ + 16 * tt * RK::RB, row0, kc));
        }
        const Frag8<BF> vf = RV::col_frag(sv, col0, 0);
        float vx[8], z[8];
        widen(vf, vx);
        mfma_fence(x[0], x[1], y[0], y[1]);
        if constexpr (!REV) {
            // ---- z = r + N r,  r = v - e^b K S
            float w[8];
            weights(kEnter, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] = fmaf(-w[i], x[i >> 2][i & 3], vx[i]);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i >> 2][i & 3] = z[i];
            if (all_finite(z)) {
                Pair<BF> r, m;
                set_pair(r, z);
#pragma unroll
                for (int tt = 0; tt < 2; ++tt) {
                    load_mat(sr + kMatN * kMatBytes, tt, lane, m);
                    x[tt] = mm(x[tt], m, r);
                }
            } else {
                mix_rows<BF, false>(x, z, sr + kMatN * kMatBytes, lane);
            }
        } else {
            // ---- D = e^{b_C - b} K G + P^T do, then dw = D + N'^T D
            float w[8];
            weights(kLeave, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i >> 2][i & 3] *= w[i];
            if (all_finite(vx)) {
                Pair<BF> m;
#pragma unroll
                for (int tt = 0; tt < 2; ++tt) {
                    load_mat(sr + kMatPT * kMatBytes, tt, lane, m);
                    x[tt] = mm(x[tt], m, vf);
                }
            } else {
                mix_rows<BF, true>(x, vx, sr + kMatPT * kMatBytes, lane);
            }
            mfma_fence(x[0], x[1]);
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] = x[i >> 2][i & 3];
            if (all_finite(z)) {
                Pair<BF> r, m;
                set_pair(r, z);
#pragma unroll
                for (int tt = 0; tt < 2; ++tt) {
                    load_mat(sr + kMatNT * kMatBytes, tt, lane, m);
                    x[tt] = mm(x[tt], m, r);
                }
            } else {
                mix_rows<BF, true>(x, z, sr + kMatNT * kMatBytes, lane);
            }
        }
        mfma_fence(x[0], x[1]);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = x[i >> 2][i & 3];

        if constexpr (MODE == kForward) {
            // ---- o^T = scale e^b S^T q + P z
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) y[tt] *= wt[kEnterScaled * C + 16 * tt + li];
            if (all_finite(z)) {
                Pair<BF> zp, m;
                set_pair(zp, z);
#pragma unroll
                for (int tt = 0; tt < 2; ++tt) {
                    load_mat(sr + kMatP * kMatBytes, tt, lane, m);
                    y[tt] = mm(y[tt], zp, m);
                }
            } else {
                mix_cols<BF>(y, z, sr + kMatP * kMatBytes, lane);
            }
            mfma_fence(y[0], y[1]);
            const int64_t t = sq.t0 + (int64_t)c * C;
            const int m = (int)(sq.t1 - t < C ? sq.t1 - t : C);
            // the hardware drops the stores behind the chunk's last row (past the buffer's end)
            const auto out = __builtin_amdgcn_make_buffer_rsrc(
                reinterpret_cast<char *>(A.o) + (t * A.c.H + h) * V * EB, 0, (m - 1) * lv + V * EB, 0x00027000);
            const uint32_t at = li * lv + (uint32_t)(col + 4 * g) * EB;
#pragma unroll
            for (int tt = 0; tt < 2; ++tt)
                if constexpr (BF)
                    __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack_bf16(y[tt].x, y[tt].y), pack_bf16(y[tt].z, y[tt].w)},
                                                          out, at + 16 * tt * lv, 0, 0);
                else
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, y[tt]), out, at + 16 * tt * lv, 0, 0);
        } else {
            // ---- z or dw by columns: [V][32], the parts one after the other
            char *rows = A.rows + ((sq.first + c) * A.c.H + h) * (int64_t)V * (C * 4);
            Pair<BF> zp;
            set_pair(zp, z);
            if constexpr (BF) {
                char *p = rows + (col + li) * (C * 2) + 16 * g;
                *reinterpret_cast<u32x4 *>(p) = u32x4{zp.hi.p[0], zp.hi.p[1], zp.hi.p[2], zp.hi.p[3]};
                *reinterpret_cast<u32x4 *>(p + V * (C * 2)) = u32x4{zp.lo.p[0], zp.lo.p[1], zp.lo.p[2], zp.lo.p[3]};
            } else {
                char *p = rows + (col + li) * (C * 4) + 16 * g;
                *reinterpret_cast<f32x4 *>(p) = f32x4{z[0], z[1], z[2], z[3]};
                *reinterpret_cast<f32x4 *>(p + 64) = f32x4{z[4], z[5], z[6], z[7]};
            }
        }
        // ---- the state's update
        const float total = wt[kTotal * C];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) st[kt] *= total;
        if constexpr (!REV) {
            float w[8];
            weights(kLeaveBeta, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] *= z[i];
            Frag8<BF> f[kParts<BF>];
            set_parts(f, w);
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                const Frag8<BF> a = RK::tile_frag(sk, tile0, kt);
#pragma unroll
                for (int p = 0; p < kParts<BF>; ++p) st[kt] = mma32(st[kt], a, f[p]);
            }
        } else {
            float wq[8], wk[8], be[8];
            weights(kEnterScaled, wq);
            weights(kEnter, wk);
            weights(kBeta, be);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                z[i] *= be[i];  // dL/dz, which is dL/dv
                wq[i] *= vx[i];
                wk[i] *= -z[i];
            }
            Frag8<BF> f[kParts<BF>], e[kParts<BF>];
            set_parts(f, wq);
            set_parts(e, wk);
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                const Frag8<BF> a = RK::tile_frag(sq_, tile0, kt), a2 = RK::tile_frag(sk, tile0, kt);
#pragma unroll
                for (int p = 0; p < kParts<BF>; ++p) {
                    st[kt] = mma32(st[kt], a, f[p]);
                    st[kt] = mma32(st[kt], a2, e[p]);
                }
            }
            const int64_t t = sq.t0 + (int64_t)c * C;
            const int m = (int)(sq.t1 - t < C ? sq.t1 - t : C);
            const auto out = __builtin_amdgcn_make_buffer_rsrc(
                reinterpret_cast<char *>(A.o) + (t * A.c.H + h) * V * EB, 0, (m - 1) * lv + V * EB, 0x00027000);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t at = (uint32_t)slot_token<BF>(g, i) * lv + (uint32_t)(col + li) * EB;
                if constexpr (BF) __builtin_amdgcn_raw_buffer_store_b16((uint16_t)pack_bf16(z[i], 0.f), out, at, 0, 0);
                else __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, z[i]), out, at, 0, 0);
            }
        }
        hd::mfma_fence_state(reinterpret_cast<f32x4(&)[1][KT]>(st));
    }
    if (A.s_end) put_state(A.s_end + nh * sstate);
}

}  // namespace gd
}  // namespace kda
