// The gated delta rule with one decay per head: the gradients of q, k, g and beta.
//
// Given the errors z and the gradients dw of what is written (w = beta z), the recurrence is a plain decaying sum of
// k_i w_i^T, and what is left are four such sums, two forward in time over the state S and two backward over its gradient
// G (E_ri = e^{b_r - b_i}; M_ri = dw_r.z_i):
//   dq_r = scale ( e^{b_r} S do_r + sum_{i<=r} E_ri (do_r.w_i) k_i )
//   dk_r = - beta_r ( e^{b_r} S dw_r + sum_{i<r} E_ri beta_i M_ri k_i )                                  (read)
//        + e^{b_C - b_r} beta_r G z_r + sum_{j>=r} scale E_jr (do_j.w_r) q_j - sum_{j>r} E_jr beta_j beta_r M_jr k_j
//   dbeta_r = M_rr
// Each pair and state that a token's log-decay spans is in a row's read and another's write: with db_r = q_r.dq_r +
// k_r.dk_r(read) - k_r.dk_r(rest),  dg_t = sum_{r>=t} db_r up to a border, and what the border passes on, <G, S> there.
#pragma once

#include "kda_gd_core.hpp"

namespace kda {
namespace gd {

// A tile of V channels x 32 tokens in LDS, from rows of the states' passes: 16 bytes of a row are the tokens of a lane
// group's slots. bf16: the two halves (tiles of 16 tokens) in planes of their own, rows of 32 bytes ordered so that the
// eight rows of a transposing read, and the sixteen of a row read, fall on different banks. (The planes are not a multiple
// of 512 bytes apart: the compiler would join a lane's reads of both into one instruction, whose halves then meet on the
// same banks, 8 cycles for 4.)
template <bool BF, int V, int NP> struct Tile;
template <int V, int NP> struct Tile<true, V, NP> {
    static constexpr int PLANE = V * 32 + 64, PART = 2 * PLANE;
    static __device__ __forceinline__ int at(int row, int g) {
        const int line = (row & 3) | (row & 24) >> 1 | (row & 4) << 2 | (row & ~31);
        return line * 32 + ((g ^ ((row >> 3) & 2)) << 3);
    }
    // channels 32 vc .. x tokens 16 tt + l % 16; rows of the state's tile vt x the chunk's tokens
    static __device__ __forceinline__ int cols_at(int lane) { return at(8 * (lane >> 4) + ((lane >> 2) & 3), lane & 3); }
    static __device__ __forceinline__ Frag8<true> cols(const char *t, int at, int vc, int tt) {
        return Rw<true, 32>::tr_frag(t + at + 1024 * vc + PLANE * tt, 512);  // 16 lines on: the row 4 on
    }
    static __device__ __forceinline__ int rows_at(int lane) {
        return at(8 * ((lane >> 2) & 3) + (lane & 3), lane >> 4);
    }
    static __device__ __forceinline__ Frag8<true> rows(const char *t, int at, int vt) {
        const char *p = t + at + 1024 * (vt >> 1) + 512 * (vt & 1);
        const uint2 a = *reinterpret_cast<const uint2 *>(p), b = *reinterpret_cast<const uint2 *>(p + PLANE);
        return Frag8<true>{{a.x, a.y, b.x, b.y}};
    }
    static __device__ __forceinline__ Multi<true, NP> all_cols(const char *t, int at, int vc, int tt) {
        Multi<true, NP> m;
#pragma unroll
        for (int n = 0; n < NP; ++n) m.p[n] = cols(t + n * PART, at, vc, tt);
        return m;
    }
    static __device__ __forceinline__ Multi<true, NP> all_rows(const char *t, int at, int vt) {
        Multi<true, NP> m;
#pragma unroll
        for (int n = 0; n < NP; ++n) m.p[n] = rows(t + n * PART, at, vt);
        return m;
    }
};
template <int V, int NP> struct Tile<false, V, NP> {
    using R = Rw<false, 32>;
    static constexpr int PART = R::bytes(V);
    static __device__ __forceinline__ int cols_at(int lane) { return R::col_at(lane, 0); }
    static __device__ __forceinline__ int rows_at(int lane) { return R::row_at(lane); }
    static __device__ __forceinline__ Multi<false, NP> all_cols(const char *t, int at, int vc, int tt) {
        return {{R::col_frag(t + 32 * vc * R::RB + 64 * tt, at)}};
    }
    static __device__ __forceinline__ Multi<false, NP> all_rows(const char *t, int at, int vt) {
        return {{R::row_frag(t + 16 * vt * R::RB, at, 0)}};
    }
};
// On its way there: all parts, 16 bytes a load.
template <bool BF, int V, int NP, int NT>
struct TileIn {
    using T = Tile<BF, V, NP>;
    static constexpr int UNITS = V * (BF ? 4 * NP : 8), NL = (UNITS + NT - 1) / NT;
    u32x4 w[NL];
    int to[NL];
    uint32_t from[NL];
    __device__ __forceinline__ void init(int tid) {
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int u = i * NT + tid < UNITS ? i * NT + tid : UNITS - 1;  // lanes left over bring the last once more
            from[i] = u * 16;
            if constexpr (BF) to[i] = u / (V * 4) * T::PART + T::at(u / 4 % V, u & 3);
            else to[i] = Rw<false, 32>::slot(u / 8, u & 7);
        }
    }
    __device__ __forceinline__ void take(const char *p) {
        const auto b = __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(p), 0, UNITS * 16, 0x00027000);
#pragma unroll
        for (int i = 0; i < NL; ++i) w[i] = __builtin_amdgcn_raw_buffer_load_b128(b, from[i], 0, 0);
    }
    __device__ __forceinline__ void put(char *t) const {
#pragma unroll
        for (int i = 0; i < NL; ++i)
            if constexpr (BF) {
                *reinterpret_cast<uint2 *>(t + to[i]) = make_uint2(w[i].x, w[i].y);
                *reinterpret_cast<uint2 *>(t + to[i] + T::PLANE) = make_uint2(w[i].z, w[i].w);
            } else {
                *reinterpret_cast<u32x4 *>(t + to[i]) = w[i];
            }
    }
};

// The sum of the pieces of a product over a long axis.
__device__ __forceinline__ f32x4 sum_of(const f32x4 (&x)[1]) { return x[0]; }
__device__ __forceinline__ f32x4 sum_of(const f32x4 (&x)[2]) { return x[0] + x[1]; }
__device__ __forceinline__ f32x4 sum_of(const f32x4 (&x)[4]) { return (x[0] + x[1]) + (x[2] + x[3]); }
__device__ __forceinline__ void fence_each(f32x4 (&x)[1]) { mfma_fence(x[0]); }
__device__ __forceinline__ void fence_each(f32x4 (&x)[2]) { mfma_fence(x[0], x[1]); }
__device__ __forceinline__ void fence_each(f32x4 (&x)[4]) { mfma_fence(x[0], x[1], x[2], x[3]); }

// The sum over a wavefront's four groups of 16 lanes, in all of them. A swap exchanges the odd groups (or the upper pair) of
// its first operand with the even ones (the lower pair) of its second.
__device__ __forceinline__ float sum_groups(float x) {
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const uint32_t a0 = a[0], a1 = a[1];
    const uint32_t s = __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, a0) + __builtin_bit_cast(float, a1));
    const auto b = __builtin_amdgcn_permlane32_swap(s, s, false, false);
    const uint32_t b0 = b[0], b1 = b[1];
    return __builtin_bit_cast(float, b0) + __builtin_bit_cast(float, b1);
}

template <bool BF, int K, int V, int NP>
struct GradLds {
    static constexpr int C = kChunkTokens, NM = BF ? 2 : 1, NW = K / 16;
    static constexpr int T_ = (BF ? NP : 1) * Tile<BF, V, NP>::PART, M_ = Rw<BF, C>::bytes(C);  // a tile; a part of a matrix
    static constexpr int K_ = Rw<BF, K>::bytes(C), O_ = Rw<BF, V>::bytes(C);
    // A chunk's rows, twice where there is room for one workgroup that fills the compute unit: the next chunk's come while
    // this one's are read. (Of smaller workgroups several run side by side instead.)
    static constexpr int dout = 0, z = dout + O_, dw = z + T_, k = dw + T_, q = k + K_, wt = q + K_,
                         ROWS = wt + kWeights * C * 4;
    static constexpr int MOST = segment_most(K);
    static constexpr int REST = 2 * NM * M_ + MOST * (NW * C + 12 * 16 + C) * 4 + NW * 4;
    static constexpr int NB = NW == 8 && 2 * ROWS + REST <= 160 * 1024 ? 2 : 1;
    static constexpr int m1 = NB * ROWS, m2 = m1 + NM * M_, u = m2 + NM * M_, pairs = u + MOST * NW * C * 4,
                         db = pairs + MOST * 12 * 16 * 4, red = db + MOST * C * 4, bytes = red + NW * 4;
    static_assert(bytes == NB * ROWS + REST && bytes <= 160 * 1024, "a compute unit's memory");
};

// One segment of a (sequence, head); a wavefront 16 columns of K, all V rows of the transposed states in its registers.
// YF: dq and dk in fp32 per v head. NP: bf16 parts of computed operands, two beside bf16 gates, three beside fp32 ones (dg
// is a difference of long sums: with two parts it was off by 1.4e-5 of its size, with three by 1e-6). The pairs' weights are two
// parts in either: only dq and dk are made of them, dg's pairs come from the unrounded products. GF: the gates'
// gradients in fp32. What adds to the log-decays' gradient stays in LDS by chunk until the segment's end: summed chunk by
// chunk it held up every barrier (60 of 600 us).
//
// 4096 tokens of 96 heads of 128 channels, bf16: 532 us. A chunk's q, k, do and the two tensors of the states' passes
// come once for each walk, dk's first part leaves and returns: 2.0 GB, 400 us at a copy's rate. Vector instructions issue in
// 35% of the cycles, matrix ones run in 21%, LDS in 40%; two wavefronts a SIMD, in step by their barriers, seldom fill in for
// each other. Two workgroups a CU (128 registers, no rows on the way) took 780 us, half of the wavefronts with
// the two halves of a chunk's first part exchanged 600.
template <bool BF, int K, int V, bool YF, int NP>
__global__ __launch_bounds__(K * 4, 2) void kda_gd_grad_kernel(const GradArgs A) {
    using L = GradLds<BF, K, V, NP>;
    using RK = Rw<BF, K>;
    using RV = Rw<BF, V>;
    using RC = Rw<BF, kChunkTokens>;
    using TV = Tile<BF, V, NP>;
    constexpr int NW = L::NW, NT = NW * 64, VT = V / 16, VC = V / 32, KC = K / 32;
    constexpr int C = kChunkTokens, EB = BF ? 2 : 4;
    constexpr bool GF = !BF || NP == 3;
    using Op = Multi<BF, NP>;
    __shared__ __align__(16) char smem[L::bytes];
    char *const s_m1 = smem + L::m1, *const s_m2 = smem + L::m2;
    float *const s_red = reinterpret_cast<float *>(smem + L::red);
    // the log-decays' gradient by chunk: tokens' dots by wavefront, pairs' sums by job (of rows, of sources), all of them
    float(*const s_u)[NW][C] = reinterpret_cast<float(*)[NW][C]>(smem + L::u);
    float(*const s_pairs)[12][16] = reinterpret_cast<float(*)[12][16]>(smem + L::pairs);
    float *const s_db = reinterpret_cast<float *>(smem + L::db);
    // the rows in use
    char *s_do, *s_z, *s_dw, *s_k, *s_q;
    float *s_wt;
    auto rows_of = [&](int i) __attribute__((always_inline)) {
        char *const p = smem + (i & (L::NB - 1)) * L::ROWS;
        s_do = p + L::dout;
        s_z = p + L::z;
        s_dw = p + L::dw;
        s_k = p + L::k;
        s_q = p + L::q;
        s_wt = reinterpret_cast<float *>(p + L::wt);
    };

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 4,
              li = lane & 15;
    const int64_t blk = blockIdx.x + (int64_t)blockIdx.y * gridDim.x, slot = blk / A.c.H;
    const int h = (int)(blk - slot * A.c.H), group = A.c.H / A.c.Hk;
    if (slot >= A.c.segs) return;
    const int64_t n = find_seq<true>(A.c, slot, lane);
    const Seq sq = seq_of(A.c, n);
    const int len = (int)(sq.t1 - sq.t0);  // under 2^31
    const int all = (int)(((int64_t)len + C - 1) / C);  // the sequence's chunks
    if (slot < sq.seg || (slot - sq.seg) * A.c.seg >= all) return;
    const int c0 = (int)(slot - sq.seg) * A.c.seg, c1 = c0 + A.c.seg < all ? c0 + A.c.seg : all;
    const int nch = c1 - c0, col = wave * 16;  // this wavefront's first column
    const int64_t sstate = (int64_t)K * V, nh = n * A.c.H + h;

    // a state [K][V] in memory as tiles of its transpose
    auto get_state = [&](const float *s, f32x4 (&st)[VT]) __attribute__((always_inline)) {
#pragma unroll
        for (int vt = 0; vt < VT; ++vt)
            st[vt] = s ? *reinterpret_cast<const f32x4 *>(s + (int64_t)(col + li) * V + RV::state_row(vt, g)) : zero4();
    };
    const uint32_t lk = (uint32_t)A.c.Hk * (K * EB), lv = (uint32_t)A.c.H * (V * EB);
    const char *pk = reinterpret_cast<const char *>(A.k) + (sq.t0 * A.c.Hk + h / group) * (K * EB);
    const char *pq = reinterpret_cast<const char *>(A.q) + (sq.t0 * A.c.Hk + h / group) * (K * EB);
    const char *pd = reinterpret_cast<const char *>(A.dout) + (sq.t0 * A.c.H + h) * (V * EB);
    constexpr int64_t tile = (int64_t)V * C * (BF ? 2 * NP : 4);
    RowsIn<BF, K, C, NT> rk, rq;
    RowsIn<BF, V, C, NT> rd;
    TileIn<BF, V, NP, NT> rz, rw;
    rk.init(tid, lk);
    rq.init(tid, lk);
    rd.init(tid, lv);
    rz.init(tid);
    rw.init(tid);
    u32x4 rwt;
    auto take = [&](int i) __attribute__((always_inline)) {
        const int c = c0 + i;
        const int64_t t = (int64_t)c * C, at = (sq.first + c) * A.c.H + h;
        const int m = len - (int)t < C ? len - (int)t : C;
        rk.take(pk + t * lk, m);
        rq.take(pq + t * lk, m);
        rd.take(pd + t * lv, m);
        rz.take(A.z + at * tile);
        rw.take(A.dw + at * tile);
        rwt = *reinterpret_cast<const u32x4 *>(A.c.rec + at * rec_bytes(true) + rec_weights(true) + (tid & 63) * 16);
    };
    auto put = [&](int i) __attribute__((always_inline)) {
        char *const p = smem + (i & (L::NB - 1)) * L::ROWS;
        rk.put(p + L::k);
        rq.put(p + L::q);
        rd.put(p + L::dout);
        rz.put(p + L::z);
        rw.put(p + L::dw);
        if (wave == 0) *reinterpret_cast<u32x4 *>(p + L::wt + tid * 16) = rwt;
    };
    take(0);
    f32x4 st[VT];
    const int64_t border_h = (sq.border + slot - sq.seg) * A.c.H + h;  // the border behind the segment
    get_state(c0 > 0 ? A.seed_s + (border_h - A.c.H) * sstate : A.S0 ? A.S0 + nh * sstate : nullptr, st);
    hd::mfma_fence_state(reinterpret_cast<f32x4(&)[1][VT]>(st));

    const int rowv0 = RV::row_at(lane), rowk0 = RK::row_at(lane), rowc0 = RC::row_at(lane), tilev0 = RV::tile_at(lane);
    const int tcols0 = TV::cols_at(lane), trows0 = TV::rows_at(lane);
    const int colk0 = RK::col_at(lane, wave);
    auto tile_cols = [&](const char *s, int vc, int tt) __attribute__((always_inline)) {
        return TV::all_cols(s, tcols0, vc, tt);
    };
    auto tile_rows = [&](const char *s, int vt) __attribute__((always_inline)) { return TV::all_rows(s, trows0, vt); };
    // The matrices of the pairs' weights: sixteen bytes of a row are the tokens of a lane group's slots, as in a tile.
    auto mat_row = [&](const char *s, int tt) __attribute__((always_inline)) {
        Pair<BF> p;
#pragma unroll
        for (int n = 0; n < L::NM; ++n) p.p[n] = RC::row_frag(s + n * L::M_ + 16 * tt * RC::RB, rowc0, 0);
        return p;
    };
    auto put_mat = [&](char *s, int row, int ts, const f32x4 &w) __attribute__((always_inline)) {  // sources 16 ts + 4g ..
        if constexpr (BF) {
            const int at = RC::slot(row, g) + 8 * ts;
            uint2 hi, lo;
            split_bf16(w.x, w.y, hi.x, lo.x);
            split_bf16(w.z, w.w, hi.y, lo.y);
            *reinterpret_cast<uint2 *>(s + at) = hi;
            *reinterpret_cast<uint2 *>(s + L::M_ + at) = lo;
        } else {
            *reinterpret_cast<f32x4 *>(s + RC::quad(row, 16 * ts + 4 * g)) = w;
        }
    };
    auto mat_one = [&](const char *s, int row, int j) __attribute__((always_inline)) -> float {
        if constexpr (BF) {
            const char *p = s + RC::slot(row, (j >> 2) & 3) + 8 * (j >> 4) + 2 * (j & 3);
            return bf2f(*reinterpret_cast<const uint16_t *>(p)) + bf2f(*reinterpret_cast<const uint16_t *>(p + L::M_));
        } else {
            return RC::load_one(s, row, j);
        }
    };
    auto clear_mats = [&]() __attribute__((always_inline)) {  // the tiles across the diagonal are read, never computed
        for (int i = tid; i < 2 * L::NM * L::M_ / 16; i += NT) reinterpret_cast<uint4 *>(s_m1)[i] = make_uint4(0, 0, 0, 0);
    };
    auto weights = [&](int which, float (&w)[8]) __attribute__((always_inline)) {
        *reinterpret_cast<f32x4 *>(w) = *reinterpret_cast<const f32x4 *>(s_wt + which * C + token_of(0, g));
        *reinterpret_cast<f32x4 *>(w + 4) = *reinterpret_cast<const f32x4 *>(s_wt + which * C + token_of(1, g));
    };
    // e^{b_r - b_i} of a lane's four rows against one token
    auto decays = [&](int t, int s0, bool later, f32x4 &e) __attribute__((always_inline)) {
        const float th = s_wt[kSumHi * C + t], tl = s_wt[kSumLo * C + t];
        const f32x4 sh = *reinterpret_cast<const f32x4 *>(s_wt + kSumHi * C + s0);
        const f32x4 sl = *reinterpret_cast<const f32x4 *>(s_wt + kSumLo * C + s0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            e[i] = __builtin_amdgcn_exp2f(later ? (sh[i] - th) + (sl[i] - tl) : (th - sh[i]) + (tl - sl[i]));
    };
    // a token's dot of rows x with a result y (columns 4g + i of token 16 tt + l % 16) over this wavefront's columns
    auto dot = [&](const char *x, int tt, const f32x4 &y) __attribute__((always_inline)) {
        float r[4];
        int row = 16 * tt + li;
        asm("" : "+v"(row));  // one read for both tiles would meet itself on the same banks
        RK::load_quad(x, row, col + 4 * g, r);
        float d = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) d = fmaf(r[i], y[i], d);
        return d;
    };
    auto at_of = [&](int64_t t) __attribute__((always_inline)) { return (t * A.c.H + h) * K + col + 4 * g; };
    auto store = [&](void *p, int64_t at, const f32x4 &y) __attribute__((always_inline)) {
        if constexpr (BF && !YF)
            *reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(p) + at) =
                make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
        else
            *reinterpret_cast<f32x4 *>(reinterpret_cast<float *>(p) + at) = y;
    };
    // y += the first matrix times the rows at s (f: this wavefront's columns of them); see all_finite
    auto mix = [&](f32x4 (&y)[2], const Exact<BF> (&f)[1], const float (&x)[8], const Pair<BF> (&mat)[2], const char *s,
                   bool later, int m) __attribute__((always_inline)) {
        if (all_finite(x)) {
            mmx(y, f, mat);
            return;
        }
#pragma unroll 1
        for (int j = 0; j < m; ++j) {
            float r[4];
            RK::load_quad(s, j, col + 4 * g, r);
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
                const int t = 16 * tt + li;
                const float w = mat_one(s_m1, t, j);
                if (later ? j >= t : j <= t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[tt][i] = fmaf(w, r[i], y[tt][i]);
            }
        }
    };

    // ================================================================ forward in time
    clear_mats();
    if constexpr (L::NB == 2) {
        put(0);
        if (nch > 1) take(1);
    }
    // the gradient behind the segment: for the walk back, asked for before the last chunk where registers are left
    f32x4 gt[VT];
    constexpr bool EARLY = NP == 2;
    const float *const behind =
        c1 < all ? A.seed_g + border_h * sstate : A.dS_final ? A.dS_final + nh * sstate : nullptr;
    for (int i = 0; i < nch; ++i) {
        const int64_t tc = sq.t0 + (int64_t)(c0 + i) * C;
        const int m = sq.t1 - tc < C ? (int)(sq.t1 - tc) : C;
        rows_of(i);
        __syncthreads();  // the last chunk's rows and matrices are read (NB = 2: and this one's rows are there)
        if constexpr (L::NB == 1) {
            put(i);
            if (i + 1 < nch) take(i + 1);
            else if (nch > 1) take(nch - 2);  // the walk back begins with the chunk that is here
            __syncthreads();
        }
        if (EARLY && i == nch - 1) get_state(behind, gt);
        // ---- the pairs' weights: lane holds sources i = 16 ts + 4g .. of token r = 16 tt + l % 16
        for (int p = wave; p < 6; p += NW) {
            const int which = p >= 3, x = which ? p - 3 : p, tt = x > 0, ts = x > 1;
            f32x4 part[VC], acc, prod = zero4(), e;
            const int r = 16 * tt + li, i0 = 16 * ts + 4 * g;
            Op z[VC];
#pragma unroll
            for (int vc = 0; vc < VC; ++vc) {
                part[vc] = zero4();
                z[vc] = tile_cols(s_z, vc, ts);
            }
            if (which) {
                Op w[VC];
#pragma unroll
                for (int vc = 0; vc < VC; ++vc) w[vc] = tile_cols(s_dw, vc, tt);
                mmx(part, z, w);
            } else {
                Exact<BF> d[VC];
#pragma unroll
                for (int vc = 0; vc < VC; ++vc) d[vc].p[0] = RV::row_frag(s_do + 16 * tt * RV::RB, rowv0, vc);
                mmx(part, z, d);
            }
#pragma unroll
            for (int kc = 0; kc < KC; ++kc)
                prod = mma32(prod, RK::row_frag(s_k + 16 * ts * RK::RB, rowk0, kc),
                             RK::row_frag((which ? s_k : s_q) + 16 * tt * RK::RB, rowk0, kc));
            decays(r, i0, false, e);
            const f32x4 be = *reinterpret_cast<const f32x4 *>(s_wt + kBeta * C + i0);
            const float f = which ? -s_wt[kBeta * C + r] : A.scale;
            fence_each(part);
            acc = sum_of(part);
            mfma_fence(prod);
            if (which && tt == ts && r < m) {  // M's diagonal
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i0 + i == r) {
                        const int64_t at = (tc + r) * A.c.H + h;
                        if (!GF) IO<true>::st(reinterpret_cast<uint16_t *>(A.dbeta), at, acc[i]);
                        else reinterpret_cast<float *>(A.dbeta)[at] = acc[i];
                    }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[i] = (which ? i0 + i < r : i0 + i <= r) && r < m ? f * acc[i] * e[i] * be[i] : 0.f;
            put_mat(which ? s_m2 : s_m1, r, ts, acc);
            // pairs of the log-decays' gradient: + at the row, - at the source
            float sum = 0.f;
            f32x4 by_source;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const float X = i0 + n < r ? acc[n] * prod[n] : 0.f;
                sum += X;
                by_source[n] = row_scan16(X);  // the source's sum, in its last lane
            }
            if (li == 15) *reinterpret_cast<f32x4 *>(&s_pairs[i][2 * p + 1][4 * g]) = by_source;
            sum = sum_groups(sum);
            if (g == 0) s_pairs[i][2 * p][li] = sum;
        }
        if constexpr (L::NB == 2) {
            if (i + 1 < nch) {
                put(i + 1);
                if (i + 2 < nch) take(i + 2);
                else if (nch > 2) take(nch - 3);  // the walk back finds the last two chunks here
            }
        }
        // ---- what the state gives
        f32x4 y1[2] = {zero4(), zero4()}, y2[2] = {zero4(), zero4()};
#pragma unroll
        for (int vc = 0; vc < VC; ++vc) {
            Exact<BF> d[2];
            Op w[2];
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
                d[tt].p[0] = RV::row_frag(s_do + 16 * tt * RV::RB, rowv0, vc);
                w[tt] = tile_cols(s_dw, vc, tt);
            }
            const Op s[1] = {multi_of<BF, NP>(st[2 * vc], st[2 * vc + 1])};
            mmx(y1, s, d);
            mmx(y2, s, w);
        }
        mfma_fence(y1[0], y1[1], y2[0], y2[1]);
        float dots[2];
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
            const int t = 16 * tt + li;
            y1[tt] *= s_wt[kEnterScaled * C + t];
            y2[tt] *= -s_wt[kEnter * C + t] * s_wt[kBeta * C + t];
            dots[tt] = dot(s_q, tt, y1[tt]) + dot(s_k, tt, y2[tt]);
        }
        __syncthreads();
        Pair<BF> mat1[2], mat2[2];
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
            mat1[tt] = mat_row(s_m1, tt);
            mat2[tt] = mat_row(s_m2, tt);
        }
        const Exact<BF> kf[1] = {{{RK::col_frag(s_k, colk0)}}};
        float kx[8], w[8];
        widen(kf[0].p[0], kx);
        mix(y1, kf, kx, mat1, s_k, false, m);
        mmx(y2, kf, mat2);
        // ---- the state's update
        weights(kLeaveBeta, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] *= kx[i];
        Op kp;
        set_multi(kp, w);
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
            const float d = sum_groups(dots[tt]);
            if (g == 0) s_u[i][wave][16 * tt + li] = d;
        }
        const float total = s_wt[kTotal * C];
#pragma unroll
        for (int vt = 0; vt < VT; ++vt) {
            st[vt] *= total;
            st[vt] = mmx(st[vt], tile_rows(s_z, vt), kp);
        }
        // ---- results
        mfma_fence(y1[0], y1[1], y2[0], y2[1]);
#pragma unroll
        for (int tt = 0; tt < 2; ++tt)
            if (16 * tt + li < m) {
                const int64_t at = at_of(tc + 16 * tt + li);
                store(A.dq, at, y1[tt]);
                *reinterpret_cast<f32x4 *>(A.dk_part + at) = y2[tt];
            }
        hd::mfma_fence_state(reinterpret_cast<f32x4(&)[1][VT]>(st));
    }
    // ---- what the border behind the segment passes on
    if (!EARLY) get_state(behind, gt);
    float border = 0.f;
#pragma unroll
    for (int vt = 0; vt < VT; ++vt)
#pragma unroll
        for (int i = 0; i < 4; ++i) border = fmaf(gt[vt][i], st[vt][i], border);
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) border += __shfl_xor(border, d);
    if (lane == 0) s_red[wave] = border;
    hd::mfma_fence_state(reinterpret_cast<f32x4(&)[1][VT]>(gt));

    // ================================================================ backward in time
    __syncthreads();
    clear_mats();
    for (int i = nch - 1; i >= 0; --i) {
        const int64_t tc = sq.t0 + (int64_t)(c0 + i) * C;
        const int m = sq.t1 - tc < C ? (int)(sq.t1 - tc) : C;
        rows_of(i);
        __syncthreads();
        if (L::NB == 1 && i < nch - 1) {
            put(i);
            if (i > 0) take(i - 1);
            __syncthreads();
        }
        f32x4 read[2];  // what the walk forward left for dk
#pragma unroll
        for (int tt = 0; tt < 2; ++tt)
            if (16 * tt + li < m) read[tt] = *reinterpret_cast<const f32x4 *>(A.dk_part + at_of(tc + 16 * tt + li));
        // ---- the pairs' weights the other way round: lane holds tokens j = 16 ts + 4g .. that see token r = 16 tt + l % 16
        for (int p = wave; p < 6; p += NW) {
            const int which = p >= 3, x = which ? p - 3 : p, ts = x > 0, tt = x > 1;
            f32x4 part[VC], acc, e;
            const int r = 16 * tt + li, j0 = 16 * ts + 4 * g;
            Op z[VC];
#pragma unroll
            for (int vc = 0; vc < VC; ++vc) {
                part[vc] = zero4();
                z[vc] = tile_cols(s_z, vc, tt);
            }
            if (which) {
                Op w[VC];
#pragma unroll
                for (int vc = 0; vc < VC; ++vc) w[vc] = tile_cols(s_dw, vc, ts);
                mmx(part, w, z);
            } else {
                Exact<BF> d[VC];
#pragma unroll
                for (int vc = 0; vc < VC; ++vc) d[vc].p[0] = RV::row_frag(s_do + 16 * ts * RV::RB, rowv0, vc);
                mmx(part, d, z);
            }
            decays(r, j0, true, e);
            const f32x4 be = *reinterpret_cast<const f32x4 *>(s_wt + kBeta * C + j0);
            const float f = s_wt[kBeta * C + r];
            fence_each(part);
            acc = sum_of(part);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[i] = (which ? j0 + i > r : j0 + i >= r) && j0 + i < m ? f * acc[i] * e[i] * (which ? -be[i] : A.scale) : 0.f;
            put_mat(which ? s_m2 : s_m1, r, ts, acc);
        }
        if constexpr (L::NB == 2)
            if (i > 0 && i < nch - 1) {
                put(i - 1);
                if (i > 1) take(i - 2);
            }
        f32x4 y[2] = {zero4(), zero4()};
#pragma unroll
        for (int vc = 0; vc < VC; ++vc) {
            Op z[2];
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) z[tt] = tile_cols(s_z, vc, tt);
            const Op s[1] = {multi_of<BF, NP>(gt[2 * vc], gt[2 * vc + 1])};
            mmx(y, s, z);
        }
        mfma_fence(y[0], y[1]);
        float dots[2];
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
            y[tt] *= s_wt[kLeaveBeta * C + 16 * tt + li];
            dots[tt] = dot(s_k, tt, y[tt]);
        }
        __syncthreads();
        Pair<BF> mat1[2], mat2[2];
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
            mat1[tt] = mat_row(s_m1, tt);
            mat2[tt] = mat_row(s_m2, tt);
        }
        const Exact<BF> kf[1] = {{{RK::col_frag(s_k, colk0)}}}, qf[1] = {{{RK::col_frag(s_q, colk0)}}};
        float qx[8], kx[8];
        widen(qf[0].p[0], qx);
        widen(kf[0].p[0], kx);
        mix(y, qf, qx, mat1, s_q, true, m);
        mmx(y, kf, mat2);
        // ---- the state gradient's update
        Op qp, kp;
        {
            float w[8], e[8], be[8];
            weights(kEnterScaled, w);
            weights(kEnter, e);
            weights(kBeta, be);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                w[i] *= qx[i];
                e[i] *= -be[i] * kx[i];
            }
            set_multi(qp, w);
            set_multi(kp, e);
        }
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
            const float d = sum_groups(dots[tt]);
            if (g == 0) s_u[i][wave][16 * tt + li] -= d;
        }
        const float total = s_wt[kTotal * C];
#pragma unroll
        for (int vt = 0; vt < VT; ++vt) {
            gt[vt] *= total;
            const Exact<BF> d = {{RV::tile_frag(s_do, tilev0, vt)}};
            gt[vt] = mmx(gt[vt], d, qp);
            gt[vt] = mmx(gt[vt], tile_rows(s_dw, vt), kp);
        }
        mfma_fence(y[0], y[1]);
#pragma unroll
        for (int tt = 0; tt < 2; ++tt)
            if (16 * tt + li < m) store(A.dk, at_of(tc + 16 * tt + li), y[tt] + read[tt]);
        hd::mfma_fence_state(reinterpret_cast<f32x4(&)[1][VT]>(gt));
    }
    __syncthreads();
    for (int t = tid; t < nch * C; t += NT) {
        const int i = t / C, r = t % C;
        float d = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) d += s_u[i][w][r];
        // jobs 3x + (0, 1, 2): rows of tiles 0, 1, 1, sources of tiles 0, 0, 1
#pragma unroll
        for (int x = 0; x < 6; x += 3) {
            const float *s = &s_pairs[i][2 * x][r & 15];
            d += r < 16 ? s[0] - (s[16] + s[48]) : s[32] + (s[64] - s[80]);
        }
        s_db[t] = sq.t0 + (int64_t)c0 * C + t < sq.t1 ? d : 0.f;
    }
    __syncthreads();
    // ---- dg: the sums from a token to the border, in fp64
    if (wave == 0) {
        constexpr int PER = L::MOST * C / 64;
        double own[PER], sum = 0.0;
#pragma unroll
        for (int i = PER - 1; i >= 0; --i) {
            const int t = lane * PER + i;
            sum += t < nch * C ? (double)s_db[t] : 0.0;
            own[i] = sum;
        }
        double upto = sum;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const double x = __shfl_down(upto, d);
            if (lane + d < 64) upto += x;
        }
        double b = upto - sum;
#pragma unroll
        for (int w = 0; w < NW; ++w) b += s_red[w];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int64_t t = sq.t0 + (int64_t)c0 * C + lane * PER + i;
            if (t < sq.t1 && lane * PER + i < nch * C) {
                const float x = (float)(own[i] + b);
                if (!GF) IO<true>::st(reinterpret_cast<uint16_t *>(A.dg), t * A.c.H + h, x);
                else reinterpret_cast<float *>(A.dg)[t * A.c.H + h] = x;
            }
        }
    }
}

template <bool BF, int K, int V, bool YF, int NP>
hipError_t launch_grad(const GradArgs &a, hipStream_t st) {
    hipLaunchKernelGGL((kda_gd_grad_kernel<BF, K, V, YF, NP>), hd::wide_grid(a.c.segs * a.c.H), dim3(K * 4), 0, st, a);
    return hipGetLastError();
}
template <bool BF, int K, bool YF, int NP>
hipError_t grad_by_v(const GradArgs &a, int V, hipStream_t st) {
    return V == 32   ? launch_grad<BF, K, 32, YF, NP>(a, st)
           : V == 64 ? launch_grad<BF, K, 64, YF, NP>(a, st)
                     : launch_grad<BF, K, 128, YF, NP>(a, st);
}
template <bool BF, bool YF, int NP>
hipError_t grad_by_k(const GradArgs &a, int K, int V, hipStream_t st) {
    return K == 32   ? grad_by_v<BF, 32, YF, NP>(a, V, st)
           : K == 64 ? grad_by_v<BF, 64, YF, NP>(a, V, st)
                     : grad_by_v<BF, 128, YF, NP>(a, V, st);
}

}  // namespace gd
}  // namespace kda
