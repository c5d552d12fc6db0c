// The gated delta rule with one decay per head: the chunks' records, the order of the passes of a forward or backward
// call, and the sums over heads that share q and k.
#include "kda_gd_core.hpp"

namespace kda {
namespace gd {
namespace {

// ------------------------------------------------------------------ packed sequences
// One workgroup: clamps cu_seqlens into [0, T], makes it non-decreasing (a running maximum), numbers the chunks, segments and
// borders between them, and orders up to 1024 sequences by length: one that starts late would run on alone (more of them balance by
// their number). T < 2^31. (4 us; without the order the state pass over 16 sequences of 17011 tokens, 32 heads, took 275
// us, not 227.)
__global__ __launch_bounds__(1024) void kda_gd_table_kernel(const int32_t *__restrict__ cu, int32_t N, uint32_t T,
                                                            uint32_t seg_chunks, Packed *__restrict__ seqs,
                                                            int32_t *__restrict__ order) {
    __shared__ uint32_t s_max[16], s_chunks[16], s_segs[16], s_borders[16];
    __shared__ __align__(16) uint32_t s_all[1024];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    auto entry = [&](int64_t i) -> uint32_t {
        const int32_t x = cu[i];
        return x < 0 ? 0 : (uint32_t)x > T ? T : (uint32_t)x;
    };
    uint32_t top = entry(0), first = 0, seg = 0, border = 0;
    for (int64_t base = 0; base < N; base += 1024) {
        const int64_t n = base + t;
        uint32_t end = n < N ? entry(n + 1) : 0;
        if (end < top) end = top;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t x = __shfl_up(end, d);
            if (lane >= d && x > end) end = x;
        }
        uint32_t before = __shfl_up(end, 1);
        if (lane == 0) before = top;
        if (lane == 63) s_max[wave] = end;
        __syncthreads();
        for (int w = 0; w < 16; ++w) {
            const uint32_t x = s_max[w];
            if (w < wave && x > end) end = x;
            if (w < wave && x > before) before = x;
            if (x > top) top = x;
        }
        const uint32_t chunks = (end - before + (kChunkTokens - 1)) / kChunkTokens;
        const uint32_t segs = (chunks + (seg_chunks - 1)) / seg_chunks;
        const uint32_t borders = segs ? segs - 1 : 0;
        uint32_t uc = chunks, us = segs, ub = borders;  // sums up to this sequence
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t x = __shfl_up(uc, d), y = __shfl_up(us, d), z = __shfl_up(ub, d);
            if (lane >= d) uc += x, us += y, ub += z;
        }
        if (lane == 63) s_chunks[wave] = uc, s_segs[wave] = us, s_borders[wave] = ub;
        s_all[t] = chunks;
        __syncthreads();
        if (N > 1024) {
            if (n < N) order[n] = (int32_t)n;
        } else if (n < N) {  // the longest first, of equal ones the first; lengths behind the last are 0 and come last
            int ahead = 0;
            for (int j = 0; j < N; j += 4) {
                const uint4 x = *reinterpret_cast<const uint4 *>(s_all + j);
                ahead += (x.x > chunks || (x.x == chunks && j < t)) + (x.y > chunks || (x.y == chunks && j + 1 < t)) +
                         (x.z > chunks || (x.z == chunks && j + 2 < t)) + (x.w > chunks || (x.w == chunks && j + 3 < t));
            }
            order[ahead] = (int32_t)n;
        }
        uint32_t ac = 0, as = 0, ab = 0;
        for (int w = 0; w < 16; ++w) {
            if (w < wave) uc += s_chunks[w], us += s_segs[w], ub += s_borders[w];
            ac += s_chunks[w];
            as += s_segs[w];
            ab += s_borders[w];
        }
        if (n < N)
            seqs[n] = Packed{(int64_t)before, (int64_t)end, (int64_t)(first + uc - chunks), (int32_t)(seg + us - segs),
                             (int32_t)(border + ub - borders)};
        first += ac;
        seg += as;
        border += ab;
        __syncthreads();
    }
}

// ------------------------------------------------------------------ the chunks' records
// One wavefront per (chunk, q/k head): the products k_r.k_i and q_r.k_i once, then for every v head that shares them the
// decays, A and its inverse. The inverse by blocks of 16: by substitution over all 32 rows the registers that hold them
// spilled (464 us for the 70 below). It is formed in fp32; as operands the matrices leave in two bf16 parts (2^-17 of an
// entry), for the gradients of fp32 gates in three: with two dbeta was off by 2.6e-6 of its size, with three by 2.4e-7.
// HBM bounds it: 4096 tokens of 96 heads of 128 channels, bf16, move 328 MB in 69 us (4.8 TB/s), backward 377 MB in 79.
constexpr int kPitch = kChunkTokens + 4;
template <bool BF, bool GF, int K, bool BWD>
__global__ __launch_bounds__(64) void kda_gd_prep_kernel(const Common cm, const void *__restrict__ qp,
                                                         const void *__restrict__ kp, const void *__restrict__ gp,
                                                         const void *__restrict__ bp, float scale) {
    constexpr int C = kChunkTokens, KC = K / 32, EB = BF ? 2 : 4, NM = BWD ? 2 : 1;
    using GE = typename IO<!GF>::T;
    __shared__ __align__(16) float s_a[NM][C][kPitch], s_p[C][kPitch];
    __shared__ __align__(16) float s_bh[C], s_bl[C], s_be[C];
    const int lane = threadIdx.x, g = lane >> 4, li = lane & 15;
    const int64_t blk = blockIdx.x + (int64_t)blockIdx.y * gridDim.x, slot = blk / cm.Hk;
    const int hk = (int)(blk - slot * cm.Hk), group = cm.H / cm.Hk;
    if (slot >= cm.slots) return;
    const int64_t ns = find_seq<false>(cm, slot, lane);
    const Seq sq = seq_of(cm, ns);
    const int64_t tc = sq.t0 + (slot - sq.first) * C;
    if (slot < sq.first || tc >= sq.t1) return;
    const int n = (int)(sq.t1 - tc < C ? sq.t1 - tc : C);

    // ---- the products: lane holds sources 16 ts + 4g + i of token 16 tt + l % 16
    const char *pk = reinterpret_cast<const char *>(kp) + (tc * cm.Hk + hk) * (K * EB);
    const char *pq = reinterpret_cast<const char *>(qp) + (tc * cm.Hk + hk) * (K * EB);
    const int64_t pitch = (int64_t)cm.Hk * (K * EB);
    auto row_frag = [&](const char *p, int tt, int c) __attribute__((always_inline)) {
        const int t = 16 * tt + li;
        const char *r = p + (t < n ? t : n - 1) * pitch;
        Frag8<BF> f;
        if constexpr (BF) {
            const u32x4 u = *reinterpret_cast<const u32x4 *>(r + 64 * c + 16 * g);
            f.p[0] = u.x; f.p[1] = u.y; f.p[2] = u.z; f.p[3] = u.w;
        } else {
            const f32x4 u = *reinterpret_cast<const f32x4 *>(r + 128 * c + 16 * g);
            const f32x4 w = *reinterpret_cast<const f32x4 *>(r + 128 * c + 64 + 16 * g);
            f = Frag8<false>{{u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w}};
        }
        return f;
    };
    f32x4 kk[3] = {zero4(), zero4(), zero4()}, qk[3] = {zero4(), zero4(), zero4()};  // tiles (0, 0), (1, 0), (1, 1)
#pragma unroll
    for (int c = 0; c < KC; ++c) {
        const Frag8<BF> k0 = row_frag(pk, 0, c), k1 = row_frag(pk, 1, c), q0 = row_frag(pq, 0, c), q1 = row_frag(pq, 1, c);
        kk[0] = mma32(kk[0], k0, k0);
        kk[1] = mma32(kk[1], k0, k1);
        kk[2] = mma32(kk[2], k1, k1);
        qk[0] = mma32(qk[0], k0, q0);
        qk[1] = mma32(qk[1], k0, q1);
        qk[2] = mma32(qk[2], k1, q1);
    }
    mfma_fence(kk[0], kk[1], kk[2], qk[0], qk[1], qk[2]);
    // the tile above the diagonal
    for (int i = lane; i < 16 * 16; i += 64) {
        s_a[0][i >> 4][16 + (i & 15)] = 0.f;
        if constexpr (BWD) s_a[1][i >> 4][16 + (i & 15)] = 0.f;
        s_p[i >> 4][16 + (i & 15)] = 0.f;
    }

    const int t = lane & 31;
    for (int hh = 0; hh < group; ++hh) {
        const int h = hk * group + hh;
        float gv = 0.f, bv = 0.f;
        if (t < n) {
            gv = IO<!GF>::ld(reinterpret_cast<const GE *>(gp), (tc + t) * cm.H + h);
            bv = IO<!GF>::ld(reinterpret_cast<const GE *>(bp), (tc + t) * cm.H + h);
        }
        hd::Decay d = hd::decay_base2(gv);
        d.hi = row_scan16(d.hi);
        d.lo = row_scan16(d.lo);
        const float h0 = lane_value(d.hi, 15), l0 = lane_value(d.lo, 15);
        d.hi += lane & 16 ? h0 : 0.f;
        d.lo += lane & 16 ? l0 : 0.f;
        const float hc = lane_value(d.hi, 31), lc = lane_value(d.lo, 31);
        const float enter = t < n ? __builtin_amdgcn_exp2f(d.hi + d.lo) : 0.f;
        const float leave = t < n ? __builtin_amdgcn_exp2f((hc - d.hi) + (lc - d.lo)) : 0.f;
        char *rec = cm.rec + (slot * cm.H + h) * rec_bytes(BWD);
        float *wt = reinterpret_cast<float *>(rec + rec_weights(BWD));
        __syncthreads();  // the last head's matrices are read
        if (lane < C) {
            s_bh[t] = d.hi;
            s_bl[t] = d.lo;
            s_be[t] = bv;
            wt[kEnter * C + t] = enter;
            wt[kEnterScaled * C + t] = scale * enter;
            wt[kLeave * C + t] = leave;
            wt[kLeaveBeta * C + t] = t < n ? bv * leave : 0.f;
            wt[kBeta * C + t] = bv;
            wt[kSumHi * C + t] = d.hi;
            wt[kSumLo * C + t] = d.lo;
            wt[kTotal * C + t] = __builtin_amdgcn_exp2f(hc + lc);
        }
        __syncthreads();
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            const int tt = p > 0, ts = p > 1, r = 16 * tt + li, i0 = 16 * ts + 4 * g;
            const float th = s_bh[r], tl = s_bl[r], be = s_be[r];
            const f32x4 sh = *reinterpret_cast<const f32x4 *>(s_bh + i0), sl = *reinterpret_cast<const f32x4 *>(s_bl + i0);
            const f32x4 sb = *reinterpret_cast<const f32x4 *>(s_be + i0);
            f32x4 a, a2, w;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float e = __builtin_amdgcn_exp2f((th - sh[i]) + (tl - sl[i]));
                const bool past = i0 + i < r && r < n, upto = i0 + i <= r && r < n;
                const float ka = kk[p][i] * e;
                a[i] = past ? ka * sb[i] : 0.f;
                a2[i] = past ? ka * be : 0.f;
                w[i] = upto ? scale * qk[p][i] * e * (BWD ? 1.f : sb[i]) : 0.f;
            }
            *reinterpret_cast<f32x4 *>(&s_a[0][r][i0]) = a;
            if constexpr (BWD) *reinterpret_cast<f32x4 *>(&s_a[1][r][i0]) = a2;
            *reinterpret_cast<f32x4 *>(&s_p[r][i0]) = w;
        }
        __syncthreads();
        // ---- the strict part N of (1 + A)^-1, in A's place (backward: both matrices)
        bool usual = true;
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x4 a = *reinterpret_cast<const f32x4 *>(&s_a[m][lane >> 1][16 * (lane & 1) + 4 * i]);
                s = fmaf(a.x, 0.f, fmaf(a.y, 0.f, fmaf(a.z, 0.f, fmaf(a.w, 0.f, s))));
            }
            usual = usual && s == 0.f;
        }
        if (__builtin_amdgcn_ballot_w64(!usual) == 0) {
            // The blocks on the diagonal by substitution, a column in each lane: row r is minus row r of A times the rows
            // before it. Then the block below them, -(1 + N_11) A_10 (1 + N_00).
            float inv[16];
            {
                float(*const A)[kPitch] = s_a[NM == 2 ? g >> 1 : 0];
                const int o = 16 * (g & 1);
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    f32x4 sum = zero4();
#pragma unroll
                    for (int l = 0; l < r; l += 4) {
                        const f32x4 a = *reinterpret_cast<const f32x4 *>(&A[o + r][o + l]);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (l + i < r) sum[i] = fmaf(a[i], inv[l + i], sum[i]);
                    }
                    inv[r] = r == li ? 1.f : -((sum.x + sum.y) + (sum.z + sum.w));
                }
                __syncthreads();
#pragma unroll
                for (int r = 0; r < 16; ++r) A[o + r][o + li] = inv[r];
                __syncthreads();
            }
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                float(*const A)[kPitch] = s_a[m];
                const f32x4 a = *reinterpret_cast<const f32x4 *>(&A[16 + li][4 * g]);
                const f32x4 c = *reinterpret_cast<const f32x4 *>(&A[16 + li][16 + 4 * g]);
                f32x4 x = zero4(), y = zero4();
#pragma unroll
                for (int i = 0; i < 4; ++i) x = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], A[4 * g + i][li], x, 0, 0, 0);
                mfma_fence(x);
#pragma unroll
                for (int i = 0; i < 4; ++i) y = __builtin_amdgcn_mfma_f32_16x16x4f32(c[i], x[i], y, 0, 0, 0);
                mfma_fence(y);
                __syncthreads();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    A[16 + 4 * g + i][li] = -y[i];
                    if (li == 4 * g + i) A[li][li] = A[16 + li][16 + li] = 0.f;
                }
            }
            __syncthreads();
        } else {
            // Something is not finite: row by row and no zeros times it, for the rows before it keep their values.
            for (int m = 0; m < NM; ++m)
                for (int r = 0; r < C; ++r) {
                    float s = 0.f;
                    for (int l = 0; l < r; ++l)
                        s += l == t ? s_a[m][r][l] : l > t ? s_a[m][r][l] * s_a[m][l][t] : 0.f;
                    __syncthreads();
                    if (lane < C && t < r) s_a[m][r][t] = -s;
                    __syncthreads();
                }
        }
        // ---- as operands (bf16 beside fp32 gates: what two parts leave of an entry lies by itself)
        auto put = [&](int which, int tt, const float (&x)[8]) __attribute__((always_inline)) {
            if constexpr (BF && GF && BWD) {
                Multi<true, 3> f;
                set_multi(f, x);
                store_mat(rec + which * kMatBytes, tt, lane, Pair<true>{{f.p[0], f.p[1]}});
                __builtin_memcpy(cm.third + (((slot * cm.H + h) * 3 + which) * 2 + tt) * (kThirdBytes / 2) + lane * 16,
                                 &f.p[2], 16);
            } else {
                Pair<BF> f;
                set_multi(f, x);
                store_mat(rec + which * kMatBytes, tt, lane, f);
            }
        };
        auto rows = [&](const float (&m)[C][kPitch], int r, float (&x)[8]) __attribute__((always_inline)) {
            *reinterpret_cast<f32x4 *>(x) = *reinterpret_cast<const f32x4 *>(&m[r][token_of(0, g)]);
            *reinterpret_cast<f32x4 *>(x + 4) = *reinterpret_cast<const f32x4 *>(&m[r][token_of(1, g)]);
        };
        auto cols = [&](const float (&m)[C][kPitch], int c, float (&x)[8]) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = m[slot_token(g, j)][c];
        };
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
            float x[8];
            rows(s_a[0], 16 * tt + li, x);
            put(kMatN, tt, x);
            if constexpr (!BWD) {
                rows(s_p, 16 * tt + li, x);
                put(kMatP, tt, x);
            } else {
                cols(s_a[BWD], 16 * tt + li, x);
                put(kMatNT, tt, x);
                cols(s_p, 16 * tt + li, x);
                put(kMatPT, tt, x);
            }
        }
    }
}

// out[t][hk][d] = sum over the group's heads of in[t][h][d] (fp32), for the tokens of the sequences; four d a thread.
template <bool BF>
__global__ __launch_bounds__(256) void kda_gd_group_kernel(const Common cm, const float *__restrict__ in0,
                                                           void *__restrict__ out0, const float *__restrict__ in1,
                                                           void *__restrict__ out1, int64_t per_token, int64_t D4) {
    const float *in = blockIdx.y ? in1 : in0;
    void *out = blockIdx.y ? out1 : out0;
    const int group = cm.H / cm.Hk;
    const int64_t lo = cm.seqs ? cm.seqs[0].t0 : 0, hi = cm.seqs ? cm.seqs[cm.N - 1].t1 : cm.ntok;
    const int64_t end = hi * per_token;  // per_token: Hk * D / 4
    for (int64_t e = lo * per_token + (int64_t)blockIdx.x * 256 + threadIdx.x; e < end; e += (int64_t)gridDim.x * 256) {
        const int64_t u = e / D4, d = e - u * D4;  // u: (token, q/k head)
        const f32x4 *p = reinterpret_cast<const f32x4 *>(in) + u * group * D4 + d;
        f32x4 x = p[0];
        for (int i = 1; i < group; ++i) x += p[i * D4];
        if constexpr (BF)
            reinterpret_cast<uint2 *>(out)[e] = make_uint2(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w));
        else
            reinterpret_cast<f32x4 *>(out)[e] = x;
    }
}

// ------------------------------------------------------------------ workspace
struct Layout {
    size_t seqs, order, rec, third, z, dw, seed_s, seed_g, dk_part, dq, dk, total;
};
struct Sizes {
    int64_t slots, segs, borders;
    int32_t nch, nseg, seg;
};
// The segments' length by the heads alone, so that a sequence's gradients are the same bits in every batch: about two
// workgroups of the gradients' kernel for every place on the card that a sequence of 4096 tokens finds. A segment's start and
// end cost about as much as 1.2 of its chunks and its states' way through memory (4096 x 96 heads: 533 us of 16 chunks, 554 of
// 8), a long one leaves compute units idle (1531 tokens x 12 heads of 64 channels: 282 us of 16 chunks, 146 of 8, 84 of 2).
// Short rows pay for it: a single one of 512 tokens of 96 heads is 96 workgroups (the whole call 210 us; segments of 8 chunks
// would take 149), of 64 heads 191 (of 4: 95); four rows of 512 497 (of 8: 466), one of 1024 271 (of 8: 285).
int32_t segment_chunks(int32_t H, int32_t K) {
    int32_t seg = segment_most(K);
    while (seg > 2 && (int64_t)seg * 512 > (int64_t)H * K) seg >>= 1;
    return seg;
}
Sizes sizes(int64_t B, int64_t T, int32_t N, int32_t H, int32_t K, bool packed) {
    Sizes s;
    const int64_t nch = (T + kChunkTokens - 1) / kChunkTokens;
    s.seg = segment_chunks(H, K);
    const int64_t nseg = (nch + s.seg - 1) / s.seg;
    s.nch = (int32_t)(nch ? nch : 1);
    s.nseg = (int32_t)(nseg ? nseg : 1);
    s.slots = packed ? T / kChunkTokens + N : B * nch;
    s.segs = packed ? T / (kChunkTokens * s.seg) + N : B * nseg;
    s.borders = packed ? T / (kChunkTokens * s.seg) : B * (s.nseg - 1);  // a sequence of L tokens has (L - 1) / a segment's
    return s;
}
Layout layout(const Sizes &s, int64_t ntok, int32_t H, int32_t Hk, int32_t K, int32_t V, int32_t N, bool packed, bool bwd,
              int tile_bytes) {
    Layout l{};
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    const size_t ch = (size_t)s.slots * H;
    if (packed) {
        l.seqs = take((size_t)N * sizeof(Packed));
        l.order = take((size_t)N * 4);
    }
    l.rec = take(ch * rec_bytes(bwd));
    if (bwd) {
        l.third = take(tile_bytes > 4 ? ch * 3 * kThirdBytes : 0);
        l.z = take(ch * V * kChunkTokens * tile_bytes);
        l.dw = take(ch * V * kChunkTokens * tile_bytes);
        l.seed_s = take((size_t)s.borders * H * K * V * 4);
        l.seed_g = take((size_t)s.borders * H * K * V * 4);
        l.dk_part = take((size_t)ntok * H * K * 4);
        if (Hk != H) {
            l.dq = take((size_t)ntok * H * K * 4);
            l.dk = take((size_t)ntok * H * K * 4);
        }
    }
    l.total = at ? at : 256;
    return l;
}

#define KDA_TRY(x)                            \
    do {                                      \
        const hipError_t e_ = (x);            \
        if (e_ != hipSuccess) return e_;      \
    } while (0)

// Of a value of the tiles between the backward call's passes: two bf16 parts where all that is summed from them leaves in
// bf16, three beside fp32 gates (whose gradients are sums with cancellation: 1.4e-5 off from two parts).
int tile_parts(bool io_bf16, bool gates_fp32) { return io_bf16 && gates_fp32 ? 3 : 2; }
int tile_bytes(bool io_bf16, bool gates_fp32) { return 2 * tile_parts(io_bf16, gates_fp32); }

struct Call {
    Layout l;
    char *ws;
    Common c;
};
Call prepare(const GdArgs &a, bool bwd) {
    Call x{};
    const bool packed = a.cu_seqlens != nullptr;
    const Sizes s = sizes(a.B, a.T, a.num_seqs, a.H, a.K, packed);
    x.l = layout(s, a.B * a.T, a.H, a.Hk, a.K, a.V, a.num_seqs, packed, bwd, tile_bytes(a.io_bf16, a.gates_fp32));
    x.ws = reinterpret_cast<char *>(a.workspace);
    x.c.seqs = packed ? reinterpret_cast<const Packed *>(x.ws + x.l.seqs) : nullptr;
    x.c.order = packed ? reinterpret_cast<const int32_t *>(x.ws + x.l.order) : nullptr;
    x.c.T = a.T;
    x.c.ntok = a.B * a.T;
    x.c.slots = s.slots;
    x.c.segs = s.segs;
    x.c.nch = s.nch;
    x.c.nseg = s.nseg;
    x.c.seg = s.seg;
    x.c.N = a.num_seqs;
    x.c.H = a.H;
    x.c.Hk = a.Hk;
    x.c.rec = x.ws + x.l.rec;
    x.c.third = bwd && tile_parts(a.io_bf16, a.gates_fp32) == 3 ? x.ws + x.l.third : nullptr;
    return x;
}

template <bool BF, bool GF, int K>
hipError_t prep_kb(const GdArgs &a, const Common &c, bool bwd, hipStream_t st) {
    const dim3 grid = hd::wide_grid(c.slots * a.Hk);
    if (bwd)
        hipLaunchKernelGGL((kda_gd_prep_kernel<BF, GF, K, true>), grid, dim3(64), 0, st, c, a.q, a.k, a.g, a.beta, a.scale);
    else
        hipLaunchKernelGGL((kda_gd_prep_kernel<BF, GF, K, false>), grid, dim3(64), 0, st, c, a.q, a.k, a.g, a.beta, a.scale);
    return hipGetLastError();
}
template <bool BF, bool GF>
hipError_t prep_k(const GdArgs &a, const Common &c, bool bwd, hipStream_t st) {
    return a.K == 32   ? prep_kb<BF, GF, 32>(a, c, bwd, st)
           : a.K == 64 ? prep_kb<BF, GF, 64>(a, c, bwd, st)
                       : prep_kb<BF, GF, 128>(a, c, bwd, st);
}
// The table of packed sequences and the chunks' records.
hipError_t make_records(const GdArgs &a, const Call &x, bool bwd, hipStream_t st) {
    if (x.c.seqs) {
        hipLaunchKernelGGL(kda_gd_table_kernel, dim3(1), dim3(1024), 0, st, a.cu_seqlens, a.num_seqs, (uint32_t)a.T,
                           (uint32_t)x.c.seg, const_cast<Packed *>(x.c.seqs), const_cast<int32_t *>(x.c.order));
        KDA_TRY(hipGetLastError());
    }
    if (a.T == 0) return hipSuccess;
    if (!a.io_bf16) return prep_k<false, true>(a, x.c, bwd, st);
    return a.gates_fp32 ? prep_k<true, true>(a, x.c, bwd, st) : prep_k<true, false>(a, x.c, bwd, st);
}

}  // namespace
}  // namespace gd

size_t gd_fwd_workspace_bytes(int64_t B, int64_t T, int32_t H, int32_t Hk, int32_t K, int32_t V, int32_t num_seqs,
                              bool packed, bool) {
    return gd::layout(gd::sizes(B, T, num_seqs, H, K, packed), B * T, H, Hk, K, V, num_seqs, packed, false, 0).total;
}
size_t gd_bwd_workspace_bytes(int64_t B, int64_t T, int32_t H, int32_t Hk, int32_t K, int32_t V, int32_t num_seqs,
                              bool packed, bool io_bf16) {
    return gd::layout(gd::sizes(B, T, num_seqs, H, K, packed), B * T, H, Hk, K, V, num_seqs, packed, true,
                      gd::tile_bytes(io_bf16, true)).total;
}

hipError_t launch_gd_fwd(const GdArgs &a, hipStream_t st) {
    using namespace gd;
    const Call x = prepare(a, false);
    KDA_TRY(make_records(a, x, false, st));
    StateArgs s{};
    s.c = x.c;
    s.q = a.q;
    s.k = a.k;
    s.v = a.v;
    s.s_init = a.S0;
    s.s_end = a.S_final;
    s.o = a.o;
    return forward_pass(a.io_bf16, s, a.K, a.V, st);
}

hipError_t launch_gd_bwd(const GdArgs &a, hipStream_t st) {
    using namespace gd;
    const Call x = prepare(a, true);
    KDA_TRY(make_records(a, x, true, st));
    auto at = [&](size_t off) { return x.ws + off; };
    StateArgs s{};
    s.c = x.c;
    s.q = a.q;
    s.k = a.k;
    s.parts = tile_parts(a.io_bf16, a.gates_fp32);
    // forward in time: the errors z, and the states at the segments' starts
    StateArgs e = s;
    e.v = a.v;
    e.s_init = a.S0;
    e.rows = at(x.l.z);
    e.seed = reinterpret_cast<float *>(at(x.l.seed_s));
    // backward in time: dv, the writes' gradients, and the state's at the segments' ends
    s.v = a.dout;
    s.s_init = a.dS_final;
    s.s_end = a.dS0;
    s.o = a.dv;
    s.rows = at(x.l.dw);
    s.seed = reinterpret_cast<float *>(at(x.l.seed_g));
    KDA_TRY(backward_passes(a.io_bf16, s, e, a.K, a.V, st));
    if (a.T == 0) return hipSuccess;
    const bool grouped = a.H != a.Hk;
    GradArgs g{};
    g.c = x.c;
    g.q = a.q;
    g.k = a.k;
    g.dout = a.dout;
    g.z = at(x.l.z);
    g.dw = at(x.l.dw);
    g.S0 = a.S0;
    g.dS_final = a.dS_final;
    g.seed_s = reinterpret_cast<const float *>(at(x.l.seed_s));
    g.seed_g = reinterpret_cast<const float *>(at(x.l.seed_g));
    g.dq = grouped ? at(x.l.dq) : a.dq;
    g.dk = grouped ? at(x.l.dk) : a.dk;
    g.dk_part = reinterpret_cast<float *>(at(x.l.dk_part));
    g.dg = a.dg;
    g.dbeta = a.dbeta;
    g.scale = a.scale;
    KDA_TRY(!a.io_bf16     ? grad_pass_fp32(g, a.K, a.V, st)
            : a.gates_fp32 ? grad_pass_bf16_gates_fp32(g, a.K, a.V, grouped, st)
                           : grad_pass_bf16(g, a.K, a.V, grouped, st));
    if (!grouped) return hipSuccess;
    const int64_t per = (int64_t)a.Hk * a.K / 4, n = a.B * a.T * per;
    const dim3 grid((uint32_t)((n + 255) / 256 < 8192 ? (n + 255) / 256 : 8192), 2);
    const float *iq = reinterpret_cast<const float *>(g.dq), *ik = reinterpret_cast<const float *>(g.dk);
    if (a.io_bf16)
        hipLaunchKernelGGL(kda_gd_group_kernel<true>, grid, dim3(256), 0, st, x.c, iq, a.dq, ik, a.dk, per, (int64_t)a.K / 4);
    else
        hipLaunchKernelGGL(kda_gd_group_kernel<false>, grid, dim3(256), 0, st, x.c, iq, a.dq, ik, a.dk, per, (int64_t)a.K / 4);
    return hipGetLastError();
}

}  // namespace kda
