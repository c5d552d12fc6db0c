// Layer norm over rows of C channels, its output gate, and its gradient, for gfx950.
//
//   n = (x - mean) r,  r = (mean((x - mean)^2) + eps)^(-1/2)   (mean = 0 without centering)
//   y = n w + b,  and with a gate's pre-activation z:  y sigmoid(z)
// backward, with dy the gradient of what was returned and a = sigmoid(z) (1 without a gate):
//   dz = dy (n w + b) a (1 - a);  e = dy a;  dw = sum_rows e n;  db = sum_rows e;
//   d = e w;  dx = r (d - n mean(d n) - mean(d))              (the last term only with centering)
//
// Both directions are bound by bytes: every row is read once, held in registers through its reductions (the variance
// is the mean square of the centered values, not a difference of sums), and written once. The backward recomputes
// the statistics, so nothing is kept from the forward. All arithmetic is fp32. Measured, bf16: forward of 4096 x 96
// rows of 128 with a gate (302 MB) 66 us, 4.6 TB/s; gradient of 8192 rows of 4096 (201 MB and the partial sums) 44 us
// in the row kernel and 5 us in the sums' (79 us with one round trip through LDS more per row and no row in flight).
//
// Row r has the parameters of group r % G. A row is handled by TPR threads; a thread's rows are a whole multiple of G
// apart, so its parameters, and its sums for their gradients, stay in registers over all of its rows. At the end a
// workgroup adds up its row slots of one group where G divides their number, the sums leave as partial rows, and a
// second kernel adds those in a fixed order (no atomics: the same inputs give the same bits).
#include <type_traits>

#include "kda_common.hpp"
#include "kda_layer.hpp"

namespace kda {
namespace {

constexpr int kMaxWG = 512;  // row slots of the backward's grid are at most this many workgroups (and G's multiple)

// Sums of NS values over the TPR threads of a row. Rows of several wavefronts meet in LDS, in one of two buffers in
// turn: a wavefront that is a call ahead writes the other one, and cannot be two ahead of the barrier.
template <int TPR, int NT, int NS>
__device__ __forceinline__ void row_sums(float (&x)[NS], float (*lds)[4 * (NT / 64)], int &turn) {
#pragma unroll
    for (int d = 1; d < (TPR < 64 ? TPR : 64); d <<= 1)
#pragma unroll
        for (int i = 0; i < NS; ++i) x[i] += __shfl_xor(x[i], d);
    if constexpr (TPR > 64) {
        static_assert(NS <= 4, "the buffers hold four sums");
        constexpr int NW = TPR / 64;
        const int wave = threadIdx.x >> 6, w0 = wave / NW * NW;
        float *b = lds[turn];
        turn ^= 1;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int i = 0; i < NS; ++i) b[wave * NS + i] = x[i];
        __syncthreads();
        // a lane per (wavefront, sum): NS values a wavefront, at most 64
        static_assert(NW * NS <= 64 && (NS & (NS - 1)) == 0, "one value per lane");
        const int lane = threadIdx.x & 63;
        float v = b[w0 * NS + (lane & (NW * NS - 1))];
#pragma unroll
        for (int d = NS; d < NW * NS; d <<= 1) v += __shfl_xor(v, d);
#pragma unroll
        for (int i = 0; i < NS; ++i) x[i] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), i));
    }
}

// A thread's EPT elements of a row. VEC: runs of 16 bytes, run i at 16-byte slot i * TPR + t; else element i at
// i * TPR + t (rows that are no whole number of 16-byte runs).
template <bool BF, bool VEC, int TPR, int EPT>
struct Slice {
    static constexpr int EL = BF ? 8 : 4;
    static __device__ __forceinline__ int at(int i, int t) {
        return VEC ? ((i / EL) * TPR + t) * EL + i % EL : i * TPR + t;
    }
    // as loaded: a row on its way while another is worked on
    struct Raw {
        typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
        u32x4 v[VEC ? EPT / EL : 1];
        typename IO<BF>::T e[VEC ? 1 : EPT];
    };
    static __device__ __forceinline__ void load(const void *p, int64_t row, int C, int t, Raw &x) {
        using E = typename IO<BF>::T;
        const E *r = reinterpret_cast<const E *>(p) + row * C;
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < EPT; i += EL) {
                x.v[i / EL] = typename Raw::u32x4{0, 0, 0, 0};
                if (at(i, t) < C) x.v[i / EL] = *reinterpret_cast<const typename Raw::u32x4 *>(r + at(i, t));
            }
        } else {
#pragma unroll
            for (int i = 0; i < EPT; ++i) x.e[i] = at(i, t) < C ? r[at(i, t)] : E(0);
        }
    }
    static __device__ __forceinline__ void widen(const Raw &w, float (&x)[EPT]) {
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < EPT; i += EL) {
                typename IO<BF>::T e[EL];
                __builtin_memcpy(e, &w.v[i / EL], 16);
#pragma unroll
                for (int j = 0; j < EL; ++j) x[i + j] = IO<BF>::ld(e, j);
            }
        } else {
#pragma unroll
            for (int i = 0; i < EPT; ++i) x[i] = IO<BF>::ld(w.e, i);
        }
    }
    static __device__ __forceinline__ void store(void *p, int64_t row, int C, int t, const float (&x)[EPT]) {
        using E = typename IO<BF>::T;
        E *r = reinterpret_cast<E *>(p) + row * C;
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < EPT; i += EL) {
                E e[EL];
#pragma unroll
                for (int j = 0; j < EL; ++j) IO<BF>::st(e, j, x[i + j]);
                uint4 w;
                __builtin_memcpy(&w, e, 16);
                if (at(i, t) < C) *reinterpret_cast<uint4 *>(r + at(i, t)) = w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < EPT; ++i)
                if (at(i, t) < C) IO<BF>::st(r, at(i, t), x[i]);
        }
    }
    // fp32 parameters (a row of C), or a constant where they are absent
    static __device__ __forceinline__ void param(const float *p, int64_t g, int C, int t, float absent, float (&x)[EPT]) {
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < EPT; i += 4) {
                float4 w = make_float4(absent, absent, absent, absent);
                if (p && at(i, t) < C) w = *reinterpret_cast<const float4 *>(p + g * C + at(i, t));
                x[i] = w.x; x[i + 1] = w.y; x[i + 2] = w.z; x[i + 3] = w.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < EPT; ++i) x[i] = p && at(i, t) < C ? p[g * C + at(i, t)] : absent;
        }
    }
    static __device__ __forceinline__ void store_param(float *p, int64_t row, int C, int t, const float (&x)[EPT]) {
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < EPT; i += 4)
                if (at(i, t) < C)
                    *reinterpret_cast<float4 *>(p + row * C + at(i, t)) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < EPT; ++i)
                if (at(i, t) < C) p[row * C + at(i, t)] = x[i];
        }
    }
};

// The same elements out of a checkpoint in 8 bits: a code's step is that of its 128 channels, and the value it stands
// for is of the I/O type. A row of 4096 bf16 values is 4 KB for 8; what the gradient moves goes from 201 to 169 MB for
// 8192 rows (45 us, 3.8 TB/s: as with the values themselves, the rows' rounds of sums bound it).
template <bool BF, bool VEC, int TPR, int EPT>
struct Codes {
    static constexpr int EL = BF ? 8 : 4, NR = VEC ? EPT / EL : EPT;
    struct Raw {
        int8_t e[NR][VEC ? EL : 1];
        float step[NR];
    };
    static __device__ __forceinline__ int at(int i, int t) { return Slice<BF, VEC, TPR, EPT>::at(i, t); }
    static __device__ __forceinline__ void load(const int8_t *codes, const float *scales, int64_t row, int C, int t, Raw &x) {
        const int8_t *r = codes + row * C;
        const float *s = scales + row * ((C + kCkptBlock - 1) / kCkptBlock);
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int c = at(VEC ? i * EL : i, t);
            const bool in = c < C;
            if constexpr (VEC) {
                using W = typename std::conditional<BF, uint2, uint32_t>::type;
                W w{};
                if (in) w = *reinterpret_cast<const W *>(r + c);
                __builtin_memcpy(x.e[i], &w, EL);
            } else {
                x.e[i][0] = in ? r[c] : int8_t(0);
            }
            x.step[i] = in ? s[c / kCkptBlock] : 0.f;
        }
    }
    static __device__ __forceinline__ void widen(const Raw &w, float (&x)[EPT]) {
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            const int r = VEC ? i / EL : i;
            x[i] = (float)w.e[r][VEC ? i % EL : 0] * w.step[r];
        }
        if constexpr (BF)
#pragma unroll
            for (int i = 0; i < EPT; i += 2) {
                const uint32_t p = pack_bf16(x[i], x[i + 1]);
                x[i] = bf_lo(p);
                x[i + 1] = bf_hi(p);
            }
    }
};

// A workgroup of 1024 threads with 16 elements each has no registers for a second row: no row in flight, one more round.
template <int NT, int EPT>
constexpr bool piped = NT * EPT < 1024 * 16;

// A row's reductions go in two rounds, and the second shares one with the next row's first (its values are in flight
// meanwhile and arrive by then): the sum for the mean, then everything that needs it. d = e w does not depend on the
// statistics and n = (x - mean) r only through r, so mean(d n) = r mean(d (x - mean)) needs no round of its own.
template <bool BF, bool VEC, int TPR, int NT, int EPT, bool GATE>
__global__ __launch_bounds__(NT) void kda_norm_fwd_kernel(const void *__restrict__ xp, const void *__restrict__ zp,
                                                          const float *__restrict__ wp, const float *__restrict__ bp,
                                                          void *__restrict__ yp, int64_t rows, int G, int C, float eps,
                                                          int center) {
    using SL = Slice<BF, VEC, TPR, EPT>;
    constexpr int RPW = NT / TPR;
    __shared__ float lds[2][4 * (NT / 64)];
    int turn = 0;
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const int64_t slot = (int64_t)blockIdx.x * RPW + sub, slots = (int64_t)gridDim.x * RPW;
    const float inv = 1.f / (float)C;
    float w[EPT], b[EPT];
    SL::param(wp, slot % G, C, t, 1.f, w);
    SL::param(bp, slot % G, C, t, 0.f, b);
    const int64_t turns = (rows + slots - 1) / slots;  // the same for all threads: the sums hold barriers
    auto row_of = [&](int64_t i) { const int64_t r = i * slots + slot; return r < rows ? r : rows - 1; };
    constexpr bool PIPE = piped<NT, EPT>;
    typename SL::Raw rx, rz;
    float x[EPT], z[EPT], mean[1];
    auto first_round = [&](int64_t i) __attribute__((always_inline)) {
        SL::load(xp, row_of(i), C, t, rx);
        if (GATE) SL::load(zp, row_of(i), C, t, rz);
        SL::widen(rx, x);
        if (GATE) SL::widen(rz, z);
        mean[0] = 0.f;
        if (!center) return;
#pragma unroll
        for (int e = 0; e < EPT; ++e) mean[0] += x[e];  // elements past the row are 0
        row_sums<TPR, NT>(mean, lds, turn);
    };
    first_round(0);
    for (int64_t i = 0; i < turns; ++i) {
        const bool next = PIPE && i + 1 < turns;
        if (!PIPE && i > 0) first_round(i);
        if (next) {
            SL::load(xp, row_of(i + 1), C, t, rx);
            if (GATE) SL::load(zp, row_of(i + 1), C, t, rz);
        }
        const float mu = mean[0] * inv;
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < EPT; ++e) {
            x[e] = SL::at(e, t) < C ? x[e] - mu : 0.f;
            s[0] = fmaf(x[e], x[e], s[0]);
        }
        float nx[EPT];
        if (next) {
            SL::widen(rx, nx);
            if (center)
#pragma unroll
                for (int e = 0; e < EPT; ++e) s[1] += nx[e];
        }
        row_sums<TPR, NT>(s, lds, turn);
        const float r = rsqrtf(s[0] * inv + eps);
#pragma unroll
        for (int e = 0; e < EPT; ++e) {
            x[e] = fmaf(x[e] * r, w[e], b[e]);
            if (GATE) x[e] *= sigmoid_f(z[e]);
        }
        if (i * slots + slot < rows) SL::store(yp, i * slots + slot, C, t, x);
        if (next) {
            mean[0] = s[1];
#pragma unroll
            for (int e = 0; e < EPT; ++e) x[e] = nx[e];
            if (GATE) SL::widen(rz, z);
        }
    }
}

// Partial rows that a workgroup of rpw row slots leaves: one per group where that is possible.
__host__ __device__ constexpr int parts_of(int rpw, int G) { return rpw % G == 0 ? G : rpw; }

// part: [2][partial rows][C] fp32, the sums of e n and of e over the rows of each
template <bool BF, bool VEC, int TPR, int NT, int EPT, bool GATE, bool Q8>
__global__ __launch_bounds__(NT, NT == 256 || (NT == 512 && GATE) ? 1 : 4) void kda_norm_bwd_kernel(const void *__restrict__ dyp, const void *__restrict__ xp,
                                                          const float *__restrict__ scales,
                                                          const void *__restrict__ zp, const float *__restrict__ wp,
                                                          const float *__restrict__ bp, void *__restrict__ dxp,
                                                          void *__restrict__ dzp, float *__restrict__ part,
                                                          int want_dw, int want_db, int64_t rows, int G, int C,
                                                          float eps, int center) {
    using SL = Slice<BF, VEC, TPR, EPT>;
    using SX = typename std::conditional<Q8, Codes<BF, VEC, TPR, EPT>, SL>::type;
    constexpr int RPW = NT / TPR;
    __shared__ float lds[2][4 * (NT / 64)];
    int turn = 0;
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const int64_t slot = (int64_t)blockIdx.x * RPW + sub, slots = (int64_t)gridDim.x * RPW;
    const float inv = 1.f / (float)C;
    // the parameters' sums: registers, or LDS where 1024 threads of 16 elements leave none
    constexpr bool LACC = !piped<NT, EPT>;
    __shared__ float s_acc[LACC ? 2 * EPT : 1][LACC ? NT : 1];
    float w[EPT], dw[EPT], db[EPT];
    SL::param(wp, slot % G, C, t, 1.f, w);
#pragma unroll
    for (int e = 0; e < EPT; ++e) {
        dw[e] = db[e] = 0.f;
        if constexpr (LACC) s_acc[e][threadIdx.x] = s_acc[EPT + e][threadIdx.x] = 0.f;
    }
    const int64_t turns = (rows + slots - 1) / slots;
    auto row_of = [&](int64_t i) { const int64_t r = i * slots + slot; return r < rows ? r : rows - 1; };
    constexpr bool PIPE = piped<NT, EPT>;
    typename SX::Raw rx;
    typename SL::Raw rd, rz;
    float x[EPT], mean[1];
    auto load_x = [&](int64_t row) __attribute__((always_inline)) {
        if constexpr (Q8) SX::load(reinterpret_cast<const int8_t *>(xp), scales, row, C, t, rx);
        else SL::load(xp, row, C, t, rx);
    };
    auto first_round = [&](int64_t i) __attribute__((always_inline)) {
        load_x(row_of(i));
        SL::load(dyp, row_of(i), C, t, rd);
        if (GATE) SL::load(zp, row_of(i), C, t, rz);
        SX::widen(rx, x);
        mean[0] = 0.f;
        if (!center) return;
#pragma unroll
        for (int e = 0; e < EPT; ++e) mean[0] += x[e];
        row_sums<TPR, NT>(mean, lds, turn);
    };
    first_round(0);
    for (int64_t i = 0; i < turns; ++i) {
        const bool mine = i * slots + slot < rows, next = PIPE && i + 1 < turns;
        if (!PIPE) {  // the parameters come anew, too
            if (i > 0) first_round(i);
            SL::param(wp, slot % G, C, t, 1.f, w);
        }
        float d[EPT], a[EPT];
        SL::widen(rd, d);
        if (GATE) SL::widen(rz, a);
        if (next) {
            load_x(row_of(i + 1));
            SL::load(dyp, row_of(i + 1), C, t, rd);
            if (GATE) SL::load(zp, row_of(i + 1), C, t, rz);
        }
        const float mu = mean[0] * inv;
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int e = 0; e < EPT; ++e) {
            x[e] = SL::at(e, t) < C ? x[e] - mu : 0.f;
            const float g = GATE ? sigmoid_f(a[e]) : 1.f;
            a[e] = d[e] * (1.f - g);  // what dz has beside y g
            d[e] *= g;
            const float dn = d[e] * w[e];
            s[0] = fmaf(x[e], x[e], s[0]);
            s[1] = fmaf(dn, x[e], s[1]);
            s[2] += dn;
            if (GATE) a[e] *= g;
        }
        float nx[EPT];
        if (next) {
            SX::widen(rx, nx);
            if (center)
#pragma unroll
                for (int e = 0; e < EPT; ++e) s[3] += nx[e];
        }
        row_sums<TPR, NT>(s, lds, turn);
        const float r = rsqrtf(s[0] * inv + eps);
        const float m1 = r * s[1] * inv, m2 = center ? s[2] * inv : 0.f;
#pragma unroll
        for (int e = 0; e < EPT; ++e) {
            x[e] *= r;  // n
            if (mine) {
                if constexpr (LACC) {
                    s_acc[e][threadIdx.x] = fmaf(d[e], x[e], s_acc[e][threadIdx.x]);
                    s_acc[EPT + e][threadIdx.x] += d[e];
                } else {
                    dw[e] = fmaf(d[e], x[e], dw[e]);
                    db[e] += d[e];
                }
            }
            d[e] = r * (d[e] * w[e] - fmaf(x[e], m1, m2));
        }
        if (mine) {
            SL::store(dxp, i * slots + slot, C, t, d);
            if (GATE) {
                float bb[EPT];
                SL::param(bp, slot % G, C, t, 0.f, bb);
#pragma unroll
                for (int e = 0; e < EPT; ++e) a[e] *= fmaf(x[e], w[e], bb[e]);
                SL::store(dzp, i * slots + slot, C, t, a);
            }
        }
        if (next) {
            mean[0] = s[3];
#pragma unroll
            for (int e = 0; e < EPT; ++e) x[e] = nx[e];
        }
    }
    if constexpr (LACC)
#pragma unroll
        for (int e = 0; e < EPT; ++e) {
            dw[e] = s_acc[e][threadIdx.x];
            db[e] = s_acc[EPT + e][threadIdx.x];
        }
    const int per = parts_of(RPW, G);
    if constexpr (RPW > 1) {
        __shared__ float s_sum[RPW][EPT][TPR];
        if (per < RPW) {  // uniform: slots sub, sub + G, ... of the workgroup are of one group
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                if (p == 1) __syncthreads();
#pragma unroll
                for (int e = 0; e < EPT; ++e) s_sum[sub][e][t] = p ? db[e] : dw[e];
                __syncthreads();
                if (sub < per)
                    for (int j = sub + per; j < RPW; j += per)
#pragma unroll
                        for (int e = 0; e < EPT; ++e) (p ? db : dw)[e] += s_sum[j][e][t];
            }
        }
    }
    if (sub >= per) return;
    const int64_t row = (int64_t)blockIdx.x * per + sub, all = (int64_t)gridDim.x * per;
    if (want_dw) SL::store_param(part, row, C, t, dw);
    if (want_db) SL::store_param(part + all * C, row, C, t, db);
}

// dw[g][c], db[g][c] = sum over the partial rows s with s % G == g, in order: 16 wavefronts take every 16th of them,
// 8 loads at a time, then one adds the wavefronts.
__global__ __launch_bounds__(1024) void kda_norm_param_kernel(const float *__restrict__ part, float *__restrict__ dw,
                                                              float *__restrict__ db, int64_t parts, int G, int C) {
    __shared__ float s[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t col = (int64_t)blockIdx.x * 64 + lane, cols = (int64_t)G * C;
    float *out = blockIdx.y ? db : dw;
    if (!out) return;  // uniform
    const float *p = part + (blockIdx.y ? parts * C : 0);
    float a = 0.f;
    if (col < cols) {
        const int64_t n = parts / G;
#pragma unroll 8
        for (int64_t i = wave; i < n; i += 16) a += p[i * cols + col];
    }
    s[wave][lane] = a;
    __syncthreads();
    if (wave == 0 && col < cols) {
#pragma unroll
        for (int w = 1; w < 16; ++w) a += s[w][lane];
        out[col] = a;
    }
}

// Row slots of a grid over `rows` rows: workgroups times rows per workgroup, a multiple of G.
int64_t grid_for(int64_t rows, int G, int rpw, int64_t most) {
    int64_t a = G, b = rpw;
    while (b) { const int64_t c = a % b; a = b; b = c; }
    const int64_t step = G / a;  // workgroups whose slots are a multiple of G
    int64_t wgs = (rows + rpw - 1) / rpw;
    if (wgs > most) wgs = most;
    wgs = (wgs + step - 1) / step * step;
    return wgs;
}

constexpr int kFwdWG = 2048;  // the same for the forward pass

template <bool BF, bool VEC, int TPR, int NT, int EPT, bool GATE>
hipError_t run_gate(const NormArgs &a, bool bwd, hipStream_t st) {
    constexpr int RPW = NT / TPR;
    if (!bwd) {
        const int64_t wgs = grid_for(a.rows, a.G, RPW, kFwdWG);
        hipLaunchKernelGGL((kda_norm_fwd_kernel<BF, VEC, TPR, NT, EPT, GATE>), dim3((uint32_t)wgs), dim3(NT), 0, st,
                           a.x, a.gate, a.weight, a.bias, a.y, a.rows, a.G, a.C, a.eps, (int)a.center);
        return hipGetLastError();
    }
    const int64_t wgs = grid_for(a.rows, a.G, RPW, kMaxWG);
    float *part = reinterpret_cast<float *>(a.workspace);
    auto bwd_kernel = a.codes ? kda_norm_bwd_kernel<BF, VEC, TPR, NT, EPT, GATE, true>
                              : kda_norm_bwd_kernel<BF, VEC, TPR, NT, EPT, GATE, false>;
    hipLaunchKernelGGL(bwd_kernel, dim3((uint32_t)wgs), dim3(NT), 0, st, a.dy, a.codes ? a.codes : a.x, a.scales, a.gate,
                       a.weight, a.bias, a.dx, a.dgate, part, (int)(a.dweight != nullptr), (int)(a.dbias != nullptr),
                       a.rows, a.G, a.C, a.eps, (int)a.center);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || (!a.dweight && !a.dbias)) return e;
    const int64_t cols = (int64_t)a.G * a.C;
    hipLaunchKernelGGL(kda_norm_param_kernel, dim3((uint32_t)((cols + 63) / 64), 2), dim3(1024), 0, st, part,
                       a.dweight, a.dbias, wgs * parts_of(RPW, a.G), a.G, a.C);
    return hipGetLastError();
}
template <bool BF, bool VEC, int TPR, int NT, int EPT>
hipError_t run_norm(const NormArgs &a, bool bwd, hipStream_t st) {
    return a.gate ? run_gate<BF, VEC, TPR, NT, EPT, true>(a, bwd, st) : run_gate<BF, VEC, TPR, NT, EPT, false>(a, bwd, st);
}

// The fewest threads that hold a row at 8 elements each (20000 rows of 513, bf16 with a gate: the gradient takes 66 us, on 256 threads a
// row 105).
template <bool BF, bool VEC>
hipError_t by_width(const NormArgs &a, bool bwd, hipStream_t st) {
    const int C = a.C;
    if (C <= 8 * 8) return run_norm<BF, VEC, 8, 256, 8>(a, bwd, st);
    if (C <= 16 * 8) return run_norm<BF, VEC, 16, 256, 8>(a, bwd, st);
    if (C <= 32 * 8) return run_norm<BF, VEC, 32, 256, 8>(a, bwd, st);
    if (C <= 64 * 8) return run_norm<BF, VEC, 64, 256, 8>(a, bwd, st);
    if (C <= 128 * 8) return run_norm<BF, VEC, 128, 256, 8>(a, bwd, st);
    if (C <= 256 * 8) return run_norm<BF, VEC, 256, 256, 8>(a, bwd, st);
    if (C <= 512 * 8) return run_norm<BF, VEC, 512, 512, 8>(a, bwd, st);
    if (C <= 1024 * 8) return run_norm<BF, VEC, 1024, 1024, 8>(a, bwd, st);
    return run_norm<BF, VEC, 1024, 1024, 16>(a, bwd, st);
}
hipError_t by_type(const NormArgs &a, bool bwd, hipStream_t st) {
    if (a.io_bf16) return a.C % 8 == 0 ? by_width<true, true>(a, bwd, st) : by_width<true, false>(a, bwd, st);
    return a.C % 4 == 0 ? by_width<false, true>(a, bwd, st) : by_width<false, false>(a, bwd, st);
}

}  // namespace

static int rows_per_wg(int32_t C) {  // NT / TPR of by_width
    return C <= 64 ? 32 : C <= 128 ? 16 : C <= 256 ? 8 : C <= 512 ? 4 : C <= 1024 ? 2 : 1;
}
bool norm_grid_fits(int64_t rows, int32_t G, int32_t C) {
    const int64_t threads = C <= 2048 ? 256 : C <= 4096 ? 512 : 1024;  // NT of by_width
    return grid_for(rows, G, rows_per_wg(C), kFwdWG) * threads < (int64_t)1 << 32;
}
size_t norm_bwd_workspace_bytes(int64_t rows, int32_t G, int32_t C) {
    const int rpw = rows_per_wg(C);
    return (size_t)(grid_for(rows, G, rpw, kMaxWG) * parts_of(rpw, G)) * C * 2 * sizeof(float);
}
hipError_t launch_norm_fwd(const NormArgs &a, hipStream_t st) {
    return a.rows == 0 ? hipSuccess : by_type(a, false, st);
}
hipError_t launch_norm_bwd(const NormArgs &a, hipStream_t st) {
    if (a.rows == 0) {  // no rows: the parameters' gradients are zero
        const int64_t cols = (int64_t)a.G * a.C;
        if (!a.dweight && !a.dbias) return hipSuccess;
        hipLaunchKernelGGL(kda_norm_param_kernel, dim3((uint32_t)((cols + 63) / 64), 2), dim3(1024), 0, st, nullptr,
                           a.dweight, a.dbias, (int64_t)0, a.G, a.C);
        return hipGetLastError();
    }
    return by_type(a, true, st);
}

}  // namespace kda
