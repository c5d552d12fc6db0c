// Rotary positions: channel pairs (x1, x2) of every head turn by the angle pos * freq,
//   y1 = (x1 cos - x2 sin) * scale,  y2 = (x1 sin + x2 cos) * scale,
// the first R of a head's D channels in pairs (j, j + R/2) ("half") or (2j, 2j + 1) ("interleaved"); the rest are
// copied. The gradient is the same rotation backwards (inverse).
//
// Angles. A product pos * freq in fp32 is off by 2^-24 of itself, 0.03 radians at position 2^20. Here a frequency
// becomes the fraction of a turn it advances per position as a 64-bit fixed-point number, and the product with the
// position wraps modulo one turn in integer arithmetic: exact range reduction at any 32-bit position, the error is
// that of the fp64 frequency. The top bits name the nearest quarter turn, the remainder in [-1/8, 1/8] turn goes to
// fp32 and through the Taylor series of sine (to x^11) and cosine (to x^10); the next terms are below 2e-10 at pi/4.
//
// The kernel only moves bytes: one read and one write of q and k. A thread owns a run of pairs (two 16-byte vectors)
// of one token and walks over the heads, so the sines are formed once per thread and not per head, and holds the next
// row in flight while it turns one. 16382 tokens of 64 heads of 128 channels, bf16 (537 MB): 107 us, 5.0 TB/s, where a
// plain copy of that size reaches 5.2; without the row in flight 124 us, with two heads' rows at a time 134 us.
#include "kda_common.hpp"
#include "kda_layer.hpp"

namespace kda {
namespace {

__device__ __forceinline__ uint64_t turn_fraction(double freq) {  // of a finite frequency
    double t = freq * 0.15915494309189535;  // 1 / (2 pi)
    t -= floor(t);
    return t >= 1.0 || !(t >= 0.0) ? 0ull : (uint64_t)(t * 18446744073709551616.0);
}

// sin and cos of 2 pi (turn / 2^64)
__device__ __forceinline__ void sincos_turn(uint64_t turn, float &s, float &c) {
    const uint32_t top = (uint32_t)(turn >> 32);
    const uint32_t quad = (top + 0x20000000u) >> 30;          // nearest quarter turn
    const int32_t rem = (int32_t)(top - (quad << 30));        // [-2^29, 2^29): an eighth of a turn either way
    const float x = (float)rem * 1.4629180792671596e-9f;      // 2 pi / 2^32
    const float x2 = x * x;
    float ps = -2.5052108385441720e-8f;
    ps = fmaf(ps, x2, 2.7557319223985893e-6f);
    ps = fmaf(ps, x2, -1.9841269841269841e-4f);
    ps = fmaf(ps, x2, 8.3333333333333333e-3f);
    ps = fmaf(ps, x2, -1.6666666666666667e-1f);
    ps = fmaf(ps * x2, x, x);
    float pc = -2.7557319223985888e-7f;
    pc = fmaf(pc, x2, 2.4801587301587302e-5f);
    pc = fmaf(pc, x2, -1.3888888888888889e-3f);
    pc = fmaf(pc, x2, 4.1666666666666664e-2f);
    pc = fmaf(pc, x2, -0.5f);
    pc = fmaf(pc, x2, 1.0f);
    s = (quad & 1) ? pc : ps;
    c = (quad & 1) ? ps : pc;
    if (quad & 2) s = -s;
    if ((quad + 1) & 2) c = -c;
}

// A run of E elements (a vector of E * element bytes, at most 16, which p is aligned to) as fp32 and back.
template <int BYTES> struct Words;
template <> struct Words<2> { using T = uint16_t; };
template <> struct Words<4> { using T = uint32_t; };
template <> struct Words<8> { using T = uint2; };
template <> struct Words<16> { using T = uint4; };
template <bool BF, int E>
__device__ __forceinline__ void load_run(const void *p, float (&x)[E]) {
    using W = typename Words<E * (BF ? 2 : 4)>::T;
    typename IO<BF>::T e[E];
    const W w = *reinterpret_cast<const W *>(p);
    __builtin_memcpy(e, &w, sizeof(w));
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = IO<BF>::ld(e, i);
}
template <bool BF, int E>
__device__ __forceinline__ void store_run(void *p, const float (&x)[E]) {
    using W = typename Words<E * (BF ? 2 : 4)>::T;
    typename IO<BF>::T e[E];
#pragma unroll
    for (int i = 0; i < E; ++i) IO<BF>::st(e, i, x[i]);
    W w;
    __builtin_memcpy(&w, e, sizeof(w));
    *reinterpret_cast<W *>(p) = w;
}

// E pairs of a unit: (x[i], y[i]), or adjacent channels of x followed by y. The first n turn; the others (adjacent channels
// alone have any) are copied and not turned by nothing: a channel is to keep its bits whatever its neighbour holds.
template <int E, bool INTER>
__device__ __forceinline__ void turn_run(float (&x)[E], float (&y)[E], const float (&cs)[E], const float (&sn)[E], int n) {
    auto turn = [&](float &a, float &b, int i) __attribute__((always_inline)) {
        const float r = a * cs[i] - b * sn[i], q = a * sn[i] + b * cs[i];
        a = !INTER || i < n ? r : a;
        b = !INTER || i < n ? q : b;
    };
    if constexpr (!INTER || E == 1) {
#pragma unroll
        for (int i = 0; i < E; ++i) turn(x[i], y[i], i);
    } else {
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            turn(x[2 * i], x[2 * i + 1], i);
            turn(y[2 * i], y[2 * i + 1], E / 2 + i);
        }
    }
}

// A unit is a run of E pairs or, behind them, a run of 2E copied channels; an interleaved unit that straddles R copies
// its pairs from R on. Threads of a workgroup: `units` consecutive ones per head, heads_par heads at a
// time, tok_par tokens at a time. q_out and k_out may be q and k: a thread reads its channels before it writes them.
// AXES: pair j turns by the position of axis axes[j], positions are [naxes, tokens].
template <bool BF, int E, bool INTER, bool AXES>
__global__ __launch_bounds__(256) void kda_rotary_kernel(const void *qp, const void *kp, void *qo, void *ko,
                                                         const double *__restrict__ freqs,
                                                         const int32_t *__restrict__ positions,
                                                         const int32_t *__restrict__ axes, int naxes, int64_t tokens,
                                                         int64_t T, int Hq, int Hk, int D, int R, int units,
                                                         int heads_par, int tok_par, float sgn, float scale) {
    constexpr int ES = BF ? 2 : 4;
    const int per_tok = units * heads_par;
    const int tsub = threadIdx.x / per_tok;
    if (tsub >= tok_par) return;
    const int in_tok = threadIdx.x - tsub * per_tok;
    const int hsub = in_tok / units, u = in_tok - hsub * units;
    const int np = (R / 2 + E - 1) / E;  // units with pairs to turn
    const bool pairs = u < np;
    uint64_t fr[E];
    uint32_t undefined = 0;  // pairs whose frequency is infinite or NaN: their angles are NaN at any position
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const double f = pairs && u * E + i < R / 2 ? freqs[u * E + i] : 0.0;
        fr[i] = turn_fraction(f);
        undefined |= (uint32_t)!(fabs(f) < HUGE_VAL) << i;
    }
    int64_t line[AXES ? E : 1];  // where the positions of a pair's axis begin
    if constexpr (AXES) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int a = pairs && u * E + i < R / 2 ? axes[u * E + i] : 0;
            const bool known = a >= 0 && a < naxes;
            undefined |= (uint32_t)!known << i;
            line[i] = known ? a * tokens : 0;
        }
    }
    // the two runs of a unit: (x1 run, x2 run) of "half", 2E adjacent channels otherwise
    const int c0 = INTER ? 2 * E * u : pairs ? E * u : R + 2 * E * (u - np);
    const int c1 = pairs && !INTER ? c0 + R / 2 : c0 + E;
    const bool two = c1 + E <= D;  // a last copied run may be half as long
    // A row (token, head) in flight: the next one's loads go out before this one is turned.
    struct Row {
        float x[E], y[E];
        char *d;
        bool live;
    };
    auto take = [&](int64_t t, int h, Row &r) __attribute__((always_inline)) {
        const bool isq = h < Hq;
        const char *src = isq ? (const char *)qp : (const char *)kp;
        char *dst = isq ? (char *)qo : (char *)ko;
        const int64_t row = (isq ? t * Hq + h : t * Hk + (h - Hq)) * D * ES;
        r.d = dst + row;
        r.live = t < tokens && (pairs || src != dst);  // in place there is nothing to copy
        if (!r.live) return;
        load_run<BF, E>(src + row + c0 * ES, r.x);
        if (two) load_run<BF, E>(src + row + c1 * ES, r.y);
    };
    const int64_t step = (int64_t)gridDim.x * tok_par;
    Row r = {};
    int64_t t = (int64_t)blockIdx.x * tok_par + tsub;
    take(t, hsub, r);
    int32_t at[AXES ? E : 1] = {};  // the token's positions, asked for while the one before it is turned
    auto positions_of = [&](int64_t t) __attribute__((always_inline)) {
        if (AXES && pairs && t < tokens)
#pragma unroll
            for (int i = 0; i < (AXES ? E : 1); ++i) at[i] = positions[line[i] + t];
    };
    positions_of(t);
    for (; t < tokens; t += step) {
        float cs[E], sn[E];
        if (pairs) {
            int64_t pos = 0;
            if constexpr (!AXES) {
                pos = positions ? (int64_t)positions[t]
                    : tokens <= 0xffffffffll ? (int64_t)((uint32_t)t % (uint32_t)T) : t % T;
            }
#pragma unroll
            for (int i = 0; i < E; ++i) {
                if constexpr (AXES) pos = at[i];
                sincos_turn(fr[i] * (uint64_t)pos, sn[i], cs[i]);
                sn[i] *= sgn * scale;
                cs[i] *= scale;
                if (undefined >> i & 1) sn[i] = cs[i] = __builtin_nanf("");
            }
        }
        positions_of(t + step);
        for (int h = hsub; h < Hq + Hk; h += heads_par) {
            Row next = {};
            const bool more = h + heads_par < Hq + Hk;
            take(more ? t : t + step, more ? h + heads_par : hsub, next);
            if (r.live) {
                if (pairs) turn_run<E, INTER>(r.x, r.y, cs, sn, R / 2 - u * E);
                store_run<BF, E>(r.d + c0 * ES, r.x);
                if (two) store_run<BF, E>(r.d + c1 * ES, r.y);
            }
            r = next;
        }
    }
}

template <bool BF, int E, bool INTER, bool AXES>
hipError_t launch_i(const RotaryArgs &a, hipStream_t st) {
    const int units = INTER ? (a.D + 2 * E - 1) / (2 * E) : a.R / (2 * E) + (a.D - a.R + 2 * E - 1) / (2 * E);
    const int H = a.Hq + a.Hk;
    int heads_par = 256 / units;  // D <= 512: at most 256 units
    if (heads_par > H) heads_par = H;
    if (heads_par < 1) heads_par = 1;
    // With axes of their own a thread's angles cost as much as the rows that it turns by them: where 1024 workgroups are left,
    // a thread turns several heads of a token (2 x 8191 tokens of 40 heads of 128 channels: 97 us with 32 heads side by side,
    // 77 with 8, 72 with 4: 4.7 TB/s).
    if (AXES)
        while (heads_par > 4 && a.tokens * units * (heads_par / 2) >= 256 * 1024) heads_par /= 2;
    int tok_par = 256 / (units * heads_par);
    if (tok_par < 1) tok_par = 1;
    int64_t wgs = (a.tokens + tok_par - 1) / tok_par;
    if (wgs > 4096) wgs = 4096;  // a thread's frequencies serve several tokens
    const float sgn = a.inverse ? -1.f : 1.f;
    hipLaunchKernelGGL((kda_rotary_kernel<BF, E, INTER, AXES>), dim3((uint32_t)wgs), dim3(256), 0, st, a.q, a.k, a.q_out,
                       a.k_out, a.freqs, a.positions, a.axes, a.naxes, a.tokens, a.T, a.Hq, a.Hk, a.D, a.R, units,
                       heads_par, tok_par, sgn, a.scale);
    return hipGetLastError();
}
template <bool BF, int E>
hipError_t launch_e(const RotaryArgs &a, hipStream_t st) {
    if (a.axes) return a.interleaved ? launch_i<BF, E, true, true>(a, st) : launch_i<BF, E, false, true>(a, st);
    return a.interleaved ? launch_i<BF, E, true, false>(a, st) : launch_i<BF, E, false, false>(a, st);
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs &a, hipStream_t st) {
    if (a.tokens == 0) return hipSuccess;
    // The widest runs (at most 16 bytes) that every run of a head starts on a multiple of: a head is a whole number
    // of runs, and with the pairs' halves apart each half is.
    const int64_t m = a.interleaved ? a.D : (int64_t)a.D | (a.R / 2);
    if (a.io_bf16) {
        if (m % 8 == 0) return launch_e<true, 8>(a, st);
        if (m % 4 == 0) return launch_e<true, 4>(a, st);
        return m % 2 == 0 ? launch_e<true, 2>(a, st) : launch_e<true, 1>(a, st);
    }
    if (m % 4 == 0) return launch_e<false, 4>(a, st);
    return m % 2 == 0 ? launch_e<false, 2>(a, st) : launch_e<false, 1>(a, st);
}

}  // namespace kda
