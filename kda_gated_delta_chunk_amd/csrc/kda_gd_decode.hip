// One decode step of the gated delta rule with one decay per head, for gfx950:
//   S <- e^g S;  w = beta (v - S^T k);  S <- S + k w^T;  o = scale * S^T q,
// one token per sequence, S [K, V] fp32 per (sequence, head) updated in place. One read and one write of S: both
// products with the decayed state are formed while it is in registers, S_new^T q = (e^g S)^T q + (k.q) w.
#include "kda_common.hpp"
#include "kda_gd.hpp"

namespace kda {
namespace {

// e^g of a log-decay: the rounding of g log2(e) is made up for (2^-24 of the exponent is 6e-7 of the result at g = -10).
__device__ __forceinline__ float exp_decay(float g) {
    const float x = g * 1.4426950408889634f;
    const float rest = fmaf(g, 1.4426950408889634f, -x) + g * 1.9259629911266175e-8f;
    const float e = __builtin_amdgcn_exp2f(x);
    return x < -150.f ? e : fmaf(e, rest * 0.6931471805599453f, e);  // -inf: 0, and no inf - inf in the rest
}

// A workgroup of NT threads walks the (sequence, head) pairs blockIdx.x, blockIdx.x + gridDim.x, ...; while it updates
// one it holds the next one's state and vectors in flight. Thread t owns the float4 column group t % (V/4) of every
// (4 NT / V)-th key row, so each load and store of the workgroup is one contiguous run of S (16 KB with 1024 threads).
// HBM bounds it: 512 streams of 96 heads of 128 x 128 move 6.5 GB in 1091 us, 5.95 TB/s (a copy: 4.9 to 5.3).
template <bool BF, bool GF, int K, int V, int NT>
__global__ __launch_bounds__(NT) void kda_gd_decode_kernel(const void *__restrict__ qp, const void *__restrict__ kp,
                                                           const void *__restrict__ vp, const void *__restrict__ gp,
                                                           const void *__restrict__ bp, float *__restrict__ S,
                                                           void *__restrict__ op, int H, int group, float scale,
                                                           int32_t NH) {
    constexpr int CG = V / 4, RG = NT / CG, RPT = K / RG, NW = NT / 64;
    static_assert(RPT >= 1 && RG * RPT == K && NT % 64 == 0 && NW > 1 && NT >= K, "unsupported K, V");
    using E = typename IO<BF>::T;
    using GE = typename IO<!GF>::T;
    __shared__ f32x4 s_u[NW][CG], s_y[NW][CG], s_w[CG];
    __shared__ float s_q[2][K], s_k[2][K], s_kq[NW];
    const int t = threadIdx.x, cg = t % CG, rg = t / CG, lane = t & 63, wave = t >> 6;
    struct Pair {
        f32x4 s[RPT];
        float q, k, v[4], g, b;
    };
    auto take = [&](int32_t nh, Pair &x) __attribute__((always_inline)) {
        const float *Sp = S + ((int64_t)nh * K + rg) * V + 4 * cg;
#pragma unroll
        for (int j = 0; j < RPT; ++j) x.s[j] = __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(Sp + RG * j * V));
        const int32_t n = nh / H, h = nh - n * H;
        const int64_t nk = (int64_t)n * (H / group) + h / group;
        if (t < K) {
            x.q = IO<BF>::ld(reinterpret_cast<const E *>(qp) + nk * K, t);
            x.k = IO<BF>::ld(reinterpret_cast<const E *>(kp) + nk * K, t);
        }
        if (t < CG) {
#pragma unroll
            for (int j = 0; j < 4; ++j) x.v[j] = IO<BF>::ld(reinterpret_cast<const E *>(vp) + (int64_t)nh * V + 4 * t, j);
        }
        x.g = IO<!GF>::ld(reinterpret_cast<const GE *>(gp), nh);
        x.b = IO<!GF>::ld(reinterpret_cast<const GE *>(bp), nh);
    };
    int32_t nh = blockIdx.x;  // gridDim.x <= NH
    Pair x, next;
    take(nh, x);
    for (int buf = 0;; buf ^= 1) {
        const int32_t nx = nh + gridDim.x;
        if (nx < NH) take(nx, next);
        if (t < K) {
            s_q[buf][t] = x.q;
            s_k[buf][t] = x.k;
        }
        __syncthreads();
        const float a = exp_decay(x.g);
        f32x4 u = {0.f, 0.f, 0.f, 0.f}, y = {0.f, 0.f, 0.f, 0.f};
        float kq = 0.f;
#pragma unroll
        for (int j = 0; j < RPT; ++j) {
            const float kj = s_k[buf][rg + RG * j], qj = s_q[buf][rg + RG * j];
            f32x4 &s = x.s[j];
            s *= a;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                u[i] = fmaf(s[i], kj, u[i]);
                y[i] = fmaf(s[i], qj, y[i]);
            }
            kq = fmaf(kj, qj, kq);
        }
#pragma unroll
        for (int d = CG; d < 64; d <<= 1) {  // row groups of a wavefront
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                u[i] += __shfl_xor(u[i], d);
                y[i] += __shfl_xor(y[i], d);
            }
            kq += __shfl_xor(kq, d);
        }
        if (lane < CG) {
            s_u[wave][cg] = u;
            s_y[wave][cg] = y;
            if (lane == 0) s_kq[wave] = kq;
        }
        __syncthreads();
        if (t < CG) {
            u = s_u[0][t];
            y = s_y[0][t];
            kq = s_kq[0];
#pragma unroll
            for (int w = 1; w < NW; ++w) {
                u += s_u[w][t];
                y += s_y[w][t];
                kq += s_kq[w];
            }
            f32x4 w;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[i] = x.b * (x.v[i] - u[i]);
                y[i] = scale * fmaf(kq, w[i], y[i]);
            }
            s_w[t] = w;
            const int64_t ob = (int64_t)nh * V + 4 * t;
            if constexpr (BF)
                *reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(op) + ob) =
                    make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
            else
                *reinterpret_cast<f32x4 *>(reinterpret_cast<float *>(op) + ob) = y;
        }
        __syncthreads();
        const f32x4 w = s_w[cg];
        float *Sp = S + ((int64_t)nh * K + rg) * V + 4 * cg;
#pragma unroll
        for (int j = 0; j < RPT; ++j) {
            f32x4 s = x.s[j];
            const float kj = s_k[buf][rg + RG * j];
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] = fmaf(kj, w[i], s[i]);
            __builtin_nontemporal_store(s, reinterpret_cast<f32x4 *>(Sp + RG * j * V));
        }
        if (nx >= NH) break;
        nh = nx;
        x = next;
    }
}

template <bool BF, bool GF, int K, int V>
hipError_t launch_kv(const GdDecodeArgs &a, hipStream_t st) {
    constexpr int NT = K * V / 4 < 1024 ? K * V / 4 : 1024;
    const int32_t NH = a.N * a.H;
    // up to 4096 workgroups take one pair each; above that each walks about 4 pairs (more where the grid's threads would
    // pass 32 bits)
    constexpr int32_t most = 1 << 21;
    const int32_t quarter = (NH + 3) / 4;
    const int32_t grid = NH <= 4096 ? NH : quarter < 4096 ? 4096 : quarter < most ? quarter : most;
    hipLaunchKernelGGL((kda_gd_decode_kernel<BF, GF, K, V, NT>), dim3(grid), dim3(NT), 0, st, a.q, a.k, a.v, a.g, a.beta,
                       a.S, a.o, a.H, a.H / a.Hk, a.scale, NH);
    return hipGetLastError();
}
template <bool BF, bool GF, int K>
hipError_t launch_k(const GdDecodeArgs &a, hipStream_t st) {
    switch (a.V) {
        case 32: return launch_kv<BF, GF, K, 32>(a, st);
        case 64: return launch_kv<BF, GF, K, 64>(a, st);
        default: return launch_kv<BF, GF, K, 128>(a, st);
    }
}
template <bool BF, bool GF>
hipError_t launch_b(const GdDecodeArgs &a, hipStream_t st) {
    switch (a.K) {
        case 32: return launch_k<BF, GF, 32>(a, st);
        case 64: return launch_k<BF, GF, 64>(a, st);
        default: return launch_k<BF, GF, 128>(a, st);
    }
}
}  // namespace

hipError_t launch_gd_decode(const GdDecodeArgs &a, hipStream_t st) {
    if (a.N == 0) return hipSuccess;
    if (!a.io_bf16) return launch_b<false, true>(a, st);
    return a.gates_fp32 ? launch_b<true, true>(a, st) : launch_b<true, false>(a, st);
}

}  // namespace kda
