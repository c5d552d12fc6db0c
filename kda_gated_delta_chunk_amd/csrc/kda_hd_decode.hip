// One decode step of linear attention with one decay per head, for gfx950:
//   S <- e^g S + k v^T,   o = scale * S^T q,
// one token per sequence, S [K, V] fp32 per (sequence, head) updated in place. The step is one read and one write of
// S; the read-out uses the updated rows while they are in registers, so S makes one round trip through HBM.
#include "kda_common.hpp"
#include "kda_layer.hpp"

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
// (4 NT / V)-th key row, so each load and store of the workgroup is one contiguous run of S (16 KB with 1024 threads);
// q and k pass through LDS, and so do the partial read-outs of the wavefronts (two buffers). At 512 sequences x 96
// heads of 128 x 128 (3.2 GB of S) 1024 threads move 6.15 TB/s (1055 us), 512 threads 5.6, 256 threads 5.4; runs of 8
// consecutive rows a thread, without LDS, 5.4 to 5.7.
template <bool BF, int K, int V, int NT>
__global__ __launch_bounds__(NT) void kda_hd_decode_kernel(const void *__restrict__ qp, const void *__restrict__ kp,
                                                           const void *__restrict__ vp, const void *__restrict__ gp,
                                                           float *__restrict__ S, void *__restrict__ op, int H,
                                                           int group, int decay_per_head, float scale, int32_t NH) {
    constexpr int CG = V / 4, RG = NT / CG, RPT = K / RG, NW = NT / 64;
    static_assert(RPT >= 1 && RG * RPT == K && NT % 64 == 0 && NW > 1, "unsupported K, V");
    using E = typename IO<BF>::T;
    __shared__ f32x4 s_part[2][NW][CG];
    __shared__ float s_q[2][K], s_k[2][K];
    const int t = threadIdx.x, cg = t % CG, rg = t / CG, lane = t & 63, wave = t >> 6;
    struct Pair {
        f32x4 s[RPT];
        float q, k, v[4], g;
    };
    auto take = [&](int32_t nh, Pair &x) __attribute__((always_inline)) {
        const float *Sp = S + ((int64_t)nh * K + rg) * V + 4 * cg;
#pragma unroll
        for (int j = 0; j < RPT; ++j) x.s[j] = __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(Sp + RG * j * V));
        const int32_t n = nh / H, h = nh - n * H;
        const int64_t nk = (int64_t)n * (H / group) + h / group;
        const E *q = reinterpret_cast<const E *>(qp) + nk * K;
        const E *k = reinterpret_cast<const E *>(kp) + nk * K;
        const E *v = reinterpret_cast<const E *>(vp) + (int64_t)nh * V + 4 * cg;
        if (t < K) {
            x.q = IO<BF>::ld(q, t);
            x.k = IO<BF>::ld(k, t);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) x.v[j] = IO<BF>::ld(v, j);
        x.g = decay_per_head ? reinterpret_cast<const float *>(gp)[h] : IO<BF>::ld(reinterpret_cast<const E *>(gp), nh);
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
        float *Sp = S + ((int64_t)nh * K + rg) * V + 4 * cg;
        f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < RPT; ++j) {
            f32x4 s = x.s[j];
            const float kj = s_k[buf][rg + RG * j], qj = s_q[buf][rg + RG * j];
            s.x = fmaf(s.x, a, kj * x.v[0]);
            s.y = fmaf(s.y, a, kj * x.v[1]);
            s.z = fmaf(s.z, a, kj * x.v[2]);
            s.w = fmaf(s.w, a, kj * x.v[3]);
            __builtin_nontemporal_store(s, reinterpret_cast<f32x4 *>(Sp + RG * j * V));
            y.x = fmaf(s.x, qj, y.x);
            y.y = fmaf(s.y, qj, y.y);
            y.z = fmaf(s.z, qj, y.z);
            y.w = fmaf(s.w, qj, y.w);
        }
#pragma unroll
        for (int d = CG; d < 64; d <<= 1) {  // row groups of a wavefront
            y.x += __shfl_xor(y.x, d);
            y.y += __shfl_xor(y.y, d);
            y.z += __shfl_xor(y.z, d);
            y.w += __shfl_xor(y.w, d);
        }
        if (lane < CG) s_part[buf][wave][cg] = y;
        __syncthreads();
        if (t < CG) {
            y = s_part[buf][0][t];
#pragma unroll
            for (int w = 1; w < NW; ++w) y += s_part[buf][w][t];
            y *= scale;
            const int64_t ob = (int64_t)nh * V + 4 * t;
            if constexpr (BF)
                *reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(op) + ob) =
                    make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
            else
                *reinterpret_cast<f32x4 *>(reinterpret_cast<float *>(op) + ob) = y;
        }
        if (nx >= NH) break;
        nh = nx;
        x = next;
    }
}

template <bool BF, int K, int V>
hipError_t launch_kv(const HdDecodeArgs &a, hipStream_t st) {
    constexpr int NT = K * V / 4 < 1024 ? K * V / 4 : 1024;
    const int32_t NH = a.N * a.H;
    // up to 4096 workgroups take one pair each; above that each walks about 4 pairs (more where the grid's threads would
    // pass 32 bits)
    constexpr int32_t most = 1 << 21;
    const int32_t quarter = (NH + 3) / 4;
    const int32_t grid = NH <= 4096 ? NH : quarter < 4096 ? 4096 : quarter < most ? quarter : most;
    hipLaunchKernelGGL((kda_hd_decode_kernel<BF, K, V, NT>), dim3(grid), dim3(NT), 0, st, a.q, a.k, a.v, a.g, a.S, a.o,
                       a.H, a.H / a.Hk, (int)a.decay_per_head, a.scale, NH);
    return hipGetLastError();
}
template <bool BF, int K>
hipError_t launch_k(const HdDecodeArgs &a, hipStream_t st) {
    switch (a.V) {
        case 32: return launch_kv<BF, K, 32>(a, st);
        case 64: return launch_kv<BF, K, 64>(a, st);
        default: return launch_kv<BF, K, 128>(a, st);
    }
}
template <bool BF>
hipError_t launch_b(const HdDecodeArgs &a, hipStream_t st) {
    switch (a.K) {
        case 32: return launch_k<BF, 32>(a, st);
        case 64: return launch_k<BF, 64>(a, st);
        default: return launch_k<BF, 128>(a, st);
    }
}
}  // namespace

hipError_t launch_hd_decode(const HdDecodeArgs &a, hipStream_t st) {
    if (a.N == 0) return hipSuccess;
    return a.io_bf16 ? launch_b<true>(a, st) : launch_b<false>(a, st);
}

}  // namespace kda
