// One decode step of linear attention with one decay per head, for gfx950:
//   S <- e^g S + k v^T,   o = scale * S^T q,
// one token per sequence, S [K, V] fp32 per (sequence, head) updated in place. The step is one read and one write of
// S; the read-out uses the updated rows while they are in registers, so S makes one round trip through HBM.
#include "kda_common.hpp"
#include "kda_layer.hpp"

namespace kda {
namespace {

// A workgroup takes one (sequence, head, tile of W value columns). Thread t owns the float4 column group t % (W/4) of
// the RPT consecutive key rows from RPT * (t / (W/4)) on: its q and k are one short run each, and a wavefront's
// accesses to S are whole row pieces of 4W bytes.
template <bool BF, int K, int W, int NT>
__global__ __launch_bounds__(NT) void kda_hd_decode_kernel(const void *__restrict__ qp, const void *__restrict__ kp,
                                                           const void *__restrict__ vp, const void *__restrict__ gp,
                                                           float *__restrict__ S, void *__restrict__ op, int H,
                                                           int group, int V, int decay_per_head, float scale) {
    constexpr int CG = W / 4, RG = NT / CG, RPT = K / RG, NW = NT / 64;
    static_assert(RPT >= 1 && RG * RPT == K && NT % 64 == 0, "unsupported K, W");
    using E = typename IO<BF>::T;
    __shared__ f32x4 s_part[NW][CG];
    const int t = threadIdx.x, cg = t % CG, rg = t / CG, lane = t & 63, wave = t >> 6;
    const int tiles = V / W;
    const int64_t nh = blockIdx.x / tiles;
    const int c0 = (int)(blockIdx.x % tiles) * W + 4 * cg;
    const int64_t n = nh / H;
    const int h = (int)(nh - n * H);
    const int64_t nk = n * (H / group) + h / group;
    float *Sp = S + (nh * K + (int64_t)rg * RPT) * V + c0;
    f32x4 s[RPT];
#pragma unroll
    for (int j = 0; j < RPT; ++j) s[j] = __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(Sp + j * V));
    const E *q = reinterpret_cast<const E *>(qp) + nk * K + rg * RPT;
    const E *k = reinterpret_cast<const E *>(kp) + nk * K + rg * RPT;
    const E *v = reinterpret_cast<const E *>(vp) + nh * V + c0;
    float qr[RPT], kr[RPT], vv[4];
#pragma unroll
    for (int j = 0; j < RPT; ++j) {
        qr[j] = IO<BF>::ld(q, j);
        kr[j] = IO<BF>::ld(k, j);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) vv[j] = IO<BF>::ld(v, j);
    const float g = decay_per_head ? reinterpret_cast<const float *>(gp)[h]
                                   : IO<BF>::ld(reinterpret_cast<const E *>(gp), nh);
    const float a = __builtin_amdgcn_exp2f(g * 1.4426950408889634f);
    f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < RPT; ++j) {
        s[j].x = fmaf(s[j].x, a, kr[j] * vv[0]);
        s[j].y = fmaf(s[j].y, a, kr[j] * vv[1]);
        s[j].z = fmaf(s[j].z, a, kr[j] * vv[2]);
        s[j].w = fmaf(s[j].w, a, kr[j] * vv[3]);
        __builtin_nontemporal_store(s[j], reinterpret_cast<f32x4 *>(Sp + j * V));
        y.x = fmaf(s[j].x, qr[j], y.x);
        y.y = fmaf(s[j].y, qr[j], y.y);
        y.z = fmaf(s[j].z, qr[j], y.z);
        y.w = fmaf(s[j].w, qr[j], y.w);
    }
#pragma unroll
    for (int d = CG; d < 64; d <<= 1) {  // row groups of a wavefront
        y.x += __shfl_xor(y.x, d);
        y.y += __shfl_xor(y.y, d);
        y.z += __shfl_xor(y.z, d);
        y.w += __shfl_xor(y.w, d);
    }
    if (NW > 1) {
        if (lane < CG) s_part[wave][cg] = y;
        __syncthreads();
    }
    if (t < CG) {
#pragma unroll
        for (int w = 1; w < NW; ++w) y += s_part[w][t];
        const int64_t ob = nh * V + c0;
        if constexpr (BF)
            *reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(op) + ob) =
                make_uint2(pack_bf16(scale * y.x, scale * y.y), pack_bf16(scale * y.z, scale * y.w));
        else
            *reinterpret_cast<float4 *>(reinterpret_cast<float *>(op) + ob) =
                make_float4(scale * y.x, scale * y.y, scale * y.z, scale * y.w);
    }
}

template <bool BF, int K, int W>
hipError_t launch_kw(const HdDecodeArgs &a, hipStream_t st) {
    constexpr int NT = K * W / 4 < 512 ? K * W / 4 : 512;
    const uint32_t grid = (uint32_t)((int64_t)a.N * a.H * (a.V / W));
    hipLaunchKernelGGL((kda_hd_decode_kernel<BF, K, W, NT>), dim3(grid), dim3(NT), 0, st, a.q, a.k, a.v, a.g, a.S, a.o,
                       a.H, a.H / a.Hk, a.V, (int)a.decay_per_head, a.scale);
    return hipGetLastError();
}
template <bool BF, int K>
hipError_t launch_k(const HdDecodeArgs &a, hipStream_t st) {
    switch (a.V) {
        case 32: return launch_kw<BF, K, 32>(a, st);
        case 64: return launch_kw<BF, K, 64>(a, st);
        default: return launch_kw<BF, K, 128>(a, st);
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
