// Activation checkpoints in 8 bits, for gfx950: along every row 128 values share a step, their largest size's 127th part,
//   step = max |x| / 127,  code = the nearest whole number to 127 x / max |x| (ties to even),  x ~ code * step.
// A value is off by at most half a step, 2^-8 of the block's largest, before it is rounded to its type (uniform steps: for
// values of one scale the error is a quarter of what 8-bit floating point leaves). A block that holds an infinity or a NaN
// comes back as NaN.
//
// The kernels only move bytes: x once and one byte a value. A group of lanes owns a block, eight values each, so the
// largest is found across lanes and every load and store is 8 to 32 bytes wide. 8192 x 4096 values of bf16, 102 MB either
// way: saved in 22 us (4.6 TB/s), restored in 15 to 16 (6.5 TB/s, the codes from the caches).
#include "kda_common.hpp"
#include "kda_layer.hpp"

namespace kda {
namespace {

typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;

// 127 x / top to the nearest: the quotient by the reciprocal, then what it leaves of the dividend (exact) divided once
// more, which brings a quotient that is a half exactly there. The dividend is scaled so that nothing over- or underflows.
// 127 x is exact for bf16 and rounded once for fp32, where a quotient within 2^-16 of a half can go either way.
struct Quantizer {
    float top, inv, scale;
    __device__ __forceinline__ explicit Quantizer(float largest) {
        const float s = largest > 0x1p60f ? 0x1p-80f : largest < 0x1p-60f ? 0x1p80f : 1.f;
        top = largest * s;
        inv = 1.f / top;
        scale = 127.f * s;
    }
    __device__ __forceinline__ int code(float x) const {
        const float n = x * scale, q = n * inv;
        return (int)rintf(fmaf(fmaf(-q, top, n), inv, q));
    }
};
__device__ __forceinline__ uint32_t size_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// The largest over LPB lanes next to each other, in all of them: quads by their permutations, then the other quad and the
// other eight by mirrors.
template <int LPB>
__device__ __forceinline__ uint32_t largest_of(uint32_t m) {
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xb1, 0xf, 0xf, true));
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4e, 0xf, 0xf, true));
    if constexpr (LPB >= 8) m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x141, 0xf, 0xf, true));
    if constexpr (LPB >= 16) m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x140, 0xf, 0xf, true));
    return m;
}

// LPB lanes a block, eight adjacent values each (C a multiple of 8) or the values lane, lane + LPB, ...; a workgroup
// takes 256 / LPB blocks at a time.
template <bool BF, bool VEC, int LPB>
__global__ __launch_bounds__(256) void kda_ckpt_save_kernel(const void *__restrict__ xp, int8_t *__restrict__ codes,
                                                            float *__restrict__ scales, int64_t blocks, int nb, int C) {
    using E = typename IO<BF>::T;
    constexpr int V = 8;
    const int lane = threadIdx.x % LPB;
    for (int64_t b = ((int64_t)blockIdx.x * 256 + threadIdx.x) / LPB; b < blocks; b += (int64_t)gridDim.x * (256 / LPB)) {
        const int64_t row = nb == 1 ? b : b / nb;
        const int c0 = nb == 1 ? 0 : (int)(b - row * nb) * kCkptBlock;
        const int n = C - c0 < kCkptBlock ? C - c0 : kCkptBlock;  // values of this block
        const E *p = reinterpret_cast<const E *>(xp) + row * C + c0;
        float x[V];
        if constexpr (VEC) {
            E e[V] = {};
            if (lane * V < n) {
                u32x4 w[BF ? 1 : 2];
#pragma unroll
                for (int i = 0; i < (BF ? 1 : 2); ++i)
                    w[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p + lane * V) + i);
                __builtin_memcpy(e, w, sizeof(e));
            }
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = IO<BF>::ld(e, i);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = lane + i * LPB < n ? IO<BF>::ld(p, lane + i * LPB) : 0.f;
        }
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) m = max(m, size_bits(x[i]));
        m = largest_of<LPB>(m);
        const float top = __uint_as_float(m);
        const bool bad = m >= 0x7f800000u;
        int8_t out[V];
        const Quantizer q(m == 0 || bad ? 1.f : top);
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = (int8_t)(bad ? 0 : q.code(x[i]));
        int8_t *o = codes + row * C + c0;
        if constexpr (VEC) {
            uint2 w;
            __builtin_memcpy(&w, out, 8);
            if (lane * V < n) *reinterpret_cast<uint2 *>(o + lane * V) = w;
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (lane + i * LPB < n) o[lane + i * LPB] = out[i];
        }
        // The quotient may round up: where 127 of it would pass the largest value of fp32, the scale below it (off by less
        // than one step of fp32, so that 127 of it stay under the largest).
        float scale = top / 127.f;
        if (scale * 127.f > __FLT_MAX__) scale = __uint_as_float(__float_as_uint(scale) - 1);
        if (lane == 0) scales[b] = bad ? __builtin_nanf("") : scale;
    }
}

// Eight adjacent values a thread (C a multiple of 8), or one.
template <bool BF, int V>
__global__ __launch_bounds__(256) void kda_ckpt_restore_kernel(const int8_t *__restrict__ codes,
                                                               const float *__restrict__ scales, void *__restrict__ xp,
                                                               int64_t runs, int runs_per_row, int nb) {
    using E = typename IO<BF>::T;
    const int64_t stride = (int64_t)gridDim.x * 256;
    for (int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x; r < runs; r += stride) {
        const int64_t row = runs_per_row == kCkptBlock / V ? r / (kCkptBlock / V) : r / runs_per_row;
        const int c = (int)(r - row * runs_per_row) * V;
        const float step = scales[row * nb + c / kCkptBlock];
        if constexpr (V == 8) {
            const uint2 w = *reinterpret_cast<const uint2 *>(codes + r * V);
            int8_t in[V];
            __builtin_memcpy(in, &w, 8);
            E e[V];
#pragma unroll
            for (int i = 0; i < V; ++i) IO<BF>::st(e, i, (float)in[i] * step);
            u32x4 o[BF ? 1 : 2];
            __builtin_memcpy(o, e, sizeof(e));
#pragma unroll
            for (int i = 0; i < (BF ? 1 : 2); ++i)
                *(reinterpret_cast<u32x4 *>(reinterpret_cast<E *>(xp) + r * V) + i) = o[i];
        } else {
            IO<BF>::st(reinterpret_cast<E *>(xp), r, (float)codes[r] * step);
        }
    }
}

template <bool BF, bool VEC, int LPB>
hipError_t save_l(const CkptArgs &a, int nb, hipStream_t st) {
    const int64_t blocks = a.rows * nb, wgs = (blocks + 256 / LPB - 1) / (256 / LPB);
    hipLaunchKernelGGL((kda_ckpt_save_kernel<BF, VEC, LPB>), dim3((uint32_t)(wgs < 65536 ? wgs : 65536)), dim3(256), 0,
                       st, a.x, a.codes, a.scales, blocks, nb, a.C);
    return hipGetLastError();
}
// As many lanes as a row needs where it is shorter than a block.
template <bool BF, bool VEC>
hipError_t save_c(const CkptArgs &a, int nb, hipStream_t st) {
    if (a.C <= 32) return save_l<BF, VEC, 4>(a, nb, st);
    return a.C <= 64 ? save_l<BF, VEC, 8>(a, nb, st) : save_l<BF, VEC, 16>(a, nb, st);
}
template <bool BF, int V>
hipError_t restore_v(const CkptArgs &a, int nb, hipStream_t st) {
    const int64_t runs = a.rows * (a.C / V), wgs = (runs + 255) / 256;
    hipLaunchKernelGGL((kda_ckpt_restore_kernel<BF, V>), dim3((uint32_t)(wgs < 65536 ? wgs : 65536)), dim3(256), 0, st,
                       a.codes, a.scales, a.x, runs, a.C / V, nb);
    return hipGetLastError();
}
int blocks_of(int32_t C) { return (int)(((int64_t)C + kCkptBlock - 1) / kCkptBlock); }
// Rows of whole blocks are as many rows of one block.
CkptArgs by_blocks(CkptArgs a) {
    if (a.C % kCkptBlock == 0) {
        a.rows *= a.C / kCkptBlock;
        a.C = kCkptBlock;
    }
    return a;
}

}  // namespace

hipError_t launch_ckpt_save(const CkptArgs &args, hipStream_t st) {
    if (args.rows == 0) return hipSuccess;
    const CkptArgs a = by_blocks(args);
    const int nb = blocks_of(a.C);
    if (a.io_bf16) return a.C % 8 == 0 ? save_c<true, true>(a, nb, st) : save_c<true, false>(a, nb, st);
    return a.C % 8 == 0 ? save_c<false, true>(a, nb, st) : save_c<false, false>(a, nb, st);
}
hipError_t launch_ckpt_restore(const CkptArgs &args, hipStream_t st) {
    if (args.rows == 0) return hipSuccess;
    const CkptArgs a = by_blocks(args);
    const int nb = blocks_of(a.C);
    if (a.io_bf16) return a.C % 8 == 0 ? restore_v<true, 8>(a, nb, st) : restore_v<true, 1>(a, nb, st);
    return a.C % 8 == 0 ? restore_v<false, 8>(a, nb, st) : restore_v<false, 1>(a, nb, st);
}

}  // namespace kda
