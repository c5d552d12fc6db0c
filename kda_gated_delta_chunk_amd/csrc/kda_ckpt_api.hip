// C ABI of the rotary positions with several axes and of the activation checkpoints in 8 bits (declared in
// include/kda.h). Argument validation runs on the host before any HIP call, so every error status leaves the device
// untouched (and works on a host with no GPU).

#include "kda_check.hpp"
#include "kda_layer.hpp"

namespace {

kda_status_t check_rows(int64_t rows, int32_t C) {
    if (rows < 0 || C < 1 || rows > kMaxElems / C) return KDA_ERROR_INVALID_VALUE;
    return KDA_SUCCESS;
}
int64_t scales_bytes(int64_t rows, int32_t C) {
    return rows * (((int64_t)C + kda::kCkptBlock - 1) / kda::kCkptBlock) * 4;
}

}  // namespace

extern "C" {

kda_status_t kda_rotary_axes(const void *q, const void *k, const double *freqs, const int32_t *axes,
                             const int32_t *positions, void *q_out, void *k_out, int64_t tokens, int32_t num_axes,
                             int32_t Hq, int32_t Hk, int32_t D, int32_t R, kda_dtype_t io, kda_rotary_layout_t layout,
                             int32_t inverse, float scale, void *stream) {
    if (!valid_io(io) || (layout != KDA_ROTARY_HALF && layout != KDA_ROTARY_INTERLEAVED) || !std::isfinite(scale))
        return KDA_ERROR_INVALID_VALUE;
    if (inverse != 0 && inverse != 1) return KDA_ERROR_INVALID_VALUE;
    if (tokens < 0 || num_axes < 1 || Hq < 1 || Hk < 0 || D < 2 || R < 2 || R > D || R % 2 != 0)
        return KDA_ERROR_INVALID_VALUE;
    if (D > 512 || num_axes > 16) return KDA_ERROR_NOT_SUPPORTED;
    if ((int64_t)Hq + Hk > (1 << 20) || tokens > kMaxElems / ((int64_t)Hq + Hk) / D) return KDA_ERROR_INVALID_VALUE;
    if (tokens == 0) return KDA_SUCCESS;
    if (!q || !q_out || !freqs || !axes || !positions || (Hk > 0 && (!k || !k_out))) return KDA_ERROR_INVALID_VALUE;
    if (Hk == 0) k = k_out = nullptr;
    for (const void *p : {q, k, (const void *)q_out, (const void *)k_out})
        if (!aligned(p, 16)) return KDA_ERROR_INVALID_VALUE;
    if (!aligned(freqs, 8) || !aligned(axes, 4) || !aligned(positions, 4)) return KDA_ERROR_INVALID_VALUE;
    const int64_t e = (int64_t)elem(io), nq = tokens * Hq * D * e, nk = tokens * Hk * D * e;
    // q_out may be q and k_out may be k; nothing else that is written may meet anything
    const Range in[] = {{q == q_out ? nullptr : q, nq}, {k == k_out ? nullptr : k, nk}, {freqs, (int64_t)R / 2 * 8},
                        {axes, (int64_t)R / 2 * 4}, {positions, tokens * num_axes * 4}};
    const Range out[] = {{q_out, nq}, {k_out, nk}};
    if (clash(out, in)) return KDA_ERROR_INVALID_VALUE;
    const kda_status_t st = check_device();
    if (st != KDA_SUCCESS) return st;
    kda::RotaryArgs a{};
    a.q = q; a.k = k; a.q_out = q_out; a.k_out = k_out; a.freqs = freqs; a.positions = positions;
    a.axes = axes; a.naxes = num_axes;
    a.tokens = a.T = tokens;
    a.Hq = Hq; a.Hk = Hk; a.D = D; a.R = R;
    a.io_bf16 = io == KDA_DTYPE_BF16;
    a.interleaved = layout == KDA_ROTARY_INTERLEAVED;
    a.inverse = inverse != 0;
    a.scale = scale;
    return launched(kda::launch_rotary(a, reinterpret_cast<hipStream_t>(stream)));
}

kda_status_t kda_checkpoint8_save(const void *x, int8_t *codes, float *scales, int64_t rows, int32_t C, kda_dtype_t io,
                                  void *stream) {
    if (!valid_io(io)) return KDA_ERROR_INVALID_VALUE;
    kda_status_t st = check_rows(rows, C);
    if (st != KDA_SUCCESS) return st;
    if (rows == 0) return KDA_SUCCESS;
    if (!x || !codes || !scales) return KDA_ERROR_INVALID_VALUE;
    if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 4)) return KDA_ERROR_INVALID_VALUE;
    const Range in[] = {{x, rows * C * (int64_t)elem(io)}};
    const Range out[] = {{codes, rows * C}, {scales, scales_bytes(rows, C)}};
    if (clash(out, in)) return KDA_ERROR_INVALID_VALUE;
    st = check_device();
    if (st != KDA_SUCCESS) return st;
    kda::CkptArgs a{const_cast<void *>(x), codes, scales, rows, C, io == KDA_DTYPE_BF16};
    return launched(kda::launch_ckpt_save(a, reinterpret_cast<hipStream_t>(stream)));
}

kda_status_t kda_checkpoint8_restore(const int8_t *codes, const float *scales, void *x, int64_t rows, int32_t C,
                                     kda_dtype_t io, void *stream) {
    if (!valid_io(io)) return KDA_ERROR_INVALID_VALUE;
    kda_status_t st = check_rows(rows, C);
    if (st != KDA_SUCCESS) return st;
    if (rows == 0) return KDA_SUCCESS;
    if (!x || !codes || !scales) return KDA_ERROR_INVALID_VALUE;
    if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 4)) return KDA_ERROR_INVALID_VALUE;
    const Range in[] = {{codes, rows * C}, {scales, scales_bytes(rows, C)}};
    const Range out[] = {{x, rows * C * (int64_t)elem(io)}};
    if (clash(out, in)) return KDA_ERROR_INVALID_VALUE;
    st = check_device();
    if (st != KDA_SUCCESS) return st;
    kda::CkptArgs a{x, const_cast<int8_t *>(codes), const_cast<float *>(scales), rows, C, io == KDA_DTYPE_BF16};
    return launched(kda::launch_ckpt_restore(a, reinterpret_cast<hipStream_t>(stream)));
}

kda_status_t kda_layer_norm_bwd_checkpoint8(const void *dy, const int8_t *codes, const float *scales, const float *weight,
                                            const float *bias, const void *o_gate, void *dx, float *dweight,
                                            float *dbias, void *d_o_gate, int64_t rows, int32_t groups, int32_t C,
                                            float eps, int32_t center, kda_dtype_t io, void *workspace,
                                            size_t workspace_bytes, void *stream) {
    if (!valid_io(io) || !(eps > 0.f) || !std::isfinite(eps) || (center != 0 && center != 1))
        return KDA_ERROR_INVALID_VALUE;
    const size_t need = kda_layer_norm_bwd_workspace_bytes(rows, groups, C);
    if (need == 0) return C > 16384 && rows >= 0 && groups >= 1 && rows % groups == 0 ? KDA_ERROR_NOT_SUPPORTED : KDA_ERROR_INVALID_VALUE;
    if (rows > 0 && (!dy || !codes || !scales || !dx || (o_gate && !d_o_gate))) return KDA_ERROR_INVALID_VALUE;
    if (!o_gate) d_o_gate = nullptr;
    for (const void *p : {dy, (const void *)codes, (const void *)weight, (const void *)bias, o_gate, (const void *)dx,
                          (const void *)dweight, (const void *)dbias, (const void *)d_o_gate, (const void *)workspace})
        if (!aligned(p, 16)) return KDA_ERROR_INVALID_VALUE;
    if (!aligned(scales, 4)) return KDA_ERROR_INVALID_VALUE;
    const int64_t n = rows * C * (int64_t)elem(io), w = (int64_t)groups * C * 4;
    const Range in[] = {{dy, n}, {codes, rows * C}, {scales, scales_bytes(rows, C)}, {weight, w}, {bias, w}, {o_gate, n}};
    const Range out[] = {{dx, n}, {dweight, w}, {dbias, w}, {d_o_gate, n}, {workspace, (int64_t)need}};
    if (clash(out, in)) return KDA_ERROR_INVALID_VALUE;
    if (!workspace || workspace_bytes < need) return KDA_ERROR_WORKSPACE_TOO_SMALL;
    const kda_status_t st = check_device();
    if (st != KDA_SUCCESS) return st;
    kda::NormArgs a{};
    a.codes = codes; a.scales = scales; a.gate = o_gate; a.weight = weight; a.bias = bias;
    a.rows = rows; a.G = groups; a.C = C; a.eps = eps;
    a.io_bf16 = io == KDA_DTYPE_BF16;
    a.center = center != 0;
    a.dy = dy; a.dx = dx; a.dgate = d_o_gate; a.dweight = dweight; a.dbias = dbias; a.workspace = workspace;
    return launched(kda::launch_norm_bwd(a, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
