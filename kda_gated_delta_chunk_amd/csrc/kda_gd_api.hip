// C ABI of the gated delta rule with one decay per head (declared in include/kda.h). Argument validation runs on the
// host before any HIP call, so every error status leaves the device untouched (and works on a host with no GPU).

#include "kda_check.hpp"
#include "kda_gd.hpp"

namespace {

kda_status_t check_sizes(int64_t B, int64_t T, int32_t H, int32_t Hk, int32_t K, int32_t V, int32_t num_seqs, bool packed) {
    if (B < 1 || T < 0 || H < 1 || Hk < 1 || K < 1 || V < 1 || num_seqs < 1) return KDA_ERROR_INVALID_VALUE;
    if (H % Hk != 0) return KDA_ERROR_INVALID_VALUE;
    if (packed ? (B != 1) : (num_seqs != B)) return KDA_ERROR_INVALID_VALUE;
    if (!supported_dim(K) || !supported_dim(V)) return KDA_ERROR_NOT_SUPPORTED;
    // cu_seqlens and a sequence's chunks are 32-bit; a chunk's rows of all heads (32 tokens) stay below 2^31 bytes
    if (T >= ((int64_t)1 << 31) || B > ((int64_t)1 << 31) || B * T > kMaxElems / H / 512) return KDA_ERROR_INVALID_VALUE;
    if (H >= (1 << 16) || (int64_t)num_seqs * H >= ((int64_t)1 << 26)) return KDA_ERROR_INVALID_VALUE;
    // workgroups: one per (chunk, head)
    if (B * ((T + 31) / 32) + num_seqs > ((int64_t)1 << 34) / H) return KDA_ERROR_INVALID_VALUE;
    return KDA_SUCCESS;
}
// The gates come in the I/O type, or in fp32 beside bf16.
bool valid_gates(kda_dtype_t io, kda_dtype_t gates) { return valid_io(gates) && (gates == io || gates == KDA_DTYPE_FP32); }

}  // namespace

extern "C" {

size_t kda_gd_chunk_fwd_workspace_bytes(int64_t B, int64_t T, int32_t H, int32_t Hk, int32_t K, int32_t V,
                                        int32_t num_seqs, int32_t packed, kda_dtype_t io) {
    if (!valid_io(io) || check_sizes(B, T, H, Hk, K, V, num_seqs, packed != 0) != KDA_SUCCESS) return 0;
    return kda::gd_fwd_workspace_bytes(B, T, H, Hk, K, V, num_seqs, packed != 0, io == KDA_DTYPE_BF16);
}

size_t kda_gd_chunk_bwd_workspace_bytes(int64_t B, int64_t T, int32_t H, int32_t Hk, int32_t K, int32_t V,
                                        int32_t num_seqs, int32_t packed, kda_dtype_t io) {
    if (!valid_io(io) || check_sizes(B, T, H, Hk, K, V, num_seqs, packed != 0) != KDA_SUCCESS) return 0;
    return kda::gd_bwd_workspace_bytes(B, T, H, Hk, K, V, num_seqs, packed != 0, io == KDA_DTYPE_BF16);
}

kda_status_t kda_gd_chunk_fwd(const void *q, const void *k, const void *v, const void *g, const void *beta,
                              const float *S0, const int32_t *cu_seqlens, int64_t B, int64_t T, int32_t H, int32_t Hk,
                              int32_t K, int32_t V, int32_t num_seqs, kda_dtype_t io, kda_dtype_t gates, float scale,
                              void *o, float *S_final, void *workspace, size_t workspace_bytes, void *stream) {
    if (!valid_io(io) || !valid_gates(io, gates) || !std::isfinite(scale)) return KDA_ERROR_INVALID_VALUE;
    const bool packed = cu_seqlens != nullptr;
    kda_status_t st = check_sizes(B, T, H, Hk, K, V, num_seqs, packed);
    if (st != KDA_SUCCESS) return st;
    if (T > 0 && (!q || !k || !v || !g || !beta || !o)) return KDA_ERROR_INVALID_VALUE;
    for (const void *p : {q, k, v, (const void *)S0, (const void *)o, (const void *)S_final, (const void *)workspace})
        if (!aligned(p, 16)) return KDA_ERROR_INVALID_VALUE;
    if (!aligned(g, elem(gates)) || !aligned(beta, elem(gates)) || !aligned(cu_seqlens, 4)) return KDA_ERROR_INVALID_VALUE;
    const int64_t n = B * T, e = (int64_t)elem(io), ng = n * H * (int64_t)elem(gates);
    const int64_t states = (int64_t)num_seqs * H * K * V * 4;
    const size_t need = kda::gd_fwd_workspace_bytes(B, T, H, Hk, K, V, num_seqs, packed, io == KDA_DTYPE_BF16);
    const Range in[] = {{q, n * Hk * K * e}, {k, n * Hk * K * e}, {v, n * H * V * e}, {g, ng}, {beta, ng}, {S0, states},
                        {cu_seqlens, ((int64_t)num_seqs + 1) * 4}};
    const Range out[] = {{o, n * H * V * e}, {S_final, states}, {workspace, (int64_t)need}};
    if (clash(out, in)) return KDA_ERROR_INVALID_VALUE;
    if (!workspace || workspace_bytes < need) return KDA_ERROR_WORKSPACE_TOO_SMALL;
    st = check_device();
    if (st != KDA_SUCCESS) return st;
    kda::GdArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.S0 = S0; a.cu_seqlens = cu_seqlens;
    a.B = B; a.T = T; a.H = H; a.Hk = Hk; a.K = K; a.V = V; a.num_seqs = num_seqs;
    a.io_bf16 = io == KDA_DTYPE_BF16;
    a.gates_fp32 = gates == KDA_DTYPE_FP32;
    a.scale = scale;
    a.o = o; a.S_final = S_final; a.workspace = workspace;
    return launched(kda::launch_gd_fwd(a, reinterpret_cast<hipStream_t>(stream)));
}

kda_status_t kda_gd_chunk_bwd(const void *q, const void *k, const void *v, const void *g, const void *beta,
                              const float *S0, const int32_t *cu_seqlens, const void *d_o, const float *dS_final,
                              int64_t B, int64_t T, int32_t H, int32_t Hk, int32_t K, int32_t V, int32_t num_seqs,
                              kda_dtype_t io, kda_dtype_t gates, float scale, void *dq, void *dk, void *dv, void *dg,
                              void *dbeta, float *dS0, void *workspace, size_t workspace_bytes, void *stream) {
    if (!valid_io(io) || !valid_gates(io, gates) || !std::isfinite(scale)) return KDA_ERROR_INVALID_VALUE;
    const bool packed = cu_seqlens != nullptr;
    kda_status_t st = check_sizes(B, T, H, Hk, K, V, num_seqs, packed);
    if (st != KDA_SUCCESS) return st;
    if (T > 0 && (!q || !k || !v || !g || !beta || !d_o || !dq || !dk || !dv || !dg || !dbeta))
        return KDA_ERROR_INVALID_VALUE;
    for (const void *p : {q, k, v, (const void *)S0, d_o, (const void *)dS_final, (const void *)dq, (const void *)dk,
                          (const void *)dv, (const void *)dS0, (const void *)workspace})
        if (!aligned(p, 16)) return KDA_ERROR_INVALID_VALUE;
    for (const void *p : {g, beta, (const void *)dg, (const void *)dbeta})
        if (!aligned(p, elem(gates))) return KDA_ERROR_INVALID_VALUE;
    if (!aligned(cu_seqlens, 4)) return KDA_ERROR_INVALID_VALUE;
    const int64_t n = B * T, e = (int64_t)elem(io), ng = n * H * (int64_t)elem(gates);
    const int64_t states = (int64_t)num_seqs * H * K * V * 4;
    const size_t need = kda::gd_bwd_workspace_bytes(B, T, H, Hk, K, V, num_seqs, packed, io == KDA_DTYPE_BF16);
    const Range in[] = {{q, n * Hk * K * e}, {k, n * Hk * K * e}, {v, n * H * V * e}, {d_o, n * H * V * e}, {g, ng},
                        {beta, ng}, {S0, states}, {dS_final, states}, {cu_seqlens, ((int64_t)num_seqs + 1) * 4}};
    const Range out[] = {{dq, n * Hk * K * e}, {dk, n * Hk * K * e}, {dv, n * H * V * e}, {dg, ng}, {dbeta, ng},
                         {dS0, states}, {workspace, (int64_t)need}};
    if (clash(out, in)) return KDA_ERROR_INVALID_VALUE;
    if (!workspace || workspace_bytes < need) return KDA_ERROR_WORKSPACE_TOO_SMALL;
    st = check_device();
    if (st != KDA_SUCCESS) return st;
    kda::GdArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.S0 = S0; a.cu_seqlens = cu_seqlens;
    a.B = B; a.T = T; a.H = H; a.Hk = Hk; a.K = K; a.V = V; a.num_seqs = num_seqs;
    a.io_bf16 = io == KDA_DTYPE_BF16;
    a.gates_fp32 = gates == KDA_DTYPE_FP32;
    a.scale = scale;
    a.dout = d_o; a.dS_final = dS_final;
    a.dq = dq; a.dk = dk; a.dv = dv; a.dg = dg; a.dbeta = dbeta; a.dS0 = dS0;
    a.workspace = workspace;
    return launched(kda::launch_gd_bwd(a, reinterpret_cast<hipStream_t>(stream)));
}

kda_status_t kda_gd_decode_step(const void *q, const void *k, const void *v, const void *g, const void *beta, float *S,
                                void *o, int32_t N, int32_t H, int32_t Hk, int32_t K, int32_t V, kda_dtype_t io,
                                kda_dtype_t gates, float scale, void *stream) {
    if (!valid_io(io) || !valid_gates(io, gates) || !std::isfinite(scale)) return KDA_ERROR_INVALID_VALUE;
    if (N < 0 || H < 1 || Hk < 1 || H % Hk != 0) return KDA_ERROR_INVALID_VALUE;
    if (!supported_dim(K) || !supported_dim(V)) return KDA_ERROR_NOT_SUPPORTED;
    if ((int64_t)N * H >= ((int64_t)1 << 28)) return KDA_ERROR_INVALID_VALUE;
    if (N == 0) return KDA_SUCCESS;
    if (!q || !k || !v || !g || !beta || !S || !o) return KDA_ERROR_INVALID_VALUE;
    for (const void *p : {q, k, v, (const void *)S, (const void *)o})
        if (!aligned(p, 16)) return KDA_ERROR_INVALID_VALUE;
    if (!aligned(g, elem(gates)) || !aligned(beta, elem(gates))) return KDA_ERROR_INVALID_VALUE;
    const int64_t e = (int64_t)elem(io), nh = (int64_t)N * H, nk = (int64_t)N * Hk, ng = nh * (int64_t)elem(gates);
    const Range in[] = {{q, nk * K * e}, {k, nk * K * e}, {v, nh * V * e}, {g, ng}, {beta, ng}};
    const Range out[] = {{S, nh * K * V * 4}, {o, nh * V * e}};
    if (clash(out, in)) return KDA_ERROR_INVALID_VALUE;
    const kda_status_t st = check_device();
    if (st != KDA_SUCCESS) return st;
    kda::GdDecodeArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.S = S; a.o = o;
    a.N = N; a.H = H; a.Hk = Hk; a.K = K; a.V = V;
    a.io_bf16 = io == KDA_DTYPE_BF16;
    a.gates_fp32 = gates == KDA_DTYPE_FP32;
    a.scale = scale;
    return launched(kda::launch_gd_decode(a, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
