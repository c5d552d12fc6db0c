// C ABI of the operators around the recurrence (declared in include/kda.h): linear attention with one decay per head,
// rotary positions, layer norm. Argument validation runs on the host before any HIP call, so every error status
// leaves the device untouched (and works on a host with no GPU).

#include "../../include/kda.h"
#include "kda_layer.hpp"

#include <atomic>
#include <cmath>

namespace {

constexpr int64_t kMaxElems = (int64_t)1 << 60;

bool aligned(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
bool valid_io(kda_dtype_t t) { return t == KDA_DTYPE_FP32 || t == KDA_DTYPE_BF16; }
bool valid_decay(kda_decay_t d) { return d == KDA_DECAY_PER_TOKEN || d == KDA_DECAY_PER_HEAD; }
bool supported_dim(int32_t d) { return d == 32 || d == 64 || d == 128; }
size_t elem(kda_dtype_t t) { return t == KDA_DTYPE_BF16 ? 2 : 4; }

// A range of device memory a call reads or writes; p null: absent.
struct Range {
    const void *p;
    int64_t bytes;
};
bool meet(const Range &a, const Range &b) {
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return x < y + (uintptr_t)b.bytes && y < x + (uintptr_t)a.bytes;
}
// Whether any written range meets a read one or another written one.
template <int NO, int NI>
bool clash(const Range (&out)[NO], const Range (&in)[NI]) {
    for (int i = 0; i < NO; ++i) {
        for (int j = 0; j < NI; ++j)
            if (meet(out[i], in[j])) return true;
        for (int j = i + 1; j < NO; ++j)
            if (meet(out[i], out[j])) return true;
    }
    return false;
}

kda_status_t check_device() {
    static std::atomic<bool> found{false};  // a device that was visible stays so
    if (found.load(std::memory_order_relaxed)) return KDA_SUCCESS;
    int n = 0;
    if (hipGetDeviceCount(&n) != hipSuccess || n < 1) {
        (void)hipGetLastError();
        return KDA_ERROR_NO_DEVICE;
    }
    found.store(true, std::memory_order_relaxed);
    return KDA_SUCCESS;
}
kda_status_t launched(hipError_t e) {
    if (e == hipSuccess) return KDA_SUCCESS;
    (void)hipGetLastError();
    return KDA_ERROR_HIP;
}

kda_status_t check_hd_sizes(int64_t B, int64_t T, int32_t H, int32_t Hk, int32_t K, int32_t V, int32_t num_seqs,
                            bool packed) {
    if (B < 1 || T < 0 || H < 1 || Hk < 1 || K < 1 || V < 1 || num_seqs < 1) return KDA_ERROR_INVALID_VALUE;
    if (H % Hk != 0) return KDA_ERROR_INVALID_VALUE;
    if (packed ? (B != 1) : (num_seqs != B)) return KDA_ERROR_INVALID_VALUE;
    if (!supported_dim(K) || !supported_dim(V)) return KDA_ERROR_NOT_SUPPORTED;
    // element counts; cu_seqlens and a sequence's chunks are 32-bit
    if (T >= ((int64_t)1 << 31) || T > kMaxElems / B || B * T > kMaxElems / H / 512) return KDA_ERROR_INVALID_VALUE;
    // a chunk's rows of all heads (32 tokens) stay below 2^31 bytes, the kernels' offsets within it; heads and states
    // are 32-bit
    if (H >= (1 << 16) || (int64_t)num_seqs * H >= ((int64_t)1 << 26)) return KDA_ERROR_INVALID_VALUE;
    // workgroups of a pass (at most 9 for each head of a segment, at least 128 tokens or a sequence) stay below 2^32
    if ((B * ((T + 127) / 128) + num_seqs) > ((int64_t)1 << 27) / H) return KDA_ERROR_INVALID_VALUE;
    return KDA_SUCCESS;
}

}  // namespace

extern "C" {

size_t kda_hd_chunk_fwd_workspace_bytes(int64_t B, int64_t T, int32_t H, int32_t Hk, int32_t K, int32_t V,
                                        int32_t num_seqs, int32_t packed, kda_dtype_t io) {
    if (!valid_io(io) || check_hd_sizes(B, T, H, Hk, K, V, num_seqs, packed != 0) != KDA_SUCCESS) return 0;
    return kda::hd_fwd_workspace_bytes(B, T, H, Hk, K, V, num_seqs, packed != 0, io == KDA_DTYPE_BF16);
}

size_t kda_hd_chunk_bwd_workspace_bytes(int64_t B, int64_t T, int32_t H, int32_t Hk, int32_t K, int32_t V,
                                        int32_t num_seqs, int32_t packed, kda_dtype_t io) {
    if (!valid_io(io) || check_hd_sizes(B, T, H, Hk, K, V, num_seqs, packed != 0) != KDA_SUCCESS) return 0;
    return kda::hd_bwd_workspace_bytes(B, T, H, Hk, K, V, num_seqs, packed != 0, io == KDA_DTYPE_BF16);
}

kda_status_t kda_hd_chunk_fwd(const void *q, const void *k, const void *v, const void *g, const float *S0,
                              const int32_t *cu_seqlens, int64_t B, int64_t T, int32_t H, int32_t Hk, int32_t K,
                              int32_t V, int32_t num_seqs, kda_dtype_t io, kda_decay_t decay, float scale, void *o,
                              float *S_final, void *workspace, size_t workspace_bytes, void *stream) {
    if (!valid_io(io) || !valid_decay(decay) || !std::isfinite(scale)) return KDA_ERROR_INVALID_VALUE;
    const bool packed = cu_seqlens != nullptr;
    kda_status_t st = check_hd_sizes(B, T, H, Hk, K, V, num_seqs, packed);
    if (st != KDA_SUCCESS) return st;
    if (T > 0 && (!q || !k || !v || !g || !o)) return KDA_ERROR_INVALID_VALUE;
    for (const void *p : {q, k, v, (const void *)S0, (const void *)o, (const void *)S_final, (const void *)workspace})
        if (!aligned(p, 16)) return KDA_ERROR_INVALID_VALUE;
    const bool per_head = decay == KDA_DECAY_PER_HEAD;
    if (!aligned(g, per_head ? 4 : elem(io)) || !aligned(cu_seqlens, 4)) return KDA_ERROR_INVALID_VALUE;
    const int64_t n = B * T, e = (int64_t)elem(io), states = (int64_t)num_seqs * H * K * V * 4;
    const size_t need = kda::hd_fwd_workspace_bytes(B, T, H, Hk, K, V, num_seqs, packed, io == KDA_DTYPE_BF16);
    const Range in[] = {{q, n * Hk * K * e}, {k, n * Hk * K * e}, {v, n * H * V * e},
                        {g, per_head ? (int64_t)H * 4 : n * H * e}, {S0, states},
                        {cu_seqlens, ((int64_t)num_seqs + 1) * 4}};
    const Range out[] = {{o, n * H * V * e}, {S_final, states}, {workspace, (int64_t)need}};
    if (clash(out, in)) return KDA_ERROR_INVALID_VALUE;
    if (!workspace || workspace_bytes < need) return KDA_ERROR_WORKSPACE_TOO_SMALL;
    st = check_device();
    if (st != KDA_SUCCESS) return st;
    kda::HdArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = g; a.S0 = S0; a.cu_seqlens = cu_seqlens;
    a.B = B; a.T = T; a.H = H; a.Hk = Hk; a.K = K; a.V = V; a.num_seqs = num_seqs;
    a.io_bf16 = io == KDA_DTYPE_BF16;
    a.decay_per_head = per_head;
    a.scale = scale;
    a.o = o; a.S_final = S_final; a.workspace = workspace;
    return launched(kda::launch_hd_fwd(a, reinterpret_cast<hipStream_t>(stream)));
}

kda_status_t kda_hd_chunk_bwd(const void *q, const void *k, const void *v, const void *g, const float *S0,
                              const int32_t *cu_seqlens, const void *d_o, const float *dS_final, int64_t B, int64_t T,
                              int32_t H, int32_t Hk, int32_t K, int32_t V, int32_t num_seqs, kda_dtype_t io,
                              kda_decay_t decay, float scale, void *dq, void *dk, void *dv, void *dg, float *dS0,
                              void *workspace, size_t workspace_bytes, void *stream) {
    if (!valid_io(io) || !valid_decay(decay) || !std::isfinite(scale)) return KDA_ERROR_INVALID_VALUE;
    const bool packed = cu_seqlens != nullptr, per_head = decay == KDA_DECAY_PER_HEAD;
    kda_status_t st = check_hd_sizes(B, T, H, Hk, K, V, num_seqs, packed);
    if (st != KDA_SUCCESS) return st;
    if (T > 0 && (!q || !k || !v || !g || !d_o || !dq || !dk || !dv)) return KDA_ERROR_INVALID_VALUE;
    if (dg && per_head) return KDA_ERROR_NOT_SUPPORTED;
    for (const void *p : {q, k, v, (const void *)S0, d_o, (const void *)dS_final, (const void *)dq, (const void *)dk,
                          (const void *)dv, (const void *)dS0, (const void *)workspace})
        if (!aligned(p, 16)) return KDA_ERROR_INVALID_VALUE;
    if (!aligned(g, per_head ? 4 : elem(io)) || !aligned(dg, elem(io)) || !aligned(cu_seqlens, 4))
        return KDA_ERROR_INVALID_VALUE;
    const int64_t n = B * T, e = (int64_t)elem(io), states = (int64_t)num_seqs * H * K * V * 4;
    const size_t need = kda::hd_bwd_workspace_bytes(B, T, H, Hk, K, V, num_seqs, packed, io == KDA_DTYPE_BF16);
    const Range in[] = {{q, n * Hk * K * e}, {k, n * Hk * K * e}, {v, n * H * V * e}, {d_o, n * H * V * e},
                        {g, per_head ? (int64_t)H * 4 : n * H * e}, {S0, states}, {dS_final, states},
                        {cu_seqlens, ((int64_t)num_seqs + 1) * 4}};
    const Range out[] = {{dq, n * Hk * K * e}, {dk, n * Hk * K * e}, {dv, n * H * V * e}, {dg, n * H * e},
                         {dS0, states}, {workspace, (int64_t)need}};
    if (clash(out, in)) return KDA_ERROR_INVALID_VALUE;
    if (!workspace || workspace_bytes < need) return KDA_ERROR_WORKSPACE_TOO_SMALL;
    st = check_device();
    if (st != KDA_SUCCESS) return st;
    kda::HdArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = g; a.S0 = S0; a.cu_seqlens = cu_seqlens;
    a.B = B; a.T = T; a.H = H; a.Hk = Hk; a.K = K; a.V = V; a.num_seqs = num_seqs;
    a.io_bf16 = io == KDA_DTYPE_BF16;
    a.decay_per_head = per_head;
    a.scale = scale;
    a.dout = d_o; a.dS_final = dS_final;
    a.dq = dq; a.dk = dk; a.dv = dv; a.dg = T > 0 ? dg : nullptr; a.dS0 = dS0;
    a.workspace = workspace;
    return launched(kda::launch_hd_bwd(a, reinterpret_cast<hipStream_t>(stream)));
}

kda_status_t kda_hd_decode_step(const void *q, const void *k, const void *v, const void *g, float *S, void *o,
                                int32_t N, int32_t H, int32_t Hk, int32_t K, int32_t V, kda_dtype_t io,
                                kda_decay_t decay, float scale, void *stream) {
    if (!valid_io(io) || !valid_decay(decay) || !std::isfinite(scale)) return KDA_ERROR_INVALID_VALUE;
    if (N < 0 || H < 1 || Hk < 1 || H % Hk != 0) return KDA_ERROR_INVALID_VALUE;
    if (!supported_dim(K) || !supported_dim(V)) return KDA_ERROR_NOT_SUPPORTED;
    if ((int64_t)N * H >= ((int64_t)1 << 28)) return KDA_ERROR_INVALID_VALUE;
    if (N == 0) return KDA_SUCCESS;
    if (!q || !k || !v || !g || !S || !o) return KDA_ERROR_INVALID_VALUE;
    for (const void *p : {q, k, v, (const void *)S, (const void *)o})
        if (!aligned(p, 16)) return KDA_ERROR_INVALID_VALUE;
    const bool per_head = decay == KDA_DECAY_PER_HEAD;
    if (!aligned(g, per_head ? 4 : elem(io))) return KDA_ERROR_INVALID_VALUE;
    const int64_t e = (int64_t)elem(io), nh = (int64_t)N * H, nk = (int64_t)N * Hk;
    const Range in[] = {{q, nk * K * e}, {k, nk * K * e}, {v, nh * V * e}, {g, per_head ? (int64_t)H * 4 : nh * e}};
    const Range out[] = {{S, nh * K * V * 4}, {o, nh * V * e}};
    if (clash(out, in)) return KDA_ERROR_INVALID_VALUE;
    const kda_status_t st = check_device();
    if (st != KDA_SUCCESS) return st;
    kda::HdDecodeArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = g; a.S = S; a.o = o;
    a.N = N; a.H = H; a.Hk = Hk; a.K = K; a.V = V;
    a.io_bf16 = io == KDA_DTYPE_BF16;
    a.decay_per_head = per_head;
    a.scale = scale;
    return launched(kda::launch_hd_decode(a, reinterpret_cast<hipStream_t>(stream)));
}

kda_status_t kda_rotary(const void *q, const void *k, const double *freqs, const int32_t *positions, void *q_out,
                        void *k_out, int64_t tokens, int64_t T, int32_t Hq, int32_t Hk, int32_t D, int32_t R,
                        kda_dtype_t io, kda_rotary_layout_t layout, int32_t inverse, float scale, void *stream) {
    if (!valid_io(io) || (layout != KDA_ROTARY_HALF && layout != KDA_ROTARY_INTERLEAVED) || !std::isfinite(scale))
        return KDA_ERROR_INVALID_VALUE;
    if (inverse != 0 && inverse != 1) return KDA_ERROR_INVALID_VALUE;
    if (tokens < 0 || Hq < 1 || Hk < 0 || D < 2 || R < 2 || R > D || R % 2 != 0) return KDA_ERROR_INVALID_VALUE;
    if (!positions && T < 1 && tokens > 0) return KDA_ERROR_INVALID_VALUE;
    if (D > 512) return KDA_ERROR_NOT_SUPPORTED;
    if ((int64_t)Hq + Hk > (1 << 20) || tokens > kMaxElems / ((int64_t)Hq + Hk) / D) return KDA_ERROR_INVALID_VALUE;
    if (tokens == 0) return KDA_SUCCESS;
    if (!q || !q_out || !freqs || (Hk > 0 && (!k || !k_out))) return KDA_ERROR_INVALID_VALUE;
    if (Hk == 0) k = k_out = nullptr;
    for (const void *p : {q, k, (const void *)q_out, (const void *)k_out})
        if (!aligned(p, 16)) return KDA_ERROR_INVALID_VALUE;
    if (!aligned(freqs, 8) || !aligned(positions, 4)) return KDA_ERROR_INVALID_VALUE;
    const int64_t e = (int64_t)elem(io), nq = tokens * Hq * D * e, nk = tokens * Hk * D * e;
    // q_out may be q and k_out may be k; nothing else that is written may meet anything
    const Range in[] = {{q == q_out ? nullptr : q, nq}, {k == k_out ? nullptr : k, nk}, {freqs, (int64_t)R / 2 * 8},
                        {positions, tokens * 4}};
    const Range out[] = {{q_out, nq}, {k_out, nk}};
    if (clash(out, in)) return KDA_ERROR_INVALID_VALUE;
    const kda_status_t st = check_device();
    if (st != KDA_SUCCESS) return st;
    kda::RotaryArgs a{};
    a.q = q; a.k = k; a.q_out = q_out; a.k_out = k_out; a.freqs = freqs; a.positions = positions;
    a.tokens = tokens;
    a.T = T > 0 && T < tokens ? T : tokens;  // a period past the last token changes nothing (and is 32-bit if tokens are)
    a.Hq = Hq; a.Hk = Hk; a.D = D; a.R = R;
    a.io_bf16 = io == KDA_DTYPE_BF16;
    a.interleaved = layout == KDA_ROTARY_INTERLEAVED;
    a.inverse = inverse != 0;
    a.scale = scale;
    return launched(kda::launch_rotary(a, reinterpret_cast<hipStream_t>(stream)));
}

static kda_status_t check_norm_sizes(int64_t rows, int32_t groups, int32_t C) {
    if (rows < 0 || groups < 1 || C < 1 || rows % groups != 0) return KDA_ERROR_INVALID_VALUE;
    if (C > 16384) return KDA_ERROR_NOT_SUPPORTED;
    // a workgroup of 1024 threads for 64 parameters: a grid's threads are 32-bit
    if (rows > kMaxElems / C || (int64_t)groups * C > (1 << 27)) return KDA_ERROR_INVALID_VALUE;
    if (!kda::norm_grid_fits(rows, groups, C)) return KDA_ERROR_INVALID_VALUE;
    return KDA_SUCCESS;
}

kda_status_t kda_layer_norm_fwd(const void *x, const float *weight, const float *bias, const void *o_gate, void *y,
                                int64_t rows, int32_t groups, int32_t C, float eps, int32_t center, kda_dtype_t io,
                                void *stream) {
    if (!valid_io(io) || !(eps > 0.f) || !std::isfinite(eps) || (center != 0 && center != 1))
        return KDA_ERROR_INVALID_VALUE;
    kda_status_t st = check_norm_sizes(rows, groups, C);
    if (st != KDA_SUCCESS) return st;
    if (rows == 0) return KDA_SUCCESS;
    if (!x || !y) return KDA_ERROR_INVALID_VALUE;
    for (const void *p : {x, (const void *)weight, (const void *)bias, o_gate, (const void *)y})
        if (!aligned(p, 16)) return KDA_ERROR_INVALID_VALUE;
    const int64_t n = rows * C * (int64_t)elem(io), w = (int64_t)groups * C * 4;
    const Range in[] = {{x, n}, {weight, w}, {bias, w}, {o_gate, n}};
    const Range out[] = {{y, n}};
    if (clash(out, in)) return KDA_ERROR_INVALID_VALUE;
    st = check_device();
    if (st != KDA_SUCCESS) return st;
    kda::NormArgs a{};
    a.x = x; a.gate = o_gate; a.weight = weight; a.bias = bias; a.y = y;
    a.rows = rows; a.G = groups; a.C = C; a.eps = eps;
    a.io_bf16 = io == KDA_DTYPE_BF16;
    a.center = center != 0;
    return launched(kda::launch_norm_fwd(a, reinterpret_cast<hipStream_t>(stream)));
}

size_t kda_layer_norm_bwd_workspace_bytes(int64_t rows, int32_t groups, int32_t C) {
    if (check_norm_sizes(rows, groups, C) != KDA_SUCCESS) return 0;
    const size_t n = kda::norm_bwd_workspace_bytes(rows, groups, C);
    return n ? n : 16;
}

kda_status_t kda_layer_norm_bwd(const void *dy, const void *x, const float *weight, const float *bias,
                                const void *o_gate, void *dx, float *dweight, float *dbias, void *d_o_gate,
                                int64_t rows, int32_t groups, int32_t C, float eps, int32_t center, kda_dtype_t io,
                                void *workspace, size_t workspace_bytes, void *stream) {
    if (!valid_io(io) || !(eps > 0.f) || !std::isfinite(eps) || (center != 0 && center != 1))
        return KDA_ERROR_INVALID_VALUE;
    kda_status_t st = check_norm_sizes(rows, groups, C);
    if (st != KDA_SUCCESS) return st;
    if (rows > 0 && (!dy || !x || !dx || (o_gate && !d_o_gate))) return KDA_ERROR_INVALID_VALUE;
    if (!o_gate) d_o_gate = nullptr;
    for (const void *p : {dy, x, (const void *)weight, (const void *)bias, o_gate, (const void *)dx,
                          (const void *)dweight, (const void *)dbias, (const void *)d_o_gate, (const void *)workspace})
        if (!aligned(p, 16)) return KDA_ERROR_INVALID_VALUE;
    const size_t need = kda_layer_norm_bwd_workspace_bytes(rows, groups, C);
    const int64_t n = rows * C * (int64_t)elem(io), w = (int64_t)groups * C * 4;
    const Range in[] = {{dy, n}, {x, n}, {weight, w}, {bias, w}, {o_gate, n}};
    const Range out[] = {{dx, n}, {dweight, w}, {dbias, w}, {d_o_gate, n}, {workspace, (int64_t)need}};
    if (clash(out, in)) return KDA_ERROR_INVALID_VALUE;
    if (!workspace || workspace_bytes < need) return KDA_ERROR_WORKSPACE_TOO_SMALL;
    st = check_device();
    if (st != KDA_SUCCESS) return st;
    kda::NormArgs a{};
    a.x = x; a.gate = o_gate; a.weight = weight; a.bias = bias;
    a.rows = rows; a.G = groups; a.C = C; a.eps = eps;
    a.io_bf16 = io == KDA_DTYPE_BF16;
    a.center = center != 0;
    a.dy = dy; a.dx = dx; a.dgate = d_o_gate; a.dweight = dweight; a.dbias = dbias; a.workspace = workspace;
    return launched(kda::launch_norm_bwd(a, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
