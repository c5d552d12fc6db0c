// Host-side launch interface between the layer operators' C ABI (kda_layer_api.hip) and their kernel translation
// units: linear attention with one decay per head (hd), rotary positions, layer norm. Internal to the library.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

// ------------------------------------------------------- linear attention with one decay per head
struct HdArgs {
    const void *q, *k, *v;     // q, k [B,T,Hk,K]; v [B,T,H,V]
    const void *g;             // [B,T,H] in the I/O dtype, or [H] fp32 (decay_per_head)
    const float *S0;           // [N,H,K,V] or null
    const int32_t *cu_seqlens;
    int64_t B, T;
    int32_t H, Hk, K, V, num_seqs;
    bool io_bf16, decay_per_head;
    float scale;
    void *o;
    float *S_final;            // or null
    // backward only
    const void *dout;          // dL/do [B,T,H,V]
    const float *dS_final;     // or null
    void *dq, *dk, *dv, *dg;   // I/O dtype; dg null: not wanted
    float *dS0;                // or null
    void *workspace;
};
size_t hd_fwd_workspace_bytes(int64_t B, int64_t T, int32_t H, int32_t Hk, int32_t K, int32_t V, int32_t num_seqs,
                              bool packed, bool io_bf16);
size_t hd_bwd_workspace_bytes(int64_t B, int64_t T, int32_t H, int32_t Hk, int32_t K, int32_t V, int32_t num_seqs,
                              bool packed, bool io_bf16);
hipError_t launch_hd_fwd(const HdArgs &a, hipStream_t st);
hipError_t launch_hd_bwd(const HdArgs &a, hipStream_t st);

struct HdDecodeArgs {
    const void *q, *k, *v, *g;
    float *S;
    void *o;
    int32_t N, H, Hk, K, V;
    bool io_bf16, decay_per_head;
    float scale;
};
hipError_t launch_hd_decode(const HdDecodeArgs &a, hipStream_t st);

// ------------------------------------------------------- rotary positions
struct RotaryArgs {
    const void *q, *k;         // [tokens, Hq, D], [tokens, Hk, D] (k or null with Hk = 0)
    void *q_out, *k_out;
    const double *freqs;       // [R / 2] radians per position
    const int32_t *positions;  // [tokens], or null: token index modulo T; with axes [naxes, tokens]
    const int32_t *axes;       // [R / 2] the axis whose position turns a pair, or null: one axis
    int32_t naxes;
    int64_t tokens, T;         // 1 <= T <= tokens
    int32_t Hq, Hk, D, R;
    bool io_bf16, interleaved, inverse;
    float scale;
};
hipError_t launch_rotary(const RotaryArgs &a, hipStream_t st);

// ------------------------------------------------------- layer norm
struct NormArgs {
    const void *x, *gate;      // [rows, C]; gate pre-activation [rows, C] or null
    const int8_t *codes;       // backward: x out of a checkpoint (x null), [rows, C] and [rows, ceil(C / 128)]
    const float *scales;
    const float *weight, *bias;  // [G, C] or null
    void *y;
    int64_t rows;
    int32_t G, C;
    float eps;
    bool io_bf16, center;
    // backward only
    const void *dy;
    void *dx, *dgate;
    float *dweight, *dbias;
    void *workspace;
};
bool norm_grid_fits(int64_t rows, int32_t G, int32_t C);  // a grid's threads are 32-bit (many groups of narrow rows)
size_t norm_bwd_workspace_bytes(int64_t rows, int32_t G, int32_t C);
hipError_t launch_norm_fwd(const NormArgs &a, hipStream_t st);
hipError_t launch_norm_bwd(const NormArgs &a, hipStream_t st);

// ------------------------------------------------------- activation checkpoints in 8 bits
constexpr int32_t kCkptBlock = 128;  // values along a row that share a step
struct CkptArgs {
    void *x;                   // [rows, C]
    int8_t *codes;             // [rows, C]
    float *scales;              // [rows, ceil(C / 128)]
    int64_t rows;
    int32_t C;
    bool io_bf16;
};
hipError_t launch_ckpt_save(const CkptArgs &a, hipStream_t st);
hipError_t launch_ckpt_restore(const CkptArgs &a, hipStream_t st);

}  // namespace kda
