// Linear attention with one decay per head: what its translation units share (segments, the chunk kernel's arguments).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda_layer.hpp"

namespace kda {
namespace hd {

// A sequence is cut into segments of `seg` tokens (a multiple of 64) that run as workgroups of their own. Slot i of a
// batch is segment i % nseg of row i / nseg; of packed sequences, entry i of a table that a first kernel makes from
// cu_seqlens (slots behind the last segment have seq -1). An empty sequence is one empty segment.
struct Segment {
    int32_t seq, j, nseg, pad;
    int64_t t0, t1;  // tokens of the flattened [B * T]
};

struct CoreArgs {
    const void *a, *b, *c;      // rows [B*T, H / g?, KD | KD | VD]
    int32_t ga, gb, gc;         // heads that share a row of a, b, c
    int32_t H, VD, tiles;       // heads; columns of c and y; tiles of VT columns
    int32_t share;              // adjacent heads whose workgroups are placed together
    void *y;                    // [B*T, H, VD]
    bool g_head;
    const void *g;              // [B*T, H] I/O type, or [H] fp32 (g_head)
    const float *s_init;        // state before the first segment (REV: after the last), or null
    const float *s_seg;         // states the other segments start from, per slot and head; of sequences of up to `fold`
    int32_t fold;               //   segments: what each adds
    float *s_out;               // state after the last segment (REV: before the first), or null
    float *s_inc;               // what a segment adds (the increment passes), per slot and head
    float *seg_decay;           // log2 of a segment's decay, per slot and head
    const Segment *table;       // or null: rows of T tokens
    int64_t slots, T, seg, ntok;
    int32_t nseg;
    float s_intra, s_inter, s_up;
    // the log-decays' gradient
    const void *x;              // rows [B*T, H / gx, VD] that y is multiplied with
    int32_t gx;
    float *part;                // [tiles][H][B*T]: a token's part, from these columns
    float *border;              // [tiles][slots][H]: <state gradient, state> behind a segment, from these columns
    const float *s_seg_fwd;     // the forward states the segments start from
};
struct GradArgs {
    CoreArgs dv, dk, dq;
};

#ifdef __HIPCC__
__device__ __forceinline__ Segment segment_of(const CoreArgs &A, int64_t slot) {
    if (A.table) return A.table[slot];
    Segment s;
    s.seq = (int32_t)(slot / A.nseg);
    s.j = (int32_t)(slot - (int64_t)s.seq * A.nseg);
    s.nseg = A.nseg;
    s.pad = 0;
    const int64_t row = (int64_t)s.seq * A.T, e = (int64_t)(s.j + 1) * A.seg;
    s.t0 = row + (int64_t)s.j * A.seg;
    s.t1 = row + (e < A.T ? e : A.T);
    return s;
}
#endif

// Columns of a tile: of the forward pass and the gradients (whose three workgroups have one size), of the increments
// (no weighted products to share, only the rows b: narrower tiles, more workgroups).
constexpr int fwd_tile(int V, bool bf16) { return bf16 || V < 64 ? V : 64; }
constexpr int grad_tile(int K, int V, bool bf16) { return fwd_tile(K < V ? K : V, bf16); }
constexpr int inc_tile(int V) { return V < 64 ? V : 64; }

// A grid of n workgroups (at least; under 2^32): a dimension's threads are 32-bit, and 2^20 workgroups of 1024 are within.
inline dim3 wide_grid(int64_t n) {
    const int64_t x = (int64_t)1 << 20;
    return n <= x ? dim3((uint32_t)n) : dim3((uint32_t)x, (uint32_t)((n + x - 1) / x));
}

// The passes. inc_pass: the increments of the states, and with r those of their gradients.
hipError_t fwd_pass(bool bf16, const CoreArgs &a, int K, int vt, hipStream_t st);
hipError_t inc_pass(bool bf16, const CoreArgs &f, const CoreArgs *r, int K, int vt, hipStream_t st);
hipError_t grad_pass_bf16(const GradArgs &g, int K, int V, bool dg, bool y_fp32, hipStream_t st);
hipError_t grad_pass_fp32(const GradArgs &g, int K, int V, bool dg, hipStream_t st);

}  // namespace hd
}  // namespace kda
