// The gated delta rule with one decay per head: what its translation units share. Internal to the library.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

struct GdArgs {
    const void *q, *k, *v;     // q, k [B,T,Hk,K]; v [B,T,H,V]
    const void *g, *beta;      // [B,T,H] in the I/O dtype, or fp32 (gates_fp32)
    const float *S0;           // [N,H,K,V] or null
    const int32_t *cu_seqlens;
    int64_t B, T;
    int32_t H, Hk, K, V, num_seqs;
    bool io_bf16, gates_fp32;
    float scale;
    void *o;
    float *S_final;            // or null
    // backward only
    const void *dout;          // dL/do [B,T,H,V]
    const float *dS_final;     // or null
    void *dq, *dk, *dv;        // I/O dtype
    void *dg, *dbeta;          // the gates' dtype
    float *dS0;                // or null
    void *workspace;
};
size_t gd_fwd_workspace_bytes(int64_t B, int64_t T, int32_t H, int32_t Hk, int32_t K, int32_t V, int32_t num_seqs,
                              bool packed, bool io_bf16);
size_t gd_bwd_workspace_bytes(int64_t B, int64_t T, int32_t H, int32_t Hk, int32_t K, int32_t V, int32_t num_seqs,
                              bool packed, bool io_bf16);  // for gates of either type
hipError_t launch_gd_fwd(const GdArgs &a, hipStream_t st);
hipError_t launch_gd_bwd(const GdArgs &a, hipStream_t st);

struct GdDecodeArgs {
    const void *q, *k, *v, *g, *beta;
    float *S;
    void *o;
    int32_t N, H, Hk, K, V;
    bool io_bf16, gates_fp32;
    float scale;
};
hipError_t launch_gd_decode(const GdDecodeArgs &a, hipStream_t st);

namespace gd {

constexpr int kChunkTokens = 32;
// Chunks of a workgroup of the gradients' kernel: a power of two from 2 up to this (Common::seg).
constexpr int segment_most(int K) { return K == 128 ? 16 : 8; }

// A sequence: its tokens in the flattened [B * T], the number of its first chunk and of its first segment among all, and that
// of its first border between two segments.
struct Seq {
    int64_t t0, t1, first, seg, border;
};
// The same of a packed sequence, in the workspace: 32 bytes (fewer than 2^31 tokens in all, and 2^26 sequences).
struct Packed {
    int64_t t0, t1, first;
    int32_t seg, border;
};

// A chunk's record, made once per (chunk, head) and read by the passes over the states. Matrices lie in the order in
// which a wavefront's lanes read them as operands: [16-row tile][half][lane][16 bytes], the halves a bf16 pair's parts
// or the first and last four of eight fp32 slots.
enum Mat { kMatN = 0, kMatP = 1, kMatNT = 1, kMatPT = 2 };  // forward: N, P; backward: N, its transpose, P's
constexpr int kMatBytes = 4096, kThirdBytes = 2048;
enum Weight { kEnter, kEnterScaled, kLeave, kLeaveBeta, kBeta, kSumHi, kSumLo, kTotal, kWeights };
constexpr int rec_bytes(bool bwd) { return (bwd ? 3 : 2) * kMatBytes + kWeights * kChunkTokens * 4; }
constexpr int rec_weights(bool bwd) { return (bwd ? 3 : 2) * kMatBytes; }

struct Common {
    const Packed *seqs;   // or null: rows of T tokens
    const int32_t *order;  // the sequences in the order of their workgroups, or null
    int64_t T, ntok, slots, segs;  // slots, segs: chunks and segments of all sequences (upper bounds when packed)
    int32_t nch, nseg;  // per row (not packed)
    int32_t seg;        // chunks of a segment
    int32_t N, H, Hk;
    char *rec;          // [slots][H] records
    char *third;        // backward, bf16 I/O beside fp32 gates: third parts of the records' matrices, in their order; or null
};

struct StateArgs {
    Common c;
    const void *q, *k, *v;   // v: the rows of V channels (backward: dL/do)
    const float *s_init;     // the state before the first chunk (reverse: its gradient behind the last), or null
    float *s_end;            // at the other end, or null
    void *o;                 // forward: [B,T,H,V]; reverse: dv
    char *rows;              // backward: [slots][H] tiles of [V][32]: the errors z, or the writes' gradients
    int32_t parts;           // of a tile's values, bf16 I/O: 2, or 3 for all their bits
    float *seed;             // backward: states at the borders between segments [borders][H][K][V]
    int32_t tiles;           // column tiles
};

struct GradArgs {
    Common c;
    const void *q, *k, *dout;
    const char *z, *dw;      // tiles of [V][32] per (chunk, head)
    const float *S0, *dS_final, *seed_s, *seed_g;
    void *dq, *dk;           // I/O dtype, or fp32 per v head
    float *dk_part;          // [B,T,H,K]: what the walk forward adds to dk
    void *dg, *dbeta;
    float scale;
};

enum Mode { kForward, kErrors, kReverse };  // outputs; the errors and states for the gradients; the state's gradients
hipError_t forward_pass(bool bf16, const StateArgs &a, int K, int V, hipStream_t st);
hipError_t backward_passes(bool bf16, const StateArgs &reverse, StateArgs errors, int K, int V, hipStream_t st);
hipError_t grad_pass_bf16(const GradArgs &a, int K, int V, bool y_fp32, hipStream_t st);
hipError_t grad_pass_bf16_gates_fp32(const GradArgs &a, int K, int V, bool y_fp32, hipStream_t st);
hipError_t grad_pass_fp32(const GradArgs &a, int K, int V, hipStream_t st);

#ifdef __HIPCC__
__device__ __forceinline__ Seq seq_of(const Common &c, int64_t n) {
    if (c.seqs) {
        const Packed p = c.seqs[n];
        return Seq{p.t0, p.t1, p.first, p.seg, p.border};
    }
    return Seq{n * c.T, (n + 1) * c.T, n * c.nch, n * c.nseg, n * (c.nseg - 1)};
}
// The last sequence whose first chunk (segment) is at most `slot`, by 64 entries at a time. One wavefront, all lanes.
template <bool SEG>
__device__ __forceinline__ int64_t find_seq(const Common &c, int64_t slot, int lane) {
    if (!c.seqs) return slot / (SEG ? c.nseg : c.nch);
    int64_t lo = 0, len = c.N;
    while (true) {
        const int64_t step = (len + 63) / 64, i = lo + lane * step;
        const bool at_most = i < lo + len && (SEG ? c.seqs[i].seg : c.seqs[i].first) <= slot;
        const int n = __builtin_popcountll(__builtin_amdgcn_ballot_w64(at_most));  // the entries do not decrease
        if (n == 0) return lo;
        const int64_t end = lo + len;
        lo += (n - 1) * step;
        if (step == 1) return lo;
        len = end - lo < step ? end - lo : step;
    }
}
#endif

}  // namespace gd
}  // namespace kda
