// Linear attention with one decay per head: segments, the pass that carries states over them, and the order of the
// chunk kernel's passes (kda_hd_core.hpp) in a forward or backward call.
//
// A call whose heads and column tiles do not fill the chip cuts its sequences into segments. A first pass forms what
// each segment adds to a zero state (and its total decay), a second carries the states over the segments (few segments
// of the forward pass: their workgroups do), and then every segment runs as if it were a sequence of its own. The
// backward does the same for the states' gradients, from the other end.
#include "kda_hd.hpp"

#include <cmath>

#include "kda_common.hpp"

namespace kda {
namespace hd {
namespace {

constexpr int64_t kLeastSegment = 128;
// Where a sequence has up to this many segments, a workgroup of the forward pass reads what the segments before its own
// add and forms the state that it starts from (4096 tokens of 96 heads, 5 segments: 157 -> 150 us). With more that would
// be too many reads, half the segments' states on average, and a pass of its own carries the states over them first. So
// it does for the gradients, where three workgroups would form each state (478 us either way).
constexpr int32_t kFold = 8;

struct Plan {
    int64_t seg;        // tokens per segment
    int32_t nseg;       // segments per row (not packed)
    int64_t slots;      // workgroups' slots: an upper bound when packed
    bool several;       // some sequence may have more than one segment
    int32_t fold;       // sequences of up to so many segments: workgroups form the states they start from themselves
};

int64_t round64(int64_t x) { return (x + 63) / 64 * 64; }

// How long a call with n segments per row takes, in ns as measured at K = V = 128 in bf16: the main pass's rounds over
// the workgroups that the chip holds (a token of the forward pass takes 110 ns, of the gradients 160; three quarters of
// that where no two share a CU); with several segments also the increments' rounds (80 ns), the states' traffic (50 ns
// per head and segment, twice for the gradients) and two more launches. (The forward pass's 110 is of the state read in one
// part; with the 13% more of two parts 2% of random sizes would be cut otherwise, by the model for 3% of their time.)
int64_t cost(int64_t rows, int64_t inc_rows, int64_t heads, int64_t resident, int64_t T, int64_t n, bool bwd) {
    const int64_t seg = round64((T + n - 1) / n), groups = rows * n;
    int64_t c = (groups + resident - 1) / resident * seg * (bwd ? 160 : 110);
    if (groups <= 256) c = c * 3 / 4;
    if (n > 1) c += (inc_rows * (n - 1) + 1023) / 1024 * seg * 80 + heads * n * (bwd ? 100 : 50) + 12000;
    return c;
}

// The same for N packed sequences of T tokens in all, whose lengths the host does not know. They are taken for what N - 1
// random cuts make of T: the longest is ln N + 0.6 times the average, N / (1 - e^(-seg / average)) segments of at most
// `seg` tokens. A workgroup's token takes `alone` ns where it has a CU to itself, and the longest segment that many; all
// together take what the chip's CUs can do. `scale`: percent of the times measured at K = V = 128 in bf16. Against a model
// that takes one sequence for nearly all of the batch: 1531 tokens of 5 sequences, 12 heads, fp32: gradients 99 -> 81 us;
// 6000 of 3, 8 heads, fp32: forward 115 -> 86; 50000 of 64, 96 heads: 1363 -> 1303; 8000 of 5, 32 heads: 130 -> 117.
int64_t packed_cost(int64_t T, int64_t N, int64_t H, int64_t tiles, int64_t inc_tiles, int64_t resident, int64_t seg,
                    int64_t longest, int64_t scale, int64_t state, bool bwd) {
    const int64_t segs = seg < longest ? (int64_t)(N / (1.0 - std::exp(-(double)seg * N / (T > 0 ? T : 1)))) : N;
    const int64_t groups = H * tiles * segs;
    const int64_t alone = (bwd ? 100 : 62) * scale / 100, shared = (bwd ? 160 : 110) * scale / 100;
    const int64_t more = groups <= 256 ? 0 : groups < resident ? groups - 256 : resident - 256;  // that share a CU
    const int64_t lone = seg * (alone + (shared - alone) * more / (resident - 256));
    const int64_t all = H * tiles * T / 256 * shared / 2 + (groups > resident ? lone / 4 : 0);
    int64_t c = lone > all ? lone : all;
    if (segs > N) {  // increments of all but the last segments
        const int64_t one = seg * 40, inc = (int64_t)((double)(H * inc_tiles * T / 256) * (segs - N) / segs * 20);
        c += (one > inc ? one : inc) * scale / 100 + H * segs * (bwd ? 100 : 50) * state / 16384 + 12000;
    }
    return c;
}

Plan plan(int64_t B, int64_t T, int32_t H, int32_t K, int32_t V, int32_t N, bool packed, bool bf16, bool bwd) {
    Plan p;
    const int64_t whole = round64(T > 0 ? T : 1);
    const int vt = bwd ? grad_tile(K, V, bf16) : fwd_tile(V, bf16);
    const int64_t tiles = bwd ? 2 * (K / vt) + V / vt : V / vt, inc_tiles = V / inc_tile(V) * (bwd ? 2 : 1);
    const int64_t resident = vt == 128 || bwd ? 512 : 768;
    if (packed) {
        // A batch that needs no segments still gets them, at the longest length to be expected or as much as one workgroup
        // does while the chip does all of the batch: one long sequence among short ones would otherwise run on alone (a
        // launch that finds nothing costs 2 to 7%).
        const int64_t likely = round64((int64_t)((std::log((double)N) + 0.6) * T / N) + 1);
        const int64_t longest = N > 1 && likely < whole ? likely : whole;
        const int64_t scale = bf16 ? (vt == 128 ? 100 : 75) : 180 * (bwd && V > K ? V : K) / 128;
        const int64_t meanwhile = H * tiles * T / 256 * 4 / 5;
        p.seg = round64(meanwhile > longest ? (meanwhile < whole ? meanwhile : whole) : longest);
        int64_t least = packed_cost(T, N, H, tiles, inc_tiles, resident, longest, longest, scale, (int64_t)K * V, bwd);
        for (int64_t n = 2; longest / n >= kLeastSegment && H * tiles * n < 4 * resident; ++n) {
            const int64_t seg = round64((longest + n - 1) / n);
            const int64_t c = packed_cost(T, N, H, tiles, inc_tiles, resident, seg, longest, scale, (int64_t)K * V, bwd);
            if (c < least) p.seg = seg, least = c;
        }
        p.nseg = (int32_t)(T > 0 ? (T + p.seg - 1) / p.seg : 1);
        p.slots = T / p.seg + N;
    } else {
        const int64_t heads = B * H, rows = heads * tiles;
        int64_t best = 1, least = cost(rows, heads * inc_tiles, heads, resident, whole, 1, bwd);
        for (int64_t n = 2; n <= whole / kLeastSegment && rows * (n - 1) < 4 * resident; ++n) {
            const int64_t c = cost(rows, heads * inc_tiles, heads, resident, whole, n, bwd);
            if (c < least) best = n, least = c;
        }
        p.seg = round64((whole + best - 1) / best);
        p.nseg = (int32_t)(T > 0 ? (T + p.seg - 1) / p.seg : 1);
        p.slots = B * p.nseg;
    }
    p.several = p.nseg > 1;
    p.fold = bwd ? 0 : kFold;
    return p;
}

// ------------------------------------------------------------------ segments of packed sequences
struct SeqSlots { int32_t first, count; };

// One workgroup: clamps cu_seqlens into [0, T] and makes it non-decreasing (a running maximum), numbers the segments.
// Both are scans over the sequences, 1024 at a time: within a wavefront by lanes, over its 16 wavefronts through LDS.
// T < 2^31, so tokens are 32-bit here.
__global__ __launch_bounds__(1024) void kda_hd_table_kernel(const int32_t *__restrict__ cu, int32_t N, uint32_t T,
                                                            uint32_t seg, int64_t slots, Segment *__restrict__ table,
                                                            SeqSlots *__restrict__ seqs, int64_t *__restrict__ covered) {
    __shared__ uint32_t s_max[2][16], s_sum[2][16];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    auto entry = [&](int64_t i) -> uint32_t {
        const int32_t x = cu[i];
        return x < 0 ? 0 : (uint32_t)x > T ? T : (uint32_t)x;
    };
    uint32_t top = entry(0), first = 0;
    if (t == 0) covered[0] = top;
    int turn = 0;
    for (int64_t base = 0; base < N; base += 1024, turn ^= 1) {
        const int64_t n = base + t;
        uint32_t end = n < N ? entry(n + 1) : 0;
        if (end < top) end = top;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t x = __shfl_up(end, d);
            if (lane >= d && x > end) end = x;
        }
        uint32_t before = __shfl_up(end, 1);
        if (lane == 0) before = top;
        if (lane == 63) s_max[turn][wave] = end;
        __syncthreads();
        for (int w = 0; w < 16; ++w) {
            const uint32_t x = s_max[turn][w];
            if (w < wave && x > end) end = x;
            if (w < wave && x > before) before = x;
            if (x > top) top = x;
        }
        const uint32_t segs = (end - before + (seg - 1)) / seg;  // under 2^32: seg <= 2^31
        const uint32_t count = n < N ? (segs > 1 ? segs : 1) : 0;
        uint32_t upto = count;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t x = __shfl_up(upto, d);
            if (lane >= d) upto += x;
        }
        if (lane == 63) s_sum[turn][wave] = upto;
        __syncthreads();
        uint32_t all = 0;
        for (int w = 0; w < 16; ++w) {
            const uint32_t x = s_sum[turn][w];
            if (w < wave) upto += x;
            all += x;
        }
        if (n < N) {
            const uint32_t at = first + upto - count;
            seqs[n] = SeqSlots{(int32_t)at, (int32_t)count};
            // equal parts (at most `seg`, so none is empty): workgroups of one length
            const int64_t part = (int64_t)(((end - before + (count - 1)) / count + 63) / 64) * 64;
            for (uint32_t j = 0; j < count; ++j) {
                const int64_t a = before + j * part, e = a + part;
                table[at + j] = Segment{(int32_t)n, (int32_t)j, (int32_t)count, 0, a, e < end ? e : (int64_t)end};
            }
        }
        first += all;
    }
    for (int64_t i = (int64_t)first + t; i < slots; i += 1024) table[i] = Segment{-1, 0, 0, 0, 0, 0};
    if (t == 0) covered[1] = top;
}

// ------------------------------------------------------------------ states over the segments
struct CarryArgs {
    float *seg;
    const float *decay, *init;
};
// In place: what each segment adds becomes the state it starts from (rev: the state gradient it ends with). A thread
// carries four adjacent state entries over the segments of its sequence, if they are more than `fold`.
__global__ __launch_bounds__(256) void kda_hd_carry_kernel(const CarryArgs F, const CarryArgs R,
                                                           const SeqSlots *__restrict__ seqs, int32_t N, int32_t nseg,
                                                           int32_t fold, int32_t H, int64_t kv4) {
    const int rev = blockIdx.z;
    float *seg = rev ? R.seg : F.seg;
    const float *decay = rev ? R.decay : F.decay, *init = rev ? R.init : F.init;
    const int64_t blk = blockIdx.x + (int64_t)blockIdx.y * gridDim.x;
    const int64_t runs = (kv4 + 255) / 256, nh = blk / runs, n = nh / H;
    const int64_t e = (blk - nh * runs) * 256 + threadIdx.x;
    if (e >= kv4 || n >= N) return;
    const int h = (int)(nh - n * H);
    const int32_t first = seqs ? seqs[n].first : (int32_t)(n * nseg), count = seqs ? seqs[n].count : nseg;
    if (count <= fold) return;
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
    if (init) s = reinterpret_cast<const f32x4 *>(init)[nh * kv4 + e];
#pragma unroll 4
    for (int32_t i = 0; i + 1 < count; ++i) {
        const int64_t slot = (int64_t)first + (rev ? count - 1 - i : i);
        f32x4 *p = reinterpret_cast<f32x4 *>(seg) + (slot * H + h) * kv4 + e;
        const f32x4 add = *p;
        const float d = __builtin_amdgcn_exp2f(decay[slot * H + h]);
        if (i > 0) *p = s;
        s = s * d + add;
    }
    if (count > 1) {
        const int64_t slot = (int64_t)first + (rev ? 0 : count - 1);
        (reinterpret_cast<f32x4 *>(seg) + (slot * H + h) * kv4 + e)[0] = s;
    }
}

hipError_t launch_carry(const CarryArgs &f, const CarryArgs *r, const SeqSlots *seqs, const Plan &p, const HdArgs &a,
                        hipStream_t st) {
    const int64_t kv4 = (int64_t)a.K * a.V / 4, nh = (int64_t)a.num_seqs * a.H;
    dim3 grid = wide_grid(nh * ((kv4 + 255) / 256));
    if (r) grid.z = 2;
    hipLaunchKernelGGL(kda_hd_carry_kernel, grid, dim3(256), 0, st, f, r ? *r : f, seqs, a.num_seqs, p.nseg, p.fold, a.H,
                       kv4);
    return hipGetLastError();
}

// ------------------------------------------------------------------ the gradients' last steps
// dg_t = what passes the border behind t's segment + sum over the tokens from t to there of their parts (rows' sums
// less columns' sums of the pairs, and the states' shares). A workgroup takes two heads of a segment, from its end in
// steps of 512 tokens: a wavefront sums 64 of them, then the totals of the wavefronts behind it are added.
template <bool BF>
__global__ __launch_bounds__(1024) void kda_hd_dg_kernel(const CoreArgs A, const float *__restrict__ part_q, int tiles_q,
                                                         int K, const float *__restrict__ dS, const float *__restrict__ s_end,
                                                         void *__restrict__ dg) {
    __shared__ float s_total[2][2][8];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, hsub = wave >> 3, blk = wave & 7;
    const int h = blockIdx.z * 2 + hsub;
    const int64_t slot = blockIdx.x + (int64_t)blockIdx.y * gridDim.x;
    if (slot >= A.slots) return;
    const Segment sg = segment_of(A, slot);
    if (sg.seq < 0 || sg.t1 <= sg.t0) return;
    const bool live = h < A.H;
    double behind = 0.0;
    if (sg.j == sg.nseg - 1 && dS) {  // uniform: behind the last segment the final state's
        float dot = 0.f;
        if (live) {
            const int64_t kv4 = (int64_t)K * A.VD / 4, at = ((int64_t)sg.seq * A.H + h) * kv4;
            const f32x4 *x = reinterpret_cast<const f32x4 *>(dS) + at, *y = reinterpret_cast<const f32x4 *>(s_end) + at;
#pragma unroll 4
            for (int64_t i = blk * 64 + lane; i < kv4; i += 512) {
                const f32x4 z = x[i] * y[i];
                dot += (z.x + z.y) + (z.z + z.w);
            }
        }
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) dot += __shfl_xor(dot, d);
        if (lane == 0) s_total[0][hsub][blk] = dot;
        __syncthreads();
        for (int w = 0; w < 8; ++w) behind += s_total[0][hsub][w];
        __syncthreads();
    }
    if (live)
        for (int w = 0; w < A.tiles; ++w) behind += A.border[((int64_t)w * A.slots + slot) * A.H + h];
    const int64_t plane = (int64_t)A.H * A.ntok, steps = (sg.t1 - sg.t0 + 511) / 512;
    auto take = [&](int64_t b) {
        const int64_t t = sg.t0 + b * 512 + blk * 64 + lane, at = (int64_t)h * A.ntok + t;
        float x = 0.f;
        if (b >= 0 && live && t < sg.t1) {
            for (int w = 0; w < A.tiles; ++w) x += A.part[w * plane + at];
            for (int w = 0; w < tiles_q; ++w) x += part_q[w * plane + at];
        }
        return x;
    };
    float next = take(steps - 1);
    for (int64_t b = steps - 1; b >= 0; --b) {
        float x = next;
        next = take(b - 1);
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const float y = __shfl_down(x, d);
            if (lane + d < 64) x += y;
        }
        float(*const total)[8] = s_total[b & 1];
        if (lane == 0) total[hsub][blk] = x;
        __syncthreads();
        double later = behind;
        for (int w = 7; w > blk; --w) later += total[hsub][w];
        const int64_t t = sg.t0 + b * 512 + blk * 64 + lane;
        if (live && t < sg.t1)
            IO<BF>::st(reinterpret_cast<typename IO<BF>::T *>(dg), t * A.H + h, (float)(later + x));
        for (int w = 0; w < 8; ++w) behind += total[hsub][w];
    }
}

// out[t][hk][d] = sum over the group's heads of in[t][h][d] (fp32), for the tokens of the sequences; four d a thread.
template <bool BF>
__global__ __launch_bounds__(256) void kda_hd_group_kernel(const float *__restrict__ in0, void *__restrict__ out0,
                                                           const float *__restrict__ in1, void *__restrict__ out1,
                                                           int64_t ntok, int64_t per_token, int64_t D4, int group,
                                                           const int64_t *__restrict__ covered) {
    const float *in = blockIdx.y ? in1 : in0;
    void *out = blockIdx.y ? out1 : out0;
    const int64_t lo = covered ? covered[0] : 0, hi = covered ? covered[1] : ntok;
    const int64_t n = ntok * per_token;  // per_token: Hk * D / 4
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < n; e += (int64_t)gridDim.x * 256) {
        const int64_t t = e / per_token, r = e - t * per_token, hk = r / D4, d = r - hk * D4;
        if (t < lo || t >= hi) continue;
        const f32x4 *p = reinterpret_cast<const f32x4 *>(in) + (t * (per_token / D4) * group + hk * group) * D4 + d;
        f32x4 x = p[0];
        for (int i = 1; i < group; ++i) x += p[i * D4];
        if constexpr (BF)
            reinterpret_cast<uint2 *>(out)[e] = make_uint2(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w));
        else
            reinterpret_cast<f32x4 *>(out)[e] = x;
    }
}

// ------------------------------------------------------------------ workspace
struct Layout {
    size_t table, seqs, covered, seg, decay, dseg, ddecay, s_end, part_q, part_v, border, dq, dk, total;
};
Layout layout(const Plan &p, int64_t ntok, int32_t H, int32_t Hk, int32_t K, int32_t V, int32_t N, bool packed,
              bool bf16, bool bwd) {
    Layout l{};
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    const size_t states = (size_t)H * K * V * sizeof(float);
    if (packed) {
        l.table = take((size_t)p.slots * sizeof(Segment));
        l.seqs = take((size_t)N * sizeof(SeqSlots));
        l.covered = take(2 * sizeof(int64_t));
    }
    if (p.several) {
        l.seg = take((size_t)p.slots * states);
        l.decay = take((size_t)p.slots * H * sizeof(float));
        if (bwd) {
            l.dseg = take((size_t)p.slots * states);
            l.ddecay = take((size_t)p.slots * H * sizeof(float));
        }
    }
    if (bwd) {
        l.s_end = take((size_t)N * states);
        const int gt = grad_tile(K, V, bf16);
        l.part_q = take((size_t)(K / gt) * ntok * H * sizeof(float));
        l.part_v = take((size_t)(V / gt) * ntok * H * sizeof(float));
        l.border = take((size_t)(V / gt) * p.slots * H * sizeof(float));
        if (Hk != H) {
            l.dq = take((size_t)ntok * H * K * sizeof(float));
            l.dk = take((size_t)ntok * H * K * sizeof(float));
        }
    }
    l.total = at ? at : 256;
    return l;
}

#define KDA_TRY(x)                            \
    do {                                      \
        const hipError_t e_ = (x);            \
        if (e_ != hipSuccess) return e_;      \
    } while (0)

struct Call {
    Plan p;
    Layout l;
    char *ws;
    const Segment *table;
    const SeqSlots *seqs;
    const int64_t *covered;
};

Call prepare(const HdArgs &a, bool bwd) {
    Call c;
    const bool packed = a.cu_seqlens != nullptr;
    c.p = plan(a.B, a.T, a.H, a.K, a.V, a.num_seqs, packed, a.io_bf16, bwd);
    c.l = layout(c.p, a.B * a.T, a.H, a.Hk, a.K, a.V, a.num_seqs, packed, a.io_bf16, bwd);
    c.ws = reinterpret_cast<char *>(a.workspace);
    c.table = packed ? reinterpret_cast<const Segment *>(c.ws + c.l.table) : nullptr;
    c.seqs = packed ? reinterpret_cast<const SeqSlots *>(c.ws + c.l.seqs) : nullptr;
    c.covered = packed ? reinterpret_cast<const int64_t *>(c.ws + c.l.covered) : nullptr;
    return c;
}
hipError_t make_table(const HdArgs &a, const Call &c, hipStream_t st) {
    if (!c.table) return hipSuccess;
    hipLaunchKernelGGL(kda_hd_table_kernel, dim3(1), dim3(1024), 0, st, a.cu_seqlens, a.num_seqs, (uint32_t)a.T,
                       (uint32_t)c.p.seg,
                       c.p.slots, const_cast<Segment *>(c.table), const_cast<SeqSlots *>(c.seqs),
                       const_cast<int64_t *>(c.covered));
    return hipGetLastError();
}
CoreArgs base(const HdArgs &a, const Call &c) {
    CoreArgs x{};
    x.ga = x.gb = x.gc = x.gx = 1;
    x.H = a.H;
    // Heads that share q and k go to one XCD where there are enough of them for all eight (17011 tokens of 32 heads, 4 to
    // a row of q and k: the forward
    // pass fetches 171 MB instead of 380, the increments 58 instead of 115).
    x.share = c.p.slots * a.Hk >= 128 ? a.H / a.Hk : 1;
    x.g_head = a.decay_per_head;
    x.g = a.g;
    x.table = c.table;
    x.slots = c.p.slots;
    x.T = a.T;
    x.seg = c.p.seg;
    x.ntok = a.B * a.T;
    x.nseg = c.p.nseg;
    x.fold = c.p.fold;
    x.s_intra = x.s_inter = x.s_up = 1.f;
    x.VD = a.V;
    return x;
}
// What the segments add to the states (to their gradients).
CoreArgs increments(const HdArgs &a, const Call &c, bool rev) {
    CoreArgs x = base(a, c);
    x.tiles = a.V / inc_tile(a.V);
    x.b = rev ? a.q : a.k;
    x.gb = a.H / a.Hk;
    x.c = rev ? a.dout : a.v;
    x.s_up = rev ? a.scale : 1.f;
    x.s_inc = reinterpret_cast<float *>(c.ws + (rev ? c.l.dseg : c.l.seg));
    x.seg_decay = reinterpret_cast<float *>(c.ws + (rev ? c.l.ddecay : c.l.decay));
    return x;
}
hipError_t segment_states(const HdArgs &a, const Call &c, bool bwd, hipStream_t st) {
    if (!c.p.several) return hipSuccess;
    const CoreArgs f = increments(a, c, false);
    const CarryArgs cf{f.s_inc, f.seg_decay, a.S0};
    if (!bwd) {
        KDA_TRY(inc_pass(a.io_bf16, f, nullptr, a.K, inc_tile(a.V), st));
        if (c.p.nseg <= c.p.fold) return hipSuccess;
        return launch_carry(cf, nullptr, c.seqs, c.p, a, st);
    }
    const CoreArgs r = increments(a, c, true);
    const CarryArgs cr{r.s_inc, r.seg_decay, a.dS_final};
    KDA_TRY(inc_pass(a.io_bf16, f, &r, a.K, inc_tile(a.V), st));
    return launch_carry(cf, &cr, c.seqs, c.p, a, st);
}

}  // namespace
}  // namespace hd

size_t hd_fwd_workspace_bytes(int64_t B, int64_t T, int32_t H, int32_t Hk, int32_t K, int32_t V, int32_t num_seqs,
                              bool packed, bool io_bf16) {
    const hd::Plan p = hd::plan(B, T, H, K, V, num_seqs, packed, io_bf16, false);
    return hd::layout(p, B * T, H, Hk, K, V, num_seqs, packed, io_bf16, false).total;
}
size_t hd_bwd_workspace_bytes(int64_t B, int64_t T, int32_t H, int32_t Hk, int32_t K, int32_t V, int32_t num_seqs,
                              bool packed, bool io_bf16) {
    const hd::Plan p = hd::plan(B, T, H, K, V, num_seqs, packed, io_bf16, true);
    return hd::layout(p, B * T, H, Hk, K, V, num_seqs, packed, io_bf16, true).total;
}

hipError_t launch_hd_fwd(const HdArgs &a, hipStream_t st) {
    using namespace hd;
    const Call c = prepare(a, false);
    KDA_TRY(make_table(a, c, st));
    KDA_TRY(segment_states(a, c, false, st));
    CoreArgs x = base(a, c);
    const int vt = fwd_tile(a.V, a.io_bf16);
    x.tiles = a.V / vt;
    x.a = a.q;
    x.b = a.k;
    x.ga = x.gb = a.H / a.Hk;
    x.c = a.v;
    x.y = a.o;
    x.s_init = a.S0;
    x.s_seg = reinterpret_cast<const float *>(c.ws + c.l.seg);
    x.seg_decay = reinterpret_cast<float *>(c.ws + c.l.decay);
    x.s_out = a.S_final;
    x.s_intra = x.s_inter = a.scale;
    return fwd_pass(a.io_bf16, x, a.K, vt, st);
}

hipError_t launch_hd_bwd(const HdArgs &a, hipStream_t st) {
    using namespace hd;
    const Call c = prepare(a, true);
    const int group = a.H / a.Hk, gt = grad_tile(a.K, a.V, a.io_bf16);
    const int64_t ntok = a.B * a.T;
    const bool grouped = group > 1;
    KDA_TRY(make_table(a, c, st));
    KDA_TRY(segment_states(a, c, true, st));
    const float *seg = reinterpret_cast<const float *>(c.ws + c.l.seg);
    const float *dseg = reinterpret_cast<const float *>(c.ws + c.l.dseg);
    float *s_end = reinterpret_cast<float *>(c.ws + c.l.s_end);
    void *dq = grouped ? c.ws + c.l.dq : a.dq, *dk = grouped ? c.ws + c.l.dk : a.dk;
    GradArgs g;
    // dv: backward in time, rows k against q, summing do
    g.dv = base(a, c);
    g.dv.tiles = a.V / gt;
    g.dv.a = a.k;
    g.dv.b = a.q;
    g.dv.ga = g.dv.gb = group;
    g.dv.c = a.dout;
    g.dv.y = a.dv;
    g.dv.s_init = a.dS_final;
    g.dv.s_seg = dseg;
    g.dv.s_out = a.dS0;
    g.dv.s_intra = g.dv.s_up = a.scale;
    g.dv.x = a.v;
    g.dv.part = reinterpret_cast<float *>(c.ws + c.l.part_v);
    g.dv.border = reinterpret_cast<float *>(c.ws + c.l.border);
    g.dv.s_seg_fwd = seg;
    // dk: backward in time, rows v against do, summing q; the state gradient transposed
    g.dk = base(a, c);
    g.dk.a = a.v;
    g.dk.b = a.dout;
    g.dk.c = a.q;
    g.dk.gc = group;
    g.dk.VD = a.K;
    g.dk.tiles = a.K / gt;
    g.dk.y = dk;
    g.dk.s_init = a.dS_final;
    g.dk.s_seg = dseg;
    g.dk.s_intra = g.dk.s_up = a.scale;
    // dq: forward in time, rows do against v, summing k; the state transposed
    g.dq = base(a, c);
    g.dq.a = a.dout;
    g.dq.b = a.v;
    g.dq.c = a.k;
    g.dq.gc = group;
    g.dq.VD = a.K;
    g.dq.tiles = a.K / gt;
    g.dq.y = dq;
    g.dq.s_init = a.S0;
    g.dq.s_seg = seg;
    g.dq.s_out = a.dg && a.dS_final ? s_end : nullptr;
    g.dq.s_intra = g.dq.s_inter = a.scale;
    g.dq.x = a.q;
    g.dq.gx = group;
    g.dq.part = reinterpret_cast<float *>(c.ws + c.l.part_q);
    KDA_TRY(a.io_bf16 ? grad_pass_bf16(g, a.K, a.V, a.dg != nullptr, grouped, st)
                      : grad_pass_fp32(g, a.K, a.V, a.dg != nullptr, st));
    if (ntok == 0) return hipSuccess;
    if (a.dg) {
        dim3 grid = wide_grid(c.p.slots);
        grid.z = (uint32_t)((a.H + 1) / 2);
        if (a.io_bf16)
            hipLaunchKernelGGL(kda_hd_dg_kernel<true>, grid, dim3(1024), 0, st, g.dv, g.dq.part, g.dq.tiles, a.K,
                               a.dS_final, s_end, a.dg);
        else
            hipLaunchKernelGGL(kda_hd_dg_kernel<false>, grid, dim3(1024), 0, st, g.dv, g.dq.part, g.dq.tiles, a.K,
                               a.dS_final, s_end, a.dg);
        KDA_TRY(hipGetLastError());
    }
    if (grouped) {
        const int64_t per = (int64_t)a.Hk * a.K / 4, n = ntok * per;
        const dim3 grid((uint32_t)((n + 255) / 256 < 8192 ? (n + 255) / 256 : 8192), 2);
        const float *iq = reinterpret_cast<const float *>(dq), *ik = reinterpret_cast<const float *>(dk);
        if (a.io_bf16)
            hipLaunchKernelGGL(kda_hd_group_kernel<true>, grid, dim3(256), 0, st, iq, a.dq, ik, a.dk, ntok, per,
                               (int64_t)a.K / 4, group, c.covered);
        else
            hipLaunchKernelGGL(kda_hd_group_kernel<false>, grid, dim3(256), 0, st, iq, a.dq, ik, a.dk, ntok, per,
                               (int64_t)a.K / 4, group, c.covered);
        KDA_TRY(hipGetLastError());
    }
    return hipSuccess;
}

}  // namespace kda
