// Linear attention with one decay per head: segments, the pass that carries states over them, and the order of the
// chunk kernel's passes (kda_hd_core.hpp) in a forward or backward call.
//
// A call whose heads and column tiles do not fill the chip cuts its sequences into segments. A first pass forms what
// each segment adds to a zero state (and its total decay), a second carries the states over the segments, and then
// every segment runs as if it were a sequence of its own. The backward does the same for the states' gradients, from
// the other end.
#include "kda_hd.hpp"

#include "kda_common.hpp"

namespace kda {
namespace hd {
namespace {

constexpr int64_t kResident = 512;  // workgroups of the chunk kernel that run at a time: two per CU
constexpr int64_t kLeastSegment = 256;

struct Plan {
    int64_t seg;        // tokens per segment
    int32_t nseg;       // segments per row (not packed)
    int64_t slots;      // workgroups' slots: an upper bound when packed
    bool several;       // some sequence may have more than one segment
    int vk, vv;         // column tile over K and over V columns
};

int tile_of(int cols, bool bf16) { return bf16 || cols < 64 ? cols : 64; }

// The increment passes have no weighted products to share, only the rows b: narrower tiles, more workgroups.
int inc_tile_of(int cols) { return cols < 64 ? cols : 64; }

int64_t round64(int64_t x) { return (x + 63) / 64 * 64; }

// How long a call with n segments per row takes, in tokens of one workgroup: its rounds over the chip's resident
// workgroups; with several segments also the increments' rounds (about a third of the work), two more launches and the
// states' traffic.
int64_t cost(int64_t rows, int64_t T, int64_t n) {
    const int64_t seg = round64((T + n - 1) / n);
    int64_t c = (rows * n + kResident - 1) / kResident * seg;
    if (n > 1) c += (rows * (n - 1) + kResident - 1) / kResident * seg / 3 + 100 + rows * n / 3;
    return c;
}

Plan plan(int64_t B, int64_t T, int32_t H, int32_t K, int32_t V, int32_t N, bool packed, bool bf16) {
    Plan p;
    p.vk = tile_of(K, bf16);
    p.vv = tile_of(V, bf16);
    const int64_t whole = round64(T > 0 ? T : 1);
    // workgroups of one segment per row (packed: one sequence may be nearly all of the batch)
    const int64_t rows = (packed ? 1 : B) * H * (V / p.vv);
    int64_t best = 1;
    for (int64_t n = 2; n <= whole / kLeastSegment && rows * (n - 1) < 2 * kResident; ++n)
        if (cost(rows, whole, n) < cost(rows, whole, best)) best = n;
    p.seg = round64((whole + best - 1) / best);
    p.nseg = (int32_t)(T > 0 ? (T + p.seg - 1) / p.seg : 1);
    p.slots = packed ? T / p.seg + N : B * p.nseg;
    p.several = p.nseg > 1;
    return p;
}

// ------------------------------------------------------------------ segments of packed sequences
struct SeqSlots { int32_t first, count; };

// One workgroup: clamps cu_seqlens into [0, T] and makes it non-decreasing (a running maximum), numbers the segments.
__global__ __launch_bounds__(1024) void kda_hd_table_kernel(const int32_t *__restrict__ cu, int32_t N, int64_t T,
                                                            int64_t seg, int64_t slots, Segment *__restrict__ table,
                                                            SeqSlots *__restrict__ seqs, int64_t *__restrict__ covered) {
    __shared__ int64_t s_max[1024];
    __shared__ int32_t s_sum[1024];
    const int t = threadIdx.x;
    auto entry = [&](int64_t i) {
        const int64_t x = cu[i];
        return x < 0 ? 0 : x > T ? T : x;
    };
    int64_t top = entry(0);
    int64_t first = 0;
    if (t == 0) covered[0] = top;
    for (int64_t base = 0; base < N; base += 1024) {
        const int64_t n = base + t;
        s_max[t] = n < N ? entry(n + 1) : 0;
        __syncthreads();
        for (int d = 1; d < 1024; d <<= 1) {
            const int64_t x = t >= d ? s_max[t - d] : 0;
            __syncthreads();
            if (x > s_max[t]) s_max[t] = x;
            __syncthreads();
        }
        const int64_t before = t > 0 && s_max[t - 1] > top ? s_max[t - 1] : top;
        const int64_t end = s_max[t] > top ? s_max[t] : top;
        const int64_t segs = (end - before + seg - 1) / seg;
        const int32_t count = n < N ? (int32_t)(segs > 1 ? segs : 1) : 0;
        s_sum[t] = count;
        __syncthreads();
        for (int d = 1; d < 1024; d <<= 1) {
            const int32_t x = t >= d ? s_sum[t - d] : 0;
            __syncthreads();
            s_sum[t] += x;
            __syncthreads();
        }
        if (n < N) {
            const int64_t at = first + s_sum[t] - count;
            seqs[n] = SeqSlots{(int32_t)at, count};
            for (int32_t j = 0; j < count; ++j) {
                const int64_t a = before + j * seg, e = a + seg;
                table[at + j] = Segment{(int32_t)n, j, count, 0, a, e < end ? e : end};
            }
        }
        first += s_sum[1023];
        if (s_max[1023] > top) top = s_max[1023];
        __syncthreads();
    }
    for (int64_t i = first + t; i < slots; i += 1024) table[i] = Segment{-1, 0, 0, 0, 0, 0};
    if (t == 0) covered[1] = top;
}

// ------------------------------------------------------------------ states over the segments
// In place: what each segment adds becomes the state it starts from (rev: the state gradient it ends with). A thread
// carries four adjacent state entries over the segments of its sequence.
__global__ __launch_bounds__(256) void kda_hd_carry_kernel(float *__restrict__ seg, const float *__restrict__ decay,
                                                           const float *__restrict__ init, const SeqSlots *__restrict__ seqs,
                                                           int32_t nseg, int32_t H, int64_t kv4, int rev) {
    const int64_t runs = (kv4 + 255) / 256, nh = blockIdx.x / runs, n = nh / H;
    const int64_t e = (blockIdx.x - nh * runs) * 256 + threadIdx.x;
    if (e >= kv4) return;
    const int h = (int)(nh - n * H);
    const int32_t first = seqs ? seqs[n].first : (int32_t)(n * nseg), count = seqs ? seqs[n].count : nseg;
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

hipError_t launch_carry(float *seg, const float *decay, const float *init, const SeqSlots *seqs, const Plan &p,
                        const HdArgs &a, bool rev, hipStream_t st) {
    const int64_t kv4 = (int64_t)a.K * a.V / 4, nh = (int64_t)a.num_seqs * a.H;
    // heads of all sequences times runs of 256 state entries: num_seqs * H < 2^28, K * V / 1024 <= 16
    const int64_t x = (kv4 + 255) / 256;
    if (nh * x >= ((int64_t)1 << 31)) return hipErrorInvalidValue;
    hipLaunchKernelGGL(kda_hd_carry_kernel, dim3((uint32_t)(nh * x)), dim3(256), 0, st, seg, decay, init, seqs, p.nseg,
                       a.H, kv4, (int)rev);
    return hipGetLastError();
}

// ------------------------------------------------------------------ the gradients' last steps
// dg[t][h] = sum of the column tiles' parts [tiles][H][ntok], for the tokens of the sequences.
template <bool BF>
__global__ __launch_bounds__(256) void kda_hd_dg_kernel(const float *__restrict__ part, int tiles, int32_t H,
                                                        int64_t ntok, const int64_t *__restrict__ covered,
                                                        void *__restrict__ dg) {
    __shared__ float s[64][65];
    const int64_t t0 = (int64_t)blockIdx.x * 64;
    const int h0 = blockIdx.y * 64, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t lo = covered ? covered[0] : 0, hi = covered ? covered[1] : ntok;
    for (int i = wave; i < 64; i += 4) {
        float x = 0.f;
        if (h0 + i < H && t0 + lane >= lo && t0 + lane < hi)
            for (int w = 0; w < tiles; ++w) x += part[((int64_t)w * H + h0 + i) * ntok + t0 + lane];
        s[i][lane] = x;
    }
    __syncthreads();
    for (int i = wave; i < 64; i += 4) {
        const int64_t t = t0 + i;
        if (t >= lo && t < hi && h0 + lane < H)
            IO<BF>::st(reinterpret_cast<typename IO<BF>::T *>(dg), t * H + h0 + lane, s[lane][i]);
    }
}

// out[t][hk][d] = sum over the group's heads of in[t][h][d] (fp32), for the tokens of the sequences; four d a thread.
template <bool BF>
__global__ __launch_bounds__(256) void kda_hd_group_kernel(const float *__restrict__ in, void *__restrict__ out,
                                                           int64_t ntok, int64_t per_token, int64_t D4, int group,
                                                           const int64_t *__restrict__ covered) {
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
    size_t table, seqs, covered, seg, decay, dseg, ddecay, s_end, share, dg_part, dq, dk, total;
};
Layout layout(const Plan &p, int64_t ntok, int32_t H, int32_t Hk, int32_t K, int32_t V, int32_t N, bool packed,
              bool bwd) {
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
        l.share = take((size_t)(K / p.vk) * ntok * H * sizeof(float));
        l.dg_part = take((size_t)(V / p.vv) * ntok * H * sizeof(float));
        if (Hk != H) {
            l.dq = take((size_t)ntok * H * K * sizeof(float));
            l.dk = take((size_t)ntok * H * K * sizeof(float));
        }
    }
    l.total = at ? at : 256;
    return l;
}

hipError_t core(const HdArgs &a, const CoreArgs &c, int kd, int vt, Kind k, hipStream_t st) {
    return a.io_bf16 ? core_bf16(c, kd, vt, k, st) : core_fp32(c, kd, vt, k, st);
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
    c.p = plan(a.B, a.T, a.H, a.K, a.V, a.num_seqs, packed, a.io_bf16);
    c.l = layout(c.p, a.B * a.T, a.H, a.Hk, a.K, a.V, a.num_seqs, packed, bwd);
    c.ws = reinterpret_cast<char *>(a.workspace);
    c.table = packed ? reinterpret_cast<const Segment *>(c.ws + c.l.table) : nullptr;
    c.seqs = packed ? reinterpret_cast<const SeqSlots *>(c.ws + c.l.seqs) : nullptr;
    c.covered = packed ? reinterpret_cast<const int64_t *>(c.ws + c.l.covered) : nullptr;
    return c;
}
hipError_t make_table(const HdArgs &a, const Call &c, hipStream_t st) {
    if (!c.table) return hipSuccess;
    hipLaunchKernelGGL(kda_hd_table_kernel, dim3(1), dim3(1024), 0, st, a.cu_seqlens, a.num_seqs, a.T, c.p.seg,
                       c.p.slots, const_cast<Segment *>(c.table), const_cast<SeqSlots *>(c.seqs),
                       const_cast<int64_t *>(c.covered));
    return hipGetLastError();
}
CoreArgs base(const HdArgs &a, const Call &c) {
    CoreArgs x{};
    x.ga = x.gb = x.gc = x.gx = 1;
    x.H = a.H;
    x.g_head = a.decay_per_head;
    x.g = a.g;
    x.table = c.table;
    x.slots = c.p.slots;
    x.T = a.T;
    x.seg = c.p.seg;
    x.ntok = a.B * a.T;
    x.nseg = c.p.nseg;
    x.s_intra = x.s_inter = x.s_up = 1.f;
    x.sr = a.V;
    x.sc = 1;
    x.VD = a.V;
    x.tiles = a.V / c.p.vv;
    return x;
}
// the states that the segments start from
hipError_t forward_states(const HdArgs &a, const Call &c, hipStream_t st) {
    if (!c.p.several) return hipSuccess;
    CoreArgs x = base(a, c);
    x.b = a.k;
    x.gb = a.H / a.Hk;
    x.c = a.v;
    x.s_inc = reinterpret_cast<float *>(c.ws + c.l.seg);
    x.seg_decay = reinterpret_cast<float *>(c.ws + c.l.decay);
    x.tiles = a.V / inc_tile_of(a.V);
    KDA_TRY(core(a, x, a.K, inc_tile_of(a.V), Kind::fwd_inc, st));
    return launch_carry(x.s_inc, x.seg_decay, a.S0, c.seqs, c.p, a, false, st);
}

}  // namespace
}  // namespace hd

size_t hd_fwd_workspace_bytes(int64_t B, int64_t T, int32_t H, int32_t Hk, int32_t K, int32_t V, int32_t num_seqs,
                              bool packed, bool io_bf16) {
    const hd::Plan p = hd::plan(B, T, H, K, V, num_seqs, packed, io_bf16);
    return hd::layout(p, B * T, H, Hk, K, V, num_seqs, packed, false).total;
}
size_t hd_bwd_workspace_bytes(int64_t B, int64_t T, int32_t H, int32_t Hk, int32_t K, int32_t V, int32_t num_seqs,
                              bool packed, bool io_bf16) {
    const hd::Plan p = hd::plan(B, T, H, K, V, num_seqs, packed, io_bf16);
    return hd::layout(p, B * T, H, Hk, K, V, num_seqs, packed, true).total;
}

hipError_t launch_hd_fwd(const HdArgs &a, hipStream_t st) {
    using namespace hd;
    const Call c = prepare(a, false);
    KDA_TRY(make_table(a, c, st));
    KDA_TRY(forward_states(a, c, st));
    CoreArgs x = base(a, c);
    x.a = a.q;
    x.b = a.k;
    x.ga = x.gb = a.H / a.Hk;
    x.c = a.v;
    x.y = a.o;
    x.s_init = a.S0;
    x.s_seg = reinterpret_cast<const float *>(c.ws + c.l.seg);
    x.s_out = a.S_final;
    x.s_intra = x.s_inter = a.scale;
    return core(a, x, a.K, c.p.vv, Kind::fwd, st);
}

hipError_t launch_hd_bwd(const HdArgs &a, hipStream_t st) {
    using namespace hd;
    const Call c = prepare(a, true);
    const int group = a.H / a.Hk;
    const int64_t ntok = a.B * a.T;
    KDA_TRY(make_table(a, c, st));
    KDA_TRY(forward_states(a, c, st));
    float *dseg = reinterpret_cast<float *>(c.ws + c.l.dseg), *s_end = reinterpret_cast<float *>(c.ws + c.l.s_end);
    if (c.p.several) {  // the state gradients that the segments end with
        CoreArgs x = base(a, c);
        x.b = a.q;
        x.gb = group;
        x.c = a.dout;
        x.s_up = a.scale;
        x.s_inc = dseg;
        x.seg_decay = reinterpret_cast<float *>(c.ws + c.l.ddecay);
        x.tiles = a.V / inc_tile_of(a.V);
        KDA_TRY(core(a, x, a.K, inc_tile_of(a.V), Kind::rev_inc, st));
        KDA_TRY(launch_carry(dseg, x.seg_decay, a.dS_final, c.seqs, c.p, a, true, st));
    }
    const bool grouped = group > 1;
    void *dq = grouped ? c.ws + c.l.dq : a.dq, *dk = grouped ? c.ws + c.l.dk : a.dk;
    {  // dq: forward in time, rows do against v, summing k; the state transposed
        CoreArgs x = base(a, c);
        x.a = a.dout;
        x.b = a.v;
        x.c = a.k;
        x.gc = group;
        x.VD = a.K;
        x.tiles = a.K / c.p.vk;
        x.sr = 1;
        x.sc = a.V;
        x.y = dq;
        x.y_fp32 = grouped;
        x.s_init = a.S0;
        x.s_seg = reinterpret_cast<const float *>(c.ws + c.l.seg);
        x.s_intra = x.s_inter = a.scale;
        x.x = a.q;
        x.gx = group;
        x.share = reinterpret_cast<float *>(c.ws + c.l.share);
        x.s_out = a.dg && a.dS_final ? s_end : nullptr;
        KDA_TRY(core(a, x, a.V, c.p.vk, a.dg ? Kind::fwd_dg : Kind::fwd, st));
    }
    {  // dv: backward in time, rows k against q, summing do
        CoreArgs x = base(a, c);
        x.a = a.k;
        x.b = a.q;
        x.ga = x.gb = group;
        x.c = a.dout;
        x.y = a.dv;
        x.s_init = a.dS_final;
        x.s_seg = dseg;
        x.s_out = a.dS0;
        x.s_intra = x.s_up = a.scale;
        x.x = a.v;
        x.share = reinterpret_cast<float *>(c.ws + c.l.share);
        x.share_tiles = a.K / c.p.vk;
        x.dg_part = reinterpret_cast<float *>(c.ws + c.l.dg_part);
        x.s_end = s_end;
        x.s_seg_fwd = reinterpret_cast<const float *>(c.ws + c.l.seg);
        KDA_TRY(core(a, x, a.K, c.p.vv, a.dg ? Kind::rev_dg : Kind::rev, st));
    }
    {  // dk: backward in time, rows v against do, summing q; the state gradient transposed
        CoreArgs x = base(a, c);
        x.a = a.v;
        x.b = a.dout;
        x.c = a.q;
        x.gc = group;
        x.VD = a.K;
        x.tiles = a.K / c.p.vk;
        x.sr = 1;
        x.sc = a.V;
        x.y = dk;
        x.y_fp32 = grouped;
        x.s_init = a.dS_final;
        x.s_seg = dseg;
        x.s_intra = x.s_up = a.scale;
        KDA_TRY(core(a, x, a.V, c.p.vk, Kind::rev, st));
    }
    if (ntok == 0) return hipSuccess;
    if (a.dg) {
        const dim3 grid((uint32_t)((ntok + 63) / 64), (uint32_t)((a.H + 63) / 64));
        const float *part = reinterpret_cast<const float *>(c.ws + c.l.dg_part);
        const int tiles = a.V / c.p.vv;
        if (a.io_bf16)
            hipLaunchKernelGGL(kda_hd_dg_kernel<true>, grid, dim3(256), 0, st, part, tiles, a.H, ntok, c.covered, a.dg);
        else
            hipLaunchKernelGGL(kda_hd_dg_kernel<false>, grid, dim3(256), 0, st, part, tiles, a.H, ntok, c.covered, a.dg);
        KDA_TRY(hipGetLastError());
    }
    if (grouped) {
        const int64_t per = (int64_t)a.Hk * a.K / 4, n = ntok * per;
        const uint32_t wgs = (uint32_t)((n + 255) / 256 < 8192 ? (n + 255) / 256 : 8192);
        for (int i = 0; i < 2; ++i) {
            const float *in = reinterpret_cast<const float *>(i ? dk : dq);
            void *out = i ? a.dk : a.dq;
            if (a.io_bf16)
                hipLaunchKernelGGL(kda_hd_group_kernel<true>, dim3(wgs), dim3(256), 0, st, in, out, ntok, per,
                                   (int64_t)a.K / 4, group, c.covered);
            else
                hipLaunchKernelGGL(kda_hd_group_kernel<false>, dim3(wgs), dim3(256), 0, st, in, out, ntok, per,
                                   (int64_t)a.K / 4, group, c.covered);
            KDA_TRY(hipGetLastError());
        }
    }
    return hipSuccess;
}

}  // namespace kda
