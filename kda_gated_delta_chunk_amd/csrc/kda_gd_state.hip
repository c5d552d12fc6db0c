// The gated delta rule with one decay per head: the passes over the states.
#include "kda_gd_core.hpp"

namespace kda {
namespace gd {
namespace {
template <bool BF, int K, int VT>
hipError_t launch(StateArgs a, StateArgs *e, int V, hipStream_t st) {
    a.tiles = V / VT;
    if (e) e->tiles = a.tiles;
    const int64_t blocks = ((int64_t)a.c.N * a.c.H + 7) / 8 * 8 * a.tiles;
    const dim3 grid = hd::wide_grid(e ? 2 * blocks : blocks);
    if (e && a.c.third)
        hipLaunchKernelGGL((kda_gd_states_kernel<BF, K, VT, BF && !(K == 128 && VT == 128) ? 3 : 2>), grid, dim3(VT * 6), 0, st,
                           a, *e, V, blocks);
    else if (e)
        hipLaunchKernelGGL((kda_gd_states_kernel<BF, K, VT, 2>), grid, dim3(VT * 6), 0, st, a, *e, V, blocks);
    else
        hipLaunchKernelGGL((kda_gd_state_kernel<BF, K, VT>), grid, dim3(VT * 6), 0, st, a, V);
    return hipGetLastError();
}
// Tiles of 64 columns occupy a compute unit each. Where there are more of them than compute units, the two of a head share
// one: their products overlap, and they read the same rows (4096 tokens of 256 heads: 318 us for 401; of 64 heads 184 us
// and 300). Packed sequences are balanced as they come, which takes several pieces for every compute unit (16 of 17011 tokens,
// 32 heads: 251 us for 226). With three parts and K = 128 the registers of both tiles' wavefronts spill (backward passes of
// 4096 tokens of 96 heads: 907 us for 531): one tile then. Of the others at K = V = 128 two tiles spill 2 (forward) and 4
// (backward) of 168 registers in bf16, which shows nowhere (forward 17 to 20% faster), and 19 and 23 in fp32, which costs the
// forward call what sharing gains (whole calls of 1024 tokens, two tiles for one: 160 heads 341 us for 351, 256 heads 388 for
// 387, 512 heads 781 for 760) and the backward call less (96 heads 695 for 682, 256 heads 1326 for 1401; 8000 packed tokens
// of 16 sequences, 64 heads 2768 for 2926). K = 32 in fp32 is the rule's worst: 160 to 256 heads forward 6 to 8% slower than
// one tile, 512 heads 10% faster.
template <bool BF, int K>
hipError_t by_tile(const StateArgs &a, StateArgs *e, int V, hipStream_t st) {
    constexpr int64_t kUnits = 256;
    const int64_t items = (int64_t)a.c.N * a.c.H * (e ? 2 : 1);
    const bool fits = !(K == 128 && a.c.third), many = fits && (a.c.seqs ? items >= 4 * kUnits : 2 * items > kUnits);
    return V == 32            ? launch<BF, K, 32>(a, e, V, st)
           : V == 64 || !many ? launch<BF, K, 64>(a, e, V, st)
                              : launch<BF, K, 128>(a, e, V, st);
}
template <bool BF>
hipError_t by_k(const StateArgs &a, StateArgs *e, int K, int V, hipStream_t st) {
    return K == 32   ? by_tile<BF, 32>(a, e, V, st)
           : K == 64 ? by_tile<BF, 64>(a, e, V, st)
                     : by_tile<BF, 128>(a, e, V, st);
}
}  // namespace

hipError_t forward_pass(bool bf16, const StateArgs &a, int K, int V, hipStream_t st) {
    return bf16 ? by_k<true>(a, nullptr, K, V, st) : by_k<false>(a, nullptr, K, V, st);
}
hipError_t backward_passes(bool bf16, const StateArgs &reverse, StateArgs errors, int K, int V, hipStream_t st) {
    return bf16 ? by_k<true>(reverse, &errors, K, V, st) : by_k<false>(reverse, &errors, K, V, st);
}
}  // namespace gd
}  // namespace kda
