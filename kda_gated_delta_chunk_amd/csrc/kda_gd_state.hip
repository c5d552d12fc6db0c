// The gated delta rule with one decay per head: the passes over the states.
#include "kda_gd_core.hpp"

namespace kda {
namespace gd {
namespace {
template <bool BF, int K, int VT>
hipError_t launch(const StateArgs &a, const StateArgs *e, int V, hipStream_t st) {
    const int64_t blocks = ((int64_t)a.c.N * a.c.H + 7) / 8 * 8 * a.tiles;
    if (e)
        hipLaunchKernelGGL((kda_gd_states_kernel<BF, K, VT>), hd::wide_grid(2 * blocks), dim3(VT * 6), 0, st, a, *e, V, blocks);
    else
        hipLaunchKernelGGL((kda_gd_state_kernel<BF, K, VT>), hd::wide_grid(blocks), dim3(VT * 6), 0, st, a, V);
    return hipGetLastError();
}
template <bool BF, int K>
hipError_t by_tile(const StateArgs &a, const StateArgs *e, int V, hipStream_t st) {
    return state_tile(V) == 32 ? launch<BF, K, 32>(a, e, V, st) : launch<BF, K, 64>(a, e, V, st);
}
template <bool BF>
hipError_t by_k(const StateArgs &a, const StateArgs *e, int K, int V, hipStream_t st) {
    return K == 32   ? by_tile<BF, 32>(a, e, V, st)
           : K == 64 ? by_tile<BF, 64>(a, e, V, st)
                     : by_tile<BF, 128>(a, e, V, st);
}
}  // namespace

hipError_t forward_pass(bool bf16, const StateArgs &a, int K, int V, hipStream_t st) {
    return bf16 ? by_k<true>(a, nullptr, K, V, st) : by_k<false>(a, nullptr, K, V, st);
}
hipError_t backward_passes(bool bf16, const StateArgs &reverse, const StateArgs &errors, int K, int V, hipStream_t st) {
    return bf16 ? by_k<true>(reverse, &errors, K, V, st) : by_k<false>(reverse, &errors, K, V, st);
}
}  // namespace gd
}  // namespace kda
