// The gated delta rule with one decay per head: the passes over the states.
#include "kda_gd_core.hpp"

namespace kda {
namespace gd {
namespace {
template <bool BF, int K, int VT, int MODE>
hipError_t launch(const StateArgs &a, int V, hipStream_t st) {
    const int64_t items = (int64_t)a.c.N * a.c.H;
    hipLaunchKernelGGL((kda_gd_state_kernel<BF, K, VT, MODE>), hd::wide_grid((items + 7) / 8 * 8 * a.tiles),
                       dim3(VT * 8), 0, st, a, V);
    return hipGetLastError();
}
template <bool BF, int K, int VT>
hipError_t by_mode(Mode mode, const StateArgs &a, int V, hipStream_t st) {
    return mode == kForward ? launch<BF, K, VT, kForward>(a, V, st)
         : mode == kErrors  ? launch<BF, K, VT, kErrors>(a, V, st)
                            : launch<BF, K, VT, kReverse>(a, V, st);
}
template <bool BF, int K>
hipError_t by_tile(Mode mode, const StateArgs &a, int V, hipStream_t st) {
    return state_tile(V) == 32 ? by_mode<BF, K, 32>(mode, a, V, st) : by_mode<BF, K, 64>(mode, a, V, st);
}
template <bool BF>
hipError_t by_k(Mode mode, const StateArgs &a, int K, int V, hipStream_t st) {
    return K == 32   ? by_tile<BF, 32>(mode, a, V, st)
           : K == 64 ? by_tile<BF, 64>(mode, a, V, st)
                     : by_tile<BF, 128>(mode, a, V, st);
}
}  // namespace

hipError_t state_pass(bool bf16, Mode mode, const StateArgs &a, int K, int V, hipStream_t st) {
    return bf16 ? by_k<true>(mode, a, K, V, st) : by_k<false>(mode, a, K, V, st);
}
}  // namespace gd
}  // namespace kda
