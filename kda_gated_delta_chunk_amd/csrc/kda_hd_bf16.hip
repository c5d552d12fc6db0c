// The chunk kernel of linear attention with one decay per head, bf16 I/O.
#include "kda_hd_core.hpp"

namespace kda {
namespace hd {
hipError_t core_bf16(const CoreArgs &a, int kd, int vt, Kind k, hipStream_t st) {
    return launch_core<true>(a, kd, vt, k, st);
}
}  // namespace hd
}  // namespace kda
