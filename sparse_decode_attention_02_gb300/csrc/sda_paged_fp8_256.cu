// The paged attention kernels for head size 256 over an E4M3 cache.
#include "sda_paged.cuh"

namespace sda {
namespace paged {

__attribute__((visibility("hidden"))) sda_status launch_fp8_256(const CUtensorMap &tmap, const Params &p, void *stream)
{
    return launch_dim<kE4m3, 256>(tmap, p, stream);
}

}  // namespace paged
}  // namespace sda
