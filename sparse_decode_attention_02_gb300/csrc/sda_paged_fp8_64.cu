// The paged attention kernels for head size 64 over an E4M3 cache.
#include "sda_paged.cuh"

namespace sda {
namespace paged {

__attribute__((visibility("hidden"))) sda_status launch_fp8_64(const CUtensorMap &tmap, const Params &p, void *stream)
{
    return launch_dim<true, 64>(tmap, p, stream);
}

}  // namespace paged
}  // namespace sda
