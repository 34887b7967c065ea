// The paged attention kernels for head size 192 over a quantised cache of E4M3 elements,
// whole caches and regions.
#include "sda_paged.cuh"

namespace sda {
namespace paged {

__attribute__((visibility("hidden"))) sda_status launch_qe4m3_192(const CUtensorMap &tmap, const Params &p, void *stream)
{
    return launch_dim<kScaledE4m3, 192>(tmap, p, stream);
}

__attribute__((visibility("hidden"))) sda_status regions_qe4m3_192(const CUtensorMap &tmap, const Params &p, void *stream)
{
    return launch_regions<kScaledE4m3, 192>(tmap, p, stream);
}

}  // namespace paged
}  // namespace sda
