// The paged attention kernels for head size 64 over a quantised cache of 8-bit integers,
// whole caches and regions.
#include "sda_paged.cuh"

namespace sda {
namespace paged {

__attribute__((visibility("hidden"))) sda_status launch_qint8_64(const CUtensorMap &tmap, const Params &p, void *stream)
{
    return launch_dim<kScaledInt8, 64>(tmap, p, stream);
}

__attribute__((visibility("hidden"))) sda_status regions_qint8_64(const CUtensorMap &tmap, const Params &p, void *stream)
{
    return launch_regions<kScaledInt8, 64>(tmap, p, stream);
}

}  // namespace paged
}  // namespace sda
