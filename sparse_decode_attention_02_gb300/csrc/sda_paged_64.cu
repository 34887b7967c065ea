// The paged attention kernels for head size 64.
#include "sda_paged.cuh"

namespace sda {
namespace paged {

__attribute__((visibility("hidden"))) sda_status launch_64(bool fp8, const CUtensorMap &tmap, const Params &p,
                                                            void *stream)
{
    return launch_dim<64>(fp8, tmap, p, stream);
}

}  // namespace paged
}  // namespace sda
