// The paged attention kernels for head size 192 over a bf16 cache.
#include "sda_paged.cuh"

namespace sda {
namespace paged {

__attribute__((visibility("hidden"))) sda_status launch_bf16_192(const CUtensorMap &tmap, const Params &p, void *stream)
{
    return launch_dim<kBf16, 192>(tmap, p, stream);
}

}  // namespace paged
}  // namespace sda
