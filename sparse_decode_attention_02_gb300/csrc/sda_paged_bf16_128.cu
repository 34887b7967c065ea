// The paged attention kernels for head size 128 over a bf16 cache.
#include "sda_paged.cuh"

namespace sda {
namespace paged {

__attribute__((visibility("hidden"))) sda_status launch_bf16_128(const CUtensorMap &tmap, const Params &p, void *stream)
{
    return launch_dim<kBf16, 128>(tmap, p, stream);
}

}  // namespace paged
}  // namespace sda
