// moe_b3.cu — the expert kernels of ttq_moe_lowbit for 3-bit codes.
#include "moe_tile.cuh"

namespace ttq {
namespace moe {
template ttq_status launch_bits<3>(const UpArgs&, const DownArgs&,
                                    cudaStream_t);
}  // namespace moe
}  // namespace ttq
