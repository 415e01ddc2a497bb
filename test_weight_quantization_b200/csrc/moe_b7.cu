// moe_b7.cu — the expert kernels of ttq_moe_lowbit for 7-bit codes.
#include "moe_tile.cuh"

namespace ttq {
namespace moe {
template ttq_status launch_bits<7, UpArgs>(const UpArgs&, cudaStream_t);
template ttq_status launch_bits<7, DownArgs>(const DownArgs&, cudaStream_t);
}  // namespace moe
}  // namespace ttq
