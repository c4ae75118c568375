// ra_norm_inst.cu -- the block end's kernels for one type of activations and
// one of the residual stream (RA_INST_D, RA_INST_RD); compiled once for each pair.
#include "ra_norm.cuh"

namespace ra {
namespace norm {

template cudaError_t run_forward<RA_INST_D, RA_INST_RD>(const Shape&, bool, const NormForward&, OptedIn&, unsigned,
                                                        cudaStream_t);
template cudaError_t run_backward<RA_INST_D, RA_INST_RD>(const Shape&, bool, const NormBackward&, const Deal&, OptedIn&,
                                                         unsigned, cudaStream_t);

}  // namespace norm
}  // namespace ra
