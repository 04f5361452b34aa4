#include "mv_norm_grad.cuh"

namespace mvblock {
template int run_norm_grad<__nv_bfloat16>(const NormArgs &, const NormShape &, u64, u32, bool, bool, cudaStream_t);
}  // namespace mvblock
