// The layer norm that writes a product's operand (dgp_layernorm_quantize): the
// kernel and its launch rule are those of norm.h.  HBM-bound: 4096 x 8192 bf16
// with residual and bias, e4m3 codes and fp32 block scales, 236 MB in 39 us, 6.0
// TB/s; one row of 7168 to mxfp8 3.3 us, the latency of one workgroup and of one
// sum more than the root-mean-square norm's.
#include "common.h"
#include "launch.h"
#include "norm.h"

namespace dgp {

hipError_t launch_layernorm(const NormArgs &a, int x_type, int mode, hipStream_t s)
{
    return launch_norm_typed<true>(a, x_type, mode, s);
}

}  // namespace dgp
