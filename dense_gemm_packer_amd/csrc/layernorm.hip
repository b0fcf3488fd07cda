// The layer norm that writes a product's operand (dgp_layernorm_quantize): the
// kernel and its launch rule are those of norm.h.
#include "common.h"
#include "launch.h"
#include "norm.h"

namespace dgp {

hipError_t launch_layernorm(const NormArgs &a, int x_type, int mode, hipStream_t s)
{
    return launch_norm_typed<true>(a, x_type, mode, s);
}

}  // namespace dgp
