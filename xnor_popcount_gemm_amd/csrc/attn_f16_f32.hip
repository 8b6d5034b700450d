// Tree attention: instantiation for the cache type F16, output float.
#include "attn_kernel.hpp"

namespace bnn {

hipError_t attn_f16_f32(const KvCache& c, const KvBatch& b, const AttnArgs& a, const AttnPlan& pl, hipStream_t s) {
    return launch_type<F16, 2, float>(c, b, a, pl, s);
}

}  // namespace bnn
