// Tree attention: instantiation for the cache type Bf16, output float.
#include "attn_kernel.hpp"

namespace bnn {

hipError_t attn_bf16_f32(const KvCache& c, const KvBatch& b, const AttnArgs& a, const AttnPlan& pl, hipStream_t s) {
    return launch_type<Bf16, 3, float>(c, b, a, pl, s);
}

}  // namespace bnn
