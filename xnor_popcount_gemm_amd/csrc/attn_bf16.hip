// Tree attention: instantiation for the cache type Bf16, output __bf16.
#include "attn_kernel.hpp"

namespace bnn {

hipError_t attn_bf16(const KvCache& c, const KvBatch& b, const AttnArgs& a, const AttnPlan& pl, hipStream_t s) {
    return launch_type<Bf16, 1, __bf16>(c, b, a, pl, s);
}

}  // namespace bnn
