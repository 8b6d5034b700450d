// Tree attention: instantiation for the cache type F16, output _Float16.
#include "attn_kernel.hpp"

namespace bnn {

hipError_t attn_f16(const KvCache& c, const KvBatch& b, const AttnArgs& a, const AttnPlan& pl, hipStream_t s) {
    return launch_type<F16, 1, _Float16>(c, b, a, pl, s);
}

}  // namespace bnn
