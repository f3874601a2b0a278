// expert_w4_4.cu - 4-bit products 4 rows at a time (expert_w4.cuh).
#include "expert_w4.cuh"

namespace ep {

cudaError_t launch_expert_w4_4(const W4Args& a, int num_sms, const LaunchOpts& o)
{
    return launch_w4_rows<4>(a, a.codes, num_sms, o);
}

}  // namespace ep
