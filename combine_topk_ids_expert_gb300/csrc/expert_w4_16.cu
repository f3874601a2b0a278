// expert_w4_16.cu - 4-bit products 16 rows at a time (expert_w4.cuh).
#include "expert_w4.cuh"

namespace ep {

cudaError_t launch_expert_w4_16(const W4Args& a, int num_sms, const LaunchOpts& o)
{
    return launch_w4_rows<16>(a, a.codes, num_sms, o);
}

}  // namespace ep
