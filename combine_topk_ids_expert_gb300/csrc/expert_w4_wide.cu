// expert_w4_wide.cu - 4-bit products 16 rows at a time (expert_w4.cuh).
#include "expert_w4.cuh"

namespace ep {

cudaError_t launch_expert_w4_wide(const W4Args& a, bool glu, const void* x, int64_t rows,
                                  const void* codes, int num_sms, const LaunchOpts& o)
{
    return launch_w4_rows<16>(a, glu, x, rows, codes, num_sms, o);
}

}  // namespace ep
