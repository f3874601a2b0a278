// expert_w4.cu - 4-bit products for experts with a few rows each: 8 rows at a time
// (expert_w4.cuh). Calls that route more rows per expert go to expert_w4_wide.cu.
#include "expert_w4.cuh"

namespace ep {

cudaError_t launch_expert_w4(const W4Args& a, bool glu, bool wide, const void* x, int64_t rows,
                             const void* codes, int num_sms, const LaunchOpts& o)
{
    if (a.din % 32 != 0 || a.dout % 8 != 0 || a.din % a.group != 0) return cudaErrorInvalidValue;
    return wide ? launch_expert_w4_wide(a, glu, x, rows, codes, num_sms, o)
                : launch_w4_rows<8>(a, glu, x, rows, codes, num_sms, o);
}

}  // namespace ep
