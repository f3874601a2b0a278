// expert_w4.cu - 4-bit products 8 rows at a time, and the choice among 8, 16 and 32
// (expert_w4.cuh).
#include "expert_w4.cuh"

namespace ep {

// Rows taken at once: more rows per chunk read the weights fewer times (the chunks
// after the first find them in L2), fewer leave room for all of a row of x (a panel
// of it is converted again for every tile otherwise) and cost less per scale group.
// So: as many as the caller expects per expert, as long as x fits whole.
cudaError_t launch_expert_w4(const W4Args& a, int64_t expected_rows, int num_sms,
                             const LaunchOpts& o)
{
    if ((a.group != 32 && a.group != 64 && a.group != 128) || a.din % a.group != 0 ||
        a.dout % 8 != 0)
        return cudaErrorInvalidValue;
    if (expected_rows > 16 && w4_plan<W4Cfg<32, 32>>(a.din, a.E).panel >= a.din)
        return launch_expert_w4_32(a, num_sms, o);
    if (expected_rows > 8 && w4_plan<W4Cfg<16, 32>>(a.din, a.E).panel >= a.din)
        return launch_expert_w4_16(a, num_sms, o);
    return launch_w4_rows<8>(a, a.codes, num_sms, o);
}

}  // namespace ep
