// expert_w4.cu - 4-bit products 8 rows at a time, and the choice between 4, 8 and 16
// (expert_w4.cuh).
#include "expert_w4.cuh"

namespace ep {

// Rows taken at once. 16 read the weights fewer times (the second chunk finds them in
// L2) and share a tile's barriers and unpacking: 283 against 413 us (64 rows to each of
// 64 experts, 2048 x 4096, groups of 128), 73 against 81 us (8 rows to each), 25.4 against
// 28.1 us (7.5 rows to each of 8, 4096 x 4096), and lose 23.8 to 22.4 us with 5. 8 leave room
// for all of a longer row of x (a panel of it is converted again for every tile
// otherwise) and win where experts have one row more than 16 holds: 43 against 45 us (64
// tokens, 2 of 8 experts each, 4096 x 4096, groups of 64). 32 at once were no faster than
// 16 anywhere: the drain's time goes with the rows.
// 4, where 1.6 times the mean is at most 2, take half the MMAs and multiplications of 8: 113
// against 116 us (8 tokens, 8 of 64 experts each, 7168 x 4096, groups of 128), 15.5
// against 16.0 us (groups of 32); with a mean of 2 rows, some experts' second chunks cost
// what that saves, 155 against 148 us.
cudaError_t launch_expert_w4(const W4Args& a, int64_t expected_rows, int num_sms,
                             const LaunchOpts& o)
{
    if ((a.group != 32 && a.group != 64 && a.group != 128) || a.din % a.group != 0 ||
        a.dout % 8 != 0)
        return cudaErrorInvalidValue;
    if (expected_rows > 8 && w4_plan<W4Cfg<16, 32>>(a.din, a.E).panel >= a.din)
        return launch_expert_w4_16(a, num_sms, o);
    if (expected_rows <= 2) return launch_expert_w4_4(a, num_sms, o);
    return launch_w4_rows<8>(a, a.codes, num_sms, o);
}

}  // namespace ep
