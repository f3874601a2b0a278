// expert_w4.cu - 4-bit products 8 rows at a time, and the choice between 4, 8 and 16
// (expert_w4.cuh).
#include "expert_w4.cuh"

namespace ep {

// Rows taken at once, by expected_rows (1.6 times the mean, which few experts exceed).
// 16 read the weights fewer times (the second chunk finds them in L2) and share a tile's
// barriers and unpacking: 288 against 418 us (64 rows to each of 64 experts, 4096 -> 2048,
// groups of 128), 74.7 against 81.7 us (8 rows to each), 26.3 against 29.0 us (7.5 rows to
// each of 8, 4096 -> 4096), and lose 24.4 to 23.1 us with 5. They also lose where the mean
// is 16, so that about half of the experts have a second chunk all the same: 46.6 against
// 43.1 us (64 tokens, 2 of 8 experts each, 4096 -> 4096, groups of 64). Where x of 16 rows
// would not fit whole beside the ring (asked for groups of 32, the least that fits: above
// 4096 elements, less with hundreds of experts) 8 are taken: a panel of it is converted
// again for every tile, 98.2 against 60.5 us (64 tokens, 2 of 8, 7168 -> 4096, groups of
// 128). 32 at once were no faster than 16 anywhere: the drain's time goes with the rows.
// 4, where expected_rows is at most 2, take half the MMAs and multiplications of 8: 114.4
// against 116.7 us (8 tokens, 8 of 64 experts each, 7168 -> 4096, groups of 128), 203.7
// against 210.0 us (groups of 32); with a mean of 2 rows, some experts' second chunks cost
// what that saves, 156.7 against 148.7 us.
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
