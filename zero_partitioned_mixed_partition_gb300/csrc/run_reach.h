// run_reach.h -- how far a run of equal keys goes on in a sorted list, looked at 32
// places at a time.  Without CUDA's headers, so that a test on the host can count the looks.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define ZS_HOST_DEVICE __host__ __device__
#else
#define ZS_HOST_DEVICE
#endif

namespace zs {

// The ones before the first zero, from the lowest bit up.
ZS_HOST_DEVICE inline int ones(uint32_t bits) {
    if (bits == 0xffffffffu) return 32;
#ifdef __CUDA_ARCH__
    return __ffs((int)~bits) - 1;
#else
    return __builtin_ctz(~bits);
#endif
}

// votes(at, stride): bit i is whether place at + stride (i + 1) belongs to the run, counted from
// where it was met (at = 0), and 0 past the list's end.  The bits are 1 up to some place and 0 from
// there on.  Returns that many places.  A run that ends within 31 places is one look; a longer one
// is measured in steps 32 times as wide each, then as much finer again: 2 log_32 looks.
template <typename Votes>
ZS_HOST_DEVICE int64_t run_reach(Votes votes) {
    int64_t reach = 0, stride = 1;
    for (bool more = true; more;) {
        const uint32_t in = votes(reach, stride);
        more = in == 0xffffffffu;
        reach += ones(in) * stride;
        if (more) stride *= 32;
    }
    for (; stride > 1;) {  // (the place `stride` further is not in the run)
        stride /= 32;
        reach += ones(votes(reach, stride)) * stride;
    }
    return reach;
}

}  // namespace zs
