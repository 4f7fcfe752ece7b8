// rope.cuh -- rotary helpers shared by the kernels that turn q and k: the
// reduced-angle sine and cosine, and a row's positions.
#pragma once

#include "common.cuh"

namespace dit {

// angle mod 2*pi in fp64, then single precision: keeps the angle exact to
// ~1e-7 rad for any position.  On the reduced angle, in [-pi, pi], the
// hardware sine and cosine (__sincosf, absolute error ~1e-6 there) replace
// the full-range sincosf: with 24 q + 4 k heads of 128 per row the per-row
// setup is a large share of the work (long video 143.8 -> 141.3 us), and the
// outputs move by at most one bf16 unit in ~1e-4 of the elements.
__device__ __forceinline__ void pair_cos_sin(double angle, float& c, float& s)
{
    constexpr double kTwoPi = 6.283185307179586476925286766559;
    constexpr double kInvTwoPi = 0.15915494309189533576888376337251;
    const double red = angle - kTwoPi * rint(angle * kInvTwoPi);
    __sincosf((float)red, &s, &c);
}

// Positions of a row: a row inside its sequence's T x H x W video grid
// (t-major, then h, then w) is 3D; every later row is 1D, counted from the
// end of the grid.  Without a grid every row is 1D.
struct RowPosition {
    bool is3d;
    long long t, h, w;  // 3D
    long long line;     // 1D
};

// g >= 0: the row's index in its whole sequence; grid: the sequence's T, H, W
// or null.
__device__ __forceinline__ RowPosition row_position(long long g, const int32_t* __restrict__ grid)
{
    RowPosition r{false, 0, 0, 0, g};
    if (grid == nullptr)
        return r;
    const long long T = __ldg(grid), H = __ldg(grid + 1), W = __ldg(grid + 2);
    const long long thw = T * H * W;
    if (g >= thw) {
        r.line = g - thw;
        return r;
    }
    // g >= 0, so the grid is non-empty here
    r.is3d = true;
    const long long hw = H * W;
    if (hw > 0 && hw <= 0xffffffffLL) {
        // 32-bit divisions (g < 2^32 always): the row setup is a large share
        // of a narrow row's work (24 q + 4 k heads: 146.4 -> 144.2 us, results
        // unchanged)
        const unsigned gu = (unsigned)g, hwu = (unsigned)hw, wu = (unsigned)W;
        const unsigned t = gu / hwu, rem = gu - t * hwu, h = rem / wu;
        r.t = t;
        r.h = h;
        r.w = rem - h * wu;
    } else {
        r.t = g / hw;
        r.h = (g / W) % H;
        r.w = g % W;
    }
    return r;
}

}  // namespace dit
