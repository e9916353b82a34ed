// Which kernel a scored routing and its gradient take: a function of the sizes
// alone, on the host.
#pragma once

#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kMaxList = 16;  // the longest list: larger k go to the whole wave's choice

// A token's lanes, the experts per lane, whether rows are whole 16-byte loads, and the
// length of a lane's list of keys.  list 0: a whole wave per token.
struct RouteKernel {
    int lanes, per_lane;
    bool words;
    int list;
};

// The fewest lanes that hold the experts, 8 each, 16 each beyond 128 (wider lists, fewer
// steps between lanes).  The wave's choice where k is more than fits a list (32768 x 256:
// k = 16 33 us by lists, k = 24 126 us by waves), or rows are shorter than a load.
RouteKernel route_kernel(const moe_gating_t& g) {
    if (g.k > kMaxList || g.E < 4) return {64, MOE_MAX_EXPERTS / 64, false, 0};
    return {g.E <= 32 ? 4 : (g.E <= 64 ? 8 : 16), g.E <= 128 ? 8 : 16, g.E % 4 == 0, g.k <= 4 ? 4 : (g.k <= 8 ? 8 : kMaxList)};
}

// The gradient: 8 experts per lane.
struct RouteBackKernel {
    int lanes;
    bool words;
};
RouteBackKernel route_back_kernel(const moe_gating_t& g) {
    return {g.E <= 32 ? 4 : (g.E <= 64 ? 8 : (g.E <= 128 ? 16 : 32)), g.E % 4 == 0};
}

}  // namespace

}  // namespace moe
