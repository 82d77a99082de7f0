// What norm.cu offers the other translation units of libredmoe.
#pragma once

#include "../../include/redmoe.h"

namespace redmoe {

// The argument checks of redmoe_norm_forward, without its launch.
redmoe_status norm_forward_check(const redmoe_norm* N, const void* h, const void* y, const void* gate, int T,
                                 const void* h_out, const void* x);

}  // namespace redmoe
