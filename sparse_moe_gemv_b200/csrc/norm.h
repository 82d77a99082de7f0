// What norm.cu offers the other translation units of libredmoe.
#pragma once

#include "../../include/redmoe.h"

namespace redmoe {

// The argument checks of redmoe_norm_forward, without its launch.
redmoe_status norm_forward_check(const redmoe_norm* N, const void* h, const void* y, const void* gate, int T,
                                 const void* h_out, const void* x);

// Bytes of a gate for T rows, and of one weight.
size_t norm_gate_bytes(const redmoe_norm* N, int T);
size_t norm_weight_bytes(const redmoe_norm* N);

}  // namespace redmoe
