// mx_activate.cuh -- the MLP's activations and their slopes, without act.cu's kernels.  They
// stay in act.cu because a test reads the polynomials of GELU's tail from its text.
#pragma once
#define MX_ACTIVATE_ONLY
#include "act.cu"
#undef MX_ACTIVATE_ONLY
