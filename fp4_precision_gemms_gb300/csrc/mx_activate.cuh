// mx_activate.cuh -- the MLP's activations and their slopes, without act.cu's kernels.
#pragma once
#define MX_ACTIVATE_ONLY
#include "act.cu"
#undef MX_ACTIVATE_ONLY
