// attention_wide.h — the tcgen05 kernel of attention over a paged cache (larger query blocks).
#pragma once

#include "serving.h"

namespace dspark {

// Scratch bytes for the sizes (0: the kernel does not take them).
size_t attention_wide_scratch(int Hq, int Hkv, int D, int max_q);

// Launches it into `e` and returns true; false if these types, sizes or strides are not its own.
bool launch_attention_wide(const AttentionArgs& a, void* scratch, cudaStream_t s, cudaError_t& e);

}  // namespace dspark
