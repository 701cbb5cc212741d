// What the entry points with activations and experts share with the others.
#pragma once

#include <cstdint>

namespace fp8lite {

// The largest extent: the epilogues count a tile's rows and columns, up to 256
// past the last one, in 32 bits.
constexpr int64_t kMaxExtent = (int64_t(1) << 31) - 1024;

// The device error words of the source files that wait on the device (one
// each, see gemm_kernel.cuh). Reads and clears the word; false if that failed.
bool gemm_act_error(uint32_t* v);
bool experts_error(uint32_t* v);

}  // namespace fp8lite
