// The device error words of the source files that wait on the device (one
// each, see gemm_kernel.cuh). Reads and clears the word; false if that failed.
#pragma once

#include <cstdint>

namespace fp8lite {

bool gemm_act_error(uint32_t* v);
bool experts_error(uint32_t* v);

}  // namespace fp8lite
