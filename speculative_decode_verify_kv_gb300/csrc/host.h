// host.h -- host-side helpers shared by the files that implement the C ABI
// (abi.cu: verify path; abi_rows.cu: staging, prompt, tree and commit calls).
#pragma once

#include <cudaTypedefs.h>
#include <stddef.h>
#include <stdint.h>

namespace trtv {

constexpr size_t kSmemOptin = 232448;  // opt-in shared memory per block on sm_103
constexpr size_t kAlignSlack = 1024;

int sm_count();                               // of the current device; 0 on error
int* err_word();                              // device error word of the current device; null on error
PFN_cuTensorMapEncodeTiled_v12000 encoder();  // null when the driver has none
uint64_t wait_limit_ns();                     // bounded-wait settings of the next launches
int withheld_pages();

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace trtv
