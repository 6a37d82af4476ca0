// host.h -- host-side helpers shared by the files that implement the C ABI
// (abi.cu: verify path; abi_rows.cu: staging, prompt, tree and commit calls).
#pragma once

#include <cudaTypedefs.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/trtv.h"

namespace trtv {

constexpr size_t kSmemOptin = 232448;  // opt-in shared memory per block on sm_103
constexpr size_t kAlignSlack = 1024;

int sm_count();                               // of the current device; 0 on error
int* err_word();                              // device error word of the current device; null on error
PFN_cuTensorMapEncodeTiled_v12000 encoder();  // null when the driver has none
uint64_t wait_limit_ns();                     // bounded-wait settings of the next launches
int withheld_pages();

struct RowsGeom;
// Geometry checks of the packed-row and page calls (abi_rows.cu).
trtv_status rows_geometry(const trtv_geom* g, const int32_t* indptr, int32_t num_tokens, RowsGeom* r);

// Dense ladder attention over an E2M1 cache (abi_rows.cu); g is not null.
trtv_status ladder_fp4(const trtv_geom* g, const void* q, const void* pool, const int32_t* page_table,
                       const int32_t* kv_lens, void* out, int32_t out_dtype, void* ws, size_t ws_bytes, void* stream);
size_t ladder_fp4_workspace(const trtv_geom* g);

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace trtv
