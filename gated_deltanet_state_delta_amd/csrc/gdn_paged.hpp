// gdn_paged.hpp -- internal launch entry points of the calls over paged
// caches (arguments already checked, as in gdn_kernels.hpp).
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/libgdn.h"

namespace gdn {

// Workspace with which launch_attn_decode splits the rows (0: it does not); sizes
// already checked.
size_t attn_workspace_bytes(const gdn_attn_decode_args& args);
hipError_t launch_attn_decode(const gdn_attn_decode_args& args, hipStream_t stream);
hipError_t launch_kv_append(const gdn_kv_append_args& args, hipStream_t stream);

hipError_t launch_pages_copy(void* pool, int64_t page_bytes, int64_t stride, int n_pages, const int32_t* src,
                             const int32_t* dst, int64_t n, hipStream_t stream);
size_t pages_workspace_bytes(int64_t rows, int64_t n_pages);
hipError_t launch_pages_extend(const gdn_pages_args& args, const int32_t* add, int32_t* ok, hipStream_t stream);
hipError_t launch_pages_fork(const gdn_pages_args& args, const int32_t* parent, int32_t* src, int32_t* dst,
                             hipStream_t stream);
hipError_t launch_pages_free(const gdn_pages_args& args, const uint8_t* mask, hipStream_t stream);
hipError_t launch_pages_compact(const gdn_pages_args& args, int32_t* src, int32_t* dst, int32_t* n_live,
                                hipStream_t stream);

}  // namespace gdn
