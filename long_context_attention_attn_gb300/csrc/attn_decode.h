#pragma once
#include "internal.h"

namespace gb300 {

// launch_attn_decode with the cache's copies withheld (attn_decode_test_timeout):
// cudaErrorNotSupported, and nothing launched, where the kernel has no bounded waits.
cudaError_t launch_attn_decode(const attn_decode_params& p, bool withhold, cudaStream_t st);

// ---- attn_decode_shared.cu
cudaError_t decode_shared_workspace(const attn_decode_shared_params& p, size_t* bytes);
// (withhold: the shared keys' copies)
cudaError_t launch_attn_decode_shared(const attn_decode_shared_params& p, bool withhold, cudaStream_t st);

}  // namespace gb300
