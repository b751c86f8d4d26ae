// The gated delta rule over prompts: token by token, as the recurrent form.
#include "delta_common.h"

namespace bqmm {

uint64_t delta_workspace_bytes(uint32_t tokens, uint32_t count, uint32_t hk, uint32_t hv, uint32_t dk) {
  const uint64_t chunks = tokens / 64u + (uint64_t)count;
  return chunks * (hv * 42240ull + hk * (dk <= 64u ? 8192ull : 16384ull));
}

hipError_t launch_delta_chunked(const DeltaArgs &a, hipStream_t s) { return launch_delta_recurrent(a, s); }

}  // namespace bqmm
