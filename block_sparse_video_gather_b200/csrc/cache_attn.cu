// cache_attn.cu -- attention over the 4-bit key/value cache: which kernel a
// call runs.
#include "cache_kernels.h"

namespace vsa {

namespace {

constexpr int kWorkers = 160;  // CTAs of a call at most: one per SM, B200 has 148

}  // namespace

size_t cache_attn_workspace_bytes(int, int, int) { return cache_attn_small_workspace(kWorkers); }

cudaError_t launch_cache_attn(const cache::AttnArgs& a, bool f16, int max_q, int num_sms, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  const int workers = num_sms < kWorkers ? num_sms : kWorkers;
  const long long rows = static_cast<long long>(max_q) * a.G;
  return launch_cache_attn_small(a, 0, 0x7fffffff, f16, rows > 16 ? 16 : static_cast<int>(rows), workers, stream);
}

}  // namespace vsa
