// cache_attn.cu -- attention over the 4-bit key/value cache: which kernel takes
// which request.
#include "cache_kernels.h"

namespace vsa {

namespace {

constexpr int kWorkers = 160;  // CTAs of a call at most: one per SM, B200 has 148

// Requests of up to this many rows (new tokens times query heads of a key head)
// run the kernel for few rows, others the 256-row tiles of the tensor cores.
// Measured over 8000 cached tokens, causal, 4 query heads a key head, us on the
// device, the whole batch on few rows / on tensor cores:
//   requests x heads     24 rows     40 rows     64 rows     96 rows
//   1 x 12             23.7/26.8   30.1/27.5   33.3/27.5   41.2/28.2
//   9 x 3              33.5/41.0   44.9/41.4   52.8/41.6   71.7/42.6
//   32 x 8               186/293     272/294     358/295     526/298
//   9 x 3, ragged      29.4/41.0   33.3/41.2   41.4/41.6   53.3/42.5
//   32 x 8, ragged       133/292     171/293     231/294     327/295
// (ragged: lengths spread below the given one).  Even batches cross between 24 and
// 50 rows, ragged ones between 64 and 90.  One border serves both, and it lies where
// ragged batches cross, which are the usual ones; from there on a ragged batch runs
// both kernels in line (96 rows: 9 x 3 61.5, 32 x 8 281).
constexpr int kFewRows = 64;

}  // namespace

size_t cache_attn_workspace_bytes(int Hq, int Hkv, int max_q) {
  const bool many = static_cast<long long>(max_q) * (Hq / Hkv) > kFewRows;
  return cache_attn_small_workspace(kWorkers) + (many ? cache_attn_chunk_workspace(kWorkers) : 0);
}

cudaError_t launch_cache_attn(const cache::AttnArgs& a, bool f16, int max_q, int num_sms, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  const int workers = num_sms < kWorkers ? num_sms : kWorkers;
  const long long rows = static_cast<long long>(max_q) * a.G;
  if (rows <= kFewRows)
    return launch_cache_attn_small(a, 0, 0x7fffffff, f16, static_cast<int>(rows), workers, stream);
  // A batch of one request that may have many rows needs no second kernel for requests with few.
  const int over = a.R == 1 ? 0 : kFewRows;
  cache::AttnArgs b = a;
  b.ws = static_cast<char*>(a.ws) + cache_attn_small_workspace(kWorkers);
  if (over != 0) b.fill = 0;  // the second kernel does it
  cudaError_t e = launch_cache_attn_chunk(b, over, f16, workers, stream);
  if (e != cudaSuccess || over == 0) return e;
  return launch_cache_attn_small(a, 0, kFewRows, f16, kFewRows, workers, stream);
}

}  // namespace vsa
