// cache.cu -- the 4-bit key/value cache outside its attention: block tables and
// slot map of a growing batch, pages given back, tokens quantised into their
// records, and read back.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache.cuh"
#include "cache_kernels.h"

namespace vsa {

namespace {

using namespace cache;

// ---------------------------------------------------------------------------
// Block tables and slot map
// ---------------------------------------------------------------------------
//
// Two prefix sums over the requests (their new tokens, their new pages) say
// which request a token or a taken page belongs to.  Every CTA makes them for
// itself in shared memory -- R <= 4096 lengths are 32 KB out of L2 -- and then
// fills its share of the slots and of the new table entries, finding the
// request by bisection; so the call is one launch with nothing to wait for.
// The bound is latency: the largest call writes some MB.  8 requests 4.4 to 5.0 us,
// 4096 requests with 1.02 M new tokens 11.9 to 12.3 us, of which the slots take half
// (four CTAs' worth of passes side by side, or eight tokens a thread, were slower).

// Threads of a CTA: with many requests the sums and look-ups of a thread are a
// chain, and twice the threads shorten it (4096 requests 11.8 us, 13.9 with 512);
// with few, more threads only cost (8 requests 4.4 us, 5.4 with 1024).
constexpr int kTabThreads = 512, kTabThreadsMany = 1024;

// Inclusive sum over the threads of a CTA of one value each.
__device__ __forceinline__ long long block_scan(long long v, long long* part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += u;
  }
  __syncthreads();  // part may still be read from the scan before
  if (lane == 31) part[warp] = v;
  __syncthreads();
  long long p = lane < static_cast<int>(blockDim.x >> 5) ? part[lane] : 0;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, p, d);
    if (lane >= d) p += u;
  }
  const long long before = __shfl_sync(0xffffffffu, p, warp > 0 ? warp - 1 : 0);
  return v + (warp > 0 ? before : 0);
}

// Place of entry i of an array in shared memory: neighbouring threads of the
// release, with 8 entries each at 4096 requests, start 9 words apart, in different
// banks; those of the tables, twice as many with 4 entries, 4 or 5 words, two to a
// bank.
__host__ __device__ constexpr int spread(int i) { return i + (i >> 3); }

// Largest i in [0, n) with a[i] <= x, given a[0] <= x.
__device__ __forceinline__ int last_at_most(const int* a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[spread(mid)] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kTabThreadsMany) cache_tables_kernel(const __grid_constant__ CacheTablesArgs a) {
  extern __shared__ int tab_smem[];
  __shared__ long long part[kTabThreadsMany / 32];
  __shared__ int s_pages;
  int* tok = tab_smem;            // [R + 1] first new token
  const int words = spread(a.R) + 1;
  int* pag = tok + words;         // [R + 1] first new page, from free_start
  int* len = pag + words;         // [R] cached tokens; -1: refused
  int* fresh = len + words;       // [R] new tokens, then new pages
  const int threads = blockDim.x;
  const int per = (a.R + threads - 1) / threads;
  const int r0 = min(static_cast<int>(threadIdx.x) * per, a.R), r1 = min(r0 + per, a.R);
  const int P = 1 << a.log_page;
  const long long cap = static_cast<long long>(a.max_pages) << a.log_page;
  const int start = __ldg(a.free_start);
  const bool lead = blockIdx.x == 0;
  if (threadIdx.x == 0) s_pages = 0;

  // lengths come in whole lines, then each thread looks after `per` requests
  for (int r = threadIdx.x; r < a.R; r += threads) {
    len[spread(r)] = __ldg(a.kv_len + r);
    fresh[spread(r)] = __ldg(a.new_len + r);
  }
  __syncthreads();

  // first new token of each request, cut at max_tokens
  long long sum = 0;
  for (int r = r0; r < r1; ++r) sum += max(fresh[spread(r)], 0);
  long long at = block_scan(sum, part) - sum, need_sum = 0;
  for (int r = r0; r < r1; ++r) {
    const int kv = len[spread(r)], nw = fresh[spread(r)];
    tok[spread(r)] = static_cast<int>(min(at, static_cast<long long>(a.max_tokens)));
    at += max(nw, 0);
    const long long end = static_cast<long long>(kv) + nw;
    const bool fits = kv >= 0 && nw >= 0 && end <= cap && at <= a.max_tokens;
    // new pages; -1: refused
    fresh[spread(r)] = fits ? static_cast<int>(((end + P - 1) >> a.log_page) - ((static_cast<long long>(kv) + P - 1) >> a.log_page)) : -1;
    need_sum += max(fresh[spread(r)], 0);
    if (lead) a.kv_len_out[r] = fits ? static_cast<int>(end) : kv;  // unless pages run out
  }
  if (r0 < r1 && r1 == a.R) tok[spread(a.R)] = static_cast<int>(min(at, static_cast<long long>(a.max_tokens)));

  // first new page of each request
  at = block_scan(need_sum, part) - need_sum;
  // free pages; a free_start outside [0, n_free] leaves none
  const long long have = start >= 0 && start <= a.n_free ? a.n_free - start : 0;
  int taken = 0;
  for (int r = r0; r < r1; ++r) {
    const int need = fresh[spread(r)], kv = len[spread(r)];
    pag[spread(r)] = static_cast<int>(min(at, have));
    if (need > 0) {
      at += need;
      if (at <= have) taken = static_cast<int>(at);
    }
    const bool ok = need == 0 || (need > 0 && at <= have);
    if (!ok) {
      len[spread(r)] = -1;
      if (lead) {
        a.kv_len_out[r] = kv;
        atomicCAS(a.status, 0u, (unsigned)VSA_ERR_CAPACITY);
      }
    }
  }
  if (r0 < r1 && r1 == a.R) pag[spread(a.R)] = static_cast<int>(min(at, have));
  if (taken > 0) atomicMax(&s_pages, taken);
  __syncthreads();
  const int pages = s_pages, tokens = tok[spread(a.R)];
  if (lead) {
    for (int r = threadIdx.x; r <= a.R; r += threads) a.cu[r] = tok[spread(r)];
    if (threadIdx.x == 0) *a.free_next = start + pages;
  }

  // entries of the pages taken: page i of a request's new ones follows those it has
  for (int e = blockIdx.x * threads + threadIdx.x; e < pages; e += gridDim.x * threads) {
    const int r = last_at_most(pag, a.R, e);
    const int had = (len[spread(r)] + P - 1) >> a.log_page;
    a.table[static_cast<long long>(r) * a.max_pages + had + (e - pag[spread(r)])] = __ldg(a.free_pages + start + e);
  }

  // slots; a token of a page taken now reads its id from the stack, not from the entry above
  const int page_limit = 0x7fffffff >> a.log_page;
  for (long long i0 = static_cast<long long>(blockIdx.x) * threads * 4 + threadIdx.x * 4; i0 < a.max_tokens;
       i0 += static_cast<long long>(gridDim.x) * threads * 4) {
    int4 out = make_int4(-1, -1, -1, -1);
    int* ov = &out.x;
    int r = i0 < tokens ? last_at_most(tok, a.R, static_cast<int>(i0)) : 0;
    int known_r = -1, known_pi = -1, page = -1;  // neighbours are mostly in one page
    for (int j = 0; j < 4; ++j) {
      if (i0 + j >= tokens) break;
      const int i = static_cast<int>(i0) + j;
      while (tok[spread(r + 1)] <= i) ++r;  // ends: tok[R] = tokens > i
      const int kv = len[spread(r)];
      if (kv < 0) continue;
      const int pos = kv + (i - tok[spread(r)]);
      const int pi = pos >> a.log_page;
      if (r != known_r || pi != known_pi) {
        known_r = r;
        known_pi = pi;
        const int had = (kv + P - 1) >> a.log_page;
        page = pi < had ? __ldg(a.table + static_cast<long long>(r) * a.max_pages + pi)
                        : __ldg(a.free_pages + start + pag[spread(r)] + (pi - had));
        if (page < 0 || page >= page_limit) {
          atomicCAS(a.status, 0u, (unsigned)VSA_ERR_BAD_INDEX);
          page = -1;
        }
      }
      if (page >= 0) ov[j] = (page << a.log_page) + (pos & (P - 1));
    }
    if (i0 + 4 <= a.max_tokens) {
      *reinterpret_cast<int4*>(a.slots + i0) = out;
    } else {
      for (int j = 0; i0 + j < a.max_tokens; ++j) a.slots[i0 + j] = ov[j];
    }
  }
}

// ---------------------------------------------------------------------------
// Pages given back
// ---------------------------------------------------------------------------

__global__ void __launch_bounds__(kTabThreads) cache_release_kernel(const uint8_t* __restrict__ drop, int R,
                                                                    int log_page, int32_t* kv_len,
                                                                    const int32_t* __restrict__ table, int max_pages,
                                                                    int32_t* free_pages, int n_free,
                                                                    int32_t* free_start, unsigned int* status) {
  extern __shared__ int tab_smem[];
  __shared__ long long part[kTabThreads / 32];
  __shared__ long long total;
  int* pag = tab_smem;  // [R + 1] first page given back
  const int per = (R + kTabThreads - 1) / kTabThreads;
  const int r0 = min(static_cast<int>(threadIdx.x) * per, R), r1 = min(r0 + per, R);
  const int P = 1 << log_page;
  const long long cap = static_cast<long long>(max_pages) << log_page;
  const int start = *free_start;
  if (threadIdx.x == 0) total = 0;
  auto pages_of = [&](int r) -> int {
    if (!drop[r]) return 0;
    const int kv = kv_len[r];
    if (kv < 0 || kv > cap) {
      atomicCAS(status, 0u, (unsigned)VSA_ERR_CAPACITY);
      return 0;
    }
    return static_cast<int>((static_cast<long long>(kv) + P - 1) >> log_page);
  };
  long long sum = 0;
  for (int r = r0; r < r1; ++r) sum += pages_of(r);
  const long long incl = block_scan(sum, part);
  if (threadIdx.x == kTabThreads - 1) total = incl;
  __syncthreads();
  const long long m = total;
  if (start < 0 || start > n_free || m > start) {
    if (threadIdx.x == 0) atomicCAS(status, 0u, (unsigned)VSA_ERR_CAPACITY);
    return;  // the whole CTA
  }
  long long at = incl - sum;
  for (int r = r0; r < r1; ++r) {
    pag[spread(r)] = static_cast<int>(at);
    at += pages_of(r);
  }
  if (threadIdx.x == 0) pag[spread(R)] = static_cast<int>(m);
  __syncthreads();
  const int base = start - static_cast<int>(m);
  for (int e = threadIdx.x; e < static_cast<int>(m); e += kTabThreads) {
    const int r = last_at_most(pag, R, e);
    free_pages[base + e] = table[static_cast<long long>(r) * max_pages + (e - pag[spread(r)])];
  }
  for (int r = r0; r < r1; ++r)
    if (drop[r]) kv_len[r] = 0;
  if (threadIdx.x == 0) *free_start = base;
}

// ---------------------------------------------------------------------------
// Append and read back
// ---------------------------------------------------------------------------
//
// A CTA takes 16 tokens x 2 heads: a warp holds 4 tokens of a head, 8 threads a
// token, a thread one 16-channel block of its K and of its V (64 bytes in, 16
// bytes of codes and 2 scales out).  Head pairs are the fast index of the grid:
// CTAs that run together move the same tokens' rows.  The scale of a block is the thread's own
// maximum, so nothing is exchanged but the 8 K scales of a token, which become
// two words.  Tokens are the warp's fast index because 16 tokens of a head
// share a record: its lines are written from one CTA.
// Bound: HBM (512 B in, 144 out a token and head).  27280 tokens x 24 heads: append
// 72 us and read back 74 us for 430 MB each, 6.0 and 5.8 TB/s.

constexpr int kPutThreads = 256;
constexpr int kPutTokens = 16, kPutHeads = 2;

template <bool F16>
__device__ __forceinline__ void unpack16(uint4 w0, uint4 w1, float (&f)[16]) {
  const uint32_t wd[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (F16) {
      const float2 x = f16x2_to_f32(wd[i]);
      f[2 * i] = x.x;
      f[2 * i + 1] = x.y;
    } else {
      f[2 * i] = bf16_lo(wd[i]);
      f[2 * i + 1] = bf16_hi(wd[i]);
    }
  }
}

// Codes of 16 values and their scale byte: s = E4M3(fl32(amax / 6)), code =
// E2M1(fl32(x * fl32(1 / s))), the rounding of vsa_quantize_nvfp4.  The quotient
// by 6 is q = amax c, q + c (amax - 6 q) with c = fl32(1 / 6) (Markstein's
// correction), which is the rounded one for every fp16 and bf16 amax between
// 2^-20 and 2^20; below, s is 0 either way, and above 2688 it saturates, so
// amax is cut at 3000.  `inverse` holds fl32(1 / s) of the 127 scales.
__device__ __forceinline__ uint2 quantise16(const float (&f)[16], const float* inverse, uint32_t& sb) {
  float m[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 16; i += 2) m[(i >> 1) & 3] = max3f(m[(i >> 1) & 3], fabsf(f[i]), fabsf(f[i + 1]));
  const float amax = fminf(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])), 3000.0f);
  constexpr float c = 1.0f / 6.0f;
  const float q = __fmul_rn(amax, c);
  sb = to_e4m3(__fmaf_rn(__fmaf_rn(-6.0f, q, amax), c, q));
  const float inv = inverse[sb];
  float y[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) y[i] = __fmul_rn(f[i], inv);
  return make_uint2(to_e2m1x8(y), to_e2m1x8(y + 8));
}

template <bool F16>
__global__ void __launch_bounds__(kPutThreads) cache_append_kernel(
    const uint16_t* __restrict__ k, const uint16_t* __restrict__ v, long long k_stride, long long v_stride,
    const int32_t* __restrict__ slots, int T, int Hkv, int pairs, uint8_t* __restrict__ pages, int num_pages,
    int log_page, unsigned int* status) {
  const int g = threadIdx.x & 7;  // 16-channel block
  const int group = blockIdx.x / pairs;
  const int t = group * kPutTokens + ((threadIdx.x >> 3) & 15);
  const int h = (blockIdx.x - group * pairs) * kPutHeads + (threadIdx.x >> 7);
  const bool in = t < T && h < Hkv;
  const int slot = in ? __ldg(slots + t) : -1;
  const bool bad = slot >= 0 && (slot >> log_page) >= num_pages;
  if (bad && g == 0) atomicCAS(status, 0u, (unsigned)VSA_ERR_BAD_INDEX);
  const bool put = slot >= 0 && !bad;
  __shared__ float inverse[128];
  uint4 w[4];
  if (put) {
    const uint4* kp = reinterpret_cast<const uint4*>(k + t * k_stride + h * 128 + g * 16);
    const uint4* vp = reinterpret_cast<const uint4*>(v + t * v_stride + h * 128 + g * 16);
    w[0] = __ldg(kp), w[1] = __ldg(kp + 1), w[2] = __ldg(vp), w[3] = __ldg(vp + 1);
  }
  if (threadIdx.x < 128) {
    const float s = f16x2_to_f32(from_e4m3x2(threadIdx.x)).x;
    inverse[threadIdx.x] = s == 0.0f ? 0.0f : __frcp_rn(s);
  }
  __syncthreads();
  uint32_t ks = 0, vs = 0;
  uint2 kc = make_uint2(0, 0), vc = make_uint2(0, 0);
  if (put) {
    float f[16];
    unpack16<F16>(w[0], w[1], f);
    kc = quantise16(f, inverse, ks);
    unpack16<F16>(w[2], w[3], f);
    vc = quantise16(f, inverse, vs);
  }
  // a token's eight K scales as two words
  uint32_t word = ks;
  word |= __shfl_down_sync(0xffffffffu, ks, 1) << 8;
  word |= __shfl_down_sync(0xffffffffu, ks, 2) << 16;
  word |= __shfl_down_sync(0xffffffffu, ks, 3) << 24;
  if (!put) return;
  const int p = slot & 15;
  uint8_t* rec = pages + record_of(slot, h, Hkv, log_page);
  reinterpret_cast<uint2*>(rec)[p * 8 + g] = kc;
  reinterpret_cast<uint2*>(rec + kRecV)[p * 8 + g] = vc;
  if ((g & 3) == 0) reinterpret_cast<uint32_t*>(rec + kRecKS)[p * 2 + (g >> 2)] = word;
  rec[kRecVS + g * 16 + (p & 3) * 4 + (p >> 2)] = static_cast<uint8_t>(vs);
}

// Eight values from a word of codes and their scale byte.
template <bool F16>
__device__ __forceinline__ uint4 values8(uint32_t codes, uint32_t sb) {
  const uint32_t s = dup_lo(from_e4m3x2(sb));
  uint32_t r[4];
  from_e2m1x8(codes, r);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[i] = mul_f16x2(r[i], s);
    if (!F16) {
      const float2 x = f16x2_to_f32(r[i]);
      r[i] = pack_bf16x2(x.x, x.y);
    }
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// Read back: 16 threads a token and head, so that a store is one whole row; a
// CTA takes 16 tokens x 2 heads, a thread one word of K and of V of both.
template <bool F16>
__global__ void __launch_bounds__(kPutThreads) cache_read_kernel(const int32_t* __restrict__ slots, int T, int Hkv,
                                                                 int pairs, const uint8_t* __restrict__ pages,
                                                                 int num_pages, int log_page, uint4* __restrict__ k,
                                                                 uint4* __restrict__ v, unsigned int* status) {
  const int x = threadIdx.x & 15, g = x >> 1;
  const int group = blockIdx.x / pairs;
  const int t = group * kPutTokens + (threadIdx.x >> 4);
  const int h0 = (blockIdx.x - group * pairs) * kPutHeads;
  if (t >= T) return;
  const int slot = __ldg(slots + t);
  if (slot < 0) return;
  if ((slot >> log_page) >= num_pages) {
    if (x == 0) atomicCAS(status, 0u, (unsigned)VSA_ERR_BAD_INDEX);
    return;
  }
  const int p = slot & 15;
#pragma unroll
  for (int i = 0; i < kPutHeads; ++i) {
    const int h = h0 + i;
    if (h >= Hkv) break;
    const uint8_t* rec = pages + record_of(slot, h, Hkv, log_page);
    const uint32_t kc = __ldg(reinterpret_cast<const uint32_t*>(rec) + p * 16 + x);
    const uint32_t vc = __ldg(reinterpret_cast<const uint32_t*>(rec + kRecV) + p * 16 + x);
    const uint32_t ks = __ldg(rec + kRecKS + p * 8 + g), vs = __ldg(rec + kRecVS + g * 16 + (p & 3) * 4 + (p >> 2));
    const long long dst = (static_cast<long long>(t) * Hkv + h) * 16 + x;
    k[dst] = values8<F16>(kc, ks);
    v[dst] = values8<F16>(vc, vs);
  }
}

int head_pairs(int Hkv) { return (Hkv + kPutHeads - 1) / kPutHeads; }
long long put_grid(int T, int Hkv) {
  return (static_cast<long long>(T) + kPutTokens - 1) / kPutTokens * head_pairs(Hkv);
}

}  // namespace

cudaError_t launch_cache_tables(const CacheTablesArgs& a, int num_sms, cudaStream_t stream) {
  const int threads = a.R > kTabThreads ? kTabThreadsMany : kTabThreads;
  const long long passes = (static_cast<long long>(a.max_tokens) + 4 * threads - 1) / (4 * threads);
  const int grid = static_cast<int>(passes < 1 ? 1 : passes < num_sms ? passes : num_sms);
  const int smem = 4 * (spread(a.R) + 1) * 4;
  if (smem > 40 * 1024) {  // more than the default limit only for R > 2275
    static SmemAllowed allowed;
    const cudaError_t e =
        allowed.ensure(reinterpret_cast<const void*>(cache_tables_kernel), 4 * (spread(kMaxRequests) + 1) * 4);
    if (e != cudaSuccess) return e;
  }
  cache_tables_kernel<<<grid, threads, smem, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_cache_release(const uint8_t* drop, int R, int log_page, int32_t* kv_len, const int32_t* table,
                                 int max_pages, int32_t* free_pages, int n_free, int32_t* free_start,
                                 unsigned int* status, cudaStream_t stream) {
  cache_release_kernel<<<1, kTabThreads, (spread(R) + 1) * 4, stream>>>(drop, R, log_page, kv_len, table, max_pages,
                                                                free_pages, n_free, free_start, status);
  return cudaGetLastError();
}

cudaError_t launch_cache_append(bool f16, const uint16_t* k, const uint16_t* v, long long k_stride,
                                long long v_stride, const int32_t* slots, int T, int Hkv, uint8_t* pages,
                                int num_pages, int log_page, unsigned int* status, cudaStream_t stream) {
  if (T == 0) return cudaSuccess;
  const long long grid = put_grid(T, Hkv);
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  auto kern = f16 ? cache_append_kernel<true> : cache_append_kernel<false>;
  kern<<<static_cast<unsigned>(grid), kPutThreads, 0, stream>>>(k, v, k_stride, v_stride, slots, T, Hkv,
                                                                head_pairs(Hkv), pages, num_pages, log_page, status);
  return cudaGetLastError();
}

cudaError_t launch_cache_read(bool f16, const int32_t* slots, int T, int Hkv, const uint8_t* pages, int num_pages,
                              int log_page, uint16_t* k, uint16_t* v, unsigned int* status, cudaStream_t stream) {
  if (T == 0) return cudaSuccess;
  const long long grid = put_grid(T, Hkv);
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  auto kern = f16 ? cache_read_kernel<true> : cache_read_kernel<false>;
  kern<<<static_cast<unsigned>(grid), kPutThreads, 0, stream>>>(slots, T, Hkv, head_pairs(Hkv), pages, num_pages,
                                                                log_page, reinterpret_cast<uint4*>(k),
                                                                reinterpret_cast<uint4*>(v), status);
  return cudaGetLastError();
}

}  // namespace vsa
