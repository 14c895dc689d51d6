// cache.cuh -- what the kernels of the 4-bit key/value cache share: the record
// of 16 tokens, the conversions from and to its codes and scales, and the
// requests of an attention call.
//
// The cache holds keys and values as NVFP4, the format of the fine stage's
// quantised Q and K (fp4.cu): E2M1 codes and one E4M3 scale per 16 channels.
// 16 tokens of one page and head are one record of 2304 contiguous bytes, so
// that a kernel fetches the keys, the values and their scales of 16 tokens with
// one bulk copy whatever the page size:
//   [   0,1024)  K codes, 64 B per token
//   [1024,2048)  V codes, 64 B per token
//   [2048,2176)  K scales, byte 8 t + g
//   [2176,2304)  V scales, byte 16 g + 4 (t % 4) + t / 4: the four tokens c,
//                c + 4, c + 8, c + 12 whose values one thread multiplies are
//                one word
//
// A code times its scale has at most 6 significant bits and lies between 2^-10
// and 2688 in magnitude, so every cached value is exact in fp16 and in bf16.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace vsa {
namespace cache {

constexpr int kRecTokens = 16;
constexpr int kRecBytes = 2304;
constexpr int kRecV = 1024, kRecKS = 2048, kRecVS = 2176;
constexpr int kMaxRequests = 4096;
// Softmax numerators are fp16 on their way into P V, and 2^8 at most against the
// maximum in use, which moves only when a score exceeds it by 8 (log2).  Taken
// against that maximum less kLift, with which the parts of a row and its lse are
// kept too, they reach 2^15, and what fp16 drops at its lower end is 2^-32 of the
// largest instead of 2^-25: over 126360 tokens a tail there can weigh 4e-3 of a
// row, and only P V would lose it, not the denominator.
constexpr float kLift = 7.0f;
// The longest wait of the attention kernels at one barrier; a call that waited
// longer ends with VSA_ERR_TIMEOUT.  A test's build sets it to nothing to see
// the way out; copies in flight are always given kDrainNs to land.
#ifndef VSA_CACHE_WAIT_NS
#define VSA_CACHE_WAIT_NS 2000000000
#endif
constexpr uint64_t kWaitNs = VSA_CACHE_WAIT_NS;
constexpr uint64_t kDrainNs = 2000000000;

// Eight fp32 values -> eight E2M1 codes in one word; value 0 in the low nibble
// of byte 0.  Round to nearest, ties to even, saturate at +-6.
__device__ __forceinline__ uint32_t to_e2m1x8(const float* x) {
  uint32_t r;
  asm("{\n\t.reg .b8 c0, c1, c2, c3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c3, %8, %7;\n\t"
      "mov.b32 %0, {c0, c1, c2, c3};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

// fp32 -> E4M3 bits (nearest, ties to even, saturating at 448).
__device__ __forceinline__ uint32_t to_e4m3(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(x), "f"(0.0f));
  return r & 0xffu;
}

// The four code pairs of a word as fp16x2 (exact): byte j's low nibble in the
// low half of r[j].
__device__ __forceinline__ void from_e2m1x8(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}

// Two E4M3 scales (the low 16 bits) as fp16x2, the low byte in the low half.
__device__ __forceinline__ uint32_t from_e4m3x2(uint32_t b) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<unsigned short>(b)));
  return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// One half of a pair in both places.
__device__ __forceinline__ uint32_t dup_lo(uint32_t x) {
  uint32_t d;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {l, l};\n\t}" : "=r"(d) : "r"(x));
  return d;
}
__device__ __forceinline__ uint32_t dup_hi(uint32_t x) {
  uint32_t d;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {h, h};\n\t}" : "=r"(d) : "r"(x));
  return d;
}
__device__ __forceinline__ float2 f16x2_to_f32(uint32_t x) {
  return __half22float2(*reinterpret_cast<const __half2*>(&x));
}

// Byte offset of the record of a slot's 16 tokens for head h.
__device__ __forceinline__ long long record_of(int slot, int h, int Hkv, int log_page) {
  const int page = slot >> log_page, in = slot & ((1 << log_page) - 1);
  return ((static_cast<long long>(page) * Hkv + h) * ((1 << log_page) >> 4) + (in >> 4)) * kRecBytes;
}

// One attention call, as the kernels see it.
struct AttnArgs {
  const uint16_t* q;
  long long q_stride;
  const int32_t* cu;
  const int32_t* kv_len;
  int R, T;
  int Hq, Hkv, G;  // G = Hq / Hkv query heads share a key head
  const uint8_t* pages;
  int num_pages, log_page;
  const int32_t* table;
  int max_pages;
  int causal;
  uint16_t* o;
  float* lse;
  void* ws;
  unsigned int* status;
  float scale_log2;  // log2(e) / sqrt(D)
  int fill;          // rows outside every request: 1: o = 0, 2: lse = -inf, 0: left as they were
};

// A request's new tokens [q0, q0 + n) of the batch and its cached tokens, cut
// to what the buffers hold.
struct Request {
  int q0, n, kv;
};
__device__ __forceinline__ Request load_request(const AttnArgs& a, int r, bool report) {
  const int c0 = __ldg(a.cu + r), c1 = __ldg(a.cu + r + 1), kv = __ldg(a.kv_len + r);
  Request q;
  q.q0 = min(max(c0, 0), a.T);
  q.n = min(max(c1, q.q0), a.T) - q.q0;
  const long long cap = static_cast<long long>(a.max_pages) << a.log_page;
  q.kv = static_cast<int>(min(static_cast<long long>(max(kv, 0)), cap));
  if (report && (q.q0 != c0 || q.q0 + q.n != c1 || q.kv != kv)) atomicCAS(a.status, 0u, (unsigned)VSA_ERR_BAD_INDEX);
  return q;
}

// The rows before the first request and behind the last, as a.fill says: one
// pass over them by all threads of the grid.  A call, because inlined it makes
// the kernel for few rows spill.
static __device__ __noinline__ void fill_rows(const AttnArgs& a) {
  const long long before = min(max(__ldg(a.cu), 0), a.T);
  const long long behind = min(max(static_cast<long long>(__ldg(a.cu + a.R)), before), static_cast<long long>(a.T));
  const long long rows = before + a.T - behind;
  const int grid = gridDim.x * gridDim.y, cta = blockIdx.y * gridDim.x + blockIdx.x;
  const long long first = static_cast<long long>(cta) * blockDim.x + threadIdx.x;
  const long long step = static_cast<long long>(grid) * blockDim.x;
  const int chunks = a.Hq * 16;  // of 16 bytes in a row of o
  if (a.fill & 1)
    for (long long i = first; i < rows * chunks; i += step)
      reinterpret_cast<uint4*>(a.o)[i < before * chunks ? i : i + (behind - before) * chunks] = make_uint4(0, 0, 0, 0);
  if (a.fill & 2)
    for (long long i = first; i < rows * a.Hq; i += step)
      a.lse[i < before * a.Hq ? i : i + (behind - before) * a.Hq] = -INFINITY;
}

// The cached positions that a request's new token i sees: [0, limit).
__device__ __forceinline__ int visible(const AttnArgs& a, const Request& q, int i) {
  return a.causal ? max(0, q.kv - q.n + i + 1) : q.kv;
}

}  // namespace cache
}  // namespace vsa
