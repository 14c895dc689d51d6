// cache_attn_small.cu -- attention over the 4-bit cache for few rows a request:
// a decoded token, or some drafted ones.
//
// Bound: HBM.  A cached token and head are 144 bytes, 0.022 ns at 6561 GB/s;
// the work beside the loads is to make 256 fp16 values of them.  What the
// design does about both:
//  - The line of 16-token units (cache_sched.cuh) is cut evenly over the CTAs,
//    one per SM, and a CTA's share evenly over its warps.  A warp works alone:
//    its own ring of records (one bulk copy of 2304 bytes each, four in
//    flight, 36 KB or more per SM), its own softmax state.
//  - Rows are the narrow side of the products: S^T = K Q^T and O^T = V^T P^T
//    with m16n8k16, 16 keys or channels by 8 rows.  At one row to a key head
//    that leaves 7/8 of a product unused, and the tensor pipe still idles; the
//    128-row products of tcgen05 would leave 127/128 (and its operands would
//    have to go through shared memory).  Codes become A fragments in
//    registers, from the words as they lie: which 32 channels a thread
//    multiplies, and which four keys, is free as long as Q, P and the output
//    agree, so that K is read as one 16-byte word a key and V as one 8-byte
//    word a key with no bank conflict, and the two keys of a fragment are
//    joined nibble by nibble before they are converted.
//  - A value is code * scale in fp16, exact (cache.cuh).  q is exact too: fp16
//    as it is, bf16 times a power of two per row that brings its largest
//    magnitude to [2^14, 2^15) (what underflows there is below 2^-39 of the
//    largest).  Only the numerators are rounded, to fp16.
//  - Online softmax in the log2 domain; the maximum moves (and the output is
//    rescaled) only when a score exceeds it by 8, so one vote per unit takes
//    the place of the reduction.
// Sums, maxima and denominators are fp32.  Parts are joined in a fixed order:
// the result does not depend on which CTA comes last.
#include <cuda_fp16.h>

#include "cache.cuh"
#include "cache_kernels.h"
#include "cache_sched.cuh"

namespace vsa {

namespace {

using namespace cache;

constexpr int kStages = 4;                       // records in flight per warp
constexpr uint64_t kTimeoutNs = 2000000000ull;   // 2 s per wait
constexpr int kMinUnits = 4;                     // units a warp gets at least

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Transpose of an 8 x 8 matrix of 16-bit values held two to a lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
  return d;
}
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// Part of an item that a warp or CTA holds; item0 < 0: none.
struct PieceMeta {
  long long item0;
  int nu, r, h, j;
};

template <int NT, int W>
struct Smem {
  static constexpr int kRows = 8 * NT;
  static constexpr size_t kPieceBytes = part_floats<kRows>() * 4;
  alignas(16) uint8_t ring[W][kStages][kRecBytes];
  alignas(16) uint8_t piece[W][kPieceBytes];  // a warp's first item, begun before its range
  PieceMeta meta[2 * W];                      // [2 w]: that item, [2 w + 1]: one that goes on after its range
  long long part[W];
  uint64_t full[W][kStages];
  int have[W][kStages];  // 1: the record was loaded
  int abort;
  int join[2];
};

// One row of a part: 128 sums (4 to a lane), maximum and denominator.
struct RowPart {
  float4 o;
  float m, l;
};
__device__ __forceinline__ void add_part(RowPart& t, float4 o, float w, float l) {
  t.o.x += w * o.x;
  t.o.y += w * o.y;
  t.o.z += w * o.z;
  t.o.w += w * o.w;
  t.l += w * l;
}
// Weight of a part with maximum m under the joint maximum.
__device__ __forceinline__ float part_weight(float m, float joint) {
  return m == -INFINITY ? 0.0f : ex2_approx(m - joint);
}

template <bool F16>
__device__ __forceinline__ void write_row(const AttnArgs& a, const Request& req, int h, int row, const RowPart& t) {
  const int lane = threadIdx.x & 31;
  const int token = row / a.G;
  const long long dst = (static_cast<long long>(req.q0) + token) * a.Hq + h * a.G + (row - token * a.G);
  const float inv = t.l != 0.0f ? 1.0f / t.l : 0.0f;
  uint2 w;
  w.x = pack_half2<F16>(t.o.x * inv, t.o.y * inv);
  w.y = pack_half2<F16>(t.o.z * inv, t.o.w * inv);
  reinterpret_cast<uint2*>(a.o + dst * 128)[lane] = w;
  if (lane == 0) a.lse[dst] = t.l != 0.0f ? (t.m + __log2f(t.l)) * 0.69314718055994531f : -INFINITY;
}

template <int NT, bool F16, int W>
__global__ void __launch_bounds__(W * 32, 1)
    cache_attn_small_kernel(const __grid_constant__ AttnArgs a, const Share share) {
  constexpr int RT = 8 * NT;
  using S = Sched<RT, kRecTokens>;
  using Sm = Smem<NT, W>;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Sm& sm = *reinterpret_cast<Sm*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;

  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&sm.full[warp][s], 1);
    sm.meta[2 * warp].item0 = sm.meta[2 * warp + 1].item0 = -1;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (threadIdx.x == 0) {
    sm.abort = 0;
    sm.join[0] = sm.join[1] = 0;
  }
  // the sums over requests take the place of the warps' pieces until every warp has found its own
  long long* pre = reinterpret_cast<long long*>(&sm.piece[0][0]);
  static_assert(sizeof(sm.piece) >= (kMaxRequests + 1) * 8, "the requests' sums must fit");
  scan_units<S, W * 32>(a, share, pre, sm.part);
  const long long U = pre[a.R];
  if (U == 0) return;
  const long long wanted = (U + W * kMinUnits - 1) / (W * kMinUnits);
  const int N = wanted < gridDim.x ? static_cast<int>(wanted) : static_cast<int>(gridDim.x);
  const int cta = blockIdx.x;
  if (cta >= N) return;
  const long long cs = range_start(U, cta, N), ce = range_start(U, cta + 1, N);
  const long long ws = cs + (ce - cs) * warp / W, we = cs + (ce - cs) * (warp + 1) / W;
  const int total = static_cast<int>(we - ws);

  Cursor<S> cc;
  if (total > 0) cc.seek(a, pre, ws);
  __syncthreads();

  bool ok = true;
  int issued = 0;
  if (total > 0) {
    // ---- loads: a cursor of their own, kStages units ahead
    Cursor<S> lc = cc;
    int lkeys = S::keys(a, lc.req, lc.j);
    int cache_r = -1, cache_p = 0, my_page = -1;  // 32 entries of the request's row of the table, one a lane
    const int rec_per_page = 1 << (a.log_page - 4);
    auto issue = [&]() {
      const int s = issued % kStages;
      const int key0 = lc.k * kRecTokens;
      bool load = key0 < lkeys;
      int page = -1;
      if (load) {
        const int pi = key0 >> a.log_page;
        if (lc.r != cache_r || pi < cache_p || pi >= cache_p + 32) {
          cache_r = lc.r;
          cache_p = pi;
          const int last = (lc.req.kv - 1) >> a.log_page;
          my_page = pi + lane <= last ? __ldg(a.table + static_cast<long long>(lc.r) * a.max_pages + pi + lane) : -1;
        }
        page = __shfl_sync(0xffffffffu, my_page, pi - cache_p);
        load = page >= 0 && page < a.num_pages;
        if (!load && lane == 0) atomicCAS(a.status, 0u, (unsigned)VSA_ERR_BAD_INDEX);
      }
      if (lane == 0) {
        sm.have[warp][s] = load;
        if (load) {
          const uint8_t* src =
              a.pages + ((static_cast<long long>(page) * a.Hkv + lc.h) * rec_per_page + (lc.k & (rec_per_page - 1))) *
                            kRecBytes;
          mbar_arrive_expect_tx(&sm.full[warp][s], kRecBytes);
          bulk_load(sm.ring[warp][s], src, kRecBytes, &sm.full[warp][s]);
        } else {
          mbar_arrive(&sm.full[warp][s]);
        }
      }
      ++issued;
      if (issued < total && ++lc.k == lc.nu) {
        lc.next_item(a, share);
        lkeys = S::keys(a, lc.req, lc.j);
      }
    };
    for (int i = 0; i < kStages && i < total; ++i) issue();

    uint32_t qf[NT][16];
    float rs[NT][2], m[NT][2], l[NT][2];
    int lim[NT][2];
    float acc[NT][8][4];
    int lim_min = 0;
    bool from_start = false;

    for (int i = 0; i < total; ++i) {
      if (i == 0 || cc.k == 0) {
        // ---- a new item: its rows of q as B fragments, thread (g, c) channels 32 c .. 32 c + 31 of row g
        from_start = cc.k == 0;
        const int rows = cc.req.n * a.G;
        lim_min = visible(a, cc.req, cc.j * RT / a.G);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int row = cc.j * RT + n * 8 + g;
          const int token = row / a.G;
          float amax = 0.0f;
          if (row < rows) {
            const uint4* src = reinterpret_cast<const uint4*>(
                a.q + (static_cast<long long>(cc.req.q0) + token) * a.q_stride + (cc.h * a.G + row - token * a.G) * 128 +
                c * 32);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint4 w = __ldg(src + x);
              qf[n][4 * x] = w.x, qf[n][4 * x + 1] = w.y, qf[n][4 * x + 2] = w.z, qf[n][4 * x + 3] = w.w;
            }
          } else {
#pragma unroll
            for (int x = 0; x < 16; ++x) qf[n][x] = 0u;
          }
          float inv = 1.0f;
          if (!F16) {
#pragma unroll
            for (int x = 0; x < 16; ++x) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(qf[n][x])), fabsf(bf16_hi(qf[n][x]))));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            const int e = __float_as_uint(amax) >> 23;
            const int up = amax == 0.0f || e == 255 ? 0 : min(141 - e, 100);  // 2^up * amax in [2^14, 2^15)
            const float f = __uint_as_float((up + 127) << 23);
            inv = __uint_as_float((127 - up) << 23);
#pragma unroll
            for (int x = 0; x < 16; ++x) qf[n][x] = pack_f16x2(bf16_lo(qf[n][x]) * f, bf16_hi(qf[n][x]) * f);
          }
          // scores are held by (key, rows 2c and 2c + 1)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            rs[n][e] = a.scale_log2 * __shfl_sync(0xffffffffu, inv, 8 * c + 4 * e);
            const int r2 = cc.j * RT + n * 8 + 2 * c + e;
            lim[n][e] = visible(a, cc.req, min(r2, rows - 1) / a.G);
            m[n][e] = -INFINITY;
            l[n][e] = 0.0f;
          }
#pragma unroll
          for (int x = 0; x < 8; ++x) acc[n][x][0] = acc[n][x][1] = acc[n][x][2] = acc[n][x][3] = 0.0f;
        }
      }

      const int s = i % kStages;
      ok = mbar_wait(&sm.full[warp][s], (i / kStages) & 1, &sm.abort, a.status, kTimeoutNs);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      if (sm.have[warp][s]) {
        const uint8_t* rec = sm.ring[warp][s];
        const int key0 = cc.k * kRecTokens;
        // ---- S^T = K Q^T: row x of the 16 keys is token 8 (x / 8) + 4 (x & 1) + ((x & 7) >> 1)
        float sc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.0f;
        const int ta = 4 * (g & 1) + (g >> 1);
        {
          const uint4 ka = *reinterpret_cast<const uint4*>(rec + ta * 64 + c * 16);
          const uint4 kb = *reinterpret_cast<const uint4*>(rec + (ta + 8) * 64 + c * 16);
          const uint32_t sa = from_e4m3x2(*reinterpret_cast<const uint16_t*>(rec + kRecKS + ta * 8 + 2 * c));
          const uint32_t sb = from_e4m3x2(*reinterpret_cast<const uint16_t*>(rec + kRecKS + (ta + 8) * 8 + 2 * c));
          const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t s1 = x < 2 ? dup_lo(sa) : dup_hi(sa), s2 = x < 2 ? dup_lo(sb) : dup_hi(sb);
            uint32_t va[4], vb[4];
            from_e2m1x8(wa[x], va);
            from_e2m1x8(wb[x], vb);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint32_t f[4] = {mul_f16x2(va[2 * y], s1), mul_f16x2(vb[2 * y], s2), mul_f16x2(va[2 * y + 1], s1),
                                     mul_f16x2(vb[2 * y + 1], s2)};
#pragma unroll
              for (int n = 0; n < NT; ++n) mma16816(sc[n], f, qf[n][4 * x + 2 * y], qf[n][4 * x + 2 * y + 1]);
            }
          }
        }
        // ---- softmax over the keys
        bool grow = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[n][e] *= rs[n][e & 1];
          if (key0 + kRecTokens > lim_min) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (key0 + ta + 8 * (e >> 1) >= lim[n][e & 1]) sc[n][e] = -INFINITY;
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) grow |= fmaxf(sc[n][e], sc[n][e + 2]) > m[n][e] + 8.0f;
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float t = fmaxf(sc[n][e], sc[n][e + 2]);
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
              if (t > m[n][e] + 8.0f) {
                const float alpha = part_weight(m[n][e], t);
                m[n][e] = t;
                l[n][e] *= alpha;
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                  acc[n][x][e] *= alpha;
                  acc[n][x][e + 2] *= alpha;
                }
              }
            }
        }
        uint32_t pb[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float base = m[n][e] == -INFINITY ? 0.0f : m[n][e];
            sc[n][e] = ex2_approx(sc[n][e] - base);
            sc[n][e + 2] = ex2_approx(sc[n][e + 2] - base);
            l[n][e] += sc[n][e] + sc[n][e + 2];
          }
          pb[n][0] = transpose8x8(pack_f16x2(sc[n][0], sc[n][1]));
          pb[n][1] = transpose8x8(pack_f16x2(sc[n][2], sc[n][3]));
        }
        // ---- O^T += V^T P^T: thread (g, c) has channels 16 g .. 16 g + 15 of tokens c, c + 4, c + 8, c + 12
        {
          uint2 w[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) w[x] = *reinterpret_cast<const uint2*>(rec + kRecV + (c + 4 * x) * 64 + g * 8);
          uint32_t vs = *reinterpret_cast<const uint32_t*>(rec + kRecVS + g * 16 + c * 4);
          if (key0 + kRecTokens > cc.req.kv) {
            // nothing was stored behind the last token: its scales may be NaN
            const int left = cc.req.kv - key0;
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (c + 4 * x >= left) vs &= ~(0xffu << (8 * x));
          }
          const uint32_t s01 = from_e4m3x2(vs & 0xffffu), s23 = from_e4m3x2(vs >> 16);
          constexpr uint32_t lo = 0x0f0f0f0fu, hi = 0xf0f0f0f0u;
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t w0 = y ? w[0].y : w[0].x, w1 = y ? w[1].y : w[1].x;
            const uint32_t w2 = y ? w[2].y : w[2].x, w3 = y ? w[3].y : w[3].x;
            uint32_t e01[4], o01[4], e23[4], o23[4];  // even and odd channels, two tokens to a word
            from_e2m1x8((w0 & lo) | ((w1 << 4) & hi), e01);
            from_e2m1x8(((w0 >> 4) & lo) | (w1 & hi), o01);
            from_e2m1x8((w2 & lo) | ((w3 << 4) & hi), e23);
            from_e2m1x8(((w2 >> 4) & lo) | (w3 & hi), o23);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint32_t f[4] = {mul_f16x2(e01[x], s01), mul_f16x2(o01[x], s01), mul_f16x2(e23[x], s23),
                                     mul_f16x2(o23[x], s23)};
#pragma unroll
              for (int n = 0; n < NT; ++n) mma16816(acc[n][4 * y + x], f, pb[n][0], pb[n][1]);
            }
          }
        }
      }
      __syncwarp();  // the record has been read
      if (issued < total) issue();

      const bool done = cc.k + 1 == cc.nu;
      if (done || i + 1 == total) {
        // ---- the item, or the warp's share of it, is complete: thread (g, c) holds channels 16 g .. of rows 2c, 2c + 1
        const int rows = cc.req.n * a.G - cc.j * RT;
        float* piece = reinterpret_cast<float*>(from_start ? sm.ring[warp][0] : sm.piece[warp]);
        static_assert(Sm::kPieceBytes <= kStages * kRecBytes, "the last piece takes the place of the ring");
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float t = l[n][e];
            t += __shfl_xor_sync(0xffffffffu, t, 4);
            t += __shfl_xor_sync(0xffffffffu, t, 8);
            t += __shfl_xor_sync(0xffffffffu, t, 16);
            const int row = n * 8 + 2 * c + e;
            if (row >= rows) continue;
            if (from_start && done) {
              const int rr = cc.j * RT + row, token = rr / a.G;
              const long long dst =
                  (static_cast<long long>(cc.req.q0) + token) * a.Hq + cc.h * a.G + (rr - token * a.G);
              const float inv = t != 0.0f ? 1.0f / t : 0.0f;
              uint32_t w[8];
#pragma unroll
              for (int x = 0; x < 8; ++x) w[x] = pack_half2<F16>(acc[n][x][e] * inv, acc[n][x][e + 2] * inv);
              uint4* out = reinterpret_cast<uint4*>(a.o + dst * 128 + g * 16);
              out[0] = make_uint4(w[0], w[1], w[2], w[3]);
              out[1] = make_uint4(w[4], w[5], w[6], w[7]);
              if (g == 0) a.lse[dst] = t != 0.0f ? (m[n][e] + __log2f(t)) * 0.69314718055994531f : -INFINITY;
            } else {
              float4* out = reinterpret_cast<float4*>(piece + row * 128 + g * 16);
#pragma unroll
              for (int x = 0; x < 4; ++x)
                out[x] = make_float4(acc[n][2 * x][e], acc[n][2 * x][e + 2], acc[n][2 * x + 1][e], acc[n][2 * x + 1][e + 2]);
              if (g == 0) {
                piece[RT * 128 + row] = m[n][e];
                piece[RT * 129 + row] = t;
              }
            }
          }
        if (!(from_start && done) && lane == 0)
          sm.meta[2 * warp + (from_start ? 1 : 0)] = PieceMeta{cc.item0, cc.nu, cc.r, cc.h, cc.j};
        if (i + 1 < total) cc.next_item(a, share);
      } else {
        ++cc.k;
      }
    }
    if (!ok) {
      // a wait ran out: every copy issued must land before the CTA's shared memory is released
      for (int s = 0; s < kStages; ++s)
        if (issued > s) {
          const int last = issued - 1 - ((issued - 1 - s) % kStages);
          mbar_wait_drain(&sm.full[warp][s], (last / kStages) & 1, kTimeoutNs);
        }
    }
  }
  __syncthreads();
  if (sm.abort) return;

  // ---- join the warps' pieces of each item, all warps over its rows
  int* counters = static_cast<int*>(a.ws);
  float* parts = reinterpret_cast<float*>(counters + kMaxWorkers);
  constexpr size_t kPart = part_floats<RT>();
  PieceMeta cross[2];  // items that go beyond the CTA: begun before it, going on after it
  cross[0].item0 = cross[1].item0 = -1;
  for (int p0 = 0; p0 < 2 * W;) {
    const PieceMeta mt = sm.meta[p0];
    if (mt.item0 < 0) {
      ++p0;
      continue;
    }
    int p1 = p0 + 1;
    while (p1 < 2 * W && (sm.meta[p1].item0 < 0 || sm.meta[p1].item0 == mt.item0)) ++p1;
    const Request req = load_request(a, mt.r, false);
    const int rows = min(RT, req.n * a.G - mt.j * RT);
    const bool whole = mt.item0 >= cs && mt.item0 + mt.nu <= ce;
    const int slot = mt.item0 < cs ? 0 : 1;
    if (!whole) cross[slot] = mt;
    for (int row = warp; row < rows; row += W) {
      RowPart t;
      t.m = -INFINITY;
      t.l = 0.0f;
      t.o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      auto piece_of = [&](int p) -> const float* {
        return reinterpret_cast<const float*>(p & 1 ? &sm.ring[p >> 1][0][0] : &sm.piece[p >> 1][0]);
      };
      for (int p = p0; p < p1; ++p)
        if (sm.meta[p].item0 >= 0) t.m = fmaxf(t.m, piece_of(p)[RT * 128 + row]);
      for (int p = p0; p < p1; ++p)
        if (sm.meta[p].item0 >= 0) {
          const float* f = piece_of(p);
          // a piece without a maximum has nothing but zeros, or the NaN of its scores
          const float pm = f[RT * 128 + row], w = pm == -INFINITY ? 1.0f : part_weight(pm, t.m);
          add_part(t, reinterpret_cast<const float4*>(f + row * 128)[lane], w, f[RT * 129 + row]);
        }
      if (whole) {
        write_row<F16>(a, req, mt.h, mt.j * RT + row, t);
      } else {
        float* f = parts + (static_cast<size_t>(cta) * 2 + slot) * kPart;
        reinterpret_cast<float4*>(f + row * 128)[lane] = t.o;
        if (lane == 0) {
          f[RT * 128 + row] = t.m;
          f[RT * 129 + row] = t.l;
        }
      }
    }
    p0 = p1;
  }
  if (cross[0].item0 < 0 && cross[1].item0 < 0) return;

  // ---- join the CTAs' parts: the last of an item's CTAs to arrive, in the order of the line
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int x = 0; x < 2; ++x)
      if (cross[x].item0 >= 0) {
        const int first = worker_of(U, cross[x].item0, N), last = worker_of(U, cross[x].item0 + cross[x].nu - 1, N);
        if (atomicAdd(counters + first, 1) == last - first) {
          counters[first] = 0;  // as the next call finds it
          sm.join[x] = 1;
        }
      }
    __threadfence();
  }
  __syncthreads();
  for (int x = 0; x < 2; ++x) {
    if (!sm.join[x]) continue;
    const PieceMeta mt = cross[x];
    const Request req = load_request(a, mt.r, false);
    const int first = worker_of(U, mt.item0, N), last = worker_of(U, mt.item0 + mt.nu - 1, N);
    const int rows = min(RT, req.n * a.G - mt.j * RT);
    for (int row = warp; row < rows; row += W) {
      auto part_of = [&](int w) { return parts + (static_cast<size_t>(w) * 2 + (w == first ? 1 : 0)) * kPart; };
      RowPart t;
      t.m = -INFINITY;
      t.l = 0.0f;
      t.o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int w = first + lane; w <= last; w += 32) t.m = fmaxf(t.m, __ldcg(part_of(w) + RT * 128 + row));
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) t.m = fmaxf(t.m, __shfl_xor_sync(0xffffffffu, t.m, d));
#pragma unroll 4
      for (int w = first; w <= last; ++w) {
        const float* f = part_of(w);
        const float pm = __ldcg(f + RT * 128 + row), pw = pm == -INFINITY ? 1.0f : part_weight(pm, t.m);
        add_part(t, __ldcg(reinterpret_cast<const float4*>(f + row * 128) + lane), pw, __ldcg(f + RT * 129 + row));
      }
      write_row<F16>(a, req, mt.h, mt.j * RT + row, t);
    }
  }
}

template <int NT, int W>
cudaError_t launch_small(const AttnArgs& a, const Share& share, bool f16, int num_sms, cudaStream_t stream) {
  auto kern = f16 ? cache_attn_small_kernel<NT, true, W> : cache_attn_small_kernel<NT, false, W>;
  constexpr int smem = static_cast<int>(sizeof(Smem<NT, W>));
  static_assert(smem <= 227 * 1024, "shared memory of a CTA");
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<num_sms < kMaxWorkers ? num_sms : kMaxWorkers, W * 32, smem, stream>>>(a, share);
  return cudaGetLastError();
}

}  // namespace

size_t cache_attn_small_workspace(int num_workers) {
  return kMaxWorkers * sizeof(int) + static_cast<size_t>(num_workers) * 2 * part_floats<16>() * sizeof(float);
}

cudaError_t launch_cache_attn_small(const cache::AttnArgs& a, int over, int upto, bool f16, int rows, int num_sms,
                                    cudaStream_t stream) {
  const Share share{over, upto};
  return rows <= 8 ? launch_small<1, 16>(a, share, f16, num_sms, stream)
                   : launch_small<2, 12>(a, share, f16, num_sms, stream);
}

}  // namespace vsa
