// cache_attn_small.cu -- attention over the 4-bit cache for few rows a request:
// a decoded token, or some drafted ones.
//
// Bound: HBM on paper, latency in fact.  A cached token and head are 144 bytes,
// 0.022 ns at 6561 GB/s; the work beside the loads is to make 256 fp16 values of
// them, some 290 warp instructions per 16 tokens.  126360 tokens x 12 heads: 51 us,
// 4.3 TB/s, two thirds of HBM, with 0.55 instructions issued a cycle and scheduler
// and no pipe above half.  About 10 us of it are the launch, finding the place, the
// first loads and the joins, which are nearly all of the 10 us of a single token
// over 777; in the rest a unit is a chain (wait, scores, vote, exponentials,
// transposes, products) on the four warps of a scheduler.  Adding a unit's values
// beside the next one's scores and units of 16 tokens were no faster.  What the
// design does:
//  - The line of 32-token units (cache_sched.cuh) is cut evenly over the CTAs,
//    one per SM, and a CTA's share evenly over its warps.  A warp works alone:
//    its own ring of units (a bulk copy of 4608 bytes each, or two where a page
//    ends between), its own softmax state.  One more warp fills the rings, a
//    lane for each: pages, addresses and bounds of as many units as there are
//    warps cost it the instructions of one.
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
//    the place of the reduction.  Numerators are taken against the maximum less
//    kLift (cache.cuh).
// Sums, maxima and denominators are fp32.  Parts are joined in a fixed order:
// the result does not depend on which CTA comes last.
#include <cuda_fp16.h>

#include "cache.cuh"
#include "cache_kernels.h"
#include "cache_sched.cuh"

namespace vsa {

namespace {

using namespace cache;

constexpr int kUnit = 32;                        // keys of a unit: two records
constexpr int kUnitBytes = 2 * kRecBytes;
constexpr int kAtOnce = 16;                      // parts of a row that a warp loads at once when it joins them
constexpr int kMinUnits = 2;                     // units a warp gets at least

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
__device__ __forceinline__ bool mbar_test_wait(uint32_t addr, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(addr), "r"(parity)
      : "memory");
  return ok != 0;
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
  int nu, h, j;
  int q0, rows;  // the request's first new token, the item's rows
};

// Where a warp's share of the line begins, for the loads.
struct Start {
  int r, h, j, k, nu, nt, total;
  Request req;
};

template <int NT, int W, int STAGES>
struct Smem {
  static constexpr int kRows = 8 * NT;
  static constexpr size_t kPieceBytes = part_floats<kRows>() * 4;
  alignas(16) uint8_t ring[W][STAGES][kUnitBytes];
  alignas(16) uint8_t piece[W][kPieceBytes];  // a warp's first item, begun before its range
  PieceMeta meta[2 * W];                      // [2 w]: that item, [2 w + 1]: one that goes on after its range
  long long part[W + 1];
  uint64_t full[W][STAGES], empty[W][STAGES];
  int have[W][STAGES];  // bit i: record i of the unit was loaded, or lies behind the last key
  Start start[W];
  int abort;
  int join[2][2];  // items this CTA joins: first and last CTA, or -1
};

// One row of a part: 128 sums (4 to a lane), maximum and denominator; w: the
// weight of the part that this lane looks after.
struct RowPart {
  float4 o;
  float m, l, w;
};
// Weight of a part with maximum m under the joint maximum.  Without a maximum a
// part has nothing but zeros, or the NaN of its scores.
__device__ __forceinline__ float part_weight(float m, float joint) {
  return m == -INFINITY ? 1.0f : ex2_approx(m - joint);
}
// Joint maximum and denominator of up to 32 parts, one a lane (absent: -inf, 0).
__device__ __forceinline__ RowPart join_weights(float m, float l) {
  RowPart t;
  t.m = m;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) t.m = fmaxf(t.m, __shfl_xor_sync(0xffffffffu, t.m, d));
  t.w = part_weight(m, t.m);
  t.l = t.w * l;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) t.l += __shfl_xor_sync(0xffffffffu, t.l, d);
  t.o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  return t;
}
__device__ __forceinline__ void add_part(RowPart& t, float4 o, float w) {
  t.o.x += w * o.x;
  t.o.y += w * o.y;
  t.o.z += w * o.z;
  t.o.w += w * o.w;
}

template <bool F16>
__device__ __forceinline__ void write_row(const AttnArgs& a, const PieceMeta& mt, int row, const RowPart& t) {
  const int lane = threadIdx.x & 31;
  const int token = row / a.G;
  const long long dst = (static_cast<long long>(mt.q0) + token) * a.Hq + mt.h * a.G + (row - token * a.G);
  const float inv = t.l != 0.0f ? 1.0f / t.l : 0.0f;
  uint2 w;
  w.x = pack_half2<F16>(t.o.x * inv, t.o.y * inv);
  w.y = pack_half2<F16>(t.o.z * inv, t.o.w * inv);
  reinterpret_cast<uint2*>(a.o + dst * 128)[lane] = w;
  if (lane == 0) a.lse[dst] = t.l != 0.0f ? (t.m + __log2f(t.l)) * 0.69314718055994531f : -INFINITY;
}

template <int NT, bool F16, int W, int STAGES>
__global__ void __launch_bounds__((W + 1) * 32, 1)
    cache_attn_small_kernel(const __grid_constant__ AttnArgs a, const Share share) {
  constexpr int RT = 8 * NT;
  using S = Sched<RT, kUnit, 0>;
  using Sm = Smem<NT, W, STAGES>;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Sm& sm = *reinterpret_cast<Sm*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;

  if (lane == 0 && warp < W) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&sm.full[warp][s], 1);
      mbar_init(&sm.empty[warp][s], 1);
    }
    sm.meta[2 * warp].item0 = sm.meta[2 * warp + 1].item0 = -1;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (threadIdx.x == 0) {
    sm.abort = 0;
    sm.join[0][0] = sm.join[1][0] = -1;
  }
  if (a.fill) fill_rows(a);
  // the sums over many requests take the place of the warps' pieces until every warp has found its own
  long long* pre = reinterpret_cast<long long*>(&sm.piece[0][0]);
  static_assert(sizeof(sm.piece) >= (kMaxRequests + 1) * 8, "the requests' sums must fit");
  const Line line = make_line<S, (W + 1) * 32>(a, share, pre, sm.part);
  const long long U = line.total;
  if (U == 0) return;
  const long long wanted = (U + W * kMinUnits - 1) / (W * kMinUnits);
  int N = wanted < gridDim.x ? static_cast<int>(wanted) : static_cast<int>(gridDim.x);
  // a batch that does not fill the GPU: whole CTAs for an item, so that items of one length need no joining between CTAs
  if (N < static_cast<int>(gridDim.x) && line.items > 0 && line.items <= static_cast<int>(gridDim.x))
    N = line.items * max(1, N / line.items);
  const int cta = blockIdx.x;
  if (cta >= N) return;
  const Cut cut(U, N);
  const long long cs = cut.start(cta), ce = cut.start(cta + 1);
  const int mine = static_cast<int>(ce - cs);
  const int ws = static_cast<long long>(mine) * warp / W, we = static_cast<long long>(mine) * (warp + 1) / W;
  const int total = warp < W ? we - ws : 0;

  Cursor<S> cc;
  if (total > 0) cc.seek(a, line, cs + ws);
  if (lane == 0 && warp < W) sm.start[warp] = Start{cc.r, cc.h, cc.j, cc.k, cc.nu, cc.nt, total, cc.req};
  __syncthreads();  // the sums over requests are no longer needed; the flags above are set

  if (warp == W) {
    // ---- loads, lane w for warp w: each lane walks that warp's share and fills the stages it has emptied
    const bool mine = lane < W && sm.start[lane < W ? lane : 0].total > 0;
    const Start st = sm.start[mine ? lane : 0];
    const int w = mine ? lane : 0;
    Cursor<S> lc;
    lc.r = st.r, lc.h = st.h, lc.j = st.j, lc.k = st.k, lc.nu = st.nu, lc.nt = st.nt, lc.req = st.req;
    lc.item0 = 0;
    const int log_rec = a.log_page - 4;  // records of a page
    const uint32_t page_bytes = static_cast<uint32_t>(a.Hkv) * kRecBytes << log_rec;
    int lkeys = 0;
    const uint8_t* head_base = nullptr;
    const int32_t* row = nullptr;
    unsigned page0 = 0, page1 = 0;  // of the next unit's records
    auto item = [&]() {
      lkeys = S::keys(a, lc.req, lc.j);
      head_base = a.pages + (static_cast<long long>(lc.h) * kRecBytes << log_rec);
      row = a.table + static_cast<long long>(lc.r) * a.max_pages;
    };
    auto ask = [&]() {
      const int rec = lc.k * 2;
      if (rec * kRecTokens < lkeys) page0 = static_cast<unsigned>(__ldg(row + (rec >> log_rec)));
      if (log_rec == 0 && (rec + 1) * kRecTokens < lkeys) page1 = static_cast<unsigned>(__ldg(row + rec + 1));
    };
    if (mine) {
      item();
      ask();
    }
    int issued = 0, s = 0, idle = 0;
    uint32_t parity = 1;
    uint64_t since = 0;
    while (true) {
      const bool want = mine && issued < st.total;
      if (!__any_sync(0xffffffffu, want)) break;
      const bool ready = want && mbar_test_wait(smem_u32(&sm.empty[w][s]), parity);
      if (ready) {
        uint64_t* bar = &sm.full[w][s];
        uint8_t* dst = sm.ring[w][s];
        const bool in0 = lc.k * kUnit < lkeys, in1 = lc.k * kUnit + kRecTokens < lkeys;
        const bool ok0 = in0 && page0 < static_cast<unsigned>(a.num_pages);
        const bool bad0 = in0 && !ok0;
        const uint8_t* s0 = head_base + static_cast<unsigned long long>(page0) * page_bytes;
        if (log_rec > 0) {
          // both records lie in one page; the second may hold no key, but is there
          sm.have[w][s] = bad0 ? 0 : 3;
          if (ok0) {
            mbar_arrive_expect_tx(bar, kUnitBytes);
            bulk_load(dst, s0 + (lc.k * 2 & ((1 << log_rec) - 1)) * kRecBytes, kUnitBytes, bar);
          }
          if (bad0) atomicCAS(a.status, 0u, (unsigned)VSA_ERR_BAD_INDEX);
          if (!ok0) mbar_arrive(bar);
        } else {
          const bool ok1 = in1 && page1 < static_cast<unsigned>(a.num_pages);
          sm.have[w][s] = (bad0 ? 0 : 1) | (in1 && !ok1 ? 0 : 2);
          if (bad0 || (in1 && !ok1)) atomicCAS(a.status, 0u, (unsigned)VSA_ERR_BAD_INDEX);
          if (ok0 || ok1) {
            mbar_arrive_expect_tx(bar, (ok0 ? kRecBytes : 0) + (ok1 ? kRecBytes : 0));
            if (ok0) bulk_load(dst, s0, kRecBytes, bar);
            if (ok1)
              bulk_load(dst + kRecBytes, head_base + static_cast<unsigned long long>(page1) * page_bytes, kRecBytes, bar);
          } else {
            mbar_arrive(bar);
          }
        }
        if (++s == STAGES) {
          s = 0;
          parity ^= 1;
        }
        if (++issued < st.total) {
          if (++lc.k == lc.nu) {
            lc.next_item(a, share);
            item();
          }
          ask();
        }
      }
      if (__any_sync(0xffffffffu, ready)) {
        idle = 0;
      } else {
        // bounded like every wait: give up when another warp has, or after kWaitNs without an emptied stage; by
        // vote, because lanes that read the flag or the clock at different times must not part
        const uint64_t now = globaltimer_ns();
        if (idle == 0) since = now;
        idle = 1;
        if (__any_sync(0xffffffffu, *static_cast<volatile int*>(&sm.abort) != 0 || now - since > kWaitNs)) {
          if (lane == 0) {
            sm.abort = 1;
            atomicCAS(a.status, 0u, (unsigned)VSA_ERR_TIMEOUT);
          }
          // every copy issued must land before the CTA's shared memory is released
          for (int x = 0; x < STAGES; ++x)
            if (mine && issued > x) {
              const int last = issued - 1 - ((issued - 1 - x) % STAGES);
              mbar_wait_drain(&sm.full[w][x], (last / STAGES) & 1, kDrainNs);
            }
          break;
        }
        __nanosleep(40);
      }
    }
    __syncwarp();
  }

  bool ok = true;
  if (total > 0) {
    uint32_t qf[NT][16];
    float rs[NT][2], m[NT][2], l[NT][2], base[NT][2];  // m: the maximum less kLift; base: -m, or 0 where there is none yet
    int lim[NT][2];
    float acc[NT][8][4];
    int lim_min = 0, seen = 0;
    bool from_start = false;
    int s = 0;
    uint32_t parity = 0;

    // the rows of q of the item at cc: thread (g, c) channels 32 c .. 32 c + 31 of row g
    auto load_q = [&]() {
      const int rows = cc.req.n * a.G;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int row = cc.j * RT + n * 8 + g;
        const int token = row / a.G;
        const uint4* src = reinterpret_cast<const uint4*>(
            a.q + (static_cast<long long>(cc.req.q0) + token) * a.q_stride + (cc.h * a.G + row - token * a.G) * 128 +
            c * 32);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint4 w = make_uint4(0, 0, 0, 0);
          if (row < rows) w = __ldg(src + x);
          qf[n][4 * x] = w.x, qf[n][4 * x + 1] = w.y, qf[n][4 * x + 2] = w.z, qf[n][4 * x + 3] = w.w;
        }
      }
    };
    load_q();

    for (int i = 0; i < total; ++i) {
      if (i == 0 || cc.k == 0) {
        // ---- a new item: its rows of q as B fragments
        if (i > 0) load_q();
        from_start = cc.k == 0;
        const int rows = cc.req.n * a.G;
        lim_min = visible(a, cc.req, cc.j * RT / a.G);
        seen = S::keys(a, cc.req, cc.j);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float amax = 0.0f;
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
            l[n][e] = base[n][e] = 0.0f;
          }
#pragma unroll
          for (int x = 0; x < 8; ++x) acc[n][x][0] = acc[n][x][1] = acc[n][x][2] = acc[n][x][3] = 0.0f;
        }
      }

      ok = mbar_wait(&sm.full[warp][s], parity, &sm.abort, a.status, kWaitNs);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      const uint32_t have = sm.have[warp][s];
      const int key0 = cc.k * kUnit;
      if (key0 < seen) {
        const uint8_t* unit = sm.ring[warp][s];
        // ---- S^T = K Q^T: row x of a record's 16 keys is token 8 (x / 8) + 4 (x & 1) + ((x & 7) >> 1)
        float sc[NT][2][4];
        const int ta = 4 * (g & 1) + (g >> 1);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint8_t* rec = unit + u * kRecBytes;
          const uint4 ka = *reinterpret_cast<const uint4*>(rec + ta * 64 + c * 16);
          const uint4 kb = *reinterpret_cast<const uint4*>(rec + (ta + 8) * 64 + c * 16);
          const uint32_t sa = from_e4m3x2(*reinterpret_cast<const uint16_t*>(rec + kRecKS + ta * 8 + 2 * c));
          const uint32_t sb = from_e4m3x2(*reinterpret_cast<const uint16_t*>(rec + kRecKS + (ta + 8) * 8 + 2 * c));
          const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
          // two chains of products, joined below: half the wait for one
          float even[NT][4], odd[NT][4];
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) even[n][e] = odd[n][e] = 0.0f;
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
              for (int n = 0; n < NT; ++n)
                mma16816(y ? odd[n] : even[n], f, qf[n][4 * x + 2 * y], qf[n][4 * x + 2 * y + 1]);
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[n][u][e] = even[n][e] + odd[n][e];
        }
        // ---- softmax over the keys, in units of 1 / rs (a power of two times log2(e) / sqrt(D))
        const unsigned key1 = key0 + static_cast<unsigned>(kUnit);  // may be 2^31
        if (key1 > static_cast<unsigned>(lim_min) || have != 3) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (key0 + 16 * u + ta + 8 * (e >> 1) >= lim[n][e & 1] || !(have >> u & 1)) sc[n][u][e] = -INFINITY;
        }
        bool grow = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float t = fmaxf(max3f(sc[n][0][e], sc[n][0][e + 2], sc[n][1][e]), sc[n][1][e + 2]) * rs[n][e];
            grow |= t > m[n][e] + (8.0f + kLift);
          }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float t = fmaxf(max3f(sc[n][0][e], sc[n][0][e + 2], sc[n][1][e]), sc[n][1][e + 2]) * rs[n][e];
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
              if (t > m[n][e] + (8.0f + kLift)) {
                t -= kLift;
                const float alpha = ex2_approx(m[n][e] - t);  // 0 for the first maximum
                m[n][e] = t;
                base[n][e] = -t;
                l[n][e] *= alpha;
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                  acc[n][x][e] *= alpha;
                  acc[n][x][e + 2] *= alpha;
                }
              }
            }
        }
        uint32_t pb[2][NT][2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) p[e] = ex2_approx(__fmaf_rn(sc[n][u][e], rs[n][e & 1], base[n][e & 1]));
            l[n][0] += p[0] + p[2];
            l[n][1] += p[1] + p[3];
            pb[u][n][0] = transpose8x8(pack_f16x2(p[0], p[1]));
            pb[u][n][1] = transpose8x8(pack_f16x2(p[2], p[3]));
          }
        // ---- O^T += V^T P^T: thread (g, c) has channels 16 g .. 16 g + 15 of tokens c, c + 4, c + 8, c + 12
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint8_t* rec = unit + u * kRecBytes;
          uint2 w[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) w[x] = *reinterpret_cast<const uint2*>(rec + kRecV + (c + 4 * x) * 64 + g * 8);
          uint32_t vs = *reinterpret_cast<const uint32_t*>(rec + kRecVS + g * 16 + c * 4);
          if (key1 > static_cast<unsigned>(seen) || have != 3) {
            // behind the last token, or in a record that was not loaded, the scales may be NaN
            const int left = have >> u & 1 ? seen - key0 - 16 * u : 0;
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
              for (int n = 0; n < NT; ++n) mma16816(acc[n][4 * y + x], f, pb[u][n][0], pb[u][n][1]);
            }
          }
        }
      }
      __syncwarp();  // the unit has been read
      if (lane == 0) mbar_arrive(&sm.empty[warp][s]);
      if (++s == STAGES) {
        s = 0;
        parity ^= 1;
      }

      const bool done = cc.k + 1 == cc.nu;
      if (done || i + 1 == total) {
        // ---- the item, or the warp's share of it, is complete: thread (g, c) holds channels 16 g .. of rows 2c, 2c + 1
        const int rows = cc.req.n * a.G - cc.j * RT;
        float* piece = reinterpret_cast<float*>(from_start ? sm.ring[warp][0] : sm.piece[warp]);
        static_assert(Sm::kPieceBytes <= STAGES * kUnitBytes, "the last piece takes the place of the ring");
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
          sm.meta[2 * warp + (from_start ? 1 : 0)] = PieceMeta{cc.item0, cc.nu, cc.h, cc.j, cc.req.q0, min(RT, rows)};
        if (i + 1 < total) cc.next_item(a, share);
      } else {
        ++cc.k;
      }
    }
  }
  __syncthreads();
  if (sm.abort) return;

  // ---- join the warps' pieces of each item, all warps over its rows; lane p looks after piece p
  static_assert(2 * W <= 32, "one lane per piece");
  int* counters = static_cast<int*>(a.ws);
  float* parts = reinterpret_cast<float*>(counters + kMaxWorkers);
  constexpr size_t kPart = part_floats<RT>();
  const long long key = lane < 2 * W ? sm.meta[lane].item0 : -1;
  const float* mine_at = reinterpret_cast<const float*>(lane & 1 ? &sm.ring[lane / 2 % W][0][0] : &sm.piece[lane / 2 % W][0]);
  // the pieces are in the order of the line: an item's are neighbours among those that are there
  const unsigned there = __ballot_sync(0xffffffffu, key >= 0);
  const unsigned below = there & ((1u << lane) - 1);
  const long long before = __shfl_sync(0xffffffffu, key, below ? 31 - __clz(below) : lane);
  unsigned leaders = __ballot_sync(0xffffffffu, key >= 0 && (below == 0 || before != key));
  PieceMeta cross[2];  // items that go beyond the CTA: begun before it, going on after it
  cross[0].item0 = cross[1].item0 = -1;
  while (leaders) {
    const int lead = __ffs(leaders) - 1;
    leaders &= leaders - 1;
    // from the leader to the next
    const unsigned group = there & (~0u << lead) & (leaders ? (leaders & -leaders) - 1 : ~0u);
    const PieceMeta mt = sm.meta[lead];
    const bool whole = mt.item0 >= cs && mt.item0 + mt.nu <= ce;
    const int slot = mt.item0 < cs ? 0 : 1;
    if (!whole) cross[slot] = mt;
    for (int row = warp; row < mt.rows; row += W + 1) {
      const bool in = group >> lane & 1;
      RowPart t = join_weights(in ? mine_at[RT * 128 + row] : -INFINITY, in ? mine_at[RT * 129 + row] : 0.0f);
      for (unsigned left = group; left; left &= left - 1) {
        const int p = __ffs(left) - 1;
        const float* f = reinterpret_cast<const float*>(p & 1 ? &sm.ring[p >> 1][0][0] : &sm.piece[p >> 1][0]);
        add_part(t, reinterpret_cast<const float4*>(f + row * 128)[lane], __shfl_sync(0xffffffffu, t.w, p));
      }
      if (whole) {
        write_row<F16>(a, mt, mt.j * RT + row, t);
      } else {
        float* f = parts + (static_cast<size_t>(cta) * 2 + slot) * kPart;
        reinterpret_cast<float4*>(f + row * 128)[lane] = t.o;
        if (lane == 0) {
          f[RT * 128 + row] = t.m;
          f[RT * 129 + row] = t.l;
        }
      }
    }
  }
  if (cross[0].item0 < 0 && cross[1].item0 < 0) return;

  // ---- join the CTAs' parts: the last of an item's CTAs to arrive, in the order of the line
  __syncthreads();
  if (threadIdx.x < 2 && cross[threadIdx.x].item0 >= 0) {
    const PieceMeta& mt = threadIdx.x ? cross[1] : cross[0];
    const int first = cut.worker_of(mt.item0), last = cut.worker_of(mt.item0 + mt.nu - 1);
    __threadfence();  // the CTA's parts before the count
    if (atomicAdd(counters + first, 1) == last - first) {
      counters[first] = 0;  // as the next call finds it
      __threadfence();
      sm.join[threadIdx.x][0] = first;
      sm.join[threadIdx.x][1] = last;
    }
  }
  __syncthreads();
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int first = sm.join[x][0], last = sm.join[x][1];
    if (first < 0) continue;
    const PieceMeta mt = cross[x];
    for (int row = warp; row < mt.rows; row += W + 1) {
      auto part_of = [&](int w) { return parts + (static_cast<size_t>(w) * 2 + (w == first ? 1 : 0)) * kPart; };
      RowPart t;
      t.m = -INFINITY;
      t.l = 0.0f;
      t.o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int w0 = first; w0 <= last; w0 += kAtOnce) {
        const int n = min(kAtOnce, last - w0 + 1);
        float4 o[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
          o[i] = i < n ? __ldcg(reinterpret_cast<const float4*>(part_of(w0 + i) + row * 128) + lane)
                       : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const float* f = part_of(w0 + min(lane, n - 1));
        RowPart u = join_weights(lane < n ? __ldcg(f + RT * 128 + row) : -INFINITY, lane < n ? __ldcg(f + RT * 129 + row) : 0.0f);
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) add_part(u, o[i], __shfl_sync(0xffffffffu, u.w, i));
        // their sum joins those before it
        const float m = fmaxf(t.m, u.m), wt = part_weight(t.m, m), wu = part_weight(u.m, m);
        t.o = make_float4(wt * t.o.x + wu * u.o.x, wt * t.o.y + wu * u.o.y, wt * t.o.z + wu * u.o.z,
                          wt * t.o.w + wu * u.o.w);
        t.l = wt * t.l + wu * u.l;
        t.m = m;
      }
      write_row<F16>(a, mt, mt.j * RT + row, t);
    }
  }
}

template <int NT, int W, int STAGES>
cudaError_t launch_small(const AttnArgs& a, const Share& share, bool f16, int num_sms, cudaStream_t stream) {
  auto kern = f16 ? cache_attn_small_kernel<NT, true, W, STAGES> : cache_attn_small_kernel<NT, false, W, STAGES>;
  constexpr int smem = static_cast<int>(sizeof(Smem<NT, W, STAGES>));
  static_assert(smem <= 227 * 1024, "shared memory of a CTA");
  static SmemAllowed allowed[2];  // fp16, bf16
  cudaError_t e = allowed[f16 ? 0 : 1].ensure(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  kern<<<num_sms < kMaxWorkers ? num_sms : kMaxWorkers, (W + 1) * 32, smem, stream>>>(a, share);
  return cudaGetLastError();
}

}  // namespace

size_t cache_attn_small_workspace(int num_workers) {
  return kMaxWorkers * sizeof(int) + static_cast<size_t>(num_workers) * 2 * part_floats<16>() * sizeof(float);
}

cudaError_t launch_cache_attn_small(const cache::AttnArgs& a, int over, int upto, bool f16, int rows, int num_sms,
                                    cudaStream_t stream) {
  const Share share{over, upto};
  return rows <= 8 ? launch_small<1, 15, 2>(a, share, f16, num_sms, stream)
                   : launch_small<2, 7, 4>(a, share, f16, num_sms, stream);
}

}  // namespace vsa
