// cache_attn_chunk.cu -- attention over the 4-bit cache for many rows a
// request: a chunk of a video or a piece of a prompt, on the tensor cores
// (tcgen05, accumulators in tensor memory).
//
// Work: the line of (request, key head, 256-row tile) x 128-key units of
// cache_sched.cuh, cut evenly over one persistent CTA per SM.  The pipeline is
// the fine stage's (attn_fwd.cu): two 128-row query tiles, S and P in the same
// tensor memory, PV(t) and S(t + 1) of one tile under the softmax of the other.
// What differs is where the operands come from.  Q is read by the softmax
// threads, a row each, which bring it to fp16 (bf16: times a power of two per
// row, so that nothing is lost; cache_attn_small.cu) and write the swizzled
// tile that TMA would have; K and V are made from codes by a warpgroup of their
// own, which loads the words of a 128-key tile one tile ahead into registers,
// converts them (code * scale, exact in fp16) and writes the same tiles.
//
// Warp roles (512 threads):
//   warp 0       tensor-memory owner and MMA issuer
//   warp 1       walks the CTA's share of the line and hands its segments (an
//                item's units, or part of them) to the others through a ring in
//                shared memory, so that their registers hold no schedule
//                (warps 2 and 3 idle)
//   warps 4-7    K and V tiles from codes: a thread 32 channels of 4 keys
//   warps 8-11   rows of query tile 0: Q, softmax, output
//   warps 12-15  rows of query tile 1
// Bound: no one unit is full (tensor pipe 42%, issue slots 42%).  A tile's
// softmax and the products that wait for it are a chain, as in the fine stage,
// and the conversion (256 values a key and CTA, whatever its rows) takes issue
// slots beside it: 6240 tokens over 32760, 12 heads, run in 1.29 to 1.35 ms, 930
// to 970 TFLOP/s of 16-bit products, 6 to 11% below the fine stage (1006 to
// 1049).  Every fourth exponential by a polynomial was 7% slower.
//
// An item cut between CTAs leaves its rows' sums, maxima and denominators in
// the workspace, and a second kernel joins them in the order of the line.
// Every mbarrier wait is bounded, as in the fine stage.
#include <cuda_fp16.h>

#include "cache.cuh"
#include "cache_kernels.h"
#include "cache_sched.cuh"

namespace vsa {

namespace {

using namespace cache;

constexpr int kThreads = 512;
constexpr int kRowTile = 256, kKeyTile = 128;
constexpr int kStagesK = 3, kStagesV = 2, kSegs = 4;
// An item's rows of Q, first product and output take a CTA some 6 to 9 us, a unit 2.4 us (4 x 1023 on 5000: 157 us with
// 4, 162 with 3, 170 with 2, 196 with 0, a pass; one long item does not care).  Measured on that one shape only.
constexpr int kItemCost = 4;
// Places of the line that a CTA gets at least.  Shorter shares end sooner but have more parts to join: 3 requests of
// 78 rows on 1483, 8 heads, 58.2 us with 8, 50.8 with 4, 45.3 with 2; one of 61 x 3 rows on 19525 32.3 with 4, 34.5
// with 2 (27.3 now, with the join spread wider).
constexpr int kMinPlaces = 3;
constexpr uint32_t kHalfBytes = 128 * 128;       // 128 rows x 64 fp16 (one 128-B swizzle column)
constexpr uint32_t kTileBytes = 2 * kHalfBytes;  // 128 rows x 128 fp16
constexpr uint32_t kSmemQ = 0;
constexpr uint32_t kSmemK = kSmemQ + 2 * kTileBytes;
constexpr uint32_t kSmemV = kSmemK + kStagesK * kTileBytes;
constexpr uint32_t kSmemBar = kSmemV + kStagesV * kTileBytes;
constexpr uint32_t kSmemTotal = kSmemBar + 512 + 1024;  // barriers, segments + 1 KB alignment slack
// Register split: launched at 128 per thread; 128 x (40 + 88) + 256 x 192 = 512 x 128.
constexpr int kRegsMma = 40, kRegsLoad = 88, kRegsRows = 192;
static_assert(128 * (kRegsMma + kRegsLoad) + 256 * kRegsRows == kThreads * 128, "register split must match the launch");

using S = Sched<kRowTile, kKeyTile, kItemCost>;

// Units [k0, k0 + n) of an item; n = 0: the end.
struct Seg {
  int r, h, j;        // request, key head, row tile
  int k0, n;
  int whole;          // the whole item
  int q0, tokens, kv; // the request
  int last;           // an item that starts here and goes on after the CTA's share: the CTA of its last unit; else -1
};

struct Barriers {
  uint64_t q_full, q_empty;
  uint64_t k_full[kStagesK], k_empty[kStagesK];
  uint64_t v_full[kStagesV], v_empty[kStagesV];
  uint64_t s_full[2], p_full[2], o_full[2], o_empty[2];
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  Seg seg[kSegs];
};
static_assert(sizeof(Barriers) <= 512, "barrier block too large");
constexpr int kSegReaders = 13;  // warps: the MMA issuer, 4 of the tiles, 8 of the rows

// What the join kernel needs of an item that starts in a CTA's range and goes
// on after it: in the workspace, one per CTA; last < 0: none.
struct Joint {
  int last;  // the CTA that holds the item's last unit
  int h, j, q0, rows;
  int pad[3];
};

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, Barriers* bars, unsigned int* status) {
  const bool ok = mbar_wait(bar, parity, &bars->abort, status, kWaitNs);
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ float* parts_of(void* ws, int workers) {
  return reinterpret_cast<float*>(static_cast<Joint*>(ws) + workers);
}

// The next segment, for a warp; n = 0 at the end or when a wait ran out.
struct SegReader {
  int at = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ Seg next(Barriers* bars, unsigned int* status) {
    Seg seg;
    seg.n = 0;
    if (!warp_wait(&bars->seg_full[at], parity, bars, status)) return seg;
    seg = bars->seg[at];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&bars->seg_empty[at]);
    if (++at == kSegs) {
      at = 0;
      parity ^= 1;
    }
    return seg;
  }
};

// The eight K = 16 products of a tile, one lane issuing.  Descriptors are put
// together from their low words inside the block: with 64-bit operands handed
// in one by one the compiler keeps all of them in registers, spills, and the
// issue (5200 cycles per unit where the products take 2050) bounds the kernel.
#define VSA_MMA_SS(OFF, ACC)                                                          \
  "add.u32 x, %1, " #OFF ";\n\tadd.u32 y, %2, " #OFF ";\n\t"                           \
  "mov.b64 da, {x, %3};\n\tmov.b64 db, {y, %3};\n\t"                                  \
  "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, " #ACC ";\n\t"
// D[tmem] = A[smem] B[smem], both K-major: 32 bytes of a 128-byte column a step, then the other column.
__device__ __forceinline__ void mma8_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t desc_hi, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred e, yes, no;\n\t.reg .b32 x, y;\n\t.reg .b64 da, db;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.eq.b32 yes, %3, %3;\n\tsetp.ne.b32 no, %3, %3;\n\t" VSA_MMA_SS(0, no) VSA_MMA_SS(2, yes)
          VSA_MMA_SS(4, yes) VSA_MMA_SS(6, yes) VSA_MMA_SS(1024, yes) VSA_MMA_SS(1026, yes) VSA_MMA_SS(1028, yes)
              VSA_MMA_SS(1030, yes) "}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(desc_hi), "r"(idesc)
      : "memory");
}
#undef VSA_MMA_SS
#define VSA_MMA_TS(STEP, ACC)                                                         \
  "add.u32 x, %1, 8 * " #STEP ";\n\tadd.u32 y, %2, 128 * " #STEP ";\n\t"              \
  "mov.b64 db, {y, %3};\n\t"                                                          \
  "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], db, %4, " #ACC ";\n\t"
// D[tmem] (+)= A[tmem] B[smem], B MN-major: 16 rows (2048 bytes) a step.
__device__ __forceinline__ void mma8_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t desc_hi, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, yes, acc;\n\t.reg .b32 x, y;\n\t.reg .b64 db;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.eq.b32 yes, %3, %3;\n\tsetp.ne.b32 acc, %5, 0;\n\t" VSA_MMA_TS(0, acc) VSA_MMA_TS(1, yes)
          VSA_MMA_TS(2, yes) VSA_MMA_TS(3, yes) VSA_MMA_TS(4, yes) VSA_MMA_TS(5, yes) VSA_MMA_TS(6, yes)
              VSA_MMA_TS(7, yes) "}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(desc_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
#undef VSA_MMA_TS

// 16 channels of a key, code times scale, as two 16-byte chunks of a tile.
__device__ __forceinline__ void put_chunk(uint8_t* dst, uint32_t word, uint32_t scale) {
  uint32_t v[4];
  from_e2m1x8(word, v);
  *reinterpret_cast<uint4*>(dst) =
      make_uint4(mul_f16x2(v[0], scale), mul_f16x2(v[1], scale), mul_f16x2(v[2], scale), mul_f16x2(v[3], scale));
}

template <bool F16>
__global__ void __launch_bounds__(kThreads, 1)
    cache_attn_chunk_kernel(const __grid_constant__ AttnArgs a, const Share share) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem + kSmemQ;
  uint8_t* sK = smem + kSmemK;
  uint8_t* sV = smem + kSmemV;
  Barriers* bars = reinterpret_cast<Barriers*>(smem + kSmemBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;

  // the sums over many requests use the K ring before anything else does
  const Line line = make_line<S, kThreads>(a, share, reinterpret_cast<long long*>(sK),
                                           reinterpret_cast<long long*>(sQ));
  const long long U = line.total;
  Joint* joint = static_cast<Joint*>(a.ws) + cta;
  if (threadIdx.x == 0) joint->last = -1;
  const int N = static_cast<int>(min(static_cast<long long>(gridDim.x), (U + kMinPlaces - 1) / kMinPlaces));
  if (cta >= N) return;  // N = 0: no request for this kernel
  const Cut cut(U, N);
  const long long cs = cut.start(cta), ce = cut.start(cta + 1);
  Cursor<S> cur;
  if (warp == 1) cur.seek(a, line, cs);
  __syncthreads();

  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 256);
    mbar_init(&bars->q_empty, 1);
    for (int s = 0; s < kStagesK; ++s) {
      mbar_init(&bars->k_full[s], 128);
      mbar_init(&bars->k_empty[s], 1);
    }
    for (int s = 0; s < kStagesV; ++s) {
      mbar_init(&bars->v_full[s], 128);
      mbar_init(&bars->v_empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->p_full[i], 128);
      mbar_init(&bars->o_full[i], 1);
      mbar_init(&bars->o_empty[i], 128);
    }
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(&bars->seg_full[i], 1);
      mbar_init(&bars->seg_empty[i], kSegReaders);
    }
    mbar_init(&bars->drain, 1);
    bars->abort = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 0) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  if (warp < 4) {
    regs_dec<kRegsMma>();
    if (warp == 1) {
      // ------------------------------------------------------------ the CTA's segments
      int at = 0;
      uint32_t parity = 1;
      int left = static_cast<int>(ce - cs);
      bool end = false;
      while (!end) {
        const int places = min(left, cur.nu - cur.k);
        const int units = cur.nu - kItemCost, k0 = max(0, cur.k - kItemCost), k1 = cur.k + places - kItemCost;
        end = left == 0;
        if (end || k1 > k0) {
          if (!warp_wait(&bars->seg_empty[at], parity, bars, a.status)) break;
          if (lane == 0) {
            Seg g;
            g.r = cur.r, g.h = cur.h, g.j = cur.j;
            g.k0 = k0, g.n = end ? 0 : k1 - k0;
            g.whole = k0 == 0 && k1 == units;
            g.q0 = cur.req.q0, g.tokens = cur.req.n, g.kv = cur.req.kv;
            g.last = k0 == 0 && k1 < units ? cut.worker_of(cur.item0 + cur.nu - 1) : -1;
            bars->seg[at] = g;
            mbar_arrive(&bars->seg_full[at]);
          }
          __syncwarp();
          if (++at == kSegs) {
            at = 0;
            parity ^= 1;
          }
        }
        left -= places;
        if (left > 0) cur.next_item(a, share);
      }
    } else if (warp == 0) {
      // ------------------------------------------------------------ MMA issuer
      // shared-memory descriptors (128-byte swizzle), low words; the high word is the same for all
      const uint64_t dq = sdesc_sw128(smem_u32(sQ), 16, 1024);
      const uint32_t dq0 = static_cast<uint32_t>(dq), desc_hi = static_cast<uint32_t>(dq >> 32);
      const uint32_t dk0 = static_cast<uint32_t>(sdesc_sw128(smem_u32(sK), 16, 1024));
      const uint32_t dv0 = static_cast<uint32_t>(sdesc_sw128(smem_u32(sV), kHalfBytes, 1024));
      constexpr uint32_t kTileDesc = kTileBytes >> 4;
      constexpr uint32_t kIdescS = idesc_f16_f32(128, 128, 0, 0), kIdescPV = idesc_f16_f32(128, 128, 0, 1);
      int sk = 0, sv = 0;                // ring places
      uint32_t pk = 0, pv = 0;           // and their parities
      uint32_t pq = 0, pp[2] = {0, 0}, po[2] = {1, 1};
      bool ok = true;
      auto issue_s = [&](int i) {
        mma8_ss(tmem + i * 128, dq0 + i * kTileDesc, dk0 + sk * kTileDesc, desc_hi, kIdescS);
        mma_commit_w(&bars->s_full[i]);
      };
      auto issue_pv = [&](int i, bool acc) {
        mma8_ts(tmem + 256 + i * 128, tmem + i * 128, dv0 + sv * kTileDesc, desc_hi, kIdescPV, acc);
      };
      auto k_done = [&]() {
        mma_commit_w(&bars->k_empty[sk]);
        if (++sk == kStagesK) {
          sk = 0;
          pk ^= 1;
        }
      };
      SegReader segs;
      while (ok) {
        const Seg cur = segs.next(bars, a.status);
        const int n = cur.n;
        if (n == 0) break;
        const int tiles = cur.tokens * a.G - cur.j * kRowTile > 128 ? 2 : 1;
        if (!(ok = warp_wait(&bars->q_full, pq, bars, a.status))) break;
        pq ^= 1;
        if (!(ok = warp_wait(&bars->k_full[sk], pk, bars, a.status))) break;
        tc_fence_after();
        issue_s(0);
        if (tiles == 2) issue_s(1);
        k_done();
        for (int t = 0; t < n; ++t) {
          const bool more = t + 1 < n;
          if (!(ok = warp_wait(&bars->v_full[sv], pv, bars, a.status))) break;
          if (!(ok = warp_wait(&bars->p_full[0], pp[0], bars, a.status))) break;
          pp[0] ^= 1;
          if (t == 0) {
            if (!(ok = warp_wait(&bars->o_empty[0], po[0], bars, a.status))) break;
            po[0] ^= 1;
          }
          tc_fence_after();
          issue_pv(0, t > 0);
          if (!more) mma_commit_w(&bars->o_full[0]);
          if (more) {
            if (!(ok = warp_wait(&bars->k_full[sk], pk, bars, a.status))) break;
            tc_fence_after();
            issue_s(0);
          }
          if (tiles == 2) {
            if (!(ok = warp_wait(&bars->p_full[1], pp[1], bars, a.status))) break;
            pp[1] ^= 1;
            if (t == 0) {
              if (!(ok = warp_wait(&bars->o_empty[1], po[1], bars, a.status))) break;
              po[1] ^= 1;
            }
            tc_fence_after();
            issue_pv(1, t > 0);
          }
          mma_commit_w(&bars->v_empty[sv]);
          if (++sv == kStagesV) {
            sv = 0;
            pv ^= 1;
          }
          if (tiles == 2 && !more) mma_commit_w(&bars->o_full[1]);
          if (more) {
            if (tiles == 2) issue_s(1);
            k_done();
          }
        }
        if (!ok) break;
        mma_commit_w(&bars->q_empty);
      }
      // Drain: wait for every MMA issued by this thread before TMEM and smem go away.
      mma_commit_w(&bars->drain);
      mbar_wait_drain(&bars->drain, 0, kDrainNs);
    }
  } else if (warp < 8) {
    regs_dec<kRegsLoad>();
    // ------------------------------------------------------------ K and V tiles from codes
    // Lane (g, c) of warp w: channels 32 c .. 32 c + 31 of keys 32 w + 8 x + g, x = 0 .. 3 (records 2 w and
    // 2 w + 1 of the tile).  Its four 16-byte chunks of a key go to places (4 (c & 1) + y) ^ (key & 7) of half
    // c >> 1; lanes of the upper half take y ^ 2 first, so that eight lanes always write eight different places.
    const int w = warp - 4, g = lane >> 2, c = lane & 3;
    const int log_rec = a.log_page - 4;
    const unsigned page_bytes = static_cast<unsigned>(a.Hkv) * kRecBytes << log_rec;
    uint32_t kw[16], vw[16], ks[4], vs[4];
    int live = 0;  // keys of the record pair that hold a token, from 0; bad pages hold none
    const uint8_t* rec[2];
    unsigned page[2];  // pages of the warp's two records of the next tile, asked for one tile before
    auto ask = [&](const Seg& cu, int t) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = t * 8 + w * 2 + x;  // record of the request
        page[x] = r * kRecTokens < cu.kv
                      ? static_cast<unsigned>(__ldg(a.table + static_cast<long long>(cu.r) * a.max_pages + (r >> log_rec)))
                      : 0u;
      }
    };
    auto place = [&](const Seg& cu, int t) {
      live = cu.kv - (t * kKeyTile + w * 32);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = t * 8 + w * 2 + x;
        rec[x] = nullptr;
        if (page[x] < static_cast<unsigned>(a.num_pages))
          rec[x] = a.pages + static_cast<unsigned long long>(page[x]) * page_bytes +
                   ((static_cast<long long>(cu.h) << log_rec) + (r & ((1 << log_rec) - 1))) * kRecBytes;
        else if (lane == 0)
          atomicCAS(a.status, 0u, (unsigned)VSA_ERR_BAD_INDEX);
      }
    };
    auto load_k = [&]() {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const uint8_t* p = rec[x >> 1];
        const int tok = (x & 1) * 8 + g;
        uint4 v = make_uint4(0, 0, 0, 0);
        ks[x] = 0;
        if (p != nullptr && (x * 8 + g) < live) {
          v = __ldg(reinterpret_cast<const uint4*>(p + tok * 64 + c * 16));
          ks[x] = __ldg(reinterpret_cast<const uint16_t*>(p + kRecKS + tok * 8 + 2 * c));
        }
        kw[4 * x] = v.x, kw[4 * x + 1] = v.y, kw[4 * x + 2] = v.z, kw[4 * x + 3] = v.w;
      }
    };
    auto load_v = [&]() {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const uint8_t* p = rec[x >> 1];
        const int tok = (x & 1) * 8 + g;
        uint4 v = make_uint4(0, 0, 0, 0);
        vs[x] = 0;
        if (p != nullptr && (x * 8 + g) < live) {
          v = __ldg(reinterpret_cast<const uint4*>(p + kRecV + tok * 64 + c * 16));
          const uint8_t* sp = p + kRecVS + 2 * c * 16 + (tok & 3) * 4 + (tok >> 2);
          vs[x] = static_cast<uint32_t>(__ldg(sp)) | static_cast<uint32_t>(__ldg(sp + 16)) << 8;
        }
        vw[4 * x] = v.x, vw[4 * x + 1] = v.y, vw[4 * x + 2] = v.z, vw[4 * x + 3] = v.w;
      }
    };
    auto store = [&](uint8_t* tile, const uint32_t (&word)[16], const uint32_t (&sc)[4]) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int key = w * 32 + x * 8 + g;
        uint8_t* row = tile + (c >> 1) * kHalfBytes + key * 128;
        const uint32_t s2 = from_e4m3x2(sc[x]), s_lo = dup_lo(s2), s_hi = dup_hi(s2);
        const bool up = c >> 1;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int z = up ? y ^ 2 : y;
          put_chunk(row + (((4 * (c & 1) + z) ^ (key & 7)) << 4), up ? word[4 * x + (y ^ 2)] : word[4 * x + y],
                    z < 2 ? s_lo : s_hi);
        }
      }
      fence_proxy_async_smem();
    };
    int sk = 0, sv = 0;
    uint32_t pk = 1, pv = 1;
    bool ok = true;
    SegReader segs;
    Seg cur = segs.next(bars, a.status);
    int t = 0;
    auto first_of = [&]() {  // the first tile of a segment: its pages, and the next tile's
      ask(cur, cur.k0);
      place(cur, cur.k0);
      if (cur.n > 1) ask(cur, cur.k0 + 1);
    };
    if (cur.n > 0) {
      first_of();
      load_k();
    }
    while (cur.n > 0 && ok) {
      load_v();
      if (!(ok = warp_wait(&bars->k_empty[sk], pk, bars, a.status))) break;
      store(sK + sk * kTileBytes, kw, ks);
      mbar_arrive(&bars->k_full[sk]);
      if (++sk == kStagesK) {
        sk = 0;
        pk ^= 1;
      }
      if (++t == cur.n) {
        t = 0;
        cur = segs.next(bars, a.status);
        if (cur.n > 0) first_of();
      } else {
        place(cur, cur.k0 + t);
        if (t + 1 < cur.n) ask(cur, cur.k0 + t + 1);
      }
      if (cur.n > 0) load_k();
      if (!(ok = warp_wait(&bars->v_empty[sv], pv, bars, a.status))) break;
      store(sV + sv * kTileBytes, vw, vs);
      mbar_arrive(&bars->v_full[sv]);
      if (++sv == kStagesV) {
        sv = 0;
        pv ^= 1;
      }
    }
  } else {
    regs_inc<kRegsRows>();
    // ------------------------------------------------------------ Q, softmax and output, one thread per row
    const int wg = (warp - 8) >> 2;
    const int quarter = warp & 3;  // tensor-memory lane quarter of this warp
    const int r = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_off + wg * 128;
    const uint32_t tO = tmem + lane_off + 256 + wg * 128;
    const int log_rec = a.log_page - 4;
    uint32_t ps = 0, po = 0, pq = 1;
    bool ok = true;
    SegReader segs;
    while (ok) {
      const Seg cur = segs.next(bars, a.status);
      const int n = cur.n;
      if (n == 0) break;
      const int rows = cur.tokens * a.G - cur.j * kRowTile;  // of the item, from this tile on
      const bool active = wg == 0 || rows > 128;
      const int row = wg * 128 + r;
      const bool real = row < rows;
      const int rr = cur.j * kRowTile + (real ? row : 0);
      const int token = rr / a.G;
      const int head = cur.h * a.G + (rr - token * a.G);
      const long long dst = (static_cast<long long>(cur.q0) + token) * a.Hq + head;
      const int lim = visible(a, Request{cur.q0, cur.tokens, cur.kv}, token);

      // ---- Q rows -> fp16, swizzled; a row's scale goes into its thread's softmax.  The warp loads two rows a step,
      // 16 lanes a row, so that every access takes whole rows; each lane knows where its own row is.
      float inv = 1.0f;
      const long long q_at =
          real ? (static_cast<long long>(cur.q0) + token) * a.q_stride + static_cast<long long>(head) * 128 : -1;
      if (!(ok = warp_wait(&bars->q_empty, pq, bars, a.status))) break;
      pq ^= 1;
      uint8_t* q_rows = sQ + wg * kTileBytes + quarter * 32 * 128;  // the warp's 32 rows, two columns
      const int sub = lane & 15, upper = lane >> 4;
      if (active) {
        uint4 qv[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const long long at = __shfl_sync(0xffffffffu, q_at, 2 * i + upper);
          qv[i] = make_uint4(0, 0, 0, 0);
          if (at >= 0) qv[i] = __ldg(reinterpret_cast<const uint4*>(a.q + at) + sub);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int row2 = 2 * i + upper;
          const uint4 v = qv[i];
          uint32_t qw[4] = {v.x, v.y, v.z, v.w};
          if (!F16) {
            float amax = 0.0f;
#pragma unroll
            for (int x = 0; x < 4; ++x) amax = max3f(amax, fabsf(bf16_lo(qw[x])), fabsf(bf16_hi(qw[x])));
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
            const int e = __float_as_uint(amax) >> 23;
            const int upb = amax == 0.0f || e == 255 ? 0 : min(141 - e, 100);  // 2^upb * amax in [2^14, 2^15)
            const float f = __uint_as_float((upb + 127) << 23);
#pragma unroll
            for (int x = 0; x < 4; ++x) qw[x] = pack_f16x2(bf16_lo(qw[x]) * f, bf16_hi(qw[x]) * f);
            const float back = __shfl_sync(0xffffffffu, __uint_as_float((127 - upb) << 23), (lane & 1) * 16);
            if (lane >> 1 == i) inv = back;
          }
          *reinterpret_cast<uint4*>(q_rows + (sub >> 3) * kHalfBytes + row2 * 128 + (((sub & 7) ^ (row2 & 7)) << 4)) =
              make_uint4(qw[0], qw[1], qw[2], qw[3]);
        }
        fence_proxy_async_smem();
      }
      mbar_arrive(&bars->q_full);
      const float sl2 = a.scale_log2 * inv;

      // pages of a tile's eight records, one a lane, asked for one tile before
      auto page_at = [&](int t) -> unsigned {
        const int rec = (cur.k0 + t) * (kKeyTile / kRecTokens) + lane;
        if (lane >= 8 || rec * kRecTokens >= cur.kv) return 0u;
        return static_cast<unsigned>(__ldg(a.table + static_cast<long long>(cur.r) * a.max_pages + (rec >> log_rec)));
      };
      unsigned page = page_at(0);
      float m_used = -INFINITY, l = 0.0f;  // m_used: a maximum less kLift
      for (int t = 0; t < n && active; ++t) {
        const int key0 = (cur.k0 + t) * kKeyTile;
        const unsigned bad_recs = __ballot_sync(0xffffffffu, page >= static_cast<unsigned>(a.num_pages));
        if (t + 1 < n) page = page_at(t + 1);
        if (!(ok = warp_wait(&bars->s_full[wg], ps, bars, a.status))) break;
        ps ^= 1;
        tc_fence_after();
        float alpha = 1.0f;
        bool rescale = false;
        uint32_t sv[128];
        tmem_ld32(tS + 0, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
        tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
        tmem_ld32(tS + 64, *reinterpret_cast<uint32_t(*)[32]>(&sv[64]));
        tmem_ld32(tS + 96, *reinterpret_cast<uint32_t(*)[32]>(&sv[96]));
        tmem_wait_ld();
        const int see = lim - key0;  // columns this row sees
        if (see < kKeyTile || bad_recs) {
#pragma unroll
          for (int x = 0; x < 128; ++x)
            if (x >= see || (bad_recs >> (x >> 4) & 1)) sv[x] = 0xff800000u;
        }
        // The numerators are taken against the maximum so far while the tile's own is found; only where a row's
        // exceeds it by more than 8 (always in a segment's first tile) are they taken again.
        float part;
        while (true) {
          const float msub = (m_used == -INFINITY) ? 0.0f : m_used;
          const uint64_t c2 = f2pack(sl2, sl2), nm2 = f2pack(-msub, -msub);
          uint64_t acc[2] = {0, 0};
          float a0 = -INFINITY, a1 = -INFINITY;
          const bool first = t == 0 && m_used == -INFINITY;
          if (__all_sync(0xffffffffu, first)) {
#pragma unroll
            for (int x = 0; x < 128; x += 4) {
              a0 = max3f(a0, __uint_as_float(sv[x + 0]), __uint_as_float(sv[x + 1]));
              a1 = max3f(a1, __uint_as_float(sv[x + 2]), __uint_as_float(sv[x + 3]));
            }
            const float mt = fmaxf(a0, a1) * sl2;
            if (mt > -INFINITY) m_used = mt - kLift;
            if (__any_sync(0xffffffffu, mt > -INFINITY)) continue;
          }
#pragma unroll
          for (int hf = 0; hf < 4; ++hf) {
            uint32_t pk[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const uint32_t u = sv[32 * hf + 2 * j], v = sv[32 * hf + 2 * j + 1];
              if (j & 1) a1 = max3f(a1, __uint_as_float(u), __uint_as_float(v));
              else a0 = max3f(a0, __uint_as_float(u), __uint_as_float(v));
              const uint64_t x = fma2(u2pack(u, v), c2, nm2);
              float xa, xb;
              f2unpack(x, xa, xb);
              const float p0 = ex2_approx(xa), p1 = ex2_approx(xb);
              pk[j] = pack_f16x2(p0, p1);
              acc[j & 1] = add2(acc[j & 1], f2pack(p0, p1));
            }
            tmem_st16(tS + 16 * hf, pk);
          }
          float s0, s1, s2, s3;
          f2unpack(acc[0], s0, s1);
          f2unpack(acc[1], s2, s3);
          part = (s0 + s1) + (s2 + s3);
          const float mt = fmaxf(a0, a1) * sl2;
          const bool grow = mt > m_used + (8.0f + kLift);
          if (!__any_sync(0xffffffffu, grow)) break;
          if (grow) {
            rescale = t > 0 && m_used != -INFINITY;
            alpha = rescale ? ex2_approx(m_used - (mt - kLift)) : 1.0f;
            m_used = mt - kLift;
          }
        }
        l = l * alpha + part;
        // Rescale this row of O when its maximum moved.  PV(t-1) is complete: the s_full commit just waited on
        // follows it in issue order.
        if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t ov[32];
            tmem_ld32(tO + x * 32, ov);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * alpha);
            tmem_st32(tO + x * 32, ov);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bars->p_full[wg]);
      }
      if (!ok) break;
      if (active) {
        if (!(ok = warp_wait(&bars->o_full[wg], po, bars, a.status))) break;
        po ^= 1;
        tc_fence_after();
        if (cur.whole) {
          // through the warp's rows of Q, which no product reads any more, so that whole rows are stored
          const float scale = l != 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t ov[32];
            tmem_ld32(tO + x * 32, ov);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t w[4];
#pragma unroll
              for (int y = 0; y < 4; ++y)
                w[y] = pack_half2<F16>(__uint_as_float(ov[8 * j + 2 * y]) * scale, __uint_as_float(ov[8 * j + 2 * y + 1]) * scale);
              const int chunk = 4 * x + j;
              *reinterpret_cast<uint4*>(q_rows + (chunk >> 3) * kHalfBytes + lane * 128 + (((chunk & 7) ^ (lane & 7)) << 4)) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          __syncwarp();
          const long long o_at = real ? dst : -1;
#pragma unroll 4
          for (int i = 0; i < 16; ++i) {
            const int row2 = 2 * i + upper;
            const long long at = __shfl_sync(0xffffffffu, o_at, row2);
            const uint4 v = *reinterpret_cast<const uint4*>(q_rows + (sub >> 3) * kHalfBytes + row2 * 128 +
                                                            (((sub & 7) ^ (row2 & 7)) << 4));
            if (at >= 0) reinterpret_cast<uint4*>(a.o + at * 128)[sub] = v;
          }
          if (real) a.lse[dst] = l != 0.0f ? (m_used + __log2f(l)) * 0.69314718055994531f : -INFINITY;
          __syncwarp();  // read before the next item's Q takes the rows
        } else {
          // four channels of 256 rows after another: the threads of a warp store 512 bytes in a row
          float* part = parts_of(a.ws, gridDim.x) + (static_cast<size_t>(cta) * 2 + (cur.k0 > 0 ? 0 : 1)) * part_floats<kRowTile>();
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t ov[32];
            tmem_ld32(tO + x * 32, ov);
            tmem_wait_ld();
            if (real) {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                reinterpret_cast<uint4*>(part)[(x * 8 + j) * kRowTile + row] =
                    make_uint4(ov[4 * j], ov[4 * j + 1], ov[4 * j + 2], ov[4 * j + 3]);
            }
          }
          if (real) {
            part[kRowTile * 128 + row] = m_used;
            part[kRowTile * 129 + row] = l;
          }
        }
        tc_fence_before();
        mbar_arrive(&bars->o_empty[wg]);
      }
      if (wg == 0 && r == 0 && cur.last >= 0) *joint = Joint{cur.last, cur.h, cur.j, cur.q0, min(kRowTile, rows), {0, 0, 0}};
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the rows of the items that more than one CTA worked on.  A CTA takes 32
// rows, a lane a row (reads of 512 bytes in a row).  Up to 8 parts, as of long
// batches, a warp takes 16 channels and goes through the parts; more, as of one
// item over many CTAs (148 parts one after another took 70 us), a warp takes
// every eighth part, and the warps' sums are joined; the next three CTAs, which
// have no item of their own then, take 32 channels each, as the first does.
constexpr int kJoinRows = 32, kJoinWarps = 8;
struct RowSum {
  float m, l;
};
// Scales of what is there and of a part under their joint maximum; without a
// maximum a part has nothing but zeros, or the NaN of its scores.
__device__ __forceinline__ void join_scales(RowSum& t, float pm, float pl, float& w0, float& w1) {
  const float mn = fmaxf(t.m, pm);
  w0 = t.m == -INFINITY ? 1.0f : ex2_approx(t.m - mn);
  w1 = pm == -INFINITY ? 1.0f : ex2_approx(pm - mn);
  t.l = w0 * t.l + w1 * pl;
  t.m = mn;
}
__device__ __forceinline__ float4 scaled_sum(float w0, float4 a, float w1, float4 b) {
  return make_float4(w0 * a.x + w1 * b.x, w0 * a.y + w1 * b.y, w0 * a.z + w1 * b.z, w0 * a.w + w1 * b.w);
}

template <bool F16>
__global__ void __launch_bounds__(kJoinWarps * 32)
    cache_attn_join_kernel(const __grid_constant__ AttnArgs a, int workers) {
  __shared__ float4 sums[kJoinWarps][8][kJoinRows];
  __shared__ RowSum row_sums[kJoinWarps][kJoinRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.y * kJoinRows + lane;
  if (a.fill) fill_rows(a);
  const Joint* joints = static_cast<const Joint*>(a.ws);
  int first = blockIdx.x, quarter = 0;
  if (joints[first].last < 0) {
    for (int k = 1; k < 4 && k <= first && quarter == 0; ++k)
      if (joints[first - k].last - (first - k) >= 8) quarter = k;
    if (quarter == 0) return;
    first -= quarter;
  }
  const Joint jt = joints[first];
  if (static_cast<int>(blockIdx.y) * kJoinRows >= jt.rows) return;  // the whole CTA
  const bool real = row < jt.rows;
  constexpr size_t kPart = part_floats<kRowTile>();
  const float* parts = parts_of(a.ws, workers);
  auto part = [&](int w) { return parts + (static_cast<size_t>(w) * 2 + (w == first ? 1 : 0)) * kPart; };
  const int rr = jt.j * kRowTile + row, token = rr / a.G;
  const long long dst = (static_cast<long long>(jt.q0) + token) * a.Hq + jt.h * a.G + (rr - token * a.G);
  RowSum t{-INFINITY, 0.0f};
  if (jt.last - first < 8) {
    float4 o[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) o[x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (!real) return;
#pragma unroll 2
    for (int w = first; w <= jt.last; ++w) {
      const float* f = part(w);
      float4 p[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) p[x] = reinterpret_cast<const float4*>(f)[(warp * 4 + x) * kRowTile + row];
      float w0, w1;
      join_scales(t, f[kRowTile * 128 + row], f[kRowTile * 129 + row], w0, w1);
#pragma unroll
      for (int x = 0; x < 4; ++x) o[x] = scaled_sum(w0, o[x], w1, p[x]);
    }
    const float inv = t.l != 0.0f ? 1.0f / t.l : 0.0f;
    uint32_t w[8];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      w[2 * x] = pack_half2<F16>(o[x].x * inv, o[x].y * inv);
      w[2 * x + 1] = pack_half2<F16>(o[x].z * inv, o[x].w * inv);
    }
    uint4* out = reinterpret_cast<uint4*>(a.o + dst * 128 + warp * 16);
    out[0] = make_uint4(w[0], w[1], w[2], w[3]);
    out[1] = make_uint4(w[4], w[5], w[6], w[7]);
  } else {
    const int group0 = quarter * 8;  // groups of 4 channels
    float4 s[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) s[x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (real) {
#pragma unroll 2
      for (int w = first + warp; w <= jt.last; w += kJoinWarps) {
        const float* f = part(w);
        float4 p[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) p[x] = reinterpret_cast<const float4*>(f)[(group0 + x) * kRowTile + row];
        float w0, w1;
        join_scales(t, f[kRowTile * 128 + row], f[kRowTile * 129 + row], w0, w1);
#pragma unroll
        for (int x = 0; x < 8; ++x) s[x] = scaled_sum(w0, s[x], w1, p[x]);
      }
    }
#pragma unroll
    for (int x = 0; x < 8; ++x) sums[warp][x][lane] = s[x];
    row_sums[warp][lane] = t;
    __syncthreads();
    t = RowSum{-INFINITY, 0.0f};
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < kJoinWarps; ++i) {
      float w0, w1;
      join_scales(t, row_sums[i][lane].m, row_sums[i][lane].l, w0, w1);
      o = scaled_sum(w0, o, w1, sums[i][warp][lane]);
    }
    const float inv = t.l != 0.0f ? 1.0f / t.l : 0.0f;
    uint2 w;
    w.x = pack_half2<F16>(o.x * inv, o.y * inv);
    w.y = pack_half2<F16>(o.z * inv, o.w * inv);
    if (real) reinterpret_cast<uint2*>(a.o + dst * 128)[group0 + warp] = w;
  }
  if (real && warp == 0 && quarter == 0) a.lse[dst] = t.l != 0.0f ? (t.m + __log2f(t.l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace

size_t cache_attn_chunk_workspace(int num_workers) {
  return num_workers * (sizeof(Joint) + 2 * part_floats<kRowTile>() * sizeof(float));
}

cudaError_t launch_cache_attn_chunk(const cache::AttnArgs& a, int over, bool f16, int num_workers,
                                    cudaStream_t stream) {
  const Share share{over, 0x7fffffff};
  auto kern = f16 ? cache_attn_chunk_kernel<true> : cache_attn_chunk_kernel<false>;
  static SmemAllowed allowed[2];  // fp16, bf16
  cudaError_t e = allowed[f16 ? 0 : 1].ensure(reinterpret_cast<const void*>(kern), kSmemTotal);
  if (e != cudaSuccess) return e;
  kern<<<num_workers, kThreads, kSmemTotal, stream>>>(a, share);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  auto join = f16 ? cache_attn_join_kernel<true> : cache_attn_join_kernel<false>;
  join<<<dim3(num_workers, kRowTile / kJoinRows), kJoinWarps * 32, 0, stream>>>(a, num_workers);
  return cudaGetLastError();
}

}  // namespace vsa
