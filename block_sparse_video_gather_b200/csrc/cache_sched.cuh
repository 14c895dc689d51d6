// cache_sched.cuh -- how the attention kernels of the 4-bit cache divide a batch.
//
// The rows of a request and key head are its new tokens times the query heads
// that share the key head, row = token * G + head in the group, cut into tiles
// of RT rows; an item is one (request, key head, tile).  Its cached tokens, as
// far as the tile's last row sees them, are cut into units of KT keys (an item
// that sees nothing has one unit, which writes its rows).  All units of the
// batch in item order form one line, and each of N workers takes U / N of them,
// the first U % N one more: lengths as uneven as they may be, each worker reads the same amount to
// within a unit.  Items that end up in several workers are joined by their
// running maxima and sums.  Every worker finds its place by itself from cu and
// kv_len, so lengths stay on the device and a captured call takes new ones.
#pragma once

#include "cache.cuh"

namespace vsa {
namespace cache {

// sum_{i < n} floor((a i + b) / m) for n, a, b >= 0, m > 0: the Euclid-like
// recursion on (m, a) for counting lattice points under a line.
__device__ __forceinline__ long long floor_sum(long long n, long long m, long long a, long long b) {
  long long s = 0;
  while (n > 0) {
    s += (n - 1) * n / 2 * (a / m) + n * (b / m);
    a %= m;
    b %= m;
    const long long y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const long long t = m;
    m = a;
    a = t;
  }
  return s;
}

// a / b for a >= 0, b > 0, in 32 bits where both fit.
__device__ __forceinline__ long long div_small(long long a, long long b) {
  if ((a | b) >> 32 == 0) return static_cast<unsigned>(a) / static_cast<unsigned>(b);
  return a / b;
}

// COST: places of the line that an item takes before its first unit, for the
// time a worker spends on an item whatever its length (its rows of Q, the first
// product, the output); they hold no work.
template <int RT, int KT, int COST>
struct Sched {
  static constexpr int kCost = COST;
  static __device__ __forceinline__ int tiles(const AttnArgs& a, const Request& q) { return (q.n * a.G + RT - 1) / RT; }
  // Cached tokens that tile j's last row sees.
  static __device__ __forceinline__ int keys(const AttnArgs& a, const Request& q, int j) {
    const int last = min((j + 1) * RT, q.n * a.G) - 1;
    return visible(a, q, last / a.G);
  }
  // Units of n >= 0 keys; n + KT - 1 may pass 2^31.
  static __device__ __forceinline__ int units_of(int n) {
    return max(1, static_cast<int>((static_cast<unsigned>(n) + KT - 1) / KT));
  }
  static __device__ __forceinline__ int units(const AttnArgs& a, const Request& q, int j) {
    return COST + units_of(keys(a, q, j));
  }
  // Places of tiles 0 .. j-1.
  static __device__ __forceinline__ long long units_before(const AttnArgs& a, const Request& q, int j) {
    if (!a.causal) return static_cast<long long>(COST + units_of(q.kv)) * j;
    if (j <= 1) return j == 0 ? 0 : units(a, q, 0);
    // whole tiles i: the last row's token is floor((RT (i + 1) - 1) / G), it sees kv - n + 1 more than that many
    // tokens, which is floor((RT (i + 1) - 1 + G (kv - n + KT)) / (G KT)) units, or 1 where that is less
    const int whole = (q.n * a.G) / RT, n = min(j, whole);
    const long long G = a.G, c = q.kv - q.n;
    const long long short_of = 1 - G * c;  // RT (i + 1) must reach this for the first whole unit
    const long long i0 = min(static_cast<long long>(n), short_of <= RT ? 0 : (short_of + RT - 1) / RT - 1);
    long long s = static_cast<long long>(COST) * n + i0 + floor_sum(n - i0, G * KT, RT, RT * (i0 + 1) - 1 + G * (c + KT));
    if (j > whole) s += units(a, q, whole);
    return s;
  }
};

// Which requests a kernel takes: those of more than `over` and at most `upto` rows a key head.
struct Share {
  int over, upto;
};
__device__ __forceinline__ bool takes(const Share& s, const AttnArgs& a, const Request& q) {
  const int rows = q.n * a.G;
  return rows > s.over && rows <= s.upto;
}

// Where each request's units begin in the line.  Up to 32 requests: lane r of
// every warp holds request r's, and nothing goes through shared memory; more:
// one array of sums in shared memory, made by the whole CTA.
struct Line {
  long long total;     // U
  int items;           // (request, key head, tile)s where known (R <= 32), else 0
  long long at, units; // lane r: first unit and units of request r (R <= 32)
  Request own;         // lane r: request r (R <= 32)
  const long long* pre;  // [R + 1] first units (R > 32)

  // Request r.  All lanes of a warp, r the same in all.
  __device__ __forceinline__ Request request(const AttnArgs& a, int r) const {
    if (a.R > 32) return load_request(a, r, false);
    return Request{__shfl_sync(0xffffffffu, own.q0, r), __shfl_sync(0xffffffffu, own.n, r),
                   __shfl_sync(0xffffffffu, own.kv, r)};
  }

  // The request that holds unit u < U, and its first unit.  All lanes of a warp.
  __device__ __forceinline__ int request_of(int R, long long u, long long& first) const {
    if (R <= 32) {
      const int lane = threadIdx.x & 31;
      const int r = __ffs(__ballot_sync(0xffffffffu, lane < R && u >= at && u < at + units)) - 1;
      first = __shfl_sync(0xffffffffu, at, r);
      return r;
    }
    int lo = 0, hi = R;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= u) lo = mid;
      else hi = mid;
    }
    first = pre[lo];
    return lo;
  }
};

__device__ __forceinline__ long long warp_scan(long long v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += u;
  }
  return v;
}

// All threads of the CTA; `pre` [R + 1] and `part` [warps] in shared memory are
// used for more than 32 requests only, and then the call ends with a barrier.
template <class S, int THREADS>
__device__ __forceinline__ Line make_line(const AttnArgs& a, const Share& share, long long* pre, long long* part) {
  Line line;
  line.pre = pre;
  line.at = line.units = 0;
  line.items = 0;
  line.own = Request{0, 0, 0};
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto units_of = [&](int r, bool report) -> long long {
    const Request q = load_request(a, r, report);
    return takes(share, a, q) ? S::units_before(a, q, S::tiles(a, q)) * a.Hkv : 0;
  };
  if (a.R <= 32) {
    if (lane < a.R) {
      line.own = load_request(a, lane, blockIdx.x == 0 && warp == 0);
      if (takes(share, a, line.own)) {
        line.items = S::tiles(a, line.own);
        line.units = S::units_before(a, line.own, line.items) * a.Hkv;
      }
    }
    const long long v = warp_scan(line.units);
    line.items = __reduce_add_sync(0xffffffffu, line.items) * a.Hkv;
    line.at = v - line.units;
    line.total = __shfl_sync(0xffffffffu, v, 31);
    return line;
  }
  const int per = (a.R + THREADS - 1) / THREADS;
  const int r0 = min(static_cast<int>(threadIdx.x) * per, a.R), r1 = min(r0 + per, a.R);
  long long sum = 0;
  for (int r = r0; r < r1; ++r) {
    pre[r] = sum;
    sum += units_of(r, blockIdx.x == 0);
  }
  const long long v = warp_scan(sum);
  if (lane == 31) part[warp] = v;
  __syncthreads();
  long long before = v - sum;
  for (int w = 0; w < warp; ++w) before += part[w];
  for (int r = r0; r < r1; ++r) pre[r] += before;
  if (threadIdx.x == THREADS - 1) pre[a.R] = before + sum;
  __syncthreads();
  line.total = pre[a.R];
  return line;
}

// A place in the line.
template <class S>
struct Cursor {
  int r, h, j;         // item
  int k, nu;           // place in it, and its places (units and S::kCost)
  int nt;              // tiles of the request
  Request req;
  long long item0;     // the item's first unit in the line

  // Unit u of the line.  All lanes of a warp.
  __device__ __forceinline__ void seek(const AttnArgs& a, const Line& line, long long u) {
    long long first;
    r = line.request_of(a.R, u, first);
    req = line.request(a, r);
    nt = S::tiles(a, req);
    const long long head = S::units_before(a, req, nt);
    long long rem = u - first;
    h = static_cast<int>(div_small(rem, head));
    rem -= h * head;
    // the last tile that begins at or before rem: 32 places a step, a lane each
    const int lane = threadIdx.x & 31;
    int tl = 0, left = nt;
    long long before = 0;
    while (left > 1) {
      const int step = (left + 31) >> 5, at = lane * step;
      const long long x = at < left ? S::units_before(a, req, tl + at) : 0;
      const int hit = 31 - __clz(__ballot_sync(0xffffffffu, at < left && x <= rem));  // lane 0's is
      before = __shfl_sync(0xffffffffu, x, hit);
      tl += hit * step;
      left = min(step, left - hit * step);
    }
    j = tl;
    k = static_cast<int>(rem - before);
    nu = S::units(a, req, j);
    item0 = u - k;
  }
  // The next item; the caller knows that there is one.
  __device__ __forceinline__ void next_item(const AttnArgs& a, const Share& share) {
    item0 += nu;
    k = 0;
    if (++j == nt) {
      j = 0;
      if (++h == a.Hkv) {
        h = 0;
        do {
          ++r;
          req = load_request(a, r, false);
        } while (r + 1 < a.R && !takes(share, a, req));
        nt = S::tiles(a, req);
      }
    }
    nu = S::units(a, req, j);
  }
};

// The line cut for n workers: the first U % n get one unit more than the others.
struct Cut {
  long long size, more;  // U / n, U % n
  __device__ __forceinline__ Cut(long long U, int n) {
    size = div_small(U, n);
    more = U - size * n;
  }
  __device__ __forceinline__ long long start(int i) const { return i * size + min(static_cast<long long>(i), more); }
  // The worker that holds unit u.
  __device__ __forceinline__ int worker_of(long long u) const {
    const long long big = more * (size + 1);
    return static_cast<int>(u < big ? div_small(u, size + 1) : more + div_small(u - big, size));
  }
};

// Workspace: counters of joined items, then the workers' parts.  A worker's
// range cuts at most two items, its first (slot 0) and the one that starts in
// it and goes on (slot 1); a part holds RT rows of 128 sums, then RT maxima and
// RT denominators.
constexpr int kMaxWorkers = 1024;
template <int RT>
__host__ __device__ constexpr size_t part_floats() {
  return static_cast<size_t>(RT) * 130;
}

}  // namespace cache
}  // namespace vsa
