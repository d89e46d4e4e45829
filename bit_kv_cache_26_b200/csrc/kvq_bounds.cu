// Bounds of a page's keys and the pages worth attending to.
//
// kvq_page_bounds keeps, per page and KV head, the minimum and maximum of the raw keys in every
// channel, updated as tokens arrive: bounds[page][head][0 / 1][128] in the input type (a choice of
// input values, so exact).
//
// kvq_select_pages ranks the pages of a (sequence, KV head) by the sum over its query heads of
// the largest q_g . k a key inside the page's bounds could have:
//   sum_g sum_d max(q_gd lo_d, q_gd hi_d) = sum_d W+_d hi_d + W-_d lo_d,
//   W+_d = sum_g max(q_gd, 0),  W-_d = sum_g min(q_gd, 0)
// (hi multiplies what is positive of q, lo what is negative), one product of length 256 per page
// whatever the number of query heads.  Every operation is fp32 in a fixed order, so that the
// choice is the same on every run and can be restated bit for bit:
//   W: the query heads in 16 places (absent ones 0), halved: places i and i + 8, + 4, + 2, + 1;
//   term_d = fl(fl(W+_d hi_d) + fl(W-_d lo_d)); 8 neighbouring channels halved (4, 2, 1), then
//   the 16 sums halved (8, 4, 2, 1).  Equal scores: the lower page.  NaN ranks above all.
//
// Bound: HBM.  One B200: bounds of 8 x 32768 keys x 8 heads 93 us (6.1 TB/s, 0.93 of the copy
// bandwidth); selection over 256 sequences x 8 heads x 512 pages 98 us (5.5 TB/s, 0.84), for one
// sequence of 1024 pages 10.6 us of latency (lengths, page ids, bounds, the last CTA's choice).  The
// query heads are loaded before the first is used: 16 heads a group in turn took 12.8 us for 9.2 there.
#include <algorithm>
#include <atomic>

#include "kvq_common.cuh"
#include "kvq_internal.h"
#include "kvq_pipe.cuh"

namespace kvq {

namespace {

// ---- bounds ----------------------------------------------------------------------------------

constexpr int kBoundsWarps = 8;

template <bool BF16>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (BF16) asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <bool BF16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (BF16) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// One warp per (page, KV head, sequence): 16 lanes hold a row of 128 channels, the warp two rows
// per load; all of the page's rows are in flight at once.
template <bool BF16>
__global__ void __launch_bounds__(kBoundsWarps * 32) page_bounds_kernel(Geom g, const uint16_t* __restrict__ k_new, int n_new,
                                                                        uint16_t* bounds) {
  const int lane = threadIdx.x & 31, half = lane >> 4, c = lane & 15;
  const int64_t item = (int64_t)blockIdx.x * kBoundsWarps + (threadIdx.x >> 5);
  const int b = blockIdx.y, h = (int)(item % g.H);
  const int L = g.seq_len[b];
  if (L < 0 || (int64_t)L + n_new > (int64_t)g.maxp * kG) {
    if (item == 0 && lane == 0) set_status(g.status, KVQ_DEV_OVERFLOW);
    return;
  }
  const int64_t pg = L / kG + item / g.H;
  if (pg * kG >= (int64_t)L + n_new) return;
  const int phys = g.page_table[(int64_t)b * g.maxp + pg];
  if (phys < 0 || phys >= g.npages) {
    if (lane == 0) set_status(g.status, KVQ_DEV_BAD_PAGE);
    return;
  }
  // slots [s0, s1) of the page are new
  const int s0 = max(0, (int)(L - pg * kG)), s1 = (int)min((int64_t)kG, (int64_t)L + n_new - pg * kG);
  const uint32_t inf = BF16 ? 0x7f807f80u : 0x7c007c00u, ninf = inf | 0x80008000u;
  const uint16_t* src = k_new + (((int64_t)b * n_new + (pg * kG - L)) * g.H + h) * kD + 8 * c;
  uint4 row[kG / 2];
#pragma unroll
  for (int i = 0; i < kG / 2; ++i) {
    const int slot = 2 * i + half;
    if (slot >= s0 && slot < s1) row[i] = __ldcs(reinterpret_cast<const uint4*>(src + (int64_t)slot * g.H * kD));
  }
  uint4 lo = make_uint4(inf, inf, inf, inf), hi = make_uint4(ninf, ninf, ninf, ninf);
  uint16_t* dst = bounds + ((int64_t)phys * g.H + h) * 2 * kD + 8 * c;
  if (s0 > 0 && half == 0) {  // the page's earlier tokens
    lo = *reinterpret_cast<const uint4*>(dst);
    hi = *reinterpret_cast<const uint4*>(dst + kD);
  }
#pragma unroll
  for (int i = 0; i < kG / 2; ++i) {
    const int slot = 2 * i + half;
    if (slot >= s0 && slot < s1) {
      lo = make_uint4(min2<BF16>(lo.x, row[i].x), min2<BF16>(lo.y, row[i].y), min2<BF16>(lo.z, row[i].z), min2<BF16>(lo.w, row[i].w));
      hi = make_uint4(max2<BF16>(hi.x, row[i].x), max2<BF16>(hi.y, row[i].y), max2<BF16>(hi.z, row[i].z), max2<BF16>(hi.w, row[i].w));
    }
  }
  uint32_t* l = &lo.x;
  uint32_t* u = &hi.x;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    l[e] = min2<BF16>(l[e], __shfl_xor_sync(kFull, l[e], 16));
    u[e] = max2<BF16>(u[e], __shfl_xor_sync(kFull, u[e], 16));
  }
  *reinterpret_cast<uint4*>(dst + half * kD) = half ? hi : lo;
}

// ---- selection -------------------------------------------------------------------------------

constexpr int kSelThreads = 128;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelAhead = 4;           // pages of a round per 16 lanes
constexpr int kSelRounds = 2;          // rounds in flight
constexpr int kSelRing = kSelRounds * kSelAhead * 2 * kSelThreads * 16;  // bytes: 16 of lo and of hi per lane and page
constexpr int kLocalKeys = 1024;       // keys that stay in shared memory when one CTA scores all pages
constexpr int kSelKeys = kSelRing / 4; // keys that fit in the ring's place when the scores are all there

// fp32 -> unsigned with the same order; -0 is +0, NaN above all.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t u = __float_as_uint(__fadd_rn(x, 0.0f));
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

template <bool BF16>
__device__ __forceinline__ unsigned long long widen(uint32_t u) {
  if constexpr (BF16) return pk(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u));
  return pk(f.x, f.y);
}

// Scores of pages [p0, p1) of (b, h) as ordered keys, keys[p - lo_page]: 16 lanes per page, 8 channels per lane.  Every lane
// copies its own 32 bytes of a page into its own places of the ring (so it waits for its own copies only) and has two
// rounds of four pages in flight; the four sums over the lanes share the exchanges (after a step that halves the lanes a
// value is spread over, each half of the lanes goes on with half of the values).
template <bool BF16>
__device__ void score_pages(const Geom& g, const uint16_t* __restrict__ q, int Gq, const uint16_t* __restrict__ bounds, int b,
                            int h, int p0, int p1, int lo_page, uint32_t* keys, float* W, uint8_t* ring,
                            float minus_zero) {
  static_assert(kSelAhead == 4 && kSelRounds == 2, "the exchanges and waits below are written for these");
  constexpr int kStep = 2 * kSelAhead * kSelWarps;  // pages of a round of the block
  const int lane = threadIdx.x & 31, c = lane & 15, sub = lane >> 4;
  const int32_t* table = g.page_table + (int64_t)b * g.maxp;
  const int first = p0 + 2 * kSelAhead * (threadIdx.x >> 5) + kSelAhead * sub;
  int phys[kSelAhead];
  auto load_ids = [&](int p) {
#pragma unroll
    for (int i = 0; i < kSelAhead; ++i) {
      phys[i] = p + i < p1 ? table[p + i] : -1;
      if (p + i < p1 && (unsigned)phys[i] >= (unsigned)g.npages) {
        set_status(g.status, KVQ_DEV_BAD_PAGE);
        phys[i] = -1;
      }
    }
  };
  const uint16_t* mine = bounds + (int64_t)h * 2 * kD + 8 * c;
  const int64_t page_stride = (int64_t)g.H * 2 * kD;
  uint8_t* place = ring + threadIdx.x * 16;  // + (round, page, lo / hi) * the block's threads * 16
  unsigned gone[kSelRounds] = {0u, 0u};      // pages of the round that have no valid id
  auto issue = [&](int round) {
    unsigned none = 0;
#pragma unroll
    for (int i = 0; i < kSelAhead; ++i) {
      if (phys[i] >= 0) {
        const uint16_t* src = mine + phys[i] * page_stride;
        const uint32_t dst = smem_u32(place + (round * kSelAhead + i) * 2 * kSelThreads * 16);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + kSelThreads * 16), "l"(src + kD) : "memory");
      } else {
        none |= 1u << i;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    gone[round] = none;
  };
  load_ids(first);
  issue(0);
  load_ids(first + kStep);
  issue(1);
  load_ids(first + 2 * kStep);
  static_assert(kSelThreads == kD, "a thread per channel of W+ and W-");
  {
    float v[16];
    uint16_t raw[16];  // all loads before the first use
    const uint16_t* src = q + ((int64_t)b * g.H * Gq + (int64_t)h * Gq) * kD + threadIdx.x;
#pragma unroll
    for (int i = 0; i < 16; ++i) raw[i] = __ldg(src + min(i, Gq - 1) * kD);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = i < Gq ? bits_to_float(raw[i], BF16 ? KVQ_BF16 : KVQ_F16) : 0.f;
#pragma unroll
    for (int neg = 0; neg < 2; ++neg) {
      float w[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = v[i] != v[i] ? v[i] : neg ? fminf(v[i], 0.f) : fmaxf(v[i], 0.f);
#pragma unroll
      for (int o = 8; o; o >>= 1)
#pragma unroll
        for (int i = 0; i < o; ++i) w[i] = __fadd_rn(w[i], w[i + o]);
      W[neg * kD + threadIdx.x] = w[0];
    }
  }
  __syncthreads();
  unsigned long long up[4], dn[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    up[e] = pk(W[8 * c + 2 * e], W[8 * c + 2 * e + 1]);
    dn[e] = pk(W[kD + 8 * c + 2 * e], W[kD + 8 * c + 2 * e + 1]);
  }
  // a product and a sum of pairs may be compiled into one fused operation, which rounds once; x y + (-0), with a -0 that the
  // compiler does not see, is the rounded product and can't be
  const unsigned long long mz2 = pk(minus_zero, minus_zero);
  auto round = [&](int p, int r) {
    asm volatile("cp.async.wait_group 1;" ::: "memory");  // all but the newest round
    float x[kSelAhead];
#pragma unroll
    for (int i = 0; i < kSelAhead; ++i) {
      const uint8_t* from = place + (r * kSelAhead + i) * 2 * kSelThreads * 16;
      const uint4 lo = *reinterpret_cast<const uint4*>(from), hi = *reinterpret_cast<const uint4*>(from + kSelThreads * 16);
      const uint32_t l[4] = {lo.x, lo.y, lo.z, lo.w}, u[4] = {hi.x, hi.y, hi.z, hi.w};
      unsigned long long t[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) t[e] = add2(fma2(up[e], widen<BF16>(u[e]), mz2), fma2(dn[e], widen<BF16>(l[e]), mz2));
      float s0, s1;
      upk(add2(add2(t[0], t[2]), add2(t[1], t[3])), s0, s1);
      x[i] = __fadd_rn(s0, s1);
    }
    const unsigned none = gone[r];
    issue(r);  // the round after the next, into the places just read
    load_ids(p + 3 * kStep);
    // lanes with bit 3: pages 2 and 3; of those, lanes with bit 2: the odd one
    const bool b3 = c & 8, b2 = c & 4;
    const float y0 = __fadd_rn(b3 ? x[2] : x[0], __shfl_xor_sync(kFull, b3 ? x[0] : x[2], 8));
    const float y1 = __fadd_rn(b3 ? x[3] : x[1], __shfl_xor_sync(kFull, b3 ? x[1] : x[3], 8));
    float z = __fadd_rn(b2 ? y1 : y0, __shfl_xor_sync(kFull, b2 ? y0 : y1, 4));
    z = __fadd_rn(z, __shfl_xor_sync(kFull, z, 2));
    z = __fadd_rn(z, __shfl_xor_sync(kFull, z, 1));
    const int i = (b3 ? 2 : 0) + (b2 ? 1 : 0);
    if ((c & 3) == 0 && p + i < p1) keys[p + i - lo_page] = none >> i & 1 ? 0u : order_key(z);
  };
  for (int p = first; p - kSelAhead * sub < p1; p += 2 * kStep) {
    round(p, 0);
    if (p + kStep - kSelAhead * sub < p1) round(p + kStep, 1);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Shared memory of the choice.
struct Chooser {
  unsigned bins[256];
  uint4 sums[2];                 // one value per warp, two sets
  unsigned digit, above, count;
};

// One value per warp (the same in all its lanes) to every thread, joined by `join`; one barrier.
template <typename F>
__device__ __forceinline__ unsigned block_join(unsigned v, uint4* buf, F join) {
  static_assert(kSelWarps == 4, "one 16-byte read");
  if ((threadIdx.x & 31) == 0) reinterpret_cast<unsigned*>(buf)[threadIdx.x >> 5] = v;
  __syncthreads();
  const uint4 x = *buf;
  return join(join(x.x, x.y), join(x.z, x.w));
}
// The sum of the warps before this one.
__device__ __forceinline__ unsigned block_before(unsigned v, uint4* buf) {
  if ((threadIdx.x & 31) == 0) reinterpret_cast<unsigned*>(buf)[threadIdx.x >> 5] = v;
  __syncthreads();
  unsigned s = 0;
  for (int w = 0; w < (int)(threadIdx.x >> 5); ++w) s += reinterpret_cast<const unsigned*>(buf)[w];
  return s;
}

// The k largest of keys[0 .. m) (ties: the lower index), in index order, as `base` + index to list[0 .. k); run by the
// whole block.  The k-th largest key is found by histograms of 8 bits at a time, below the bits all keys share and until
// the keys of a bin are exactly the ones still wanted: two or three rounds where a bit-by-bit search took eleven, each
// as long as a round here.  The loops stay rolled: they run once per group, and fetching the instructions of unrolled
// ones took longer than the keys.
template <bool L2>
__device__ void take_largest(const uint32_t* keys, int m, int k, int base, int32_t* list, Chooser& s) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto load = [&](int i) -> uint32_t { return L2 ? __ldcg(keys + i) : keys[i]; };
  uint32_t top = 0u, low = ~0u;
#pragma unroll 4
  for (int i = tid; i < m; i += kSelThreads) {
    const uint32_t x = load(i);
    top = max(top, x);
    low = min(low, x);
  }
  s.bins[2 * tid] = s.bins[2 * tid + 1] = 0u;
  top = block_join(__reduce_max_sync(kFull, top), &s.sums[0], [](unsigned x, unsigned y) { return max(x, y); });
  low = block_join(__reduce_min_sync(kFull, low), &s.sums[1], [](unsigned x, unsigned y) { return min(x, y); });
  int shift = 32 - __clz(top ^ low);  // bits below the ones all keys share
  uint32_t T = shift == 32 ? 0u : top >> shift << shift;
  unsigned want = k;                  // of the keys that agree with T above `shift`
  bool exact = false;                 // they are all wanted
  while (shift > 0) {
    const int width = min(8, shift), high = shift;
    shift -= width;
    const uint32_t prefix = high == 32 ? 0u : T >> high, mask = (1u << width) - 1u;
#pragma unroll 4
    for (int i = tid; i < m; i += kSelThreads) {
      const uint32_t x = load(i);
      if ((high == 32 ? 0u : x >> high) == prefix) atomicAdd(&s.bins[x >> shift & mask], 1u);
    }
    __syncthreads();
    const int d1 = 255 - 2 * tid;  // bins d1 and d1 - 1: from the highest on
    const unsigned m1 = s.bins[d1], m0 = s.bins[d1 - 1];
    unsigned upto = m1 + m0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned v = __shfl_up_sync(kFull, upto, o);
      if (lane >= o) upto += v;
    }
    upto += block_before(__shfl_sync(kFull, upto, 31), &s.sums[0]);
    const unsigned before1 = upto - m0 - m1, before0 = upto - m0;
    if (upto >= want && before1 < want) {
      const bool first = before0 >= want;
      s.digit = first ? d1 : d1 - 1;
      s.above = first ? before1 : before0;
      s.count = first ? m1 : m0;
    }
    s.bins[d1] = s.bins[d1 - 1] = 0u;  // (each thread's own) for the next round
    __syncthreads();
    T |= s.digit << shift;
    want -= s.above;
    exact = s.count == want;
    if (exact) break;
    __syncthreads();  // before s.digit is written again
  }
  // keys > T (>= T when all of those are wanted) are taken, and the first `want` that equal T
  const uint32_t over = exact ? T - 1u : T;  // (exact leaves T > 0: there are more than k keys)
  const int rows = (m + kSelThreads - 1) / kSelThreads;  // a warp's run: rows x 32 consecutive keys
  const int a0 = warp * rows * 32 + lane;
  unsigned gt = 0, eq = 0;
#pragma unroll 4
  for (int i = 0; i < rows; ++i) {
    const int at = a0 + 32 * i;
    const uint32_t x = at < m ? load(at) : 0u;
    gt += at < m && x > over;
    eq += at < m && x == T;
  }
  unsigned out, tie;
  if (m < 65536) {  // both counts in one exchange
    const unsigned before = block_before(__reduce_add_sync(kFull, gt << 16 | eq), &s.sums[0]);
    out = before >> 16;
    tie = before & 0xffffu;
  } else {
    out = block_before(__reduce_add_sync(kFull, gt), &s.sums[0]);
    tie = block_before(__reduce_add_sync(kFull, eq), &s.sums[1]);
  }
  if (!exact) out += min(tie, want);
  const unsigned below = (1u << lane) - 1u;
  for (int i = 0; i < rows; ++i) {
    const int at = a0 + 32 * i;
    const uint32_t x = at < m ? load(at) : 0u;
    const unsigned same = __ballot_sync(kFull, !exact && at < m && x == T);
    const bool take = at < m && (x > over || ((same >> lane & 1u) && tie + __popc(same & below) < want));
    const unsigned taken = __ballot_sync(kFull, take);
    if (take) list[out + __popc(taken & below)] = base + at;
    out += __popc(taken);
    tie += __popc(same);
  }
}

// CTAs an SM holds: by shared memory (228 KB, of which each takes 1 KB besides its own).
constexpr int kSelCtas = 5;
constexpr int kSelSmem = kSelRing + 2 * kD * 4 + (int)sizeof(Chooser) + 4 * kLocalKeys + 16 + 1024;
static_assert(kSelCtas * kSelSmem <= 228 * 1024 && (kSelCtas + 1) * kSelSmem > 228 * 1024, "the CTAs an SM holds");

template <bool BF16>
__global__ void __launch_bounds__(kSelThreads, kSelCtas) select_pages_kernel(Geom g, SelectArgs a) {
  __shared__ float W[2 * kD];
  __shared__ Chooser chooser;
  __shared__ uint32_t local_keys[kLocalKeys];
  extern __shared__ __align__(16) uint8_t ring[];
  uint32_t* all_keys = reinterpret_cast<uint32_t*>(ring);  // in the ring's place, once all scores are there
  __shared__ int last;
  const int b = blockIdx.z, h = blockIdx.y, split = blockIdx.x;
  const int64_t grp = (int64_t)b * g.H + h;
  int32_t* list = a.list + grp * a.budget;
  const int L = g.seq_len[b];
  int n = (int)(((int64_t)L + kG - 1) / kG);
  if (L < 0 || L > (int64_t)g.maxp * kG) {
    if (threadIdx.x == 0) set_status(g.status, KVQ_DEV_OVERFLOW);
    n = 0;
  }
  if (n <= a.budget) {  // every page
    if (split == 0) {
      for (int i = threadIdx.x; i < a.budget; i += kSelThreads) list[i] = i < n ? i : -1;
      if (threadIdx.x == 0) a.list_len[grp] = n;
    }
    return;
  }
  const int lo = a.sink, hi = n - a.recent, m = hi - lo, k = a.budget - a.sink - a.recent;
  const bool local = a.nsplit == 1 && m <= kLocalKeys;  // the keys never leave shared memory
  uint32_t* keys = local ? local_keys : a.keys + grp * g.maxp;
  if (k > 0) {
    const int per = (m + a.nsplit - 1) / a.nsplit;
    const int p0 = min(hi, lo + split * per), p1 = min(hi, p0 + per);
    if (p0 < p1) score_pages<BF16>(g, a.q, a.Gq, a.bounds, b, h, p0, p1, lo, keys, W, ring, a.minus_zero);
  }
  if (a.nsplit > 1) {
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
      last = arrive_last(a.counters, (int)grp, a.counter_sharing, a.nsplit);
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
  } else {
    __syncthreads();
  }
  const bool fits = !local && m <= kSelKeys;
  if (fits && k > 0) {
    for (int i = threadIdx.x; i < m; i += kSelThreads) all_keys[i] = __ldcg(keys + i);
    __syncthreads();
  }
  if (k > 0) {
    if (local || fits) take_largest<false>(local ? local_keys : all_keys, m, k, lo, list + a.sink, chooser);
    else take_largest<true>(keys, m, k, lo, list + a.sink, chooser);
  }
  for (int i = threadIdx.x; i < a.sink; i += kSelThreads) list[i] = i;
  for (int i = threadIdx.x; i < a.recent; i += kSelThreads) list[a.budget - a.recent + i] = hi + i;
  if (threadIdx.x == 0) a.list_len[grp] = a.budget;
}

}  // namespace

cudaError_t launch_page_bounds(const Geom& g, const void* k_new, int n_new, void* bounds, cudaStream_t st) {
  // pages a sequence's n_new tokens can touch, wherever its length stands in a page
  const int64_t pages = ((int64_t)n_new + 2 * kG - 2) / kG;
  const dim3 grid((unsigned)((pages * g.H + kBoundsWarps - 1) / kBoundsWarps), g.B);
  if (g.dtype == KVQ_BF16)
    page_bounds_kernel<true><<<grid, kBoundsWarps * 32, 0, st>>>(g, (const uint16_t*)k_new, n_new, (uint16_t*)bounds);
  else
    page_bounds_kernel<false><<<grid, kBoundsWarps * 32, 0, st>>>(g, (const uint16_t*)k_new, n_new, (uint16_t*)bounds);
  return cudaGetLastError();
}

// Arrival counters, then the keys.
size_t select_workspace(const Geom& g) { return kCounterBytes + (size_t)g.B * g.H * (size_t)g.maxp * sizeof(uint32_t); }

cudaError_t launch_select(const Geom& g, SelectArgs a, void* ws, int num_sms, cudaStream_t st) {
  const size_t groups = (size_t)g.B * g.H;
  a.minus_zero = -0.0f;
  a.counters = (unsigned*)ws;
  a.counter_sharing = counter_sharing((int64_t)groups);
  a.keys = (uint32_t*)((uint8_t*)ws + kCounterBytes);
  // as many CTAs as the SMs hold at once, each with 32 pages (one round of its warps) or more
  const int64_t most = std::min<int64_t>(std::max(1, g.maxp / 32), most_arrivals(a.counter_sharing));
  a.nsplit = (int)std::min<int64_t>(most, std::max<int64_t>(1, kSelCtas * (int64_t)num_sms / (int64_t)groups));
  const dim3 grid(a.nsplit, g.H, g.B);
  auto* kernel = g.dtype == KVQ_BF16 ? select_pages_kernel<true> : select_pages_kernel<false>;
  // the kernel's shared-memory limit is raised once per device
  static std::atomic<bool> raised[2][64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int bf = g.dtype == KVQ_BF16;
  if (dev < 0 || dev >= 64 || !raised[bf][dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelRing);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) raised[bf][dev].store(true, std::memory_order_relaxed);
  }
  kernel<<<grid, kSelThreads, kSelRing, st>>>(g, a);
  return cudaGetLastError();
}

}  // namespace kvq
