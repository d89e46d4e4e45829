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
#include <algorithm>

#include "kvq_common.cuh"
#include "kvq_internal.h"

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

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelKeys = 16;        // keys a thread keeps in registers: up to 8192 pages
constexpr int kSelAhead = 4;        // pages in flight per 16 lanes

// fp32 -> unsigned with the same order; -0 is +0, NaN above all.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t u = __float_as_uint(__fadd_rn(x, 0.0f));
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ unsigned long long mulp(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long addp(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long packf(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
template <bool BF16>
__device__ __forceinline__ unsigned long long widen(uint32_t u) {
  if constexpr (BF16) return packf(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u));
  return packf(f.x, f.y);
}

// Block-wide sum of one value per thread; `buf` alternates between two halves so that one barrier
// per sum is enough.
__device__ __forceinline__ unsigned block_sum(unsigned v, unsigned (*buf)[kSelWarps], int& turn) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = __reduce_add_sync(kFull, v);
  if (lane == 0) buf[turn][warp] = v;
  __syncthreads();
  unsigned s = lane < kSelWarps ? buf[turn][lane] : 0u;
  turn ^= 1;
  return __reduce_add_sync(kFull, s);
}

// Exclusive block-wide prefix of one value per thread (two barriers).
__device__ __forceinline__ unsigned long long block_prefix(unsigned long long v, unsigned long long* buf) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long t = __shfl_up_sync(kFull, inc, o);
    if (lane >= o) inc += t;
  }
  __syncthreads();
  if (lane == 31) buf[warp] = inc;
  __syncthreads();
  unsigned long long before = 0;
  for (int w = 0; w < warp; ++w) before += buf[w];
  return before + inc - v;
}

// Scores of pages [p0, p1) of (b, h) as ordered keys: 16 lanes per page, 8 channels per lane.
template <bool BF16>
__device__ void score_pages(const Geom& g, const uint16_t* __restrict__ q, int Gq, const uint16_t* __restrict__ bounds, int b,
                            int h, int p0, int p1, uint32_t* keys, float* W) {
  const int lane = threadIdx.x & 31, c = lane & 15;
  if (threadIdx.x < 2 * kD) {  // W+ and W-
    const int d = threadIdx.x & (kD - 1);
    const bool neg = threadIdx.x >= kD;
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float x = 0.f;
      if (i < Gq) {
        x = load_elem(q + ((int64_t)b * g.H * Gq + (int64_t)h * Gq + i) * kD + d, g.dtype);
        x = x != x ? x : neg ? fminf(x, 0.f) : fmaxf(x, 0.f);
      }
      v[i] = x;
    }
#pragma unroll
    for (int o = 8; o; o >>= 1)
#pragma unroll
      for (int i = 0; i < o; ++i) v[i] = __fadd_rn(v[i], v[i + o]);
    W[threadIdx.x] = v[0];
  }
  __syncthreads();
  unsigned long long up[4], dn[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    up[e] = packf(W[8 * c + 2 * e], W[8 * c + 2 * e + 1]);
    dn[e] = packf(W[kD + 8 * c + 2 * e], W[kD + 8 * c + 2 * e + 1]);
  }
  const int32_t* table = g.page_table + (int64_t)b * g.maxp;
  const int hw = threadIdx.x >> 4;
  for (int q0 = p0 + (hw & ~1); q0 < p1; q0 += 2 * kSelWarps * kSelAhead) {
    uint4 lo[kSelAhead], hi[kSelAhead];
    int phys[kSelAhead];
#pragma unroll
    for (int i = 0; i < kSelAhead; ++i) {
      const int p = q0 + (hw & 1) + i * 2 * kSelWarps;
      phys[i] = p < p1 ? table[p] : -1;
      if (p < p1 && (phys[i] < 0 || phys[i] >= g.npages)) {
        set_status(g.status, KVQ_DEV_BAD_PAGE);
        phys[i] = -1;
      }
    }
#pragma unroll
    for (int i = 0; i < kSelAhead; ++i) {
      lo[i] = hi[i] = make_uint4(0u, 0u, 0u, 0u);
      if (phys[i] >= 0) {
        const uint16_t* src = bounds + ((int64_t)phys[i] * g.H + h) * 2 * kD + 8 * c;
        lo[i] = __ldg(reinterpret_cast<const uint4*>(src));
        hi[i] = __ldg(reinterpret_cast<const uint4*>(src + kD));
      }
    }
#pragma unroll
    for (int i = 0; i < kSelAhead; ++i) {
      const uint32_t* l = &lo[i].x;
      const uint32_t* u = &hi[i].x;
      unsigned long long t[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) t[e] = addp(mulp(up[e], widen<BF16>(u[e])), mulp(dn[e], widen<BF16>(l[e])));
      const unsigned long long s = addp(addp(t[0], t[2]), addp(t[1], t[3]));
      float a, bb;
      asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(bb) : "l"(s));
      float x = __fadd_rn(a, bb);
#pragma unroll
      for (int o = 8; o; o >>= 1) x = __fadd_rn(x, __shfl_xor_sync(kFull, x, o));
      const int p = q0 + (hw & 1) + i * 2 * kSelWarps;
      if (c == 0 && p < p1) keys[p] = phys[i] >= 0 ? order_key(x) : 0u;
    }
  }
}

// The k largest of keys[p0 .. p1) (ties: the lower index), in index order, to list[0 .. k).
// Thread t looks after a run of consecutive keys; up to kSelKeys of them sit in registers.  The
// k-th largest key is found bit by bit: 32 counts over the block.
__device__ void take_largest(const uint32_t* keys, int p0, int p1, int k, int32_t* list, unsigned (*buf)[kSelWarps],
                             unsigned long long* buf2) {
  const int n = p1 - p0, per = (n + kSelThreads - 1) / kSelThreads;
  const int a0 = p0 + min(n, (int)threadIdx.x * per), a1 = min(p1, a0 + per);
  const bool regs = per <= kSelKeys;
  uint32_t key[kSelKeys];
  if (regs) {
#pragma unroll
    for (int i = 0; i < kSelKeys; ++i) key[i] = a0 + i < a1 ? __ldcg(keys + a0 + i) : 0u;
  }
  uint32_t T = 0;
  int turn = 0;
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t cand = T | (1u << bit);
    unsigned cnt = 0;
    if (regs) {
#pragma unroll
      for (int i = 0; i < kSelKeys; ++i) cnt += key[i] >= cand;
    } else {
      for (int i = a0; i < a1; ++i) cnt += __ldcg(keys + i) >= cand;
    }
    if (block_sum(cnt, buf, turn) >= (unsigned)k) T = cand;
  }
  // how many above the k-th, how many equal to it (T = 0 when fewer than k keys exceed 0: all equal it)
  unsigned gt = 0, eq = 0;
  for (int i = a0; i < a1; ++i) {
    const uint32_t x = __ldcg(keys + i);
    gt += x > T;
    eq += x == T;
  }
  const unsigned above = block_sum(gt, buf, turn);
  const unsigned ties = k - above;
  const unsigned long long before = block_prefix((unsigned long long)gt << 32 | eq, buf2);
  const unsigned eq0 = (unsigned)before;
  unsigned out = (unsigned)(before >> 32) + min(eq0, ties), e = eq0;
  for (int i = a0; i < a1; ++i) {
    const uint32_t x = __ldcg(keys + i);
    const bool tie = x == T;
    if (x > T || (tie && e < ties)) list[out++] = i;
    e += tie;
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kSelThreads) select_pages_kernel(Geom g, SelectArgs a) {
  __shared__ float W[2 * kD];
  __shared__ unsigned buf[2][kSelWarps];
  __shared__ unsigned long long buf2[kSelWarps];
  __shared__ int last;
  const int b = blockIdx.z, h = blockIdx.y, split = blockIdx.x;
  const int64_t grp = (int64_t)b * g.H + h;
  int32_t* list = a.list + grp * a.budget;
  const int L = g.seq_len[b];
  int n = (L + kG - 1) / kG;
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
  const int lo = a.sink, hi = n - a.recent, m = hi - lo;
  const int per = (m + a.nsplit - 1) / a.nsplit;
  const int p0 = min(hi, lo + split * per), p1 = min(hi, p0 + per);
  uint32_t* keys = a.keys + grp * g.maxp;
  if (p0 < p1) score_pages<BF16>(g, a.q, a.Gq, a.bounds, b, h, p0, p1, keys, W);
  if (a.nsplit > 1) {
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
      last = atomicAdd(a.arrivals + grp, 1) == a.nsplit - 1;
      if (last) a.arrivals[grp] = 0;  // ready for the next call
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
  } else {
    __syncthreads();
  }
  for (int i = threadIdx.x; i < a.sink; i += kSelThreads) list[i] = i;
  for (int i = threadIdx.x; i < a.recent; i += kSelThreads) list[a.budget - a.recent + i] = hi + i;
  const int k = a.budget - a.sink - a.recent;
  if (k > 0) take_largest(keys, lo, hi, k, list + a.sink, buf, buf2);
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

// Arrival counters (first, so that their place does not depend on anything but the cache), then the keys.
size_t select_workspace(const Geom& g) {
  const size_t groups = (size_t)g.B * g.H;
  return (groups * sizeof(int) + 255) / 256 * 256 + groups * (size_t)g.maxp * sizeof(uint32_t);
}

cudaError_t launch_select(const Geom& g, SelectArgs a, void* ws, int num_sms, cudaStream_t st) {
  const size_t groups = (size_t)g.B * g.H;
  a.arrivals = (int*)ws;
  a.keys = (uint32_t*)((uint8_t*)ws + (groups * sizeof(int) + 255) / 256 * 256);
  // two CTAs per SM, each with 64 pages or more
  const int64_t most = std::max(1, g.maxp / 64);
  a.nsplit = (int)std::min<int64_t>(most, std::max<int64_t>(1, 2 * (int64_t)num_sms / (int64_t)groups));
  const dim3 grid(a.nsplit, g.H, g.B);
  if (g.dtype == KVQ_BF16) select_pages_kernel<true><<<grid, kSelThreads, 0, st>>>(g, a);
  else select_pages_kernel<false><<<grid, kSelThreads, 0, st>>>(g, a);
  return cudaGetLastError();
}

}  // namespace kvq
