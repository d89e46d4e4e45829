// Page tables, slot map and positions of a batch from its request lengths, on the GPU.
//
// Sequence b holds L_b tokens and gets n_b more: it needs ceil((L_b + n_b)/32) - ceil(L_b/32)
// new pages.  Two exclusive scans over the sequences (tokens, pages) give every token its place
// in the packed order and every new page its place on the free stack, whose top is taken first.
// A sequence is served when the scans up to and including it stay within the slot map and the
// stack; both scans only grow, so the served ones are those before the first that does not fit.
//
// Bound: latency for a decode step (256 sequences of one token: 4.6-5.0 us on one B200); for prompts 16 bytes
// written per token, after latency (256 of up to 16384 tokens, 51 MB in all: 16.0-16.4 us, 3.2 TB/s, half of the
// copy bandwidth): every CTA scans the requests before its first store and starts each chunk of 1024 tokens with
// two barriers, a search and the loads of its page ids.  Two launches, the scan and the expansion, took 17 us there
// and 7.2 us for the decode step.
#include <algorithm>

#include "kvq_common.cuh"
#include "kvq_internal.h"
#include "kvq_pipe.cuh"

namespace kvq {

namespace {

constexpr int kPlanThreads = 256;
constexpr int kPlanOnce = 2048;       // up to so many sequences every CTA makes the scans for itself: one launch
constexpr int kOnceCtas = 4;          // CTAs per SM then, at most
constexpr int kPlanAhead = 2;         // rounds of a chunk (two tokens per thread each)
constexpr int kPlanScan = 1024;       // threads of the scan when it is a launch of its own
constexpr int kPlanData = kCounterBytes / 4;  // words of the workspace before the scan's results

__device__ __forceinline__ longlong2 add2ll(longlong2 a, longlong2 b) { return make_longlong2(a.x + b.x, a.y + b.y); }

// The request of one sequence: (new tokens, new pages); flags and drops what is out of range.
__device__ __forceinline__ longlong2 request(const Geom& g, const PlanArgs& a, int b, bool& bad) {
  const int64_t L = g.seq_len[b], n = a.new_len[b];
  bad = L < 0 || n < 0 || L + n > (int64_t)g.maxp * kG;
  if (bad) return make_longlong2(0, 0);
  return make_longlong2(n, (L + n + kG - 1) / kG - (L + kG - 1) / kG);
}

__device__ __forceinline__ longlong2 warp_scan(longlong2 v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(kFull, v.x, o), y = __shfl_up_sync(kFull, v.y, o);
    if (lane >= o) v = add2ll(v, make_longlong2(x, y));
  }
  return v;
}

// The sequence of packed token i: the last s of [lo, hi] with cu[s] <= i (it has tokens).
__device__ __forceinline__ int seq_of(const int32_t* cu, int i, int lo, int hi) {
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= i) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Slot of position pos in page phys; an invalid page id, from the table or the stack, has none (-1) and is noted in `bad`.
__device__ __forceinline__ int64_t slot_of(const Geom& g, int phys, int pos, bool& bad) {
  const bool ok = (unsigned)phys < (unsigned)g.npages;
  bad = bad || !ok;
  return ok ? (int64_t)phys * kG + pos % kG : -1;
}

// Packed tokens [begin, end) of the plan, two consecutive ones per thread and round (a warp's stores are whole sectors).  cu, before (new pages of the
// sequences before) and len: in shared or global memory.
__device__ __forceinline__ void expand(const Geom& g, const PlanArgs& a, const int32_t* cu, const int32_t* before,
                                       const int32_t* len, int begin, int end, int s_lo, int s_hi, int free_n) {
  bool bad = false;
  if (s_lo == s_hi && end - begin == 2 * kPlanThreads * kPlanAhead) {
    // the whole chunk in one sequence, as in a long prompt: the page ids of all rounds first, then the stores
    const int s = s_lo, L = len[s], held = (L + kG - 1) / kG, top = free_n - 1 - (before[s] - held);
    const int pos0 = L + (begin - cu[s]) + 2 * (int)threadIdx.x;
    int32_t* row = const_cast<int32_t*>(g.page_table) + (int64_t)s * g.maxp;
    auto page_id = [&](int pos) {
      const int p = pos / kG;
      return p < held ? row[p] : a.free_pages[top - p];
    };
    int id0[kPlanAhead], id1[kPlanAhead];
#pragma unroll
    for (int u = 0; u < kPlanAhead; ++u) {
      const int pos = pos0 + 2 * kPlanThreads * u;
      id0[u] = page_id(pos);
      id1[u] = (pos + 1) % kG == 0 ? page_id(pos + 1) : id0[u];
    }
#pragma unroll
    for (int u = 0; u < kPlanAhead; ++u) {
      const int pos = pos0 + 2 * kPlanThreads * u, i0 = begin + 2 * (int)threadIdx.x + 2 * kPlanThreads * u;
      *reinterpret_cast<int2*>(a.positions + i0) = make_int2(pos, pos + 1);
      *reinterpret_cast<int2*>(a.seq_ids + i0) = make_int2(s, s);
      *reinterpret_cast<longlong2*>(a.slot_map + i0) = make_longlong2(slot_of(g, id0[u], pos, bad), slot_of(g, id1[u], pos + 1, bad));
      if (pos % kG == 0) row[pos / kG] = id0[u];
      if ((pos + 1) % kG == 0) row[(pos + 1) / kG] = id1[u];
    }
    if (bad) set_status(g.status, KVQ_DEV_BAD_PAGE);
    return;
  }
  for (int i0 = begin + 2 * (int)threadIdx.x; i0 < end; i0 += 2 * kPlanThreads) {
    int s = seq_of(cu, i0, s_lo, s_hi), base = -1, next = -1, L = 0, held = 0, page = -1, phys = 0;
    int pos[2], ids[2];
    int64_t slot[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = i0 + e;
      if (i < end) {
        if (i >= next) {
          while (cu[s + 1] <= i) ++s;  // the next sequence with new tokens
          base = cu[s];
          next = cu[s + 1];
          L = len[s];
          held = (L + kG - 1) / kG;
          page = -1;
        }
        pos[e] = L + (i - base);
        ids[e] = s;
        const int p = pos[e] / kG;
        if (p != page) {
          page = p;
          phys = p < held ? g.page_table[(int64_t)s * g.maxp + p] : a.free_pages[free_n - 1 - (before[s] + p - held)];
        }
        slot[e] = slot_of(g, phys, pos[e], bad);
        if (pos[e] % kG == 0) const_cast<int32_t*>(g.page_table)[(int64_t)s * g.maxp + p] = phys;
      }
    }
    if (i0 + 2 <= end) {
      *reinterpret_cast<int2*>(a.positions + i0) = make_int2(pos[0], pos[1]);
      *reinterpret_cast<int2*>(a.seq_ids + i0) = make_int2(ids[0], ids[1]);
      *reinterpret_cast<longlong2*>(a.slot_map + i0) = make_longlong2(slot[0], slot[1]);
    } else {
      a.positions[i0] = pos[0];
      a.seq_ids[i0] = ids[0];
      a.slot_map[i0] = slot[0];
    }
  }
  if (bad) set_status(g.status, KVQ_DEV_BAD_PAGE);
}

// One launch: every CTA scans all requests (consecutive ones per thread) into shared memory and writes its chunk of
// the tokens; the first also writes cu_new, and the last one to have read the free count writes what is left of it
// (which may be the same word).  Workspace: [0] counts the CTAs that have read it, back to 0 at the end.
template <int ITEMS>  // requests per thread, at most
__global__ void __launch_bounds__(kPlanThreads) plan_once_kernel(Geom g, PlanArgs a, int chunk) {
  __shared__ int32_t cu[kPlanThreads * ITEMS + 1], before[kPlanThreads * ITEMS], len[kPlanThreads * ITEMS];
  __shared__ longlong2 warp_tot[kPlanThreads / 32];
  __shared__ longlong2 s_tot;
  __shared__ int s_free, s_last, s_range[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    s_free = max(0, min(*reinterpret_cast<const volatile int32_t*>(a.free_count), a.free_cap));
    s_tot = make_longlong2(0, 0);
    __threadfence();
    s_last = atomicInc(reinterpret_cast<unsigned*>(a.ws), gridDim.x - 1) == gridDim.x - 1;
  }
  const int items = (g.B + kPlanThreads - 1) / kPlanThreads, b0 = tid * items;
  longlong2 mine[ITEMS], sum = make_longlong2(0, 0);
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    mine[i] = make_longlong2(0, 0);
    const int b = b0 + i;
    if (i < items && b < g.B) {
      bool bad;
      mine[i] = request(g, a, b, bad);
      len[b] = g.seq_len[b];
      if (bad && blockIdx.x == 0) set_status(g.status, KVQ_DEV_OVERFLOW);
    }
    sum = add2ll(sum, mine[i]);
  }
  longlong2 upto = warp_scan(sum, lane);
  if (lane == 31) warp_tot[warp] = upto;
  __syncthreads();
  const int64_t free_n = s_free;
  for (int w = 0; w < warp; ++w) upto = add2ll(upto, warp_tot[w]);
  longlong2 at = make_longlong2(upto.x - sum.x, upto.y - sum.y);  // before this thread's requests
  int n_mine = 0;  // served ones of them: the sums only grow, so the first
  longlong2 end = at;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int b = b0 + i;
    if (i < items && b < g.B) {
      const longlong2 next = add2ll(at, mine[i]);
      const bool served = next.x <= a.max_tokens && next.y <= free_n;
      if (served) {
        cu[b + 1] = (int32_t)next.x;
        before[b] = (int32_t)at.y;
        end = next;
        ++n_mine;
      } else if (at.x <= a.max_tokens && at.y <= free_n && blockIdx.x == 0) {  // the first that does not fit
        set_status(g.status, next.y > free_n ? KVQ_DEV_NO_PAGES : KVQ_DEV_OVERFLOW);
      }
      at = next;
    }
  }
  // the served requests are the first ones, so the last thread that has any knows the totals
  const int with_any = __syncthreads_count(n_mine > 0);
  if (tid == with_any - 1) s_tot = end;
  __syncthreads();
  const longlong2 tot = s_tot;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int b = b0 + i;
    if (i < items && b < g.B && i >= n_mine) {
      cu[b + 1] = (int32_t)tot.x;
      before[b] = (int32_t)tot.y;
    }
  }
  if (tid == 0) cu[0] = 0;
  __syncthreads();
  if (blockIdx.x == 0)
    for (int b = tid; b <= g.B; b += kPlanThreads) a.cu[b] = cu[b];
  if (tid == 0 && s_last) *a.free_left = (int32_t)(free_n - tot.y);
  for (int64_t begin = (int64_t)blockIdx.x * chunk; begin < tot.x; begin += (int64_t)gridDim.x * chunk) {
    const int last = (int)min(tot.x, (long long)(begin + chunk));
    __syncthreads();  // the range of the chunk before is read
    if (tid < 2) s_range[tid] = seq_of(cu, tid ? last - 1 : (int)begin, 0, g.B - 1);  // the chunk's sequences
    __syncthreads();
    expand(g, a, cu, before, len, (int)begin, last, s_range[0], s_range[1], (int)free_n);
  }
}

// More sequences, two launches: one CTA makes the scans, cu_new, the pages before each sequence (workspace) and the free
// count left; then the tokens.  Workspace, past the counters: [0] free ids at the start, [1] tokens of the plan, [2 + b] new
// pages before b.
__global__ void __launch_bounds__(kPlanScan) plan_scan_kernel(Geom g, PlanArgs a) {
  __shared__ longlong2 warp_tot[32];
  __shared__ longlong2 s_tot;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t free_n = max(0, min(*a.free_count, a.free_cap));
  longlong2 carry = make_longlong2(0, 0);  // sums of the rounds before
  int n_served = 0;
  if (tid == 0) s_tot = carry;
  for (int b0 = 0; b0 < g.B; b0 += blockDim.x) {
    const int b = b0 + tid;
    bool bad = false;
    const longlong2 mine = b < g.B ? request(g, a, b, bad) : make_longlong2(0, 0);
    if (bad) set_status(g.status, KVQ_DEV_OVERFLOW);
    const longlong2 in_warp = warp_scan(mine, lane);
    if (lane == 31) warp_tot[warp] = in_warp;
    __syncthreads();
    if (warp == 0) warp_tot[lane] = warp_scan(lane < nw ? warp_tot[lane] : make_longlong2(0, 0), lane);
    __syncthreads();
    longlong2 upto = add2ll(in_warp, carry);
    if (warp > 0) upto = add2ll(upto, warp_tot[warp - 1]);
    const bool served = b < g.B && upto.x <= a.max_tokens && upto.y <= free_n;
    if (served) {
      a.cu[b + 1] = (int32_t)upto.x;
      a.ws[kPlanData + 2 + b] = (int32_t)(upto.y - mine.y);
    } else if (b < g.B && upto.x - mine.x <= a.max_tokens && upto.y - mine.y <= free_n) {  // the first that does not fit
      set_status(g.status, upto.y > free_n ? KVQ_DEV_NO_PAGES : KVQ_DEV_OVERFLOW);
    }
    carry = add2ll(carry, warp_tot[nw - 1]);
    const int n = __syncthreads_count(served);  // the sums only grow: the first n of this round
    if (n > 0 && tid == n - 1) s_tot = upto;
    n_served += n;
  }
  __syncthreads();
  const longlong2 tot = s_tot;
  for (int b = n_served + tid; b < g.B; b += blockDim.x) {
    a.cu[b + 1] = (int32_t)tot.x;
    a.ws[kPlanData + 2 + b] = (int32_t)tot.y;
  }
  if (tid == 0) {
    a.cu[0] = 0;
    a.ws[kPlanData] = (int32_t)free_n;
    a.ws[kPlanData + 1] = (int32_t)tot.x;
    *a.free_left = (int32_t)(free_n - tot.y);
  }
}

__global__ void __launch_bounds__(kPlanThreads) plan_expand_kernel(Geom g, PlanArgs a, int chunk) {
  __shared__ int s_range[2];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int total = a.ws[kPlanData + 1];
  const int64_t begin = (int64_t)blockIdx.x * chunk;
  if (begin >= total) return;
  const int end = (int)min((int64_t)total, begin + chunk);
  if (threadIdx.x < 2)  // the sequences of the chunk's first and last token
    s_range[threadIdx.x] = seq_of(a.cu, threadIdx.x ? end - 1 : (int)begin, 0, g.B - 1);
  __syncthreads();
  expand(g, a, a.cu, a.ws + kPlanData + 2, g.seq_len, (int)begin, end, s_range[0], s_range[1], a.ws[kPlanData]);
}

}  // namespace

size_t plan_workspace(const Geom& g) { return ((size_t)g.B + 4 + (g.B > kPlanOnce ? kPlanData : 0)) * sizeof(int32_t); }

cudaError_t launch_plan(const Geom& g, const PlanArgs& a, int num_sms, cudaStream_t st) {
  constexpr int chunk = 2 * kPlanThreads * kPlanAhead;  // tokens of a CTA at a time
  const int64_t chunks = std::max<int64_t>(1, (a.max_tokens + chunk - 1) / chunk);
  if (g.B <= kPlanOnce) {
    // every CTA makes the scans first, so there are no more than kOnceCtas per SM
    const unsigned grid = (unsigned)std::min<int64_t>(chunks, (int64_t)kOnceCtas * num_sms);
    if (g.B <= kPlanThreads) plan_once_kernel<1><<<grid, kPlanThreads, 0, st>>>(g, a, chunk);
    else plan_once_kernel<kPlanOnce / kPlanThreads><<<grid, kPlanThreads, 0, st>>>(g, a, chunk);
    return cudaGetLastError();
  }
  plan_scan_kernel<<<1, std::min(kPlanScan, (g.B + 127) / 128 * 128), 0, st>>>(g, a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at{};  // the expansion's launch overlaps the scan
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)chunks);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = st;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, plan_expand_kernel, g, a, chunk);
}

}  // namespace kvq
