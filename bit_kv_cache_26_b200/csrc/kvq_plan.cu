// Page tables, slot map and positions of a batch from its request lengths, on the GPU.
//
// Sequence b holds L_b tokens and gets n_b more: it needs ceil((L_b + n_b)/32) - ceil(L_b/32)
// new pages.  Two exclusive scans over the sequences (tokens, pages) give every token its place
// in the packed order and every new page its place on the free stack, whose top is taken first.
// A sequence is served when the scans up to and including it stay within the slot map and the
// stack; both scans only grow, so the served ones are those before the first that does not fit.
#include "kvq_common.cuh"
#include "kvq_internal.h"

namespace kvq {

namespace {

constexpr int kPlanScan = 1024;       // threads of the scan
constexpr int kPlanThreads = 256;     // threads of an expanding CTA
constexpr int kPlanChunk = 4096;      // tokens of an expanding CTA
constexpr int64_t kPlanOneCta = 4096; // up to so many tokens the scanning CTA expands them itself

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

// Packed tokens [begin, end) of the plan, four consecutive ones per thread and round.
__device__ void expand(const Geom& g, const PlanArgs& a, int begin, int end, int s_lo, int s_hi, int free_n, int tid,
                       int nthreads) {
  const int32_t* before = a.ws + 4;  // new pages of the sequences before
  for (int i0 = begin + 4 * tid; i0 < end; i0 += 4 * nthreads) {
    int s = seq_of(a.cu, i0, s_lo, s_hi), base = -1, next = -1, L = 0, held = 0, page = -1, phys = 0;
    int pos[4], ids[4];
    int64_t slot[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = i0 + e;
      if (i < end) {
        if (i >= next) {
          if (next >= 0) ++s;
          while (a.cu[s + 1] <= i) ++s;  // sequences without new tokens
          base = a.cu[s];
          next = a.cu[s + 1];
          L = g.seq_len[s];
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
        slot[e] = (int64_t)phys * kG + pos[e] % kG;
        if (pos[e] % kG == 0) const_cast<int32_t*>(g.page_table)[(int64_t)s * g.maxp + p] = phys;
      }
    }
    if (i0 + 4 <= end) {
      *reinterpret_cast<int4*>(a.positions + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      *reinterpret_cast<int4*>(a.seq_ids + i0) = make_int4(ids[0], ids[1], ids[2], ids[3]);
      *reinterpret_cast<longlong2*>(a.slot_map + i0) = make_longlong2(slot[0], slot[1]);
      *reinterpret_cast<longlong2*>(a.slot_map + i0 + 2) = make_longlong2(slot[2], slot[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i0 + e < end) {
          a.positions[i0 + e] = pos[e];
          a.seq_ids[i0 + e] = ids[e];
          a.slot_map[i0 + e] = slot[e];
        }
    }
  }
}

// One CTA: the scans, cu_new, the pages before each sequence (workspace) and the free count left;
// with EXPAND it then writes the tokens too.  Workspace: [0] free ids at the start, [1] tokens of the plan,
// [4 + b] new pages of the sequences before b.
template <bool EXPAND>
__global__ void __launch_bounds__(kPlanScan) plan_scan_kernel(Geom g, PlanArgs a) {
  __shared__ longlong2 warp_tot[32];
  __shared__ longlong2 s_tot;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  if constexpr (!EXPAND) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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
      a.ws[4 + b] = (int32_t)(upto.y - mine.y);
    } else if (mine.x > 0) {
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
    a.ws[4 + b] = (int32_t)tot.y;
  }
  if (tid == 0) {
    a.cu[0] = 0;
    a.ws[0] = (int32_t)free_n;
    a.ws[1] = (int32_t)tot.x;
    *a.free_left = (int32_t)(free_n - tot.y);
  }
  if constexpr (EXPAND) {
    __syncthreads();
    expand(g, a, 0, (int)tot.x, 0, g.B - 1, (int)free_n, tid, blockDim.x);
  }
}

__global__ void __launch_bounds__(kPlanThreads) plan_expand_kernel(Geom g, PlanArgs a) {
  __shared__ int s_range[2];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int total = a.ws[1], begin = blockIdx.x * kPlanChunk;
  if (begin >= total) return;
  const int end = min(total, begin + kPlanChunk);
  if (threadIdx.x < 2) {  // the sequences of the chunk's first and last token
    const int i = threadIdx.x ? end - 1 : begin;
    s_range[threadIdx.x] = seq_of(a.cu, i, 0, g.B - 1);
  }
  __syncthreads();
  expand(g, a, begin, end, s_range[0], s_range[1], a.ws[0], threadIdx.x, kPlanThreads);
}

}  // namespace

size_t plan_workspace(const Geom& g) { return ((size_t)g.B + 4) * sizeof(int32_t); }

// Few tokens (a decode step): one launch.  Else the scan, and an expansion whose launch overlaps it.
cudaError_t launch_plan(const Geom& g, const PlanArgs& a, cudaStream_t st) {
  if (a.max_tokens <= kPlanOneCta) {
    plan_scan_kernel<true><<<1, kPlanScan, 0, st>>>(g, a);
    return cudaGetLastError();
  }
  plan_scan_kernel<false><<<1, kPlanScan, 0, st>>>(g, a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((a.max_tokens + kPlanChunk - 1) / kPlanChunk));
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = st;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, plan_expand_kernel, g, a);
}

}  // namespace kvq
