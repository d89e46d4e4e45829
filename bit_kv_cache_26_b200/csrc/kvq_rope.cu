// Rows of queries, keys and values as the cache wants them, from one packed projection in one
// pass: per-head RMS norm of queries and keys, the position rotation of both (the cache's
// patterns are mined on, and its append takes, post-rotation keys: "PatternKV", Section 4.1),
// and the values copied into contiguous rows.
//
//   y_d = x_d / sqrt(mean_d x_d^2 + eps) * w_d                       (no weight: y = x)
//   a_i = pos * inv_freq_i,  (u, v) = channels (i, i + rot/2), or (2i, 2i + 1) when interleaved:
//   u' = u cos a - v sin a,  v' = v cos a + u sin a;  channels >= rot pass through.
//
// Bound: HBM, one read and one write of every row.  One B200, 262144 tokens x 48 rows of bf16: 1044-1085
// us, 5.9-6.2 TB/s (0.90-0.94 of the copy bandwidth).  A row over 16 lanes with four rows in flight
// took 1557 us: its shuffles, addresses and angle reads cost more instructions than the rows' bytes
// allow; two rows or more in flight per warp take registers from the warps that hide the latency.
//
// Everything between the load and the store is fp32 with one rounding at the end.  The angle
// is formed in float64 as turns (pos * inv_freq / 2 pi, minus its integer part), so far
// positions keep their phase; the sine and cosine of the remainder are fp32.
#include <algorithm>

#include "kvq_common.cuh"
#include "kvq_internal.h"
#include "kvq_pipe.cuh"

namespace kvq {

namespace {

constexpr int kRopeWarps = 4;

template <bool BF16>
__device__ __forceinline__ unsigned long long widen2(uint32_t u) {
  if constexpr (BF16) return pk(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u));
  return pk(f.x, f.y);
}
template <bool BF16>
__device__ __forceinline__ uint32_t narrow2(unsigned long long v) {
  float a, b;
  upk(v, a, b);
  if constexpr (BF16) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  const __half2 r = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// A warp takes one token and a run of its groups of four heads (queries, keys and values apart), a row over 8 lanes:
// two pieces of 8 channels per lane, so that a lane holds both channels of each of its pairs.  Lane c of the rotated
// part has pieces c and c + rot/16 (halves) or 2c and 2c + 1 (adjacent pairs); the lanes after it share the pieces
// that pass.  The token's sines and cosines are made once per warp, two per lane, and kept in registers over the heads.
template <bool BF16, bool INTER>
__global__ void __launch_bounds__(kRopeWarps * 32) norm_rope_kernel(RopeArgs a) {
  __shared__ __align__(16) float table[kRopeWarps][2][kD / 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane & 7, row = lane >> 3;
  const int64_t item = (int64_t)blockIdx.x * kRopeWarps + warp;
  const int64_t t = item / a.parts;
  if (t >= a.tokens) return;
  const int nq = (a.rows[0].heads + 3) / 4, nk = (a.rows[1].heads + 3) / 4, nv = (a.rows[2].heads + 3) / 4;
  const int part = (int)(item % a.parts), per = (nq + nk + nv + a.parts - 1) / a.parts;
  const int g0 = part * per, g1 = min(nq + nk + nv, g0 + per);
  const int rl = a.rot / 16;  // lanes of the rotated part
  const bool turns = c < rl;
  const int pA = INTER ? 2 * c : turns ? c : 2 * rl + 2 * (c - rl);
  const int pB = INTER ? pA + 1 : turns ? c + rl : pA + 1;

  // the rows of group grp: this lane's two pieces, and where they go (null: no such head)
  auto load = [&](int grp, uint4& xA, uint4& xB) -> uint16_t* {
    const int set = grp < nq ? 0 : grp < nq + nk ? 1 : 2;
    const RopeRows& R = a.rows[set];
    const int h = 4 * (grp - (set == 0 ? 0 : set == 1 ? nq : nq + nk)) + row;
    xA = xB = make_uint4(0u, 0u, 0u, 0u);
    if (grp >= g1 || h >= R.heads) return nullptr;
    const uint16_t* src = (const uint16_t*)R.in + t * R.in_tok + h * R.in_head;
    xA = *reinterpret_cast<const uint4*>(src + 8 * pA);
    xB = *reinterpret_cast<const uint4*>(src + 8 * pB);
    return (uint16_t*)R.out + t * R.out_tok + h * R.out_head;
  };
  uint4 xA, xB;
  uint16_t* dst = load(g0, xA, xB);

  unsigned long long co[4], si[4];  // of this lane's eight pairs
  if (a.rot && g0 < nq + nk) {
    const double pos = (double)a.pos[t];
    for (int f = lane; f < a.rot / 2; f += 32) {
      const double turn = pos * (double)a.inv_freq[f] * 0.15915494309189533577;
      float s, k;
      sincospif(2.0f * (float)(turn - rint(turn)), &s, &k);
      table[warp][0][f] = k;
      table[warp][1][f] = s;
    }
    __syncwarp();
    if (turns) {
      const ulonglong2* tc = reinterpret_cast<const ulonglong2*>(&table[warp][0][8 * c]);
      const ulonglong2* ts = reinterpret_cast<const ulonglong2*>(&table[warp][1][8 * c]);
      co[0] = tc[0].x; co[1] = tc[0].y; co[2] = tc[1].x; co[3] = tc[1].y;
      si[0] = ts[0].x; si[1] = ts[0].y; si[2] = ts[1].x; si[3] = ts[1].y;
    }
  }

  for (int grp = g0; grp < g1; ++grp) {
    if (grp > g0) dst = load(grp, xA, xB);
    if (grp < nq + nk) {  // the same for the whole warp
      const void* weight = grp < nq ? a.rows[0].weight : a.rows[1].weight;
      unsigned long long y[8];  // 16 channels: piece A, then piece B
      y[0] = widen2<BF16>(xA.x); y[1] = widen2<BF16>(xA.y); y[2] = widen2<BF16>(xA.z); y[3] = widen2<BF16>(xA.w);
      y[4] = widen2<BF16>(xB.x); y[5] = widen2<BF16>(xB.y); y[6] = widen2<BF16>(xB.z); y[7] = widen2<BF16>(xB.w);
      if (weight) {
        unsigned long long ss2 = mul2(y[0], y[0]);
#pragma unroll
        for (int e = 1; e < 8; ++e) ss2 = fma2(y[e], y[e], ss2);
        float s0, s1;
        upk(ss2, s0, s1);
        float ss = s0 + s1;
        ss += __shfl_xor_sync(kFull, ss, 4);
        ss += __shfl_xor_sync(kFull, ss, 2);
        ss += __shfl_xor_sync(kFull, ss, 1);
        const float inv = rsqrtf(fmaf(ss, 1.0f / kD, a.eps));
        const unsigned long long inv2 = pk(inv, inv);
        const uint4 wA = __ldg(reinterpret_cast<const uint4*>((const uint16_t*)weight + 8 * pA));
        const uint4 wB = __ldg(reinterpret_cast<const uint4*>((const uint16_t*)weight + 8 * pB));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[e] = mul2(mul2(y[e], inv2), widen2<BF16>((&wA.x)[e]));
          y[e + 4] = mul2(mul2(y[e + 4], inv2), widen2<BF16>((&wB.x)[e]));
        }
      }
      if (turns) {
        if constexpr (INTER) {  // (u, v) sits in one pair: pair p turns by angle p
#pragma unroll
          for (int p = 0; p < 8; ++p) {
            float u, v, c0, c1, s0, s1;
            upk(y[p], u, v);
            upk(co[p / 2], c0, c1);
            upk(si[p / 2], s0, s1);
            const float cc = p & 1 ? c1 : c0, s = p & 1 ? s1 : s0;
            y[p] = fma2(pk(u, v), pk(cc, cc), mul2(pk(v, u), pk(-s, s)));
          }
        } else {
          const unsigned long long minus = pk(-1.0f, -1.0f);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const unsigned long long u = y[e], v = y[e + 4];
            y[e] = fma2(u, co[e], mul2(mul2(v, si[e]), minus));
            y[e + 4] = fma2(v, co[e], mul2(u, si[e]));
          }
        }
      }
      xA = make_uint4(narrow2<BF16>(y[0]), narrow2<BF16>(y[1]), narrow2<BF16>(y[2]), narrow2<BF16>(y[3]));
      xB = make_uint4(narrow2<BF16>(y[4]), narrow2<BF16>(y[5]), narrow2<BF16>(y[6]), narrow2<BF16>(y[7]));
    }
    if (dst) {
      *reinterpret_cast<uint4*>(dst + 8 * pA) = xA;
      *reinterpret_cast<uint4*>(dst + 8 * pB) = xB;
    }
  }
}

}  // namespace

cudaError_t launch_norm_rope(const RopeArgs& a0, int dtype, bool interleaved, int num_sms, cudaStream_t st) {
  RopeArgs a = a0;
  // With many tokens a warp takes all groups of its token; with few, the groups are dealt to more
  // warps (each makes the token's angles again), down to one group each.
  const int64_t groups = (a.rows[0].heads + 3) / 4 + (a.rows[1].heads + 3) / 4 + (a.rows[2].heads + 3) / 4;
  const int64_t warps = (int64_t)num_sms * 32;
  a.parts = (int)std::min(groups, std::max<int64_t>(1, warps / a.tokens));
  // One to three waves of warps, the last less than half full: halves even it out, where the angles made twice are little
  // beside the rows.  12 groups a token (4736 tokens a wave), whole and in halves: 4800 tokens 31 and 28 us, 6500 35 and 32,
  // 9600 49 and 47; with the last wave fuller, 7300 37 and 38, 12000 55 and 56; past three waves no better (16000: 72 and 72).
  // 6 groups: 4800 tokens 17.6 and 16.0 us, 6900 20.4 and 19.9, 8191 22 and 23; 3 groups: slower everywhere.
  if (a.parts == 1 && groups >= 6 && a.tokens < 3 * warps && a.tokens % warps > 0 && 2 * (a.tokens % warps) < warps && a.tokens > warps)
    a.parts = 2;
  const int64_t grid = (a.tokens * a.parts + kRopeWarps - 1) / kRopeWarps;
  const bool bf = dtype == KVQ_BF16;
  auto* k = bf ? (interleaved ? norm_rope_kernel<true, true> : norm_rope_kernel<true, false>)
               : (interleaved ? norm_rope_kernel<false, true> : norm_rope_kernel<false, false>);
  k<<<(unsigned)grid, kRopeWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace kvq
