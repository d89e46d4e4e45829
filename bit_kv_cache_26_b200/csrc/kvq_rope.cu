// Rows of queries, keys and values as the cache wants them, from one packed projection in one
// pass: per-head RMS norm of queries and keys, the position rotation of both (the cache's
// patterns are mined on, and its append takes, post-rotation keys: "PatternKV", Section 4.1),
// and the values copied into contiguous rows.
//
//   y_d = x_d / sqrt(mean_d x_d^2 + eps) * w_d                       (no weight: y = x)
//   a_i = pos * inv_freq_i,  (u, v) = channels (i, i + rot/2), or (2i, 2i + 1) when interleaved:
//   u' = u cos a - v sin a,  v' = v cos a + u sin a;  channels >= rot pass through.
//
// Everything between the load and the store is fp32 with one rounding at the end.  The angle
// is formed in float64 as turns (pos * inv_freq / 2 pi, minus its integer part), so far
// positions keep their phase; the sine and cosine of the remainder are fp32.
#include "kvq_common.cuh"
#include "kvq_internal.h"

namespace kvq {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeRows = kRopeThreads / 16;  // a row of 128 channels is held by 16 lanes
constexpr int kRopeBatch = 4;                 // rows in flight per 16 lanes
constexpr int kRopeTile = 8;                  // most tokens of a CTA: they share one table of angles

template <bool BF16>
__device__ __forceinline__ float2 to_f2(uint32_t u) {
  if constexpr (BF16) return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
template <bool BF16>
__device__ __forceinline__ uint32_t from_f2(float a, float b) {
  if constexpr (BF16) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  const __half2 r = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// A row's 32 granules of 4 channels over 16 lanes, two each, so that a lane holds both channels of
// each of its pairs: lane c of the rotated part takes granules c and c + rot/8 (halves) or 2c and
// 2c + 1 (adjacent pairs); the lanes after it share the granules that pass.
template <bool BF16, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_kernel(RopeArgs a) {
  __shared__ __align__(16) float2 cs[kRopeTile][kD / 2];
  const int lane16 = threadIdx.x & 15, hw = threadIdx.x >> 4;
  const int64_t t0 = (int64_t)blockIdx.x * a.tile;
  const int tn = (int)min((int64_t)a.tile, a.tokens - t0);
  const int HT = a.rows[0].heads + a.rows[1].heads + a.rows[2].heads;
  const int nrows = tn * HT;
  const int pairs = a.rot / 2, rl = a.rot / 8;  // lanes of the rotated part
  const bool turns = lane16 < rl;
  const int gA = INTER ? 2 * lane16 : turns ? lane16 : 2 * rl + 2 * (lane16 - rl);
  const int gB = INTER ? gA + 1 : turns ? lane16 + rl : gA + 1;
  uint2 wq[2], wk[2];
  if (a.rows[0].weight) {
    wq[0] = *reinterpret_cast<const uint2*>((const uint16_t*)a.rows[0].weight + 4 * gA);
    wq[1] = *reinterpret_cast<const uint2*>((const uint16_t*)a.rows[0].weight + 4 * gB);
  }
  if (a.rows[1].weight) {
    wk[0] = *reinterpret_cast<const uint2*>((const uint16_t*)a.rows[1].weight + 4 * gA);
    wk[1] = *reinterpret_cast<const uint2*>((const uint16_t*)a.rows[1].weight + 4 * gB);
  }
  const int dt = kRopeRows / HT, dh = kRopeRows % HT;  // one step of kRopeRows rows
  int tok = hw / HT, head = hw % HT;
  uint2 x[kRopeBatch][2];
  uint16_t* dst[kRopeBatch];
  int kind[kRopeBatch], at[kRopeBatch];  // 0 query, 1 key, 2 value, 3 none; token of the tile
  auto load = [&](int r0) {
#pragma unroll
    for (int i = 0; i < kRopeBatch; ++i) {
      const int r = r0 + (hw & 1) + i * kRopeRows;
      int h = head, set = 0;
      if (h >= a.rows[0].heads) { h -= a.rows[0].heads; set = 1; }
      if (set == 1 && h >= a.rows[1].heads) { h -= a.rows[1].heads; set = 2; }
      kind[i] = r < nrows ? set : 3;
      at[i] = tok;
      dst[i] = nullptr;
      x[i][0] = x[i][1] = make_uint2(0u, 0u);
      if (r < nrows) {
        const RopeRows& R = a.rows[set];
        const uint16_t* src = (const uint16_t*)R.in + (t0 + tok) * R.in_tok + h * R.in_head;
        dst[i] = (uint16_t*)R.out + (t0 + tok) * R.out_tok + h * R.out_head;
        x[i][0] = *reinterpret_cast<const uint2*>(src + 4 * gA);
        x[i][1] = *reinterpret_cast<const uint2*>(src + 4 * gB);
      }
      tok += dt;
      head += dh;
      if (head >= HT) { head -= HT; ++tok; }
    }
  };
  // the first rows are on their way while the angles of the CTA's tokens are made
  load(hw & ~1);
  for (int i = threadIdx.x; i < tn * pairs; i += kRopeThreads) {
    const int t = i / pairs, f = i % pairs;
    const double turn = (double)a.pos[t0 + t] * (double)a.inv_freq[f] * 0.15915494309189533577;
    float s, c;
    sincospif(2.0f * (float)(turn - rint(turn)), &s, &c);
    cs[t][f] = make_float2(c, s);
  }
  __syncthreads();
  // both halves of a warp run the same number of rounds (the sums shuffle across the warp)
  for (int r0 = hw & ~1; r0 < nrows; r0 += kRopeRows * kRopeBatch) {
    if (r0 != (hw & ~1)) load(r0);
#pragma unroll
    for (int i = 0; i < kRopeBatch; ++i) {
      const bool rot = kind[i] < 2;
      float2 p[4] = {to_f2<BF16>(x[i][0].x), to_f2<BF16>(x[i][0].y), to_f2<BF16>(x[i][1].x), to_f2<BF16>(x[i][1].y)};
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) ss = fmaf(p[e].x, p[e].x, fmaf(p[e].y, p[e].y, ss));
#pragma unroll
      for (int o = 8; o; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
      if (rot) {
        if (a.rows[kind[i]].weight) {
          const float inv = rsqrtf(ss * (1.0f / kD) + a.eps);
          const uint2* w = kind[i] == 0 ? wq : wk;
          const float2 f[4] = {to_f2<BF16>(w[0].x), to_f2<BF16>(w[0].y), to_f2<BF16>(w[1].x), to_f2<BF16>(w[1].y)};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[e].x = p[e].x * inv * f[e].x;
            p[e].y = p[e].y * inv * f[e].y;
          }
        }
        if (turns) {
          const float4 c01 = *reinterpret_cast<const float4*>(&cs[at[i]][4 * lane16]);
          const float4 c23 = *reinterpret_cast<const float4*>(&cs[at[i]][4 * lane16 + 2]);
          const float co[4] = {c01.x, c01.z, c23.x, c23.z}, si[4] = {c01.y, c01.w, c23.y, c23.w};
          if constexpr (INTER) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              p[e] = make_float2(p[e].x * co[e] - p[e].y * si[e], p[e].y * co[e] + p[e].x * si[e]);
          } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 u = p[e], v = p[e + 2];
              p[e] = make_float2(u.x * co[2 * e] - v.x * si[2 * e], u.y * co[2 * e + 1] - v.y * si[2 * e + 1]);
              p[e + 2] = make_float2(v.x * co[2 * e] + u.x * si[2 * e], v.y * co[2 * e + 1] + u.y * si[2 * e + 1]);
            }
          }
        }
        x[i][0] = make_uint2(from_f2<BF16>(p[0].x, p[0].y), from_f2<BF16>(p[1].x, p[1].y));
        x[i][1] = make_uint2(from_f2<BF16>(p[2].x, p[2].y), from_f2<BF16>(p[3].x, p[3].y));
      }
      if (kind[i] < 3) {
        *reinterpret_cast<uint2*>(dst[i] + 4 * gA) = x[i][0];
        *reinterpret_cast<uint2*>(dst[i] + 4 * gB) = x[i][1];
      }
    }
  }
}

}  // namespace

cudaError_t launch_norm_rope(const RopeArgs& a0, int dtype, bool interleaved, int num_sms, cudaStream_t st) {
  RopeArgs a = a0;
  // a tile of tokens shares its angles; with few tokens every token gets a CTA of its own
  a.tile = a.tokens >= (int64_t)kRopeTile * num_sms * 4 ? kRopeTile : 1;
  const int64_t grid = (a.tokens + a.tile - 1) / a.tile;
  const bool bf = dtype == KVQ_BF16;
  auto* k = bf ? (interleaved ? norm_rope_kernel<true, true> : norm_rope_kernel<true, false>)
               : (interleaved ? norm_rope_kernel<false, true> : norm_rope_kernel<false, false>);
  k<<<(unsigned)grid, kRopeThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace kvq
