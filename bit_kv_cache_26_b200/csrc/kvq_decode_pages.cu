// Decode attention over chosen pages of the quantized paged cache: per (sequence, KV head) a list
// of pages, softmax(q . K_hat^T) V_hat over their tokens only, in the cache's 2- or 4-bit codes
// ("PatternKV", Section 3.4: the fused reconstruction and attention, over a subset of the pages).
//
// Bound: the listed sub-blocks from HBM, then instruction issue.  One B200, 256 sequences x 8 KV heads
// x 128 of 512 pages in 4 bits, 4 query heads each: 338-346 us, 4.7-4.8 TB/s of page bytes (0.72-0.74 of
// the copy bandwidth); 386 us back to back, under the power cap; in 2 bits, of two thirds of the bytes, 328
// us (nearly the same instructions).  With 8 and 16 heads a group (1024 groups of 64 pages) 176 and 347 us
// for 63 of bytes: the work per page grows with the heads, and 12 and 8 warps an SM hide less of it.  The
// setup and merge of a CTA (lengths, ids, q . M_K, W . M_V) are a tenth of the first and most of the time
// of short lists: they avoid branches and loads that wait for each other (all query rows at once, four
// heads' sums exchanged together, the final sum eight patterns at a time).  Two choices cost time for
// what they keep: pattern weights as fp32 sums in a fixed order took 308 -> 334 us (of which finding the
// tokens that share a pattern 13), V operands in units that follow their size 334 -> 338.
//
// Per CTA one (sequence, KV head, split of the list); each warp streams its entries' sub-blocks
// through a ring of shared-memory stages (cp.async.bulk, bounded mbarrier waits).
//
//   K, per page with per-channel scale s_d and zero z_d, T_j = q . M_K[j] (once per CTA):
//     q.k_t = sum_d (q_d s_d) code_td + sum_d q_d z_d + T[idx_t]
//   V, per token with per-group scale s_tg and zero z_tg, W_j = sum of p over tokens with pattern j:
//     sum_t p_t v_t = sum_t (p_t s_tg) code_td + sum_t p_t z_tg + sum_j W_j M_V[j]
//
// The code sums are m16n8k16 products with the codes as the fp16 A operand.  A code field masked
// out of its word is an fp16 subnormal as it stands: code * 2^S * 2^-24 for a field at bit S of a
// half word (S <= 6, so it fits the ten mantissa bits), which the tensor cores multiply exactly.
// One AND per pair of codes; the powers of two of the four fields of a 16x16 tile separate into a
// row factor (undone on the sums) and a column factor (folded into B).  B is q s or p s in fp16
// hi + lo parts (22 bits).  The query is scaled by a power of two to [16, 32): K scales up to 2000 fit
// fp16 (past them the output is not finite and KVQ_DEV_RANGE is set); of a product too small for hi + lo
// 2^-25 is dropped, as if the key's scale were off by 2^-29 (2^-25 in columns with a factor).  p s is in
// units that follow the largest product a head has met in the warp (below 2^15 of them), so that a dominant
// token of small value, or values that are small throughout, leave the others their bits: what is dropped
// is 2^-33 of that product (2^-29 where columns have a factor).
//
// Up to four query heads per KV head: the eight columns of a product are (head, {hi, lo}).  The two
// lanes of a head's columns each form the products of half the channels (tokens for V) and give each
// other the part the other's column needs: half the shared-memory reads, which were what bounded the
// loop (68 % of the shared-memory pipe at 67 % of the copy bandwidth).  More heads: the columns are
// eight heads, and a second product adds the lo parts.
//
// The newest incomplete page takes its keys from the K tail, exact 16-bit operands of the same
// products.  W is summed in fp32, in a fixed order (a token's turn among those of its page with the same
// pattern is its lane's place among theirs), so results do not depend on timing.  A lane adds one
// token for all heads of a tile at once; in the usual page few tokens share a pattern, so there are two
// or three turns.
#include <algorithm>
#include <atomic>

#include "kvq_common.cuh"
#include "kvq_internal.h"
#include "kvq_pipe.cuh"

namespace kvq {

namespace {

constexpr int kStages = 2;   // ring stages per warp
constexpr int kNW = 4;       // warps per CTA
constexpr int kMvAhead = 64;      // pattern values in flight per thread in the final sum
constexpr int kMaxSmem = 200 * 1024;  // dynamic, of a CTA (the largest shape, 255 patterns and 16 heads a group, takes 157 KB)
constexpr int kPexRow = 36;       // padded row of the p exchange (floats)
constexpr int kVTop = 15;         // p s, as an fp16 operand, is below 2^kVTop
constexpr int kVRoom = 3;         // powers of two of room for the products to come when the unit is set, and again before it is lowered
constexpr float kVLeast = 7.8886091e-31f;  // 2^-100: V scales below it do not set the operands' unit

template <int BITS>
struct Code {
  static constexpr float kRow = BITS == 2 ? 4.0f : 16.0f;  // factor of rows 8..15 of a tile
  static constexpr float kCol = BITS == 2 ? 16.0f : 1.0f;  // factor of columns 8..15
};

// The A registers of tile half `odd` of word w (2-bit: two tiles per word; 4-bit: one); `swapped`: with the
// two columns of each register exchanged.
template <int BITS>
__device__ __forceinline__ void frag16(uint32_t w, int odd, uint32_t (&a)[4], bool swapped = false) {
  if constexpr (BITS == 2) {
    const uint32_t x = swapped ? __funnelshift_r(w, w, odd ? 24 : 16) : odd ? w >> 8 : w;
    a[0] = x & 0x00030003u;
    a[1] = x & 0x000C000Cu;
    a[2] = x & 0x00300030u;
    a[3] = x & 0x00C000C0u;
  } else {
    const uint32_t x = swapped ? __funnelshift_r(w, w, 16) : w, y = swapped ? __funnelshift_r(w, w, 24) : w >> 8;
    a[0] = x & 0x000F000Fu;
    a[1] = x & 0x00F000F0u;
    a[2] = y & 0x000F000Fu;
    a[3] = y & 0x00F000F0u;
  }
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 2^e, to the range of normal numbers.
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(127 + max(-126, min(127, e))) << 23); }
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }  // e of a normal number
// 2^e / x of a power of two x.
__device__ __forceinline__ float pow2_over(int e, float x) { return __uint_as_float(((uint32_t)(254 + e) << 23) - __float_as_uint(x)); }
// x's exponent: x < 2^(exponent(x) + 1) for a number x >= 0.
__device__ __forceinline__ int exponent(float x) { return (int)(__float_as_uint(x) >> 23 & 0xff) - 127; }

__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  uint32_t h;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(hi), "f"(lo));
  return h;
}
__device__ __forceinline__ unsigned long long less(unsigned long long v, float x, float y) {  // v - (x, y)
  return fma2(pk(x, y), pk(-1.0f, -1.0f), v);
}
// fp16 pairs of the hi parts (11 significant bits) of two fp32 values and of what is left of them.
__device__ __forceinline__ void split2(unsigned long long v, uint32_t& hi, uint32_t& lo) {
  float v0, v1;
  upk(v, v0, v1);
  hi = half2_of(v0, v1);
  const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  upk(less(v, t.x, t.y), v0, v1);
  lo = half2_of(v0, v1);
}
// The same of the pairs (first of v, first of w) and (second of v, second of w).
__device__ __forceinline__ void split2x2(unsigned long long v, unsigned long long w, uint32_t (&hi)[2], uint32_t (&lo)[2]) {
  float v0, v1, w0, w1;
  upk(v, v0, v1);
  upk(w, w0, w1);
  hi[0] = half2_of(v0, w0);
  hi[1] = half2_of(v1, w1);
  const float2 s = __half22float2(*reinterpret_cast<const __half2*>(&hi[0])), t = __half22float2(*reinterpret_cast<const __half2*>(&hi[1]));
  upk(less(v, s.x, t.x), v0, v1);
  upk(less(w, s.y, t.y), w0, w1);
  lo[0] = half2_of(v0, w0);
  lo[1] = half2_of(v1, w1);
}

// x[i] of the lanes of a quad (tig = 0 .. 3) exchanged, so that lane tig ends with the x[tig] of the four lanes in turn.
__device__ __forceinline__ void quad_transpose(float (&x)[4], int tig) {
  const bool b1 = tig & 2, b0 = tig & 1;
  const float r0 = __shfl_xor_sync(kFull, b1 ? x[0] : x[2], 2), r1 = __shfl_xor_sync(kFull, b1 ? x[1] : x[3], 2);
  x[0] = b1 ? r0 : x[0];
  x[1] = b1 ? r1 : x[1];
  x[2] = b1 ? x[2] : r0;
  x[3] = b1 ? x[3] : r1;
  const float s0 = __shfl_xor_sync(kFull, b0 ? x[0] : x[1], 1), s1 = __shfl_xor_sync(kFull, b0 ? x[2] : x[3], 1);
  x[0] = b0 ? s0 : x[0];
  x[1] = b0 ? x[1] : s0;
  x[2] = b0 ? s1 : x[2];
  x[3] = b0 ? x[3] : s1;
}

// Smallest row stride >= n whose rows start `step` banks apart.
__host__ __device__ constexpr int banked(int n, int step) { return n + ((step - n) % 32 + 32) % 32; }

constexpr int kMergeRows = 8;  // pattern weights of the final sum at a time
// Row stride (floats) of the warps' sums of p v: a quad's four heads start 8 banks apart.
__host__ __device__ constexpr int merge_row(bool wide) { return kD + (wide ? 4 : 8); }

struct PagesSmem {
  int bars, qk, qinv, T, W, pex, total;
  int wc, fsh, sum_o, sum_ml;  // of the merge, floats
  int t_row;
};
__host__ __device__ inline PagesSmem pages_smem(int sub_bytes, int NT, bool wide, int P) {
  PagesSmem s;
  const int NH = NT * (wide ? 8 : 4);
  s.t_row = banked(P, wide ? 4 : 8);
  // the ring; the merge at the end reuses its place: per warp and head 128 sums of p v, max and sum, four sums of p z
  s.wc = kNW * NH * merge_row(wide) + 2 * kNW * NH + kNW * NH * 4;
  s.fsh = s.wc + (P + kMergeRows - 1) / kMergeRows * kMergeRows * NH;
  s.sum_o = s.fsh + NH * kNW;
  s.sum_ml = s.sum_o + NH * kD;
  int o = max(kNW * kStages * sub_bytes, (s.sum_ml + 2 * NH) * 4);
  o = (o + 15) & ~15;
  s.bars = o; o += kNW * kStages * 8;
  s.qinv = o; o += NH * 4;                    // inverse power of two of the query scale per head
  s.T = o; o += NH * s.t_row * 4;             // T[head][j], scaled as the query
  s.qk = o; o += wide ? NH * kD * 4 : 0;      // query in the quantized space, scaled, KSC order
  s.pex = o; o += wide ? kNW * NH * kPexRow * 4 : 0;  // per-warp p exchange
  o = (o + 15) & ~15;
  s.W = o;                                    // per-warp pattern weights [P][NH]; first the query in natural order (and in
  const int first = NH * (kD + (wide ? 0 : kD));  // KSC order, when its users then keep it in registers)
  o += max(kNW * NH * P, first) * 4;
  if (!wide) s.qk = s.W + NH * kD * 4;
  s.total = o;
  return s;
}

// All threads of the cluster: shared memory written before is seen by the others after.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
}
// Shared memory of the CTA of rank r of the cluster, at the place of p in this one's.
__device__ __forceinline__ uint32_t peer_addr(const void* p, int r) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(r));
  return a;
}
__device__ __forceinline__ float2 peer_f2(const void* p, int r) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(peer_addr(p, r)) : "memory");
  return v;
}
__device__ __forceinline__ float4 peer_f4(const void* p, int r) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(peer_addr(p, r))
               : "memory");
  return v;
}

// What a head's sum of p v is divided by.  The sum of p is 1 or more with any token, and 0 with none, for which the output is
// 0; a query of NaN has no maximum (it is ignored) and a sum of NaN, which is left to show in the output.
__device__ __forceinline__ float sum_or_one(float l) { return l == 0.f ? 1.f : l; }

// Whether v is a finite number of the output's type (fp16 rounds to infinity from 65520 on).
__device__ __forceinline__ bool in_range(const Geom& g, float v) { return fabsf(v) < (g.dtype == KVQ_BF16 ? INFINITY : 65520.0f); }

// Output of one query head from its channels 4 lane .. 4 lane + 3 of sum p v and its sum p.
__device__ __forceinline__ void finish_head(const Geom& g, float (&o)[4], float l, const float* vcol, uint16_t* out, int lane) {
  const float inv = 1.0f / l;
#pragma unroll
  for (int k = 0; k < 4; ++k) o[k] *= inv;
  if (g.tx) {
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] *= __ldg(vcol + 4 * lane + k);
    // Walsh-Hadamard: strides 1 and 2 in the lane, 4 .. 64 across lanes
    float p0 = o[0] + o[1], p1 = o[0] - o[1], p2 = o[2] + o[3], p3 = o[2] - o[3];
    o[0] = p0 + p2; o[2] = p0 - p2; o[1] = p1 + p3; o[3] = p1 - p3;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float other = __shfl_xor_sync(kFull, o[k], s);
        o[k] = (lane & s) ? other - o[k] : o[k] + other;
      }
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] *= 0.0078125f;
  }
  if (!(in_range(g, o[0]) && in_range(g, o[1]) && in_range(g, o[2]) && in_range(g, o[3]))) set_status(g.status, KVQ_DEV_RANGE);
  uint2 r;
  if (g.dtype == KVQ_BF16) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(o[0], o[1]), y = __floats2bfloat162_rn(o[2], o[3]);
    r = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  } else {
    r = make_uint2(half2_of(o[0], o[1]), half2_of(o[2], o[3]));
  }
  reinterpret_cast<uint2*>(out)[lane] = r;
}

// NT tiles of four query heads (or eight: WIDE).  Thread (gq, tig) of a warp holds the sums of head
// 4 j + tig of tile j (WIDE: heads 8 j + 2 tig and the next) and forms the B columns of head
// 4 j + gq / 2 (WIDE: 8 j + gq).
template <int BITS, int NT, bool WIDE, bool TX>
__global__ void __launch_bounds__(kNW * 32, WIDE ? (NT == 1 ? 3 : 2) : 4) decode_pages_kernel(Geom g, PagesArgs a) {
  static_assert(WIDE || NT == 1, "more than four heads: wide tiles");
  constexpr int HPT = WIDE ? 2 : 1, TH = 4 * HPT, NH = NT * TH, WPL = BITS * 4;
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gq = lane >> 2, tig = lane & 3, part = gq & 1;
  const int split = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int64_t grp = (int64_t)b * g.H + h;
  const int Gq = a.Gq, P = g.P;
  const int sub_bytes = (int)g.sub_bytes;
  const PagesSmem sp = pages_smem(sub_bytes, NT, WIDE, P);
  const int TR = sp.t_row;
  uint8_t* ring = smem + warp * kStages * sub_bytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + sp.bars) + warp * kStages;
  float* qk = reinterpret_cast<float*>(smem + sp.qk);
  float* qinv = reinterpret_cast<float*>(smem + sp.qinv);
  float* T = reinterpret_cast<float*>(smem + sp.T);
  // pattern weights: per warp and pattern NH heads, a wide tile's even heads before its odd ones (as its lanes hold them)
  float* Wall = reinterpret_cast<float*>(smem + sp.W);
  float* Ww = Wall + warp * NH * P;
  auto w_place = [](int hh) { return WIDE ? (hh & ~7) | (hh & 1) << 2 | (hh & 7) >> 1 : hh; };
  float* qn = reinterpret_cast<float*>(smem + sp.W);  // query in natural order, until T is made
  float* pex = reinterpret_cast<float*>(smem + sp.pex) + warp * NH * kPexRow;

  // entries of this warp: split + nsplit (warp + kNW i).  Lane l of window w reads entry i = 32 w + l; the first
  // window goes out with the lengths.
  const int32_t* list = a.list + grp * a.budget;
  const int64_t stride = (int64_t)a.nsplit * kNW, e_first = split + (int64_t)a.nsplit * warp;
  auto entry = [&](int i) -> int {
    const int64_t e = e_first + stride * i;
    return e < a.budget ? __ldg(list + e) : -1;
  };
  int lp = entry(lane);
  int L = g.seq_len[b];
  int n_list = a.list_len[grp];
  const bool teller = threadIdx.x == 0 && split == 0;
  if (L < 0 || L > (int64_t)g.maxp * kG) {
    if (teller) set_status(g.status, KVQ_DEV_OVERFLOW);
    L = 0;
  }
  if (n_list < 0 || n_list > a.budget) {
    if (teller) set_status(g.status, KVQ_DEV_OVERFLOW);
    n_list = 0;
  }
  int set = g.seq_to_set ? g.seq_to_set[b] : 0;
  if (set < 0 || set >= g.S) {
    if (teller) set_status(g.status, KVQ_DEV_BAD_SET);
    set = 0;
    n_list = 0;
  }
  const int nfull = L / kG, ntail = L % kG, npages = nfull + (ntail > 0);
  // this CTA's entries: split, split + nsplit, ... (dealt so that the list can be read before its length is known)
  const int n_mine = (int)(((int64_t)n_list - split + a.nsplit - 1) / a.nsplit);
  const size_t sh = (size_t)set * g.H + h;
  const int Pe = p_eff(g, (int)sh);
  const float* MK = g.kpat + sh * P * kD;
  const int64_t row0 = ((int64_t)b * a.Hq + (int64_t)h * Gq) * a.nsplit + split;  // partial row of head 0; + hh * nsplit

  // a group's sums, when they are merged in shared memory: [NH][128] sum p v and [NH] (max, sum p), after the merge's places
  const bool in_smem = a.nsplit == 1 || a.clustered;
  const bool direct = !TX && a.nsplit == 1;  // a thread's channel is final (without the transform back): no exchange
  float* sum_o = reinterpret_cast<float*>(smem) + sp.sum_o;
  float2* sum_ml = reinterpret_cast<float2*>(reinterpret_cast<float*>(smem) + sp.sum_ml);

  if (n_mine > 0) {
    // the first of the setup's loads go out before the page copies, which would keep them waiting: this warp's
    // query rows and this thread's quarters of two pattern rows (four lanes per row, 16 bytes in turn)
    uint16_t q_raw[NH / kNW][4];
#pragma unroll
    for (int r = 0; r < NH / kNW; ++r) {
      const uint16_t* src = a.q + ((int64_t)b * a.Hq + (int64_t)h * Gq + min(warp + kNW * r, Gq - 1)) * kD + lane;
#pragma unroll
      for (int k = 0; k < 4; ++k) q_raw[r][k] = __ldg(src + 32 * k);
    }
    const int quarter = threadIdx.x & 3;
    float4 m[2][8];
    auto load_patterns = [&](int j) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float4* row = reinterpret_cast<const float4*>(MK + (size_t)min(j + 32 * r, Pe - 1) * kD) + quarter;
#pragma unroll
        for (int c = 0; c < 8; ++c) m[r][c] = __ldg(row + 4 * c);
      }
    };
    load_patterns(threadIdx.x >> 2);
    // the physical page of this lane's entry, -1 where it names none; whether it is the newest incomplete page
    const int my_n = (n_mine - warp + kNW - 1) / kNW;
    unsigned tails = 0;
    auto load_ids = [&](int base) -> int {
      if (base > 0) lp = entry(base + lane);
      int phys = -1;
      if (base + lane < my_n) {
        if (lp >= 0 && lp < npages) phys = g.page_table[(int64_t)b * g.maxp + lp];
        if (phys < 0 || phys >= g.npages) {
          set_status(g.status, KVQ_DEV_BAD_PAGE);
          phys = -1;
        }
      }
      tails = __ballot_sync(kFull, phys >= 0 && lp == nfull);
      return phys;
    };
    int ids = load_ids(0);
    auto fetch = [&](int st, int phys) {  // lane 0
      if (phys >= 0) {
        mbar_expect_tx(&bars[st], sub_bytes);
        bulk_g2s(ring + st * sub_bytes, g.pool + (size_t)phys * g.page_bytes + (size_t)h * sub_bytes, sub_bytes, &bars[st]);
      } else {
        mbar_arrive(&bars[st]);
      }
    };
    if (lane < kStages) mbar_init(&bars[lane], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncwarp();
    unsigned skips = 0, tail_st = 0;  // per stage
#pragma unroll
    for (int i = 0; i < kStages; ++i) {
      const int phys = __shfl_sync(kFull, ids, i);
      if (i < my_n) {
        if (phys < 0) skips |= 1u << i;
        if (tails >> i & 1) tail_st |= 1u << i;
        if (lane == 0) fetch(i, phys);
      }
    }

    // ---- queries, T, zeroed W (over the first copies)
#pragma unroll
    for (int r = 0; r < NH / kNW; ++r) {
      const int hh = warp + kNW * r;
      float v[4], m = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = hh < Gq ? bits_to_float(q_raw[r][k], g.dtype) : 0.f;
      if constexpr (TX) {
        fwht_warp(v, lane);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = v[k] * __ldg(g.kcol + sh * kD + lane + 32 * k) * 0.0078125f;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) m = fmaxf(m, fabsf(v[k]));
      m = warp_max(m);
      const int e = (int)(__float_as_uint(m) >> 23) - 127;  // exponent of the largest
      const bool plain = m == 0.f || e > 100 || e < -100;
      const float f = plain ? 1.f : __uint_as_float((uint32_t)(127 + 4 - e) << 23);
      if (lane == 0) qinv[hh] = plain ? 1.f : __uint_as_float((uint32_t)(127 - 4 + e) << 23);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int ch = lane + 32 * k;
        qk[hh * kD + ksc_pos(ch)] = v[k] * f * ((ch & 8) ? 1.0f / Code<BITS>::kCol : 1.0f);
        qn[hh * kD + ch] = v[k] * f;
      }
    }
    __syncthreads();
    // T: four lanes per pattern, two patterns at a time
    static_assert(kNW * 32 == 4 * 32, "32 rows per round and half");
    for (int j0 = 0; j0 < Pe; j0 += 64) {
      const int j = j0 + (threadIdx.x >> 2);
      if (j0 > 0) load_patterns(j);
#pragma unroll 1
      for (int h0 = 0; h0 < NH; h0 += 4) {
        float y[4][2];  // of heads h0 .. h0 + 3, this lane's quarter
#pragma unroll
        for (int hh = 0; hh < 4; ++hh) {
          const float4* qr = reinterpret_cast<const float4*>(qn + (h0 + hh) * kD) + quarter;
          unsigned long long s[2][2] = {{0ull, 0ull}, {0ull, 0ull}};
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const float4 x = qr[4 * c];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              s[r][0] = fma2(pk(x.x, x.y), pk(m[r][c].x, m[r][c].y), s[r][0]);
              s[r][1] = fma2(pk(x.z, x.w), pk(m[r][c].z, m[r][c].w), s[r][1]);
            }
          }
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float x0, x1, x2, x3;
            upk(s[r][0], x0, x1);
            upk(s[r][1], x2, x3);
            y[hh][r] = (x0 + x1) + (x2 + x3);
          }
        }
        // summed over the four lanes, of which each goes on with fewer heads: lane `quarter` ends with head h0 + quarter
        const bool q2 = quarter & 2, q1 = quarter & 1;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float u = (q2 ? y[2][r] : y[0][r]) + __shfl_xor_sync(kFull, q2 ? y[0][r] : y[2][r], 2);
          const float v = (q2 ? y[3][r] : y[1][r]) + __shfl_xor_sync(kFull, q2 ? y[1][r] : y[3][r], 2);
          const float w = (q1 ? v : u) + __shfl_xor_sync(kFull, q1 ? u : v, 1);
          if (j + 32 * r < Pe) T[(h0 + quarter) * TR + j + 32 * r] = w;
        }
      }
    }
    // the query of this lane's columns: narrow tiles keep the half they need in registers
    float4 qreg[4];
    if constexpr (!WIDE) {
#pragma unroll
      for (int c = 0; c < 4; ++c) qreg[c] = reinterpret_cast<const float4*>(qk + (gq >> 1) * kD)[(2 * c + part) * 4 + tig];
    }
    __syncthreads();
    for (int i = lane; i < NH / 4 * P; i += 32) reinterpret_cast<float4*>(Ww)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    __syncwarp();

    // ---- per-thread state
    float accv[NT][8][4], zacc[NT][HPT][4], mrun[NT][HPT], lrun[NT][HPT], scl[NT][HPT];
    // accv is in units of 2^-kVTop vlim, a power of two above all products p r s so far; vtop: the largest when it was set, as it
    // has shrunk since
    float vlim[NT][HPT], vtop[NT][HPT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int x = 0; x < HPT; ++x) {
        mrun[j][x] = -INFINITY;
        lrun[j][x] = 0.f;
        vlim[j][x] = pow2(-100);
        vtop[j][x] = 0.f;
        scl[j][x] = a.scale_log2 * qinv[TH * j + HPT * tig + x];
#pragma unroll
        for (int u = 0; u < 4; ++u) zacc[j][x][u] = 0.f;
      }
#pragma unroll
      for (int mt = 0; mt < 8; ++mt)
#pragma unroll
        for (int u = 0; u < 4; ++u) accv[j][mt][u] = 0.f;
    }

    int stuck_at = -1;
    for (int i = 0; i < my_n; ++i) {
      const int st = i % kStages;
      const bool ok = mbar_wait(&bars[st], (i / kStages) & 1, g.wait_limit);
      if (!__all_sync(kFull, ok)) { stuck_at = i; break; }
      uint8_t* pgp = ring + st * sub_bytes;
      if (!(skips >> st & 1)) {
        const bool tail = tail_st >> st & 1;
        float sc[NT][HPT][4];  // token gq + 8 u
        if (!tail) {
          // ---- K: scores of the page's 32 tokens
          uint32_t kw[WPL];
#pragma unroll
          for (int c = 0; c < WPL / 4; ++c) {
            const uint4 t = reinterpret_cast<const uint4*>(pgp + c * 512)[lane];
            kw[4 * c] = t.x; kw[4 * c + 1] = t.y; kw[4 * c + 2] = t.z; kw[4 * c + 3] = t.w;
          }
          const float4* ks4 = reinterpret_cast<const float4*>(pgp + g.off_ks) + tig;
          const float4* kz4 = reinterpret_cast<const float4*>(pgp + g.off_kz) + tig;
          const uint32_t kidx4 = *reinterpret_cast<const uint32_t*>(pgp + g.off_kidx + gq * 4);
          float krow[4] = {1.f, 1.f, 1.f, 1.f};
          if constexpr (TX) {
            const float4 kr = *reinterpret_cast<const float4*>(pgp + g.off_krow + gq * 16);
            krow[0] = kr.x; krow[1] = kr.y; krow[2] = kr.z; krow[3] = kr.w;
          }
          float acc[NT][2][4], zk[NT];
          unsigned long long za2[NT], zb2[NT];
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            za2[j] = zb2[j] = 0ull;
#pragma unroll
            for (int x = 0; x < 8; ++x) acc[j][x >> 2][x & 3] = 0.f;
          }
          if constexpr (!WIDE) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {  // of channel steps 2 c and 2 c + 1, one is this lane's, the other its partner's
              const float4 s4 = ks4[(2 * c + part) * 4], z4 = kz4[(2 * c + part) * 4];
              const unsigned long long qa = pk(qreg[c].x, qreg[c].y), qb = pk(qreg[c].z, qreg[c].w);
              za2[0] = fma2(qa, pk(z4.x, z4.y), za2[0]);
              zb2[0] = fma2(qb, pk(z4.z, z4.w), zb2[0]);
              uint32_t own0, own1, lo0, lo1;
              split2(mul2(qa, pk(s4.x, s4.y)), own0, lo0);
              split2(mul2(qb, pk(s4.z, s4.w)), own1, lo1);
              const uint32_t got0 = __shfl_xor_sync(kFull, lo0, 4), got1 = __shfl_xor_sync(kFull, lo1, 4);
              // (which of the two columns holds hi and which lo is the other way round in the odd steps: they are added)
#pragma unroll
              for (int s = 0; s < 2; ++s) {
                const int ks = 2 * c + s;
                const uint32_t b0 = part == s ? own0 : got0, b1 = part == s ? own1 : got1;
                uint32_t f[4];
                frag16<BITS>(BITS == 2 ? kw[ks / 2] : kw[ks], ks & 1, f);
                mma_f16(acc[0][0], f, b0, b1);
                frag16<BITS>(BITS == 2 ? kw[4 + ks / 2] : kw[8 + ks], ks & 1, f);
                mma_f16(acc[0][1], f, b0, b1);
              }
            }
          } else {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
              const float4 s4 = ks4[ks * 4], z4 = kz4[ks * 4];
              uint32_t f[2][4];
              frag16<BITS>(BITS == 2 ? kw[ks / 2] : kw[ks], ks & 1, f[0]);
              frag16<BITS>(BITS == 2 ? kw[4 + ks / 2] : kw[8 + ks], ks & 1, f[1]);
#pragma unroll
              for (int j = 0; j < NT; ++j) {
                const float4 q4 = reinterpret_cast<const float4*>(qk + (TH * j + gq) * kD)[ks * 4 + tig];
                const unsigned long long qa = pk(q4.x, q4.y), qb = pk(q4.z, q4.w);
                za2[j] = fma2(qa, pk(z4.x, z4.y), za2[j]);
                zb2[j] = fma2(qb, pk(z4.z, z4.w), zb2[j]);
                uint32_t bh0, bh1, bl0, bl1;
                split2(mul2(qa, pk(s4.x, s4.y)), bh0, bl0);
                split2(mul2(qb, pk(s4.z, s4.w)), bh1, bl1);
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
                  mma_f16(acc[j][mt], f[mt], bh0, bh1);
                  mma_f16(acc[j][mt], f[mt], bl0, bl1);
                }
              }
            }
          }
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            // zero term of this lane's column, summed over the lanes that share it
            float z0, z1, z2, z3;
            upk(za2[j], z0, z1);
            upk(zb2[j], z2, z3);
            zk[j] = fmaf(z2 + z3, Code<BITS>::kCol, z0 + z1);
            zk[j] += __shfl_xor_sync(kFull, zk[j], 1);
            zk[j] += __shfl_xor_sync(kFull, zk[j], 2);
            if constexpr (!WIDE) zk[j] += __shfl_xor_sync(kFull, zk[j], 4);
#pragma unroll
            for (int x = 0; x < HPT; ++x) {
              const float z = __shfl_sync(kFull, zk[j], WIDE ? 4 * (2 * tig + x) : 8 * tig);
              const unsigned long long f08 = pk(16777216.0f, 16777216.0f / Code<BITS>::kRow), z2 = pk(z, z), l2 = pk(scl[j][x], scl[j][x]);
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {  // tokens gq + 16 hf and the one 8 on
                const float s0 = WIDE ? acc[j][hf][x] : acc[j][hf][0] + acc[j][hf][1], s8 = WIDE ? acc[j][hf][2 + x] : acc[j][hf][2] + acc[j][hf][3];
                const int i0 = min((int)((kidx4 >> (16 * hf)) & 0xff), Pe - 1), i8 = min((int)((kidx4 >> (16 * hf + 8)) & 0xff), Pe - 1);
                const float* Th = T + (TH * j + HPT * tig + x) * TR;
                const unsigned long long s = add2(fma2(pk(s0, s8), f08, z2), pk(Th[i0], Th[i8]));
                upk(mul2(s, TX ? mul2(pk(krow[2 * hf], krow[2 * hf + 1]), l2) : l2), sc[j][x][2 * hf], sc[j][x][2 * hf + 1]);
              }
            }
          }
        } else {
          // ---- K tail: exact keys; tokens that are not there yet score -inf and store nothing of V
          const uint16_t* kt = g.k_tail + grp * kG * kD;
          if (lane >= ntail) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              reinterpret_cast<float*>(pgp + g.off_vs)[vsc_pos(lane, u)] = 0.f;
              reinterpret_cast<float*>(pgp + g.off_vz)[vzc_pos(lane, u)] = 0.f;
            }
            pgp[g.off_vidx + tok_pos(lane)] = (uint8_t)kRawIndex;
            if constexpr (TX) reinterpret_cast<float*>(pgp + g.off_vrow)[tok_pos(lane)] = 0.f;
          }
          __syncwarp();
          float acc[NT][2][4];
          const uint16_t* qr[NT];
          bool has[NT];
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const int hq = TH * j + (WIDE ? gq : gq >> 1);
            has[j] = hq < Gq && (WIDE || part == 0);
            qr[j] = a.q + ((int64_t)b * a.Hq + (int64_t)h * Gq + min(hq, Gq - 1)) * kD + 2 * tig;
#pragma unroll
            for (int x = 0; x < 8; ++x) acc[j][x >> 2][x & 3] = 0.f;
          }
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            uint32_t f[2][4];
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
              const uint16_t* kr = kt + (16 * mt + gq) * kD + 16 * ks + 2 * tig;
              f[mt][0] = *reinterpret_cast<const uint32_t*>(kr);
              f[mt][1] = *reinterpret_cast<const uint32_t*>(kr + 8 * kD);
              f[mt][2] = *reinterpret_cast<const uint32_t*>(kr + 8);
              f[mt][3] = *reinterpret_cast<const uint32_t*>(kr + 8 * kD + 8);
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              const uint32_t b0 = has[j] ? *reinterpret_cast<const uint32_t*>(qr[j] + 16 * ks) : 0u;
              const uint32_t b1 = has[j] ? *reinterpret_cast<const uint32_t*>(qr[j] + 16 * ks + 8) : 0u;
#pragma unroll
              for (int mt = 0; mt < 2; ++mt) {
                if (g.dtype == KVQ_BF16) mma_bf16(acc[j][mt], f[mt], b0, b1);
                else mma_f16(acc[j][mt], f[mt], b0, b1);
              }
            }
          }
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int x = 0; x < HPT; ++x)
#pragma unroll
              for (int u = 0; u < 4; ++u)
                sc[j][x][u] = gq + 8 * u < ntail ? acc[j][u >> 1][2 * (u & 1) + x] * a.scale_log2 : -INFINITY;
        }
        const uint32_t vidx4 = *reinterpret_cast<const uint32_t*>(pgp + g.off_vidx + gq * 4);
        float vrow[4] = {1.f, 1.f, 1.f, 1.f};
        if constexpr (TX) {
          const float4 vr = *reinterpret_cast<const float4*>(pgp + g.off_vrow + gq * 16);
          vrow[0] = vr.x; vrow[1] = vr.y; vrow[2] = vr.z; vrow[3] = vr.w;
        }
        const float4* vz4 = reinterpret_cast<const float4*>(pgp + g.off_vz) + gq;
        const float4 vz[4] = {vz4[0], vz4[8], vz4[16], vz4[24]};
        // the pattern of token gq + 8 tig, and the token's turn to add its weights to the pattern's (raw tokens have none)
        const int vi = (int)((vidx4 >> (8 * tig)) & 0xff);
        const bool aligned = vi < Pe;
        const unsigned alike = __match_any_sync(kFull, aligned ? vi : kRawIndex + 1 + lane);
        const int turn = aligned ? __popc(alike & ((1u << lane) - 1u)) : 32;
        const int turns = (int)__reduce_max_sync(kFull, aligned ? (unsigned)turn + 1u : 0u);
        // the largest V scale of token gq + 8 tig, and of the page
        float vmax;
        {
          const float4 v = reinterpret_cast<const float4*>(pgp + g.off_vs)[((tig >> 1) * 4 + (gq & 1) + 2 * (tig & 1)) * 4 + (gq >> 1)];
          vmax = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
        }
        const float page_vmax = fmaxf(__uint_as_float(__reduce_max_sync(kFull, __float_as_uint(vmax))), kVLeast);
        // ---- online softmax (base 2), per head over the 32 tokens
        float p0[4];  // narrow: p of this lane's four V columns' tokens
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          float pv[HPT][4], p[HPT][4], alpha[HPT], top[HPT], wfactor[HPT];
          bool same = true;
#pragma unroll
          for (int x = 0; x < HPT; ++x) {
            float pm = fmaxf(fmaxf(sc[j][x][0], sc[j][x][1]), fmaxf(sc[j][x][2], sc[j][x][3]));
            pm = fmaxf(pm, __shfl_xor_sync(kFull, pm, 4));
            pm = fmaxf(pm, __shfl_xor_sync(kFull, pm, 8));
            pm = fmaxf(pm, __shfl_xor_sync(kFull, pm, 16));
            const float m = fmaxf(mrun[j][x], pm), base = m == -INFINITY ? 0.f : m;
            alpha[x] = ex2(mrun[j][x] - base);
            mrun[j][x] = m;
#pragma unroll
            for (int u = 0; u < 4; u += 2) {
              float d0, d1;
              upk(add2(pk(sc[j][x][u], sc[j][x][u + 1]), pk(-base, -base)), d0, d1);
              p[x][u] = ex2(d0);  // (columns past the last head go along, unused)
              p[x][u + 1] = ex2(d1);
              pv[x][u] = TX ? p[x][u] * vrow[u] : p[x][u];
              pv[x][u + 1] = TX ? p[x][u + 1] * vrow[u + 1] : p[x][u + 1];
            }
            // (the page's largest scale stands for each token's until that is not good enough)
            top[x] = fmaxf(fmaxf(pv[x][0], pv[x][1]), fmaxf(pv[x][2], pv[x][3])) * page_vmax;
            same = same && alpha[x] == 1.0f && top[x] < vlim[j][x];
          }
          if (!__all_sync(kFull, same)) {
            bool unit_fits = true;
#pragma unroll
            for (int x = 0; x < HPT; ++x) {
              vtop[j][x] *= alpha[x];
              unit_fits = unit_fits && top[x] < vlim[j][x] && vtop[j][x] * (2 << 2 * kVRoom) >= vlim[j][x];
              wfactor[x] = alpha[x];
            }
            if (!__all_sync(kFull, unit_fits)) {
              // the units of the heads follow their largest products so far, as far as those still count
#pragma unroll
              for (int x = 0; x < HPT; ++x) {
                float most = vtop[j][x];
#pragma unroll
                for (int u = 0; u < 4; ++u) most = fmaxf(most, pv[x][u] * fmaxf(__shfl_sync(kFull, vmax, (lane & ~3) + u), kVLeast));
                most = fmaxf(most, __shfl_xor_sync(kFull, most, 4));
                most = fmaxf(most, __shfl_xor_sync(kFull, most, 8));
                most = fmaxf(most, __shfl_xor_sync(kFull, most, 16));
                const int old = exponent(vlim[j][x]), e = max(-100, min(100, exponent(most) + 1 + kVRoom));
                vlim[j][x] = pow2(e);
                vtop[j][x] = most;
                wfactor[x] *= exp2i(old - e);
              }
            }
#pragma unroll
            for (int x = 0; x < HPT; ++x) {
              const int hh = TH * j + HPT * tig + x;
              lrun[j][x] *= alpha[x];
#pragma unroll
              for (int u = 0; u < 4; ++u) zacc[j][x][u] *= alpha[x];
#pragma unroll
              for (int mt = 0; mt < 8; ++mt)
#pragma unroll
                for (int u = 0; u < 4; ++u)
                  if (!WIDE || (u & 1) == x) accv[j][mt][u] *= wfactor[x];
              for (int jj = gq; jj < Pe; jj += 8) Ww[jj * NH + w_place(hh)] *= alpha[x];
            }
            __syncwarp();
          }
          {
            float w[HPT][4];  // of token gq + 8 tig: the weights of the tile's heads x, x + HPT, ...
#pragma unroll
            for (int x = 0; x < HPT; ++x) {
#pragma unroll
              for (int u = 0; u < 4; ++u) w[x][u] = pv[x][u];
              quad_transpose(w[x], tig);
            }
            float4* row = reinterpret_cast<float4*>(Ww + (aligned ? vi : 0) * NH + TH * j);
            auto add = [&](int r) {
              if (turn == r) {
#pragma unroll
                for (int x = 0; x < HPT; ++x) {
                  const float4 y = row[x];
                  row[x] = make_float4(y.x + w[x][0], y.y + w[x][1], y.z + w[x][2], y.w + w[x][3]);
                }
              }
            };
            add(0);
#pragma unroll 1
            for (int r = 1; r < turns; ++r) {
              __syncwarp();
              add(r);
            }
          }
#pragma unroll
          for (int x = 0; x < HPT; ++x) {
            const int hh = TH * j + HPT * tig + x;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              lrun[j][x] += p[x][u];
              zacc[j][x][0] = fmaf(pv[x][u], vz[u].x, zacc[j][x][0]);
              zacc[j][x][1] = fmaf(pv[x][u], vz[u].y, zacc[j][x][1]);
              zacc[j][x][2] = fmaf(pv[x][u], vz[u].z, zacc[j][x][2]);
              zacc[j][x][3] = fmaf(pv[x][u], vz[u].w, zacc[j][x][3]);
            }
            // p to the lanes of the V columns, scaled; tokens 8..15 of each 16 are columns with a factor of their own
            const float f0 = pow2_over(kVTop, vlim[j][x]), f8 = f0 / Code<BITS>::kCol;
            if constexpr (WIDE) {
              float y[4];
              upk(mul2(pk(pv[x][0], pv[x][1]), pk(f0, f8)), y[0], y[1]);
              upk(mul2(pk(pv[x][2], pv[x][3]), pk(f0, f8)), y[2], y[3]);
              *reinterpret_cast<float4*>(pex + hh * kPexRow + gq * 4) = make_float4(y[0], y[1], y[2], y[3]);
            } else {
              // Lane (head, part) wants tokens 2 tig and 2 tig + 1 (+ 8) of the page's half `part`: u = 2 part, 2 part + 1.
              // Even token rows offer the halves in one order, odd rows in the other, so that both exchanges serve both
              // parts; part 1 gets 2 tig + 1 first (and reads its scales in that order: no bank conflict with part 0).
              const float y0 = (part ? pv[x][2] : pv[x][0]) * f0, y1 = (part ? pv[x][3] : pv[x][1]) * f8;
              const float z0 = (part ? pv[x][0] : pv[x][2]) * f0, z1 = (part ? pv[x][1] : pv[x][3]) * f8;
              const int src = 8 * tig + (gq >> 1) + 4 * part;  // row 2 tig + part
              p0[0] = __shfl_sync(kFull, y0, src);
              p0[1] = __shfl_sync(kFull, z0, src ^ 4);
              p0[2] = __shfl_sync(kFull, y1, src);
              p0[3] = __shfl_sync(kFull, z1, src ^ 4);
            }
          }
        }
        if constexpr (WIDE) __syncwarp();

        // ---- V: p-weighted codes
        uint32_t vw[WPL];
#pragma unroll
        for (int c = 0; c < WPL / 4; ++c) {
          const uint4 t = reinterpret_cast<const uint4*>(pgp + g.off_vc + c * 512)[lane];
          vw[4 * c] = t.x; vw[4 * c + 1] = t.y; vw[4 * c + 2] = t.z; vw[4 * c + 3] = t.w;
        }
        const float4* vs4 = reinterpret_cast<const float4*>(pgp + g.off_vs) + tig;
        if constexpr (!WIDE) {
          const float4 s0 = vs4[5 * part * 4], s1 = vs4[(3 * part + 1) * 4], s2 = vs4[(5 * part + 2) * 4], s3 = vs4[(3 * part + 3) * 4];
          const unsigned long long q0 = pk(p0[0], p0[0]), q1 = pk(p0[1], p0[1]), q2 = pk(p0[2], p0[2]), q3 = pk(p0[3], p0[3]);
#pragma unroll
          for (int gp = 0; gp < 2; ++gp) {  // two channel groups at a time: their scales are neighbours
            uint32_t own0[2], own1[2], lo0[2], lo1[2];
            split2x2(mul2(q0, gp ? pk(s0.z, s0.w) : pk(s0.x, s0.y)), mul2(q1, gp ? pk(s1.z, s1.w) : pk(s1.x, s1.y)), own0, lo0);
            split2x2(mul2(q2, gp ? pk(s2.z, s2.w) : pk(s2.x, s2.y)), mul2(q3, gp ? pk(s3.z, s3.w) : pk(s3.x, s3.y)), own1, lo1);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t got0 = __shfl_xor_sync(kFull, lo0[x], 4), got1 = __shfl_xor_sync(kFull, lo1[x], 4);
#pragma unroll
              for (int ks = 0; ks < 2; ++ks) {
                const uint32_t b0 = part == ks ? own0[x] : got0, b1 = part == ks ? own1[x] : got1;
#pragma unroll
                for (int mh = 0; mh < 2; ++mh) {
                  const int mt = (2 * gp + x) * 2 + mh;
                  uint32_t f[4];
                  frag16<BITS>(BITS == 2 ? vw[mt] : vw[mt * 2 + ks], ks, f, ks == 1);
                  mma_f16(accv[0][mt], f, b0, b1);
                }
              }
            }
          }
        } else {
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) {
            const float4 s0 = vs4[(ks * 4 + 0) * 4], s1 = vs4[(ks * 4 + 1) * 4], s2 = vs4[(ks * 4 + 2) * 4],
                         s3 = vs4[(ks * 4 + 3) * 4];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              const float* prow = pex + (TH * j + gq) * kPexRow + 2 * ks;
              const float2 pa = *reinterpret_cast<const float2*>(prow + (2 * tig) * 4);
              const float2 pb = *reinterpret_cast<const float2*>(prow + (2 * tig + 1) * 4);
              const unsigned long long q0 = pk(pa.x, pa.x), q1 = pk(pb.x, pb.x), q2 = pk(pa.y, pa.y), q3 = pk(pb.y, pb.y);
#pragma unroll
              for (int gp = 0; gp < 2; ++gp) {
                uint32_t bh0[2], bh1[2], bl0[2], bl1[2];
                split2x2(mul2(q0, gp ? pk(s0.z, s0.w) : pk(s0.x, s0.y)), mul2(q1, gp ? pk(s1.z, s1.w) : pk(s1.x, s1.y)), bh0, bl0);
                split2x2(mul2(q2, gp ? pk(s2.z, s2.w) : pk(s2.x, s2.y)), mul2(q3, gp ? pk(s3.z, s3.w) : pk(s3.x, s3.y)), bh1, bl1);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
#pragma unroll
                  for (int mh = 0; mh < 2; ++mh) {
                    const int mt = (2 * gp + x) * 2 + mh;
                    uint32_t f[4];
                    frag16<BITS>(BITS == 2 ? vw[mt] : vw[mt * 2 + ks], ks, f);
                    mma_f16(accv[j][mt], f, bh0[x], bh1[x]);
                    mma_f16(accv[j][mt], f, bl0[x], bl1[x]);
                  }
                }
              }
            }
          }
        }
      }
      __syncwarp();
      // refill this stage with the entry kStages ahead
      const int nxt = i + kStages;
      if ((nxt & 31) == 0) ids = load_ids(nxt);
      const int phys = __shfl_sync(kFull, ids, nxt & 31);
      if (nxt < my_n) {
        skips = (skips & ~(1u << st)) | (phys < 0 ? 1u << st : 0u);
        tail_st = (tail_st & ~(1u << st)) | ((tails >> (nxt & 31) & 1) << st);
        if (lane == 0) {
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          fetch(st, phys);
        }
      }
      __syncwarp();
    }
    if (stuck_at >= 0) {
      if (lane == 0) set_status(g.status, KVQ_DEV_TIMEOUT);
      // the copies already issued land before the shared memory is reused or released
      for (int i = stuck_at; i < my_n && i < stuck_at + kStages; ++i) (void)mbar_wait(&bars[i % kStages], (i / kStages) & 1);
    }

    // ---- merge the warps and write the partials
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int x = 0; x < HPT; ++x)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          lrun[j][x] += __shfl_xor_sync(kFull, lrun[j][x], o);
#pragma unroll
          for (int u = 0; u < 4; ++u) zacc[j][x][u] += __shfl_xor_sync(kFull, zacc[j][x][u], o);
        }
    __syncthreads();  // every warp is done with its ring
    constexpr int MO = merge_row(WIDE);
    float* mo = reinterpret_cast<float*>(smem);  // [kNW][NH][MO]
    float* mm = mo + kNW * NH * MO;              // [kNW][NH] max
    float* ml = mm + kNW * NH;                   // [kNW][NH] sum
    float* mz = ml + kNW * NH;                   // [kNW][NH][4]
    float* wc = mo + sp.wc;                      // [P, to whole kMergeRows][NH] merged pattern weights
    float* fsh = mo + sp.fsh;                    // [NH][kNW] warp weights
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int x = 0; x < HPT; ++x) {
        const int hh = TH * j + HPT * tig + x;
        const float f0 = vlim[j][x] * pow2(24 - kVTop), f8 = f0 / Code<BITS>::kRow;
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
          mo[(warp * NH + hh) * MO + 16 * mt + gq] = (WIDE ? accv[j][mt][x] : accv[j][mt][0] + accv[j][mt][1]) * f0;
          mo[(warp * NH + hh) * MO + 16 * mt + gq + 8] = (WIDE ? accv[j][mt][2 + x] : accv[j][mt][2] + accv[j][mt][3]) * f8;
        }
        if (gq == 0) {
          mm[warp * NH + hh] = mrun[j][x];
          ml[warp * NH + hh] = lrun[j][x];
#pragma unroll
          for (int u = 0; u < 4; ++u) mz[(warp * NH + hh) * 4 + u] = zacc[j][x][u];
        }
      }
    // M_V values of this thread's channel, the first of them over the merge of the weights
    const float* mv = g.vpat + sh * P * kD + threadIdx.x;
    float mval[kMvAhead];
#pragma unroll
    for (int j = 0; j < kMvAhead; ++j) mval[j] = __ldg(mv + (size_t)min(j, Pe - 1) * kD);
    __syncthreads();
    {
      // the threads of a head are NH apart; each makes the weights of the warps for itself
      const int hh = threadIdx.x % NH;
      float M = -INFINITY, Ls = 0.f, f[kNW];
#pragma unroll
      for (int w = 0; w < kNW; ++w) M = fmaxf(M, mm[w * NH + hh]);
#pragma unroll
      for (int w = 0; w < kNW; ++w) {
        f[w] = mm[w * NH + hh] == -INFINITY ? 0.f : ex2(mm[w * NH + hh] - M);
        Ls += f[w] * ml[w * NH + hh];
      }
      if (threadIdx.x < NH) {
        *reinterpret_cast<float4*>(fsh + hh * kNW) = make_float4(f[0], f[1], f[2], f[3]);
        if (direct) sum_ml[hh].x = 1.0f / sum_or_one(Ls);
        else if (in_smem) sum_ml[hh] = make_float2(M, Ls);
        else if (hh < Gq) reinterpret_cast<float2*>(a.part_ml)[row0 + (int64_t)hh * a.nsplit] = make_float2(M, Ls);
      }
      const int rows = (Pe + kMergeRows - 1) / kMergeRows * kMergeRows;
#pragma unroll 4
      for (int jj = threadIdx.x / NH; jj < rows; jj += kNW * 32 / NH) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kNW; ++w) s = fmaf(f[w], Wall[(w * P + min(jj, Pe - 1)) * NH + w_place(hh)], s);
        wc[jj * NH + hh] = jj < Pe ? s : 0.f;
      }
    }
    __syncthreads();
    // thread = channel; each M_V value is read once per CTA
    {
      const int c = threadIdx.x;
      unsigned long long o2[NH / 2];  // two heads at a time
#pragma unroll
      for (int i = 0; i < NH / 2; ++i) o2[i] = 0ull;
      for (int j0 = 0; j0 < Pe; j0 += kMvAhead) {
        if (j0 > 0) {
#pragma unroll
          for (int j = 0; j < kMvAhead; ++j) mval[j] = __ldg(mv + (size_t)min(j0 + j, Pe - 1) * kD);
        }
#pragma unroll
        for (int j = 0; j < kMvAhead; j += kMergeRows) {
          if (j0 + j >= Pe) break;
#pragma unroll
          for (int e = 0; e < kMergeRows; ++e) {  // (rows past the last one have the weight 0)
            const ulonglong2* w = reinterpret_cast<const ulonglong2*>(wc + (j0 + j + e) * NH);
            const unsigned long long m2 = pk(mval[j + e], mval[j + e]);
#pragma unroll
            for (int i = 0; i < NH / 4; ++i) {
              const ulonglong2 x = w[i];
              o2[2 * i] = fma2(x.x, m2, o2[2 * i]);
              o2[2 * i + 1] = fma2(x.y, m2, o2[2 * i + 1]);
            }
          }
        }
      }
      float o[NH];
#pragma unroll
      for (int i = 0; i < NH / 2; ++i) upk(o2[i], o[2 * i], o[2 * i + 1]);
#pragma unroll
      for (int i = 0; i < NH; ++i) {  // (heads past the last one go along, unused)
        const float4 f = *reinterpret_cast<const float4*>(fsh + i * kNW);
        const float fw[kNW] = {f.x, f.y, f.z, f.w};
#pragma unroll
        for (int w = 0; w < kNW; ++w) o[i] = fmaf(fw[w], mo[(w * NH + i) * MO + c] + mz[(w * NH + i) * 4 + (c >> 5)], o[i]);
      }
      if (direct) {
        bool bad = false;
#pragma unroll
        for (int i = 0; i < NH; ++i) {
          if (i < Gq) {
            const float v = o[i] * sum_ml[i].x;
            bad = bad || !in_range(g, v);
            a.out[((int64_t)b * a.Hq + (int64_t)h * Gq + i) * kD + c] =
                g.dtype == KVQ_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
          }
        }
        if (bad) set_status(g.status, KVQ_DEV_RANGE);
        return;
      }
#pragma unroll
      for (int i = 0; i < NH; ++i) {
        if (i < Gq) {
          if (in_smem) sum_o[i * kD + c] = o[i];
          else a.part_o[(row0 + (int64_t)i * a.nsplit) * kD + c] = o[i];
        }
      }
    }
  } else {
    // nothing of the list falls to this CTA
    for (int hh = threadIdx.x; hh < Gq; hh += blockDim.x) {
      if (in_smem) sum_ml[hh] = make_float2(-INFINITY, 0.f);
      else reinterpret_cast<float2*>(a.part_ml)[row0 + (int64_t)hh * a.nsplit] = make_float2(-INFINITY, 0.f);
    }
  }

  // ---- one split, or a cluster of them: the sums stay in shared memory, and CTA r of the group finishes heads r, r + nsplit, ...
  if (in_smem) {
    if (a.nsplit > 1) cluster_sync(); else __syncthreads();
    for (int hh = split + a.nsplit * warp; hh < Gq; hh += a.nsplit * kNW) {
      const float* row = sum_o + hh * kD + 4 * lane;
      float2 x = make_float2(-INFINITY, 0.f);
      if (lane < a.nsplit) x = a.nsplit > 1 ? peer_f2(sum_ml + hh, lane) : sum_ml[hh];
      float4 y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = a.nsplit > 1 ? peer_f4(row, min(i, a.nsplit - 1)) : *reinterpret_cast<const float4*>(row);
      const float M = warp_max(x.x);
      const float fs = x.x == -INFINITY ? 0.f : ex2(x.x - M), Ls = warp_sum(fs * x.y);
      float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // (a split without entries has written no row: its weight is 0, whatever is read; so past the last one)
        const float f = __shfl_sync(kFull, fs, i);
        o[0] += f == 0.f ? 0.f : f * y[i].x;
        o[1] += f == 0.f ? 0.f : f * y[i].y;
        o[2] += f == 0.f ? 0.f : f * y[i].z;
        o[3] += f == 0.f ? 0.f : f * y[i].w;
      }
      finish_head(g, o, sum_or_one(Ls), g.vcol + sh * kD, a.out + ((int64_t)b * a.Hq + (int64_t)h * Gq + hh) * kD, lane);
    }
    if (a.nsplit > 1) cluster_sync();  // the others' reads of this CTA's sums are done
    return;
  }

  // ---- the CTA that completes a group merges its splits and writes the output
  __shared__ int last;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    last = arrive_last(a.counters, (int)grp, a.counter_sharing, a.nsplit);
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  for (int hh = warp; hh < Gq; hh += kNW) {
    const int64_t row = (int64_t)b * a.Hq + (int64_t)h * Gq + hh, base = row * a.nsplit;
    uint16_t* outp = a.out + row * kD;
    const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + base;
    float2 x = make_float2(-INFINITY, 0.f);  // of split lane (the first 32)
    if (lane < a.nsplit) x = __ldcg(ml + lane);
    float M = x.x;
    for (int s = 32 + lane; s < a.nsplit; s += 32) M = fmaxf(M, __ldcg(ml + s).x);
    M = warp_max(M);
    float Ls = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int s0 = 0; s0 < a.nsplit; s0 += 32) {
      if (s0 > 0) x = s0 + lane < a.nsplit ? __ldcg(ml + s0 + lane) : make_float2(-INFINITY, 0.f);
      const float fs = x.x == -INFINITY ? 0.f : ex2(x.x - M);
      Ls = fmaf(fs, x.y, Ls);
      const int n = min(32, a.nsplit - s0);
      for (int i0 = 0; i0 < n; i0 += 8) {
        float4 y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          y[i] = __ldcg(reinterpret_cast<const float4*>(a.part_o + (base + min(s0 + i0 + i, a.nsplit - 1)) * kD) + lane);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // (a split without entries has written no row: its weight is 0, whatever is read; so past the last one)
          const float f = __shfl_sync(kFull, fs, i0 + i);
          o[0] += f == 0.f ? 0.f : f * y[i].x;
          o[1] += f == 0.f ? 0.f : f * y[i].y;
          o[2] += f == 0.f ? 0.f : f * y[i].z;
          o[3] += f == 0.f ? 0.f : f * y[i].w;
        }
      }
    }
    Ls = warp_sum(Ls);
    finish_head(g, o, sum_or_one(Ls), g.vcol + sh * kD, outp, lane);
  }
}

template <int BITS, int NT, bool WIDE, bool TX>
cudaError_t launch_one(const Geom& g, const PagesArgs& a, cudaStream_t st) {
  const int smem = pages_smem((int)g.sub_bytes, NT, WIDE, g.P).total;
  // the kernel's shared-memory limit is raised when a call first needs more on this device
  static std::atomic<int> allowed[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || allowed[dev].load(std::memory_order_relaxed) < smem) {
    e = cudaFuncSetAttribute(decode_pages_kernel<BITS, NT, WIDE, TX>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) allowed[dev].store(kMaxSmem, std::memory_order_relaxed);
  }
  if (!a.clustered) {
    decode_pages_kernel<BITS, NT, WIDE, TX><<<dim3(a.nsplit, g.H, g.B), kNW * 32, smem, st>>>(g, a);
    return cudaGetLastError();
  }
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = a.nsplit;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.nsplit, g.H, g.B);
  cfg.blockDim = dim3(kNW * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_pages_kernel<BITS, NT, WIDE, TX>, g, a);
}

template <int BITS, bool TX>
cudaError_t launch_bits(const Geom& g, const PagesArgs& a, cudaStream_t st) {
  if (a.Gq <= 4) return launch_one<BITS, 1, false, TX>(g, a, st);
  if (a.Gq <= 8) return launch_one<BITS, 1, true, TX>(g, a, st);
  return launch_one<BITS, 2, true, TX>(g, a, st);
}

}  // namespace

// Splits of the list: 1, 2, 4 or 8 (a cluster, whose sums meet in shared memory), or 16 and more (through the workspace).
// Model, in units of the time a lone CTA takes for a page per warp (1.3 us on one B200): k CTAs on an SM at once take
// max(1, 0.48 k) for a page per warp and 5 + 1.25 (k - 1) before and after the loop; the busiest SM runs its CTAs `occ` at a
// time; merging costs a little per split, and more per head through the workspace (8 groups of 64 pages, 8 splits and 16:
// 10.7 and 10.4 us with 4 heads a group, 13.4 and 14.4 with 8, 18.6 and 21.2 with 16).  Measured best with 4, 8 and 16 heads a
// group at 64 listed pages: for 8 groups 16, 8 and 8 splits (1: 30, 41 and 67 us; 64: 17, 34 and 52), for 64 groups 4, for 128
// groups 2, for 1024 groups 1; at 256 pages for 16 groups 16 (8: 23, 32 and 52 us for 17.5, 24 and 39); at 128 pages for 256
// groups 1 (with 4 heads 2: 62 us for 68); at 452 pages for 3 groups 47.  The model's choice is the best or within a tenth of it.
// The budget is rounded up to eight sizes per power of two first, so that the largest choice of all budgets up to one is
// found by trying few.
static int64_t rounded_budget(int64_t budget) {
  int64_t step = 1;
  while (16 * step < budget) step *= 2;
  return (budget + step - 1) / step * step;
}
int decode_pages_splits(const Geom& g, int Gq, int budget_, int num_sms) {
  const int64_t budget = rounded_budget(budget_);
  const int64_t units = std::max<int64_t>(1, (int64_t)g.B * g.H), sms = std::max(1, num_sms);
  const bool wide = Gq > 4;
  const int by_regs = !wide ? 4 : Gq <= 8 ? 3 : 2;
  const int by_smem = 233472 / (pages_smem((int)g.sub_bytes, Gq > 8 ? 2 : 1, wide, g.P).total + 1024 + 128);
  const int64_t occ = std::max(1, std::min(by_regs, by_smem));
  // (through the workspace only where the groups' counters hold the splits, which no group count past 256 wants)
  const int most = (int)std::min<int64_t>(most_arrivals(counter_sharing(units)) >= 64 ? 64 : 8, budget);
  auto round = [&](int64_t k, int64_t pages) { return 5.0 + 1.25 * (k - 1) + pages * std::max(1.0, 0.48 * k); };
  int best = 1;
  double best_cost = 1e300;
  for (int ns = 1; ns <= most; ns = ns < 16 ? 2 * ns : ns + ns / 8) {
    const int64_t per_sm = (units * ns + sms - 1) / sms, full = per_sm / occ, rem = per_sm % occ;
    const int64_t pages = ((budget + ns - 1) / ns + kNW - 1) / kNW;
    const double cost = full * round(occ, pages) + (rem ? round(rem, pages) : 0.0) + 0.05 * ns + (ns >= 16 ? 0.1 * Gq : 0.0);
    if (cost < best_cost * (1.0 - 1e-9)) { best_cost = cost; best = ns; }
  }
  return best;
}

int decode_pages_most_splits(const Geom& g, int Gq, int budget, int num_sms) {
  int most = 1;
  for (int64_t b = 1; b <= rounded_budget(budget); b = rounded_budget(b + 1))
    most = std::max(most, decode_pages_splits(g, Gq, (int)std::min<int64_t>(b, budget), num_sms));
  return most;
}

static bool meet_in_clusters(int nsplit) { return nsplit == 2 || nsplit == 4 || nsplit == 8; }

// Arrival counters, then the partials of the splits that meet in the workspace.
size_t decode_pages_workspace(const Geom& g, int Hq, int nsplit) {
  return kCounterBytes + (size_t)g.B * Hq * nsplit * (2 + kD) * sizeof(float);
}
size_t decode_pages_need(const Geom& g, int Hq, int nsplit) {
  return nsplit == 1 || meet_in_clusters(nsplit) ? (size_t)kCounterBytes : decode_pages_workspace(g, Hq, nsplit);
}

cudaError_t launch_decode_pages(const Geom& g0, PagesArgs a, void* ws, cudaStream_t st) {
  Geom g = g0;
  g.wait_limit = page_wait_limit(g0.wait_limit);
  // 64 groups of 64 pages, 4 splits: 16.9 us as clusters, 18.0 us through the workspace; 8 groups, 8 splits: 10.7 / 11.6 us
  a.clustered = meet_in_clusters(a.nsplit);
  a.counters = (unsigned*)ws;
  a.counter_sharing = counter_sharing((int64_t)g.B * g.H);
  // the rows of 128 first: they are read 16 bytes at a time, which an odd number of (max, sum) pairs before them would not allow
  a.part_o = (float*)((uint8_t*)ws + kCounterBytes);
  a.part_ml = a.part_o + kD * (size_t)g.B * a.Hq * a.nsplit;
  if (g.tx) return g.bits == 2 ? launch_bits<2, true>(g, a, st) : launch_bits<4, true>(g, a, st);
  return g.bits == 2 ? launch_bits<2, false>(g, a, st) : launch_bits<4, false>(g, a, st);
}

}  // namespace kvq
