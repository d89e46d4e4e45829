// Internal host-side interfaces between the C-ABI layer (kvq_api.cu) and the
// kernel translation units.  Not installed, not part of the ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kvq {

struct Geom;

// quantize-append (kvq_append.cu)
size_t append_workspace(const Geom& g);
cudaError_t launch_append(const Geom& g, const void* k_new, const void* v_new, int n_new, void* ws, cudaStream_t st);

// decode attention (kvq_decode.cu)
int decode_num_splits(const Geom& g, int Hq, int num_sms);
size_t decode_workspace(const Geom& g, int Hq, int nsplit);
cudaError_t launch_decode(const Geom& g, const void* q, int Hq, float sm_scale, float* out, void* ws, int nsplit,
                          cudaStream_t st);
cudaError_t launch_decode_mma(const Geom& g, const void* q, int Hq, float scale_log2, int nsplit, float* ml,
                              float* o, int* arrivals, float* out, cudaStream_t st);
size_t decode_mma_smem(const Geom& g, int Hq);
// decode step: one-token append + decode in one launch (the workspace's counters reset themselves)
size_t step_workspace(const Geom& g, int Hq, int nsplit);
cudaError_t launch_decode_step(const Geom& g, const void* k_new, const void* v_new, const void* q, int Hq,
                               float sm_scale, float* out, void* ws, int nsplit, cudaStream_t st);
cudaError_t launch_decode_step_mma(const Geom& g, const void* k_new, const void* v_new, const void* q, int Hq,
                                   float scale_log2, int nsplit, float* ml, float* o, int* arrivals, int* seqcnt,
                                   float* out, cudaStream_t st);
int decode_mma_splits(const Geom& g, int Hq, int num_sms);

uint32_t page_wait_limit(uint32_t dflt);

// attention over chosen pages (kvq_decode_pages.cu)
struct PagesArgs {
  const uint16_t* q;
  int Hq, Gq;
  float scale_log2;
  const int32_t* list;      // [B][H][budget]
  const int32_t* list_len;  // [B][H]
  int budget, nsplit, clustered;
  uint16_t* out;
  float* part_ml;
  float* part_o;
  unsigned* counters;
  int counter_sharing;
};
int decode_pages_splits(const Geom& g, int Gq, int budget, int num_sms);
int decode_pages_most_splits(const Geom& g, int Gq, int budget, int num_sms);  // of all budgets up to this one
size_t decode_pages_workspace(const Geom& g, int Hq, int nsplit);
size_t decode_pages_need(const Geom& g, int Hq, int nsplit);  // what a call with so many splits uses of it
cudaError_t launch_decode_pages(const Geom& g, PagesArgs a, void* ws, cudaStream_t st);

// page bounds and page selection (kvq_bounds.cu)
cudaError_t launch_page_bounds(const Geom& g, const void* k_new, int n_new, void* bounds, cudaStream_t st);
struct SelectArgs {
  const uint16_t* q;
  int Gq;
  const uint16_t* bounds;
  int budget, sink, recent;
  int32_t* list;
  int32_t* list_len;
  unsigned* counters;
  uint32_t* keys;
  int nsplit, counter_sharing;
  float minus_zero;
};
size_t select_workspace(const Geom& g);
cudaError_t launch_select(const Geom& g, SelectArgs a, void* ws, int num_sms, cudaStream_t st);

// page tables and slot maps (kvq_plan.cu)
struct PlanArgs {
  const int32_t* new_len;
  const int32_t* free_pages;
  int32_t free_cap;
  const int32_t* free_count;
  int32_t* free_left;
  int32_t* cu;
  int64_t* slot_map;
  int32_t* positions;
  int32_t* seq_ids;
  int64_t max_tokens;
  int32_t* ws;
};
size_t plan_workspace(const Geom& g);
cudaError_t launch_plan(const Geom& g, const PlanArgs& a, int num_sms, cudaStream_t st);

// norms and rotation (kvq_rope.cu)
struct RopeRows {
  const void* in;
  void* out;
  const void* weight;
  int heads;
  int64_t in_tok, in_head, out_tok, out_head;
};
struct RopeArgs {
  RopeRows rows[3];  // queries, keys, values
  const int32_t* pos;
  const float* inv_freq;
  int64_t tokens;
  int rot, parts;  // parts: warps a token's heads are dealt to
  float eps;
};
cudaError_t launch_norm_rope(const RopeArgs& a, int dtype, bool interleaved, int num_sms, cudaStream_t st);

// dequantize (kvq_dequant.cu)
cudaError_t launch_dequant(const Geom& g, int seq, int start, int count, float* k_out, float* v_out,
                           cudaStream_t st);

// pattern mining (kvq_mine.cu)
struct MineArgs {
  const void* x;
  int dtype;
  int64_t n;
  int sets, heads;
  int64_t tok_stride, head_stride, set_stride;
  int P, iters, transform;
  float* patterns;
  float* colscale;
  int32_t* assign;
};
size_t mine_workspace(int64_t n, int sets, int heads, int P, int transform);

// Tiled TMA tensor map (cuTensorMapEncodeTiled through the runtime's driver entry point; loads
// past the end read as zeros).  kvq_mine.cu.
cudaError_t encode_tiled_map(CUtensorMap* map, CUtensorMapDataType dt, int rank, const void* base,
                             const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box,
                             CUtensorMapSwizzle swz);

cudaError_t launch_mine(const MineArgs& a, void* ws, size_t ws_bytes, cudaStream_t st);

}  // namespace kvq
