// q8_internal.h -- declarations shared by the translation units of the 8-bit
// block-scaled cache.  Not part of the public ABI (include/tq.h is).
#pragma once
#include "tq_internal.h"

namespace tq {

// The cache of one layer: K and V codes [B][Hkv][capacity][d] and scales
// [B][Hkv][ceil(capacity / block)].
struct Q8Cache {
  uint8_t *k_codes, *v_codes;
  float *k_scales, *v_scales;
  int64_t capacity;
  int B, Hkv, d, block;
  int e4m3;  // 0: int8 codes
  __host__ __device__ int64_t n_blocks() const { return (capacity + block - 1) / block; }
};

struct Q8WriteArgs {
  Q8Cache c;
  const void *k, *v;  // [B][Hkv][n][d]
  int bf16, n;
  const int32_t* pos;      // [B] first row, or with pos_is_ctx: length including the row
  const int32_t* n_valid;  // [B] or NULL
  int pos_is_ctx, max_ctx; // row = clamp(pos[b], 0, max_ctx) - 1 (a length of 0 writes nothing)
};

struct Q8ReadArgs {
  Q8Cache c;
  void *k, *v;  // [B][Hkv][n][d]
  int bf16, n;
  const int32_t *pos, *n_valid;
};

// The kernel of an attention call, and what a CTA of the tensor-memory one holds
// (q8_tc.cu).
enum Q8Mode : int { kQ8Warps, kQ8TwoRows, kQ8TwoStreams, kQ8OneStream };

// How one attention call is split: rows of a kv head (query tokens x query
// heads per kv head) in tiles, the context in chunks.
struct Q8Plan {
  int row_tile;     // rows of one work item
  int tiles;        // ceil(n * G / row_tile)
  int chunk;        // context tokens of one work item
  int n_chunks;     // ceil(max_ctx / chunk)
  int parts;        // partial results of one work item
  int n_parts;      // n_chunks * parts; 1 = items write the output themselves
  int part_stride;  // floats of one partial: d + 4
  size_t header_bytes, ws_bytes;
  Q8Mode mode;
};

struct Q8AttendArgs {
  Q8Cache c;
  const void* q;  // [B][Hq][n][d]
  int q_bf16, Hq, n;
  const int32_t *ctx_lens, *q_lens;  // q_lens NULL: n for every sequence
  int max_ctx;
  float attn_scale;
  void* out;  // [B][Hq][n][d]
  int out_bf16;
  float* lse;  // [B][Hq][n][2] or NULL
  void* workspace;
  Q8Plan plan;
  int test_starve;
};

bool q8_head_dim_supported(int d);
bool make_q8_plan(int B, int Hq, int Hkv, int d, int n, int max_ctx, bool bf16, Q8Plan* plan);
cudaError_t launch_q8_append(const Q8WriteArgs& a, cudaStream_t stream);
cudaError_t launch_q8_read(const Q8ReadArgs& a, cudaStream_t stream);
int q8_split_slots(int d, int row_tile);  // work items of the split kernel resident on the GPU
cudaError_t launch_q8_split(const Q8AttendArgs& a, cudaStream_t stream);
int q8_tc_tile_tokens(int d);             // tokens of one step of the tensor-memory kernel
cudaError_t launch_q8_tc(const Q8AttendArgs& a, cudaStream_t stream);
cudaError_t launch_q8_merge(const Q8AttendArgs& a, cudaStream_t stream);

#ifdef __CUDACC__
// The part of a sequence that its query rows see: query i sits at position
// ctx - q_len + i and attends the rows up to it.
struct Q8Seq {
  int ctx, q_len;
  bool bad;  // a length outside its range (clamped)
  __device__ __forceinline__ Q8Seq(const Q8AttendArgs& a, int b) {
    const int c0 = a.ctx_lens[b], n0 = a.q_lens ? a.q_lens[b] : a.n;
    ctx = min(max(c0, 0), a.max_ctx);
    q_len = min(max(n0, 0), a.n);
    bad = ctx != c0 || q_len != n0;
  }
  // cache rows that query i attends (0 when it sits before the first row)
  __device__ __forceinline__ int limit(int i) const { return max(0, ctx - q_len + i + 1); }
};
#endif

}  // namespace tq
