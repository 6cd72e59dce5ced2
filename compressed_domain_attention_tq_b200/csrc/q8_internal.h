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
  int fill;
};

// The kernel of an attention call, and what a CTA of the tensor-memory one holds
// (q8_tc.cu).
enum Q8Mode : int { kQ8Warps, kQ8TwoRows, kQ8TwoStreams, kQ8OneStream };

// How one attention call is split.  A unit is one tile of rows (query tokens x query heads
// of a kv head) of one kv head; units are numbered from the last tile, which attends most.
// The first `whole` ones are one work item each and write their outputs; the others, too few
// to fill the GPU once more, are split into chunks of the context, whose partial results
// the merge joins.
struct Q8Plan {
  int row_tile;     // rows of one work item
  int tiles;        // ceil(n * G / row_tile)
  int whole, units;
  int chunk;        // context tokens of one work item of a split unit
  int n_chunks;     // ceil(max_ctx / chunk)
  int parts;        // partial results of one work item
  int n_parts;      // n_chunks * parts: of a row of a split unit
  int part_stride;  // floats of one partial: d + 4
  size_t header_bytes, ws_bytes;
  Q8Mode mode;
  int64_t items() const { return whole + (int64_t)(units - whole) * n_chunks; }
  int64_t split_rows() const { return (int64_t)(units - whole) * row_tile; }
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
int q8_split_per_sm(int d, int row_tile);  // work items of the split kernel resident on an SM
cudaError_t launch_q8_split(const Q8AttendArgs& a, cudaStream_t stream);
int q8_tc_tile_tokens(int d);             // tokens of one step of the tensor-memory kernel
cudaError_t launch_q8_tc(const Q8AttendArgs& a, cudaStream_t stream);
cudaError_t launch_q8_merge(const Q8AttendArgs& a, cudaStream_t stream);

#ifdef __CUDACC__
// The unit, and the chunk of it, that work item `id` is.
struct Q8Item {
  int unit, chunk_id, tile, bh, b, hk, G, rows, row0;
  bool split;
  __device__ __forceinline__ Q8Item(const Q8AttendArgs& a, int id) {
    const int e = id - a.plan.whole;
    split = e >= 0;
    place(a, split ? a.plan.whole + e / a.plan.n_chunks : id);
    chunk_id = split ? e % a.plan.n_chunks : 0;
  }
  __device__ __forceinline__ Q8Item() {}
  __device__ __forceinline__ void place(const Q8AttendArgs& a, int u) {
    unit = u;
    const int heads = a.c.B * a.c.Hkv;
    tile = a.plan.tiles - 1 - u / heads;
    bh = u % heads;
    b = bh / a.c.Hkv;
    hk = bh % a.c.Hkv;
    G = a.Hq / a.c.Hkv;
    rows = a.n * G;
    row0 = tile * a.plan.row_tile;
  }
  // query token and output row of the tile's row r
  __device__ __forceinline__ int token(int r) const { return (row0 + r) / G; }
  __device__ __forceinline__ int64_t out_row(const Q8AttendArgs& a, int r) const {
    return ((int64_t)b * a.Hq + hk * G + (row0 + r) % G) * a.n + token(r);
  }
  // partial p of row r
  __device__ __forceinline__ float* part(const Q8AttendArgs& a, int r, int p) const {
    return reinterpret_cast<float*>(static_cast<unsigned char*>(a.workspace) + a.plan.header_bytes) +
           (((int64_t)(unit - a.plan.whole) * a.plan.row_tile + r) * a.plan.n_parts + p) * a.plan.part_stride;
  }
};

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
