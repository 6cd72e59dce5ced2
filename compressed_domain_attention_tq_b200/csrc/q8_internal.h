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
// The first `whole` ones are one work item each and write their outputs.  The others are
// split into chunks of the context, whose partial results the merge joins: where there are
// whole units, into n_chunks of `chunk` tokens each; where there are none, into chunks of a
// length that the kernels work out from the sequences' lengths (Q8Balance), so that at most
// `target` items share the tokens of a ragged batch evenly.
struct Q8Plan {
  int row_tile;     // rows of one work item
  int merge_rows;   // of them that any unit has
  int tiles;        // ceil(n * G / row_tile)
  int whole, units;
  int chunk, n_chunks;
  int target;       // most items of a balanced split; 0: not balanced
  int per_head;     // target / (Hkv * tiles)
  int step_shift;   // chunks of a balanced split are multiples of 2^step_shift tokens
  int parts;        // partial results of one work item
  int part_stride;  // floats of one partial: d + 4
  size_t header_bytes, ws_bytes;
  Q8Mode mode;
  int64_t split_items() const { return target ? target : (int64_t)(units - whole) * n_chunks; }
  int64_t items() const { return whole + split_items(); }
  int row_parts;    // partial results of a row, about
  int64_t split_rows() const { return (int64_t)(units - whole) * merge_rows; }
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
  int test_starve, test_slow_scales;
};

bool q8_head_dim_supported(int d);
bool make_q8_plan(int B, int Hq, int Hkv, int d, int n, int max_ctx, bool bf16, Q8Plan* plan);
cudaError_t launch_q8_append(const Q8WriteArgs& a, cudaStream_t stream);
cudaError_t launch_q8_read(const Q8ReadArgs& a, cudaStream_t stream);
int q8_split_per_sm(int d, int row_tile);  // work items of the split kernel resident on an SM
cudaError_t launch_q8_split(const Q8AttendArgs& a, cudaStream_t stream);
int q8_tc_tile_tokens(int d, Q8Mode mode);  // tokens of one step of the tensor-memory kernel
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

// Block 0 reports the sequences whose lengths were out of range.
__device__ __forceinline__ void q8_write_flags(const Q8AttendArgs& a) {
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < a.c.B; b += blockDim.x) static_cast<int32_t*>(a.workspace)[b] = Q8Seq(a, b).bad;
}

// A balanced split of up to 32 sequences: the smallest chunk (in steps) found with which
// they have at most `target` items.  Every warp of both kernels works it out for itself, a
// lane per sequence, and comes to the same.
struct Q8Balance {
  int chunk, lane, steps, own;  // own: chunks of this lane's sequence
  __device__ __forceinline__ Q8Balance(const Q8AttendArgs& a) : lane(threadIdx.x & 31), steps(0) {
    if (lane < a.c.B) {
      const Q8Seq s(a, lane);
      if (s.q_len > 0) steps = (s.ctx + (1 << a.plan.step_shift) - 1) >> a.plan.step_shift;
    }
    const unsigned most = a.plan.per_head;
    const unsigned total = __reduce_add_sync(0xffffffffu, (unsigned)steps);
    chunk = max(1, (int)((total + most - 1) / most));
    for (int i = 0; i < 64; ++i) {
      own = (steps + chunk - 1) / chunk;
      const unsigned n = __reduce_add_sync(0xffffffffu, (unsigned)own);
      if (n <= most) break;
      // towards the mean of the counts; doubled at last, until each sequence is one chunk
      chunk = i < 32 ? max(chunk + 1, (int)((int64_t)chunk * (n + most) / (2 * most))) : 2 * chunk;
    }
  }
  // chunks of the sequences before b
  __device__ __forceinline__ int before(int b) const {
    return (int)__reduce_add_sync(0xffffffffu, lane < b ? (unsigned)own : 0u);
  }
  // the sequence that item `at` of `heads` for each chunk falls into; false: none
  __device__ __forceinline__ bool find(int at, int heads, int& b, int& first, int& n) const {
    int sum = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, at < sum * heads);
    b = hit ? __ffs(hit) - 1 : 0;
    n = __shfl_sync(0xffffffffu, own, b);
    first = __shfl_sync(0xffffffffu, sum, b) - n;
    return hit != 0;
  }
};

// The unit, and the chunk [begin, begin + chunk) of it, that work item `id` is (whole warps).
struct Q8Item {
  int id, chunk_id, chunk, tile, bh, b, hk, G, rows, row0;
  bool split, any;  // any: there is such an item
  __device__ __forceinline__ Q8Item() {}
  __device__ __forceinline__ Q8Item(const Q8AttendArgs& a, int item) {
    id = item - a.plan.whole;
    split = id >= 0;
    any = true;
    chunk = a.plan.chunk;
    if (a.plan.target) {
      const Q8Balance s(a);
      const int heads = a.c.Hkv * a.plan.tiles;
      int first, own, seq;
      any = s.find(id, heads, seq, first, own);
      const int r = id - first * heads, u = any ? r / own : 0;
      chunk_id = r - u * own;
      chunk = s.chunk << a.plan.step_shift;
      place(a, a.plan.tiles - 1 - u / a.c.Hkv, seq, u % a.c.Hkv);
      return;
    }
    place_unit(a, split ? a.plan.whole + id / a.plan.n_chunks : item);
    chunk_id = split ? id % a.plan.n_chunks : 0;
  }
  __device__ __forceinline__ void place_unit(const Q8AttendArgs& a, int u) {
    const int heads = a.c.B * a.c.Hkv;
    place(a, a.plan.tiles - 1 - u / heads, u % heads / a.c.Hkv, u % heads % a.c.Hkv);
  }
  __device__ __forceinline__ void place(const Q8AttendArgs& a, int t, int seq, int head) {
    tile = t;
    b = seq;
    hk = head;
    bh = seq * a.c.Hkv + head;
    G = a.Hq / a.c.Hkv;
    rows = a.n * G;
    row0 = tile * a.plan.row_tile;
  }
  // the first item of split unit u, whose place this is (for the merge, whole warps)
  __device__ __forceinline__ void first_item(const Q8AttendArgs& a, int u) {
    chunk = a.plan.chunk;
    if (a.plan.target) {
      const Q8Balance s(a);
      const int first = s.before(b), own = __shfl_sync(0xffffffffu, s.own, b);
      chunk = s.chunk << a.plan.step_shift;
      id = first * a.c.Hkv * a.plan.tiles + ((a.plan.tiles - 1 - tile) * a.c.Hkv + hk) * own;
    } else {
      id = (u - a.plan.whole) * a.plan.n_chunks;
    }
  }
  // query token and output row of the tile's row r
  __device__ __forceinline__ int token(int r) const { return (row0 + r) / G; }
  __device__ __forceinline__ int64_t out_row(const Q8AttendArgs& a, int r) const {
    return ((int64_t)b * a.Hq + hk * G + (row0 + r) % G) * a.n + token(r);
  }
  // partial p of row r; those of a row are part_step() floats apart, over items too
  __device__ __forceinline__ float* part(const Q8AttendArgs& a, int r, int p) const {
    return reinterpret_cast<float*>(static_cast<unsigned char*>(a.workspace) + a.plan.header_bytes) +
           ((int64_t)id * a.plan.parts + p) * part_step(a) + (int64_t)r * a.plan.part_stride;
  }
  static __device__ __forceinline__ int64_t part_step(const Q8AttendArgs& a) {
    return (int64_t)a.plan.row_tile * a.plan.part_stride;
  }
};
#endif

}  // namespace tq
