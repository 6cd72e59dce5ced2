// q8_api.cu -- the C ABI of the 8-bit block-scaled cache (declared in
// include/tq.h): host-side validation, the split plan, kernel dispatch.
#include <limits.h>
#include <math.h>
#include <stdio.h>
#include <stdlib.h>

#include "q8_internal.h"

namespace tq {

bool q8_head_dim_supported(int d) { return d == 64 || d == 96 || d == 128 || d == 256; }

namespace {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool misaligned(const void* p, unsigned bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0;
}

tq_status status_of(cudaError_t e, const char* where) {
  if (e == cudaSuccess) return TQ_OK;
  if (getenv("TQ_DEBUG")) fprintf(stderr, "libtq: %s: %s\n", where, cudaGetErrorString(e));
  return TQ_ERR_CUDA;
}

// The checks every call makes of its cache; fills *c.
tq_status check_cache(const void* k_codes, const float* k_scales, const void* v_codes,
                      const float* v_scales, int64_t capacity, int32_t batch, int32_t num_kv_heads,
                      int32_t head_dim, tq_q8_format format, int32_t block, Q8Cache* c) {
  if (!k_codes || !k_scales || !v_codes || !v_scales) return TQ_ERR_INVALID_ARG;
  if (format != TQ_Q8_INT8 && format != TQ_Q8_E4M3) return TQ_ERR_INVALID_ARG;
  if (batch < 1 || num_kv_heads < 1 || capacity < 1) return TQ_ERR_INVALID_ARG;
  if ((int64_t)batch * num_kv_heads > INT32_MAX) return TQ_ERR_INVALID_ARG;
  if (!q8_head_dim_supported(head_dim)) return TQ_ERR_UNSUPPORTED;
  if (block != 16 && block != 32 && block != 64 && block != 128) return TQ_ERR_UNSUPPORTED;
  if (misaligned(k_codes, 16) || misaligned(v_codes, 16) || misaligned(k_scales, 4) ||
      misaligned(v_scales, 4))
    return TQ_ERR_INVALID_ARG;
  c->k_codes = static_cast<uint8_t*>(const_cast<void*>(k_codes));
  c->v_codes = static_cast<uint8_t*>(const_cast<void*>(v_codes));
  c->k_scales = const_cast<float*>(k_scales);
  c->v_scales = const_cast<float*>(v_scales);
  c->capacity = capacity;
  c->B = batch;
  c->Hkv = num_kv_heads;
  c->d = head_dim;
  c->block = block;
  c->e4m3 = format == TQ_Q8_E4M3;
  return TQ_OK;
}

}  // namespace

namespace {

// Chunks of the context for `units` units: the count that minimises the time of the busiest
// SM, (its work items) x (tokens of one + a fixed cost per item, in tokens).  Where an SM
// holds several CTAs, two of them reach 95% of its bandwidth and one 60% (side by side, 128K,
// 64/8 heads, d 128: 55 us with two a SM, 59 with four and twice the partial results to join).
// Returns the items of an SM.
int64_t split_context(int64_t units, int per_sm, int max_ctx, int64_t step, int64_t item_cost, Q8Plan* p) {
  int64_t items = 0, best = ceil_div(max_ctx, step) * step, best_cost = -1;
  // the most chunks with which no SM has more than `most` items
  const int64_t least = ceil_div(units, kSmCount);
  for (int64_t most = least; units > 0 && most <= (least > 4 * per_sm ? least : 4 * per_sm); ++most) {
    const int64_t k = most * kSmCount / units;  // >= 1
    const int64_t chunk = ceil_div(ceil_div(max_ctx, k < 1024 ? k : 1024), step) * step;
    const int64_t each = ceil_div(units * ceil_div(max_ctx, chunk), kSmCount);
    const int64_t cost = each * (chunk + item_cost) * (per_sm == 1 || each > 2 ? 20 : each == 2 ? 21 : 33);
    if (best_cost < 0 || cost < best_cost) best_cost = cost, best = chunk, items = each;
  }
  if (best > INT32_MAX) best = INT32_MAX / step * step;
  p->chunk = (int)best;
  p->n_chunks = (int)ceil_div(max_ctx, best);
  return items;
}

}  // namespace

// bf16: queries and outputs are bf16.
bool make_q8_plan(int B, int Hq, int Hkv, int d, int n, int max_ctx, bool bf16, Q8Plan* p) {
  if (B < 1 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || n < 1 || max_ctx < 1) return false;
  if (!q8_head_dim_supported(d)) return false;
  const int64_t G = Hq / Hkv, rows = G * n;
  if (rows > INT32_MAX / 2 || (int64_t)B * Hkv > INT32_MAX || (int64_t)B * Hq * n > INT32_MAX) return false;
  int per_sm;
  int64_t step, item_cost;
  if (bf16 && rows > 16) {
    p->mode = d > 128 ? kQ8OneStream : rows > 128 ? kQ8TwoRows : kQ8TwoStreams;
    p->row_tile = p->mode == kQ8TwoRows ? 256 : 128;
    p->parts = p->mode == kQ8TwoStreams ? 2 : 1;
    per_sm = 1;
    step = p->parts * q8_tc_tile_tokens(d, p->mode);
    // queries, pipeline fill, partial results and their merge (32 heads of d = 96, 2048 tokens
    // at 8K: 312 us with 512, 262 us with this; d = 256, 1024 tokens: 297 and 261 us)
    item_cost = 2048;
  } else {
    p->mode = kQ8Warps;
    p->row_tile = rows <= 8 ? 8 : 16;
    p->parts = 1;
    per_sm = q8_split_per_sm(d, p->row_tile);
    step = 64;
    item_cost = 512;
  }
  p->tiles = (int)ceil_div(rows, p->row_tile);
  p->merge_rows = rows < p->row_tile ? (int)rows : p->row_tile;
  const int64_t units = (int64_t)B * Hkv * p->tiles;
  if (units > INT32_MAX) return false;
  p->units = (int)units;
  p->whole = p->parts > 1 ? 0 : (int)(units / (per_sm * kSmCount) * (per_sm * kSmCount));
  const int64_t each = split_context(units - p->whole, per_sm, max_ctx, step, item_cost, p);
  p->target = 0;
  p->step_shift = 31 - __builtin_clz((unsigned)step);
  if (p->n_chunks * p->parts == 1) {
    p->whole = (int)units;
  } else if (p->whole == 0 && B > 1 && B <= 32) {
    // As many items as the busiest SM has, but the same number for each kv head and tile.  A
    // warp keeps one sequence in each lane, so more than 32 are split by max_ctx: decode of
    // 64/8 heads, d 128, 32K at most, 32 sequences of 18K on average 230 us, 34 of 20K 351 us
    // (equal lengths of 16K: 199 and 217 us).
    const int64_t heads = (int64_t)Hkv * p->tiles;
    p->target = (int)(each * kSmCount / heads * heads);
    if (p->target < units) p->target = (int)units;
    p->per_head = (int)(p->target / heads);
  }
  p->row_parts = p->n_chunks * p->parts;
  p->part_stride = d + 4;
  p->header_bytes = (size_t)ceil_div(4LL * B, 256) * 256;
  p->ws_bytes = p->header_bytes;
  if (p->whole < p->units)
    p->ws_bytes += sizeof(float) * (size_t)p->split_items() * p->row_tile * p->parts * p->part_stride;
  return p->items() <= INT32_MAX && p->split_rows() <= INT32_MAX;
}

namespace {

tq_status attend(const void* q, tq_dtype q_dtype, int32_t num_q_heads, int32_t n, const Q8Cache& c,
                 const int32_t* ctx_lens, const int32_t* q_lens, int32_t max_ctx, float attn_scale,
                 void* out, tq_dtype out_dtype, float* lse, void* workspace, size_t workspace_bytes,
                 cudaStream_t stream, const Q8WriteArgs* append, const char* where) {
  if (!q || !ctx_lens || !out) return TQ_ERR_INVALID_ARG;
  if ((q_dtype != TQ_F32 && q_dtype != TQ_BF16) || (out_dtype != TQ_F32 && out_dtype != TQ_BF16))
    return TQ_ERR_INVALID_ARG;
  if (num_q_heads < c.Hkv || num_q_heads % c.Hkv != 0 || n < 1) return TQ_ERR_INVALID_ARG;
  if (max_ctx < 1 || c.capacity < max_ctx) return TQ_ERR_INVALID_ARG;
  if (!(attn_scale > 0.0f) || !isfinite(attn_scale)) return TQ_ERR_INVALID_ARG;
  if (misaligned(q, 16) || misaligned(out, 16) || misaligned(lse, 8) || misaligned(ctx_lens, 4) ||
      misaligned(q_lens, 4))
    return TQ_ERR_INVALID_ARG;
  Q8AttendArgs a;
  if (!make_q8_plan(c.B, num_q_heads, c.Hkv, c.d, n, max_ctx, q_dtype == TQ_BF16 && out_dtype == TQ_BF16, &a.plan))
    return TQ_ERR_INVALID_ARG;
  if (!workspace || misaligned(workspace, 16) || workspace_bytes < a.plan.ws_bytes)
    return TQ_ERR_WORKSPACE;
  a.c = c;
  a.q = q;
  a.q_bf16 = q_dtype == TQ_BF16;
  a.Hq = num_q_heads;
  a.n = n;
  a.ctx_lens = ctx_lens;
  a.q_lens = q_lens;
  a.max_ctx = max_ctx;
  a.attn_scale = attn_scale;
  a.out = out;
  a.out_bf16 = out_dtype == TQ_BF16;
  a.lse = lse;
  a.workspace = workspace;
  const unsigned hooks = g_test_hooks.load(std::memory_order_relaxed);
  if (hooks & TQ_TEST_HOOK_FAIL_LAUNCH) return status_of(cudaErrorLaunchFailure, where);
  a.test_starve = (hooks & TQ_TEST_HOOK_STARVE_PIPELINE) != 0;
  a.test_slow_scales = (hooks & TQ_TEST_HOOK_SLOW_SCALES) != 0;
  cudaError_t e = append ? launch_q8_append(*append, stream) : cudaSuccess;
  if (e == cudaSuccess) e = a.plan.mode == kQ8Warps ? launch_q8_split(a, stream) : launch_q8_tc(a, stream);
  if (e == cudaSuccess && a.plan.whole < a.plan.units) e = launch_q8_merge(a, stream);
  return status_of(e, where);
}

}  // namespace
}  // namespace tq

using namespace tq;

extern "C" {

tq_status tq_quantize_append_q8(const void* k, const void* v, tq_dtype in_dtype, int32_t batch,
                                int32_t num_kv_heads, int32_t n_new, int32_t head_dim,
                                tq_q8_format format, int32_t block, const int32_t* pos,
                                const int32_t* n_valid, void* k_codes, float* k_scales,
                                void* v_codes, float* v_scales, int64_t capacity,
                                void* cuda_stream) {
  Q8WriteArgs a = {};
  const tq_status st = check_cache(k_codes, k_scales, v_codes, v_scales, capacity, batch, num_kv_heads,
                                   head_dim, format, block, &a.c);
  if (st != TQ_OK) return st;
  if (!k || !v || !pos || n_new < 1 || (in_dtype != TQ_F32 && in_dtype != TQ_BF16))
    return TQ_ERR_INVALID_ARG;
  if (misaligned(k, 16) || misaligned(v, 16) || misaligned(pos, 4) || misaligned(n_valid, 4))
    return TQ_ERR_INVALID_ARG;
  if (2 * (int64_t)batch * num_kv_heads * (((int64_t)n_new + block - 2) / block + 1) > INT32_MAX ||
      n_new > INT32_MAX - block)
    return TQ_ERR_INVALID_ARG;
  a.k = k;
  a.v = v;
  a.bf16 = in_dtype == TQ_BF16;
  a.n = n_new;
  a.pos = pos;
  a.n_valid = n_valid;
  return status_of(launch_q8_append(a, static_cast<cudaStream_t>(cuda_stream)), "tq_quantize_append_q8");
}

tq_status tq_read_q8(const void* k_codes, const float* k_scales, const void* v_codes,
                     const float* v_scales, int64_t capacity, int32_t batch, int32_t num_kv_heads,
                     int32_t head_dim, tq_q8_format format, int32_t block, const int32_t* pos,
                     const int32_t* n_valid, int32_t rows, void* k_out, void* v_out,
                     tq_dtype out_dtype, int32_t fill, void* cuda_stream) {
  Q8ReadArgs a = {};
  const tq_status st = check_cache(k_codes, k_scales, v_codes, v_scales, capacity, batch, num_kv_heads,
                                   head_dim, format, block, &a.c);
  if (st != TQ_OK) return st;
  if (!k_out || !v_out || rows < 1 || (out_dtype != TQ_F32 && out_dtype != TQ_BF16))
    return TQ_ERR_INVALID_ARG;
  if (misaligned(k_out, 16) || misaligned(v_out, 16) || misaligned(pos, 4) || misaligned(n_valid, 4))
    return TQ_ERR_INVALID_ARG;
  // (a CTA takes 16 to 128 rows; row numbers are rounded up to those in 32 bits)
  if (2 * (int64_t)batch * num_kv_heads * ((int64_t)rows / 16 + 1) > INT32_MAX || rows > INT32_MAX - 128)
    return TQ_ERR_INVALID_ARG;
  a.k = k_out;
  a.v = v_out;
  a.bf16 = out_dtype == TQ_BF16;
  a.n = rows;
  a.pos = pos;
  a.n_valid = n_valid;
  a.fill = fill != 0;
  return status_of(launch_q8_read(a, static_cast<cudaStream_t>(cuda_stream)), "tq_read_q8");
}

size_t tq_sdpa_q8_workspace_bytes(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                                  int32_t head_dim, int32_t n_q, int32_t max_ctx,
                                  tq_dtype out_dtype) {
  Q8Plan p, q;  // bf16 outputs: enough for queries of either type
  if (!make_q8_plan(batch, num_q_heads, num_kv_heads, head_dim, n_q, max_ctx, false, &p)) return 0;
  if (out_dtype != TQ_BF16) return p.ws_bytes;
  if (!make_q8_plan(batch, num_q_heads, num_kv_heads, head_dim, n_q, max_ctx, true, &q)) return 0;
  return p.ws_bytes > q.ws_bytes ? p.ws_bytes : q.ws_bytes;
}

tq_status tq_sdpa_q8(const void* q, tq_dtype q_dtype, int32_t batch, int32_t num_q_heads,
                     int32_t num_kv_heads, int32_t n_q, int32_t head_dim, tq_q8_format format,
                     int32_t block, const void* k_codes, const float* k_scales, const void* v_codes,
                     const float* v_scales, int64_t capacity, const int32_t* ctx_lens,
                     const int32_t* q_lens, int32_t max_ctx, float attn_scale, void* out,
                     tq_dtype out_dtype, float* lse, void* workspace, size_t workspace_bytes,
                     void* cuda_stream) {
  Q8Cache c;
  const tq_status st = check_cache(k_codes, k_scales, v_codes, v_scales, capacity, batch, num_kv_heads,
                                   head_dim, format, block, &c);
  if (st != TQ_OK) return st;
  return attend(q, q_dtype, num_q_heads, n_q, c, ctx_lens, q_lens, max_ctx, attn_scale, out, out_dtype,
                lse, workspace, workspace_bytes, static_cast<cudaStream_t>(cuda_stream), nullptr,
                "tq_sdpa_q8");
}

tq_status tq_sdpa_q8_decode_append(
    const void* q, tq_dtype q_dtype, const void* k_new, const void* v_new, tq_dtype kv_dtype,
    int32_t batch, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, tq_q8_format format,
    int32_t block, void* k_codes, float* k_scales, void* v_codes, float* v_scales, int64_t capacity,
    const int32_t* ctx_lens, int32_t max_ctx, float attn_scale, void* out, tq_dtype out_dtype,
    float* lse, void* workspace, size_t workspace_bytes, void* cuda_stream) {
  Q8WriteArgs w = {};
  const tq_status st = check_cache(k_codes, k_scales, v_codes, v_scales, capacity, batch, num_kv_heads,
                                   head_dim, format, block, &w.c);
  if (st != TQ_OK) return st;
  if (!k_new || !v_new || (kv_dtype != TQ_F32 && kv_dtype != TQ_BF16)) return TQ_ERR_INVALID_ARG;
  if (misaligned(k_new, 16) || misaligned(v_new, 16)) return TQ_ERR_INVALID_ARG;
  if (2 * (int64_t)batch * num_kv_heads > INT32_MAX) return TQ_ERR_INVALID_ARG;
  w.k = k_new;
  w.v = v_new;
  w.bf16 = kv_dtype == TQ_BF16;
  w.n = 1;
  w.pos = ctx_lens;
  w.pos_is_ctx = 1;
  w.max_ctx = max_ctx;
  return attend(q, q_dtype, num_q_heads, 1, w.c, ctx_lens, nullptr, max_ctx, attn_scale, out, out_dtype,
                lse, workspace, workspace_bytes, static_cast<cudaStream_t>(cuda_stream), &w,
                "tq_sdpa_q8_decode_append");
}

}  // extern "C"
