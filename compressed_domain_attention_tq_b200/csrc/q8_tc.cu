// q8_tc.cu -- attention of many query rows per kv head (a prefill chunk, drafted
// tokens of grouped heads) over the 8-bit block-scaled cache, bf16 in and out,
// with both products on the fifth-generation tensor cores (tcgen05.mma, f16 in,
// fp32 sums in tensor memory).
//
// Rows.  As in q8_split.cu the query rows of a kv head are its n tokens x G query
// heads, row r = i G + g, cut into tiles of 128 (the M of one product).  With
// S = Q K^T (128 rows x T tokens) and O (128 x d) += P V a CTA holds, by mode:
//   two row tiles (d <= 128, more than 128 rows): both use each tile of T = 128
//     tokens, so a code is converted once for 256 rows;
//   two token streams (d <= 128, up to 128 rows): one row tile, the even token
//     tiles in one (S, O), the odd ones in the other; each writes its own partial;
//   one stream (d = 256, T = 64): one row tile, two S, one O.
// In each the products of one S run while the softmax of the other does.
//
// Warps.  0..3 and 4..7: softmax, a thread per row, so row statistics need no
// exchange (d = 256: 0..3 only).  8..11: conversion of codes to f16 operands in
// shared memory, loaded from global memory one tile ahead into registers.
// 12: issues the products.
//
// Numbers.  Codes and the queries (bf16, scaled by a power of two per row) are
// exact in f16, so scores carry fp32's rounding alone.  A weight is
// 2^(x - m) s_v / ref with x = S s_k scale log2(e), m the row's reference (moved
// only when a score exceeds it by 2^8) and ref the item's largest V scale; it is
// rounded to f16's 11 bits, as the bf16 output keeps 8.  The ratio enters as
// its logarithm in the exponent, so it costs nothing; it is floored at 2^-40:
// a block whose scale is that far below ref then counts with at most
// 2^-40 max|v|, far below the output's rounding.  Row sums and O are fp32.
//
// Operand layout in shared memory, without swizzle: [d / 8][rows][16 bytes], an
// 8 x 16-byte core matrix contiguous.  For K that is K-major (rows = tokens), and
// the same bytes are MN-major for V, so one converter serves both, and its
// 16-byte stores of 8 neighbouring tokens fill all banks.  int8 codes leave the
// converter in the order 0 2 1 3 of each word: Q is stored in that order, and
// O's columns are put back when they are written.
//
// Bound: the tensor cores for long chunks; HBM (codes) for few rows.
#include <limits.h>
#include <math.h>

#include "q8_common.cuh"
#include "q8_internal.h"

namespace tq {
namespace {

using namespace q8;
using namespace tc;

constexpr int kSoftmaxWarps = 8, kConvertWarps = 4, kMmaWarp = kSoftmaxWarps + kConvertWarps;
constexpr int kThreads = 32 * (kMmaWarp + 1);
constexpr float kTau = 8.0f, kShift = 7.0f;  // as in q8_split.cu: weights stay below 2^15
constexpr float kMinRatio = 0x1p-40f;
constexpr int kScaleSlots = 4;

// tokens of a tile, row tiles in shared memory
__host__ __device__ constexpr int tile_tokens(int d) { return d <= 128 ? 128 : 64; }

template <int D, int MODE>
struct Layout {
  static constexpr int T = tile_tokens(D);
  static constexpr int QT = MODE == kQ8TwoRows ? 2 : 1;
  static constexpr int Q_BYTES = 128 * D * 2, KV_BYTES = T * D * 2;
  static constexpr int Q = 0, K = Q + QT * Q_BYTES, V = K + 2 * KV_BYTES;
  static constexpr int CROW = V + 2 * KV_BYTES;             // float [QT * 128]
  static constexpr int SCALES = CROW + 4 * QT * 128;        // float4 [kScaleSlots][T / 16]
  static constexpr int BAR = SCALES + 16 * kScaleSlots * (T / 16);
  static constexpr int MISC = BAR + 8 * 32;                 // tmem base, abort, ref, warp maxima
  static constexpr int BYTES = MISC + 16 + 4 * (kMmaWarp + 1);
  static_assert(BYTES <= 227 * 1024, "shared memory");
  static __host__ __device__ constexpr uint32_t S(int b) { return (uint32_t)(b * T); }
  static __host__ __device__ constexpr uint32_t O(int u) { return (uint32_t)(2 * T + u * D); }
};

enum Bar : int {
  kKFull = 0,    // [2] K operand written (convert warps)
  kKEmpty = 2,   // [2] its products done (commit)
  kVFull = 4,
  kVEmpty = 6,
  kSFull = 8,    // [2] scores in tensor memory (commit)
  kPFull = 10,   // [2] weights in tensor memory (4 softmax warps)
  kPVDone = 12,  // [2] O up to date (commit)
  kScFull = 14,  // [kScaleSlots] block scales written (one convert warp)
  kDone = 18,    // every product complete (commit)
  kBars = 19
};

// What one CTA does: rows of one kv head, and tokens [begin, stop) in nt tiles.
struct Item {
  int chunk_id, tile, b, hk, bh, G, rows, row0, begin, stop, nt;
};

template <int D>
__device__ __forceinline__ const uint8_t* head_codes(const uint8_t* codes, const Q8AttendArgs& a, int bh) {
  return codes + (int64_t)bh * a.c.capacity * D;
}

// A warp's wait, reconverged: tensor-memory instructions need the whole warp.
__device__ __forceinline__ void warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  mbar_wait(bar, parity, abort);
  __syncwarp();
}

// Pins registers written by tcgen05.ld behind the wait before this.
__device__ __forceinline__ void tie32(uint32_t (&r)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]),
                 "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7]));
}

__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// ------------------------------------------------------------------ conversion

template <int D>
struct Pieces {  // one thread's 16-byte pieces of a tile of codes
  static constexpr int N = tile_tokens(D) * D / 16 / (32 * kConvertWarps);
  uint4 w[N];
  // piece p: token (p & 7) + 8 (rest / (D/16)), bytes 16 (rest % (D/16)) .., rest = p >> 3
  static __device__ __forceinline__ int token(int p) { return (p & 7) + 8 * ((p >> 3) / (D / 16)); }
  static __device__ __forceinline__ int c16(int p) { return (p >> 3) % (D / 16); }
  // rows behind the last one repeat it: what is multiplied is always cache content
  __device__ __forceinline__ void load(const uint8_t* codes, int tok0, int stop, int tid) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int p = tid + 32 * kConvertWarps * i;
      const uint8_t* at = codes + (int64_t)min(tok0 + token(p), stop - 1) * D + 16 * c16(p);
      asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                   : "l"(at));
    }
  }
  template <typename F>
  __device__ __forceinline__ void store(unsigned char* dst, int tid) const {
    constexpr int T = tile_tokens(D);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int p = tid + 32 * kConvertWarps * i;
      unsigned char* at = dst + (2 * c16(p) * T + token(p)) * 16;
      uint4 lo, hi;
      F::cvt_word(w[i].x, lo.x, lo.y);
      F::cvt_word(w[i].y, lo.z, lo.w);
      F::cvt_word(w[i].z, hi.x, hi.y);
      F::cvt_word(w[i].w, hi.z, hi.w);
      *reinterpret_cast<uint4*>(at) = lo;
      *reinterpret_cast<uint4*>(at + T * 16) = hi;
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
  }
};

template <typename F, int D, int MODE>
__device__ __forceinline__ void convert_role(const Q8AttendArgs& a, const Item& it, unsigned char* smem,
                                             uint64_t* bar, volatile int* abort, float ref) {
  using L = Layout<D, MODE>;
  const int tid = threadIdx.x - 32 * kSoftmaxWarps, lane = tid & 31;
  const uint8_t* kc = head_codes<D>(a.c.k_codes, a, it.bh);
  const uint8_t* vc = head_codes<D>(a.c.v_codes, a, it.bh);
  const float* ksc = a.c.k_scales + (int64_t)it.bh * a.c.n_blocks();
  const float* vsc = a.c.v_scales + (int64_t)it.bh * a.c.n_blocks();
  const int shift = 31 - __clz(a.c.block);
  // K runs ahead of V by the tiles whose scores are computed before the first P V
  constexpr int kAhead = MODE == kQ8TwoRows ? 1 : 2;
  Pieces<D> k, v;
  float sk = 0.0f, sv = 0.0f;
  auto load_scales = [&](int j) {
    if (j >= it.nt) return;
    const int blk = min(it.begin + j * L::T + 16 * tid, it.stop - 1) >> shift;
    sk = __ldg(ksc + blk);
    sv = __ldg(vsc + blk);
  };
  if (it.nt > 0) {
    k.load(kc, it.begin, it.stop, tid);
    v.load(vc, it.begin, it.stop, tid);
    if (tid < L::T / 16) load_scales(0);
  }
  for (int j = 0; j < it.nt + kAhead - 1; ++j) {
    if (j < it.nt) {
      const int s = j & 1;
      if (j >= 2) warp_wait(bar + kKEmpty + s, ((j >> 1) - 1) & 1, abort);
      if (tid < 32) {
        // scales of 16 tokens: {s_k, log2(s_v / ref), ref / s_v}.  Slot j - 4 has been
        // read: the scores of tile j - 2 came after the weights of tile j - 4.
        if (tid < L::T / 16) {
          const float ratio = ref > 0.0f ? fmaxf(sv / ref, kMinRatio) : 1.0f;
          reinterpret_cast<float4*>(smem + L::SCALES)[(j & (kScaleSlots - 1)) * (L::T / 16) + tid] =
              make_float4(sk, log2f(ratio), 1.0f / ratio, 0.0f);
          load_scales(j + 1);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar + kScFull + (j & (kScaleSlots - 1)));
      }
      k.template store<F>(smem + L::K + s * L::KV_BYTES, tid);
      if (lane == 0 && !(a.test_starve && j == 0)) mbar_arrive(bar + kKFull + s);
      if (j + 1 < it.nt) k.load(kc, it.begin + (j + 1) * L::T, it.stop, tid);
    }
    const int jv = j - (kAhead - 1);
    if (jv >= 0 && jv < it.nt) {
      const int s = jv & 1;
      if (jv >= 2) warp_wait(bar + kVEmpty + s, ((jv >> 1) - 1) & 1, abort);
      v.template store<F>(smem + L::V + s * L::KV_BYTES, tid);
      if (lane == 0) mbar_arrive(bar + kVFull + s);
      if (jv + 1 < it.nt) v.load(vc, it.begin + (jv + 1) * L::T, it.stop, tid);
    }
  }
}

// -------------------------------------------------------------------- products

template <int D, int MODE>
__device__ __forceinline__ void mma_role(const Item& it, unsigned char* smem, uint64_t* bar,
                                         volatile int* abort, uint32_t tbase) {
  using L = Layout<D, MODE>;
  constexpr uint32_t idS = idesc_f16(128, L::T, 0, 0), idO = idesc_f16(128, D, 0, 1);
  const uint64_t dq = smem_desc(smem_u32(smem + L::Q), 128 * 16, 128);
  const uint64_t dk = smem_desc(smem_u32(smem + L::K), L::T * 16, 128);
  const uint64_t dv = smem_desc(smem_u32(smem + L::V), 128, L::T * 16);
  // scores of token tile j into S[b], from row tile u of Q
  auto scores = [&](int j, int u, int b) {
    if (!*abort) {
      const uint64_t q = dq + (uint64_t)((u * L::Q_BYTES) >> 4), k = dk + (uint64_t)(((j & 1) * L::KV_BYTES) >> 4);
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
        mma_ss(tbase + L::S(b), q + (uint64_t)(c * 2 * 128), k + (uint64_t)(c * 2 * L::T), idS, c > 0);
    }
    mma_commit(bar + kSFull + b);
  };
  // O[u] += P[b] V of token tile j
  auto values = [&](int j, int u, int b, bool first) {
    if (!*abort) {
      const uint64_t v = dv + (uint64_t)(((j & 1) * L::KV_BYTES) >> 4);
#pragma unroll
      for (int c = 0; c < L::T / 16; ++c)
        mma_ts(tbase + L::O(u), tbase + L::S(b) + 8 * c, v + (uint64_t)(c * 16), idO, c > 0 || !first);
    }
    mma_commit(bar + kPVDone + u);
  };
  auto wait_k = [&](int j) {
    mbar_wait(bar + kKFull + (j & 1), (j >> 1) & 1, abort);
    fence_after();
  };
  auto wait_v = [&](int j) {
    mbar_wait(bar + kVFull + (j & 1), (j >> 1) & 1, abort);
    fence_after();
  };
  if constexpr (MODE == kQ8TwoRows) {
    wait_k(0);
    scores(0, 0, 0);
    scores(0, 1, 1);
    mma_commit(bar + kKEmpty);
    for (int j = 0; j < it.nt; ++j) {
      wait_v(j);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        mbar_wait(bar + kPFull + u, j & 1, abort);
        fence_after();
        values(j, u, u, j == 0);
        if (j + 1 < it.nt) {
          if (u == 0) wait_k(j + 1);
          scores(j + 1, u, u);
        }
      }
      mma_commit(bar + kVEmpty + (j & 1));
      if (j + 1 < it.nt) mma_commit(bar + kKEmpty + ((j + 1) & 1));
    }
  } else {
    for (int j = 0; j < 2 && j < it.nt; ++j) {
      wait_k(j);
      scores(j, 0, j);
      mma_commit(bar + kKEmpty + j);
    }
    for (int j = 0; j < it.nt; ++j) {
      const int b = j & 1;
      wait_v(j);
      mbar_wait(bar + kPFull + b, (j >> 1) & 1, abort);
      fence_after();
      values(j, MODE == kQ8TwoStreams ? b : 0, b, MODE == kQ8TwoStreams ? j < 2 : j == 0);
      mma_commit(bar + kVEmpty + b);
      if (j + 2 < it.nt) {
        wait_k(j + 2);
        scores(j + 2, 0, b);
        mma_commit(bar + kKEmpty + b);
      }
    }
  }
  mma_commit(bar + kDone);
  mbar_drain(bar + kDone, 0);
}

// --------------------------------------------------------------------- softmax

// (max over a tile's scores of one row, in log2 units): MASK where a row may end inside
template <int T, bool MASK>
__device__ __forceinline__ float tile_max(uint32_t s_col, const float4* sc, float crow, int left) {
  float mx = -INFINITY;
#pragma unroll
  for (int c = 0; c < T / 32; ++c) {
    uint32_t r[32];
    tld_x32(s_col + 32 * c, r);
    wait_ld();
    tie32(r);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float f = sc[2 * c + h].x * crow;
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const float x = __uint_as_float(r[16 * h + i]), y = __uint_as_float(r[16 * h + i + 1]);
        if constexpr (MASK)
          top = max3(top, 32 * c + 16 * h + i < left ? x : -INFINITY, 32 * c + 16 * h + i + 1 < left ? y : -INFINITY);
        else
          top = max3(top, x, y);
      }
      // a masked row's -inf is kept from meeting a scale of 0
      mx = fmaxf(mx, MASK && top == -INFINITY ? top : top * f);
    }
  }
  return mx;
}

// Weights of a tile into tensor memory over its scores; returns their sum.
template <int T, bool MASK>
__device__ __forceinline__ float tile_weights(uint32_t s_col, const float4* sc, float crow, float m, int left) {
  float sum = 0.0f;
#pragma unroll
  for (int c = 0; c < T / 32; ++c) {
    uint32_t r[32], w[16];
    tld_x32(s_col + 32 * c, r);
    wait_ld();
    tie32(r);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 k = sc[2 * c + h];
      const float f = k.x * crow, off = k.y - m;
      float part[2] = {0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        float p[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = fmaf(__uint_as_float(r[16 * h + i + e]), f, off);
          if constexpr (MASK)
            if (32 * c + 16 * h + i + e >= left) x = -INFINITY;
          p[e] = ex2(x);
          part[e] += p[e];
        }
        w[8 * h + i / 2] = f16x2(p[0], p[1]);
      }
      sum = fmaf(part[0] + part[1], k.z, sum);
    }
    tst_x16(s_col + 16 * c, w);
  }
  return sum;
}

template <typename F, int D, int MODE>
__device__ __forceinline__ void softmax_role(const Q8AttendArgs& a, const Item& it, const Q8Seq& seq,
                                             unsigned char* smem, uint64_t* bar, volatile int* abort,
                                             uint32_t tbase, float ref) {
  using L = Layout<D, MODE>;
  constexpr int T = L::T;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, u = warp >> 2, quarter = warp & 3;
  const int local = (MODE == kQ8TwoRows ? 128 * u : 0) + 32 * quarter + lane;
  const int r = it.row0 + local, i = r / it.G;
  const bool live = r < it.rows && i < seq.q_len;
  const int limit = live ? seq.limit(i) : INT_MAX;
  const bool warp_live = __any_sync(0xffffffffu, live);
  const int open = __reduce_min_sync(0xffffffffu, limit);  // tokens below are seen by the whole warp
  const float crow = reinterpret_cast<const float*>(smem + L::CROW)[local];
  const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
  float m = -INFINITY, l = 0.0f;
  // this warp's tiles: all of them, or every second
  constexpr int step = MODE == kQ8TwoStreams ? 2 : 1;
  const int ou = MODE == kQ8OneStream ? 0 : u;
  int n = 0;  // tiles done
  for (int j = MODE == kQ8TwoStreams ? u : 0; j < it.nt; j += step, ++n) {
    const int sb = MODE == kQ8TwoRows ? u : (j & 1);
    const int phase = MODE == kQ8TwoRows ? j : (j >> 1);
    const uint32_t s_col = tbase + lanes + L::S(sb);
    warp_wait(bar + kScFull + (j & (kScaleSlots - 1)), (j / kScaleSlots) & 1, abort);
    warp_wait(bar + kSFull + sb, phase & 1, abort);
    fence_after();
    if (warp_live) {
      const float4* sc = reinterpret_cast<const float4*>(smem + L::SCALES) + (j & (kScaleSlots - 1)) * (T / 16);
      const int tok0 = it.begin + j * T;
      const bool mask = tok0 + T > min(open, it.stop);
      const int left = min(limit, it.stop) - tok0;  // tokens of this tile that the row sees
      const float mx = mask ? tile_max<T, true>(s_col, sc, crow, left) : tile_max<T, false>(s_col, sc, crow, left);
      if (__any_sync(0xffffffffu, mx > m + (kTau + kShift))) {
        const float mn = fmaxf(m, mx - kShift);  // m is held 2^kShift low
        const float alpha = mn == m ? 1.0f : exp2f(m - mn);
        m = mn;
        l *= alpha;
        if (n > 0) {
          warp_wait(bar + kPVDone + ou, (n - 1) & 1, abort);
          fence_after();
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            uint32_t o[16];
            tld_x16(tbase + lanes + L::O(ou) + 16 * c, o);
            wait_ld();
            asm volatile("" : "+r"(o[0]), "+r"(o[1]), "+r"(o[2]), "+r"(o[3]), "+r"(o[4]), "+r"(o[5]), "+r"(o[6]),
                         "+r"(o[7]), "+r"(o[8]), "+r"(o[9]), "+r"(o[10]), "+r"(o[11]), "+r"(o[12]),
                         "+r"(o[13]), "+r"(o[14]), "+r"(o[15]));
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tst_x16(tbase + lanes + L::O(ou) + 16 * c, o);
          }
        }
      }
      const float mm = m == -INFINITY ? 0.0f : m;
      l += mask ? tile_weights<T, true>(s_col, sc, crow, mm, left)
                : tile_weights<T, false>(s_col, sc, crow, mm, left);
      wait_st();
    }
    fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar + kPFull + sb);
  }
  if (n > 0) warp_wait(bar + kPVDone + ou, (n - 1) & 1, abort);
  fence_after();
  if (!warp_live) return;
  const bool none = n == 0 || (m == -INFINITY && l == 0.0f);
  const int64_t orow = ((int64_t)it.b * a.Hq + it.hk * it.G + r % it.G) * a.n + i;
  const bool split = a.plan.n_parts > 1;
  if (*abort) l = __int_as_float(0x7fc00000);
  const float f = none ? 0.0f : split ? ref : ref / l;
  const int part_id = MODE == kQ8TwoStreams ? 2 * it.chunk_id + u : it.chunk_id;
  float* part = reinterpret_cast<float*>(static_cast<unsigned char*>(a.workspace) + a.plan.header_bytes) +
                (orow * a.plan.n_parts + part_id) * a.plan.part_stride;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    uint32_t o[32];
    __syncwarp();
    tld_x32(tbase + lanes + L::O(ou) + 32 * c, o);
    wait_ld();
    tie32(o);
    if (!live) continue;  // (the loop begins with a __syncwarp)
    float x[32];
#pragma unroll
    for (int w = 0; w < 8; ++w)
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          x[4 * w + F::place(p, k)] = none ? 0.0f : __uint_as_float(o[4 * w + 2 * p + k]) * f;
    if (split) {
#pragma unroll
      for (int e = 0; e < 32; e += 4)
        *reinterpret_cast<float4*>(part + 32 * c + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
    } else {
#pragma unroll
      for (int e = 0; e < 32; e += 8)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + orow * D + 32 * c + e) =
            make_uint4(bf16x2(x[e], x[e + 1]), bf16x2(x[e + 2], x[e + 3]), bf16x2(x[e + 4], x[e + 5]),
                       bf16x2(x[e + 6], x[e + 7]));
    }
  }
  if (!live) return;
  if (split)
    *reinterpret_cast<float2*>(part + D) = make_float2(m, l);
  else if (a.lse != nullptr)
    *reinterpret_cast<float2*>(a.lse + orow * 2) = make_float2(m, l);
}

// ------------------------------------------------------------------ the kernel

template <typename F, int D, int MODE>
__global__ void __launch_bounds__(kThreads, 1) tc_kernel(const Q8AttendArgs a) {
  using L = Layout<D, MODE>;
  extern __shared__ __align__(1024) unsigned char smem[];
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::BAR);
  int* misc = reinterpret_cast<int*>(smem + L::MISC);
  volatile int* abort = misc + 1;
  float* warp_max = reinterpret_cast<float*>(misc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Item it;
  it.chunk_id = blockIdx.x % a.plan.n_chunks;
  const unsigned unit = blockIdx.x / a.plan.n_chunks;
  it.tile = a.plan.tiles - 1 - (int)(unit % a.plan.tiles);  // the longest first
  it.bh = unit / a.plan.tiles;
  it.b = it.bh / a.c.Hkv;
  it.hk = it.bh % a.c.Hkv;
  it.G = a.Hq / a.c.Hkv;
  it.rows = a.n * it.G;
  it.row0 = it.tile * a.plan.row_tile;
  const Q8Seq seq(a, it.b);
  if (it.chunk_id == 0 && it.tile == 0 && it.hk == 0 && threadIdx.x == 0)
    static_cast<int32_t*>(a.workspace)[it.b] = seq.bad;
  const int first_i = it.row0 / it.G;
  const int q_last = min(min(it.rows - 1, it.row0 + a.plan.row_tile - 1) / it.G, seq.q_len - 1);
  const int stop_all = q_last < first_i ? 0 : seq.limit(q_last);
  it.begin = it.chunk_id * a.plan.chunk;
  it.stop = min(stop_all, it.begin + a.plan.chunk);
  it.nt = max(0, (it.stop - it.begin + L::T - 1) / L::T);
  // nothing to do (but a first chunk of no token still writes its rows' zeros)
  if (q_last < first_i || (it.nt == 0 && it.chunk_id > 0)) return;

  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar + kKFull + i, kConvertWarps);
      mbar_init(bar + kKEmpty + i, 1);
      mbar_init(bar + kVFull + i, kConvertWarps);
      mbar_init(bar + kVEmpty + i, 1);
      mbar_init(bar + kSFull + i, 1);
      mbar_init(bar + kPFull + i, 4);
      mbar_init(bar + kPVDone + i, 1);
    }
#pragma unroll
    for (int i = 0; i < kScaleSlots; ++i) mbar_init(bar + kScFull + i, 1);
    mbar_init(bar + kDone, 1);
    *abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) {
    tmem_alloc(reinterpret_cast<uint32_t*>(misc), 512);
    tmem_relinquish();
  }
  // the largest V scale of the item
  float top = 0.0f;
  if (it.nt > 0) {
    const float* vsc = a.c.v_scales + (int64_t)it.bh * a.c.n_blocks();
    const int shift = 31 - __clz(a.c.block), last = (it.stop - 1) >> shift;
    for (int x = (it.begin >> shift) + threadIdx.x; x <= last; x += kThreads) top = fmaxf(top, vsc[x]);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) warp_max[warp] = top;
  // queries: each row scaled so that its largest element is in [2^13, 2^14)
  float* crow = reinterpret_cast<float*>(smem + L::CROW);
  constexpr int W = (D / 4 + 31) / 32;  // words of four elements per lane
#pragma unroll 2
  for (int r = warp; r < L::QT * 128; r += kMmaWarp + 1) {
    const int row = it.row0 + r, i = row / it.G;
    const bool live = row < it.rows && i < seq.q_len;
    const uint16_t* q = static_cast<const uint16_t*>(a.q) +
                        (((int64_t)it.b * a.Hq + it.hk * it.G + row % it.G) * a.n + i) * D;
    float x[W][4];
    float big = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      uint2 v = make_uint2(0u, 0u);
      if (live && lane + 32 * w < D / 4) v = *reinterpret_cast<const uint2*>(q + 4 * (lane + 32 * w));
      x[w][0] = __uint_as_float(v.x << 16);
      x[w][1] = __uint_as_float(v.x & 0xffff0000u);
      x[w][2] = __uint_as_float(v.y << 16);
      x[w][3] = __uint_as_float(v.y & 0xffff0000u);
#pragma unroll
      for (int e = 0; e < 4; ++e) big = fmaxf(big, fabsf(x[w][e]));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
    const int e = big > 0.0f ? max(-100, min(100, 13 - ilogbf(big))) : 0;
    const float up = pow2i(e);
    unsigned char* dst = smem + L::Q + (r >> 7) * L::Q_BYTES + (r & 127) * 16;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const int word = lane + 32 * w;
      if (word < D / 4)
        *reinterpret_cast<uint2*>(dst + (word >> 1) * 2048 + (word & 1) * 8) =
            make_uint2(f16x2(x[w][F::place(0, 0)] * up, x[w][F::place(0, 1)] * up),
                       f16x2(x[w][F::place(1, 0)] * up, x[w][F::place(1, 1)] * up));
    }
    if (lane == 0) crow[r] = a.attn_scale * kLog2e * pow2i(-e);
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tbase = static_cast<uint32_t>(misc[0]);
  float ref = 0.0f;
#pragma unroll
  for (int w = 0; w <= kMmaWarp; ++w) ref = fmaxf(ref, warp_max[w]);

  if (warp < kSoftmaxWarps) {
    if (MODE != kQ8OneStream || warp < 4)
      softmax_role<F, D, MODE>(a, it, seq, smem, bar, abort, tbase, ref);
  } else if (warp < kMmaWarp) {
    convert_role<F, D, MODE>(a, it, smem, bar, abort, ref);
  } else if (it.nt > 0 && lane == 0) {
    mma_role<D, MODE>(it, smem, bar, abort, tbase);
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tbase, 512);
}

template <typename F, int D, int MODE>
cudaError_t launch_one(const Q8AttendArgs& a, cudaStream_t stream) {
  static SmemLimitSet done;
  constexpr int bytes = Layout<D, MODE>::BYTES;
  const cudaError_t e = ensure_smem_limit(tc_kernel<F, D, MODE>, bytes, done);
  if (e != cudaSuccess) return e;
  const int64_t grid = (int64_t)a.c.B * a.c.Hkv * a.plan.tiles * a.plan.n_chunks;
  tc_kernel<F, D, MODE><<<(unsigned)grid, kThreads, bytes, stream>>>(a);
  return cudaGetLastError();
}

template <typename F, int D>
cudaError_t launch_mode(const Q8AttendArgs& a, cudaStream_t stream) {
  if constexpr (D <= 128)
    return a.plan.mode == kQ8TwoRows ? launch_one<F, D, kQ8TwoRows>(a, stream)
                                     : launch_one<F, D, kQ8TwoStreams>(a, stream);
  else
    return launch_one<F, D, kQ8OneStream>(a, stream);
}

template <typename F>
cudaError_t launch_format(const Q8AttendArgs& a, cudaStream_t stream) {
  switch (a.c.d) {
    case 64: return launch_mode<F, 64>(a, stream);
    case 96: return launch_mode<F, 96>(a, stream);
    case 128: return launch_mode<F, 128>(a, stream);
    default: return launch_mode<F, 256>(a, stream);
  }
}

}  // namespace

int q8_tc_tile_tokens(int d) { return tile_tokens(d); }

cudaError_t launch_q8_tc(const Q8AttendArgs& a, cudaStream_t stream) {
  return a.c.e4m3 ? launch_format<E4m3>(a, stream) : launch_format<Int8>(a, stream);
}

}  // namespace tq
