// q8_tc.cu -- attention of many query rows per kv head (a prefill chunk, drafted
// tokens of grouped heads) over the 8-bit block-scaled cache, bf16 in and out,
// with both products on the fifth-generation tensor cores (tcgen05.mma, f16 in,
// fp32 sums in tensor memory).
//
// Rows.  As in q8_split.cu the query rows of a kv head are its n tokens x G query
// heads, row r = i G + g, cut into tiles of 128 (the M of one product).  With
// S = Q K^T (128 rows x T tokens) and O (128 x d) += P V a CTA holds, by mode:
//   two row tiles (d <= 128, more than 128 rows): both use each token tile, so a code is
//     converted once for 256 rows (T = 128; 64 and two S for each row tile at d = 64);
//   two token streams (d <= 128, up to 128 rows): one row tile, the even token
//     tiles (T = 128) in one (S, O), the odd ones in the other; each writes its own partial;
//   one stream (d = 256, T = 64): one row tile, two S, one O.
// In each the products of one S run while the softmax of the other does.
//
// Warps.  0..3 and 4..7: softmax, a thread per row, so row statistics need no
// exchange (d = 256: 0..3 only).  8..13 (K, V): conversion of codes to f16 operands in
// shared memory, loaded from global memory one tile ahead into registers.
// 14: issues the products; 15: the blocks' scales.
//
// Numbers.  Codes and the queries (bf16, scaled by a power of two per row) are
// exact in f16, so scores carry fp32's rounding alone.  A weight is
// 2^(x - m) s_v / ref with x = S s_k scale log2(e), m the row's reference (moved
// only when weights get large) and ref the item's largest V scale; it is
// rounded to f16's 11 bits, as the bf16 output keeps 8.  The ratio enters as
// its logarithm in the exponent, so it costs nothing, and m is taken from scores with it,
// so weights of a row that sees only small blocks are as exact as others.  It is floored
// at 2^-90 (sums of 2^(x - m) stay in fp32's range): a block whose scale is further below
// ref counts as if it were there, with at most 2^-90 of the item's largest value.  Row
// sums and O are fp32.
//
// Operand layout in shared memory, without swizzle: [d / 8][rows][16 bytes] (and a pad
// after each column of rows), an 8 x 16-byte core matrix contiguous.  For K that is K-major
// (rows = tokens), and the same bytes are MN-major for V, so one converter serves both.  int8
// codes leave the converter in the order 0 2 1 3 of each word: Q is stored in that order,
// and O's columns are put back when they are written.
//
// Bound: for long chunks the exponentials and the products in turn (the softmax of one
// row tile overlaps the other's products, 41% to 49% of the tensor cores' time each):
// 2048 tokens of 64/8 heads at 16K, d 128, int8, normal draws, 953 us = 1.08 PFLOP/s, 65%
// of the measured matrix-product rate (e4m3 921 us; keys and values with outliers, where
// the reference moves more often, 1050 us); d 256 (32/16 heads, 1024 tokens at 8K) 260 us
// = 0.99; d 96 (32/32, 2048 at 8K) 263 us = 0.68 and d 64 (2 x 32/8, 2048 at 8K) 426 us
// = 0.56, whose products are shorter per exponential.  For few rows
// the chain of products and softmax of a token tile, 2100 clocks where HBM would need
// 1420: 5 drafted tokens at 128K 82 us, 3.3 TB/s.
#include <limits.h>
#include <math.h>

#include "q8_common.cuh"
#include "q8_internal.h"

namespace tq {
namespace {

using namespace q8;
using namespace tc;

constexpr int kSoftmaxWarps = 8, kConvertWarps = 3;  // (3 for K and 3 for V)
constexpr int kMmaWarp = kSoftmaxWarps + 2 * kConvertWarps, kScaleWarp = kMmaWarp + 1;
constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kConvertThreads = 32 * kConvertWarps;
// Registers of a thread: 2 x 144 + 2 x 112 = 4 x 128, what the four warpgroups are launched
// with.  A softmax thread holds 64 scores; what does not fit is spilled to local memory, and
// L1, which the operands leave next to nothing, misses on half of that.
constexpr int kSoftmaxRegs = 144, kOtherRegs = 112;
// kCubic of every 8 pairs of exponentials take the cubic on the FMA pipe: 16 a clock and SM
// would bound the tile (2 x 128 x 128 of them in the 2048 clocks of its products)
constexpr int kCubic = 2;
// The reference is held 2^kShift below the maximum it was taken from, and moves when 16
// weights sum to 2^15.  With 7 it moved more often (2048-token chunk at 16K with outliers
// 1120 us against 1046); weights keep 11 bits down to 2^-18 of the largest, and 2^-28 of it
// is their last bit.
constexpr float kShift = 4.0f, kTopSum = 32768.0f;
constexpr float kMasked = -3e38f, kMinRatio = 0x1p-90f;
constexpr int kScaleSlots = 4, kPrefetch = 2;

// Tokens of a tile.  With 64 there is room for a second score tile of each row tile, so that
// the softmax does not wait for its products, but products of 64 columns read Q from shared
// memory twice as often: 434 us against 459 for a 2048-token chunk at 8K with d = 64, 1117
// against 946 at 16K with d = 128, 319 against 309 with d = 96.
__host__ __device__ constexpr int tile_tokens(int d, int mode) {
  return d > 128 || (d == 64 && mode == kQ8TwoRows) ? 64 : 128;
}
// what a column of its operands (8 dims of all tokens) is longer than them
__host__ __device__ constexpr int column_pad(int d) { return d == 96 ? 32 : 16; }

template <int D, int MODE>
struct Layout {
  static constexpr int T = tile_tokens(D, MODE), H = 64, NH = T / H;  // halves of a tile of 128
  static constexpr int QT = MODE == kQ8TwoRows ? 2 : 1;
  static constexpr int NS = D <= 128 && T == 64 ? 4 : 2;   // tiles of K and of V in shared memory
  static constexpr int kUnits = MODE == kQ8TwoRows ? 2 : 1;
  static constexpr int NB = kUnits == 2 && T == 64 ? 4 : 2;  // score tiles in tensor memory
  static constexpr int kAhead = NB / kUnits;                 // of one row tile
  // Row r of a tile sits at place r ^ kRowFlip: up to 64 rows then belong to the warps of the
  // two schedulers that have one converter each, not two (5 drafts x 8 sequences:
  // 134 -> 131 us).
  static constexpr int kRowFlip = MODE == kQ8TwoRows ? 0 : 64;
  static constexpr int Q_BYTES = 128 * D * 2, COLUMN = T * 16 + column_pad(D), KV_BYTES = D / 8 * COLUMN;
  static constexpr int Q = 0, K = Q + QT * Q_BYTES, V = K + NS * KV_BYTES;
  static constexpr int CROW = V + NS * KV_BYTES;            // float [QT * 128]
  static constexpr int SCALES = CROW + 4 * QT * 128;        // float4 [kScaleSlots][T / 16]
  static constexpr int BAR = SCALES + 16 * kScaleSlots * (T / 16);
  static constexpr int MISC = BAR + 8 * 40;                 // tmem base, abort, ref, warp maxima
  static constexpr int BYTES = MISC + 16 + 4 * kWarps;
  static_assert(BYTES <= 227 * 1024, "shared memory");
  static __host__ __device__ constexpr uint32_t S(int b) { return (uint32_t)(b * T); }
  static __host__ __device__ constexpr uint32_t O(int u) { return (uint32_t)(NB * T + u * D); }
};

enum Bar : int {
  kKFull = 0,    // [NS] K operand written (convert warps)
  kKEmpty = 4,   // [NS] its products done (commit)
  kVFull = 8,
  kVEmpty = 12,
  kSFull = 16,   // [NB] scores in tensor memory (commit)
  kPFull = 20,   // [NB][NH] weights of a half in tensor memory (4 softmax warps)
  kPVDone = 24,  // [units][NH] O up to date with that half of a tile (commit)
  kScFull = 28,  // [kScaleSlots] block scales written (one warp)
  kScEmpty = 32, // [kScaleSlots] read: every weight of the tile is there (product warp)
  kDone = 36,    // every product complete (commit)
  kBars = 37
};

// What one CTA does: a work item's rows, and tokens [begin, stop) in nt tiles.
struct Item : Q8Item {
  int begin, stop, nt;
  __device__ __forceinline__ Item(const Q8AttendArgs& a, int id) : Q8Item(a, id) {}
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

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// Pins registers written by tcgen05.ld behind the wait before this.
__device__ __forceinline__ void tie32(uint32_t (&r)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]),
                 "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7]));
}

// O of a warp's 32 rows times alpha
template <int D>
__device__ __forceinline__ void rescale(uint32_t col, float alpha) {
#pragma unroll 1
  for (int c = 0; c < D / 8; ++c) {
    uint32_t o[8];
    tld_x8(col + 8 * c, o);
    wait_ld();
    asm volatile("" : "+r"(o[0]), "+r"(o[1]), "+r"(o[2]), "+r"(o[3]), "+r"(o[4]), "+r"(o[5]), "+r"(o[6]), "+r"(o[7]));
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
    tst_x8_quiet(col + 8 * c, o);
  }
}

// ------------------------------------------------------------------ conversion

// One thread's 16-byte pieces of a tile of codes, p = thread + kConvertThreads i.  Eight
// neighbouring lanes take kC pieces of each of kT tokens: a load touches few lines (with
// eight tokens a load it took 28 clocks of the SM, not 8), and with the columns of the
// operand kPad bytes further apart their stores fill all banks.
template <int D, int T>
struct Pieces {
  static constexpr int C = D / 16, N = (T * C + kConvertThreads - 1) / kConvertThreads;
  static constexpr int kC = D == 96 ? 2 : 4, kT = 8 / kC, kPad = column_pad(D);
  static constexpr int kStep = kConvertThreads / C;  // tokens from one piece of a thread to the next
  static_assert(kConvertThreads % (8 * C / kC) == 0, "a thread's pieces are the same bytes of their tokens");
  static constexpr bool kRest = T * C % kConvertThreads != 0;  // whole warps have no last piece
  uint4 w[N];
  static __device__ __forceinline__ int token(int p) { return p / kC % kT + kT * ((p >> 3) / (C / kC)); }
  static __device__ __forceinline__ int c16(int p) { return p % kC + kC * ((p >> 3) % (C / kC)); }
  static __device__ __forceinline__ int piece(int tid, int i) { return tid + kConvertThreads * i; }
  static __device__ __forceinline__ bool has(int tid, int i) { return !kRest || i + 1 < N || piece(tid, i) < T * C; }
  __device__ __forceinline__ void load_one(int i, const uint8_t* at) {
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                 : "l"(at));
  }
  // rows of the tile behind the first `rows` repeat the last one: what is multiplied is
  // always cache content
  __device__ __forceinline__ void load(const uint8_t* tile, int rows, int tid) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int p = piece(tid, i);
      if (has(tid, i)) load_one(i, tile + min(token(p), rows - 1) * D + 16 * c16(p));
    }
  }
  // Stores the operand.  Where the next tile is whole each register is loaded again as soon
  // as its piece is stored, so that a load has the time of a whole tile to arrive.
  template <typename F, bool NEXT>
  __device__ __forceinline__ void store(unsigned char* dst, const uint8_t* next, int tid) {
    constexpr int column = T * 16 + kPad;
    unsigned char* at = dst + 2 * c16(tid) * column + token(tid) * 16;
    const uint8_t* from = next + token(tid) * D + 16 * c16(tid);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (!has(tid, i)) continue;
      uint4 lo, hi;
      F::cvt_word(w[i].x, lo.x, lo.y);
      F::cvt_word(w[i].y, lo.z, lo.w);
      F::cvt_word(w[i].z, hi.x, hi.y);
      F::cvt_word(w[i].w, hi.z, hi.w);
      *reinterpret_cast<uint4*>(at + i * kStep * 16) = lo;
      *reinterpret_cast<uint4*>(at + i * kStep * 16 + column) = hi;
      if constexpr (NEXT) load_one(i, from + i * kStep * D);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
  }
};

// K and V have converters of their own (one code, so that it stays in the instruction
// cache), which keeps two tiles in flight.
template <typename F, int D, int MODE>
__device__ __forceinline__ void convert_role(const Q8AttendArgs& a, const Item& it, unsigned char* smem,
                                             uint64_t* bar, volatile int* abort, bool is_v, int tid) {
  using L = Layout<D, MODE>;
  const int lane = tid & 31;
  const uint8_t* tile = head_codes<D>(is_v ? a.c.v_codes : a.c.k_codes, a, it.bh) + (int64_t)it.begin * D;
  uint64_t* full = bar + (is_v ? kVFull : kKFull);
  uint64_t* empty = bar + (is_v ? kVEmpty : kKEmpty);
  unsigned char* operand = smem + (is_v ? L::V : L::K);
  Pieces<D, L::T> x;
  if (it.nt > 0) x.load(tile, it.stop - it.begin, tid);
#pragma unroll 1
  for (int j = 0; j < it.nt; ++j) {
    const int s = j % L::NS;
    if (j >= L::NS) warp_wait(empty + s, (j / L::NS - 1) & 1, abort);
    tile += L::T * D;
    const int rows = it.stop - it.begin - (j + 1) * L::T;  // of the next tile
    if (rows >= L::T)
      x.template store<F, true>(operand + s * L::KV_BYTES, tile, tid);
    else
      x.template store<F, false>(operand + s * L::KV_BYTES, tile, tid);
    if (lane == 0 && !(a.test_starve && !is_v && j == 0)) mbar_arrive(full + s);
    if (rows > 0 && rows < L::T) x.load(tile, rows, tid);
  }
}

// Codes of tile j into L2, kPrefetch tiles before the converters load them (the first ones
// while the queries are prepared): their registers hold one tile of K and one of V.
template <int D, int MODE>
__device__ __forceinline__ void prefetch_tile(const Q8AttendArgs& a, const Item& it, int j) {
  constexpr int T = Layout<D, MODE>::T;
  if (j >= it.nt) return;
  const int tok0 = it.begin + j * T, bytes = min(T, it.stop - tok0) * D;
  prefetch_l2(head_codes<D>(a.c.k_codes, a, it.bh) + (int64_t)tok0 * D, bytes);
  prefetch_l2(head_codes<D>(a.c.v_codes, a, it.bh) + (int64_t)tok0 * D, bytes);
}

// For each 16 tokens of a tile {s_k, log2(s_v / ref), ref / s_v}: a warp of its own, since
// the logarithm and the divisions held a converter up for a third of its time.
template <int D, int MODE>
__device__ __forceinline__ void scale_role(const Q8AttendArgs& a, const Item& it, unsigned char* smem,
                                           uint64_t* bar, volatile int* abort, float ref, int lane) {
  using L = Layout<D, MODE>;
  const float* ksc = a.c.k_scales + (int64_t)it.bh * a.c.n_blocks();
  const float* vsc = a.c.v_scales + (int64_t)it.bh * a.c.n_blocks();
  const int shift = 31 - __clz(a.c.block);
  float sk = 0.0f, sv = 0.0f;
  auto load = [&](int j) {
    if (lane >= L::T / 16 || j >= it.nt) return;
    const int blk = min(it.begin + j * L::T + 16 * lane, it.stop - 1) >> shift;
    sk = __ldg(ksc + blk);
    sv = __ldg(vsc + blk);
  };
  load(0);
#pragma unroll 1
  for (int j = 0; j < it.nt; ++j) {
    if (lane == 0) prefetch_tile<D, MODE>(a, it, j + kPrefetch);
    const float ratio = ref > 0.0f ? fmaxf(sv / ref, kMinRatio) : 1.0f;
    const float4 k = make_float4(sk, log2f(ratio), 1.0f / ratio, 0.0f);
    load(j + 1);
    if (a.test_slow_scales) __nanosleep(20000);
    // The slot was tile j - 4's.  Its barrier cannot pass two phases while this warp is late
    // (the parity would then read as not yet): the next one takes tile j's own scales.  The
    // operands' barriers would not do, as tile j's scores need no scales.
    const int slot = j & (kScaleSlots - 1);
    if (j >= kScaleSlots) warp_wait(bar + kScEmpty + slot, (j / kScaleSlots - 1) & 1, abort);
    if (lane < L::T / 16) reinterpret_cast<float4*>(smem + L::SCALES)[slot * (L::T / 16) + lane] = k;
    __syncwarp();
    if (lane == 0) mbar_arrive(bar + kScFull + slot);
  }
}

// -------------------------------------------------------------------- products

// The whole warp runs this, so that addresses and descriptors stay in uniform registers;
// one elected thread issues.
template <int D, int MODE>
__device__ __forceinline__ void mma_role(const Item& it, unsigned char* smem, uint64_t* bar,
                                         volatile int* abort, uint32_t tbase) {
  using L = Layout<D, MODE>;
  constexpr uint32_t idS = idesc_f16(128, L::T, 0, 0), idO = idesc_f16(128, D, 0, 1);
  // descriptors: the upper words are constants, the lower ones add (bytes / 16) offsets
  constexpr uint64_t q0 = smem_desc(0, 128 * 16, 128), k0 = smem_desc(0, L::COLUMN, 128), v0 = smem_desc(0, 128, L::COLUMN);
  const uint32_t at = smem_u32(smem) >> 4;
  const bool leader = elect_one();
  auto commit = [&](int b) {
    if (leader) mma_commit(bar + b);
  };
  // scores of token tile j into S[b], from row tile u of Q
  auto scores = [&](int j, int u, int b) {
    const uint32_t q = at + ((L::Q + u * L::Q_BYTES) >> 4), k = at + ((L::K + j % L::NS * L::KV_BYTES) >> 4);
    if (leader && !*abort) {
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
        mma_ss(tbase + L::S(b), q0 | (q + c * 2 * 128), k0 | (k + c * 2 * (L::COLUMN >> 4)), idS, c > 0);
    }
    commit(kSFull + b);
  };
  // O[u] += P[b] V of token tile j, half by half as their weights come
  auto values = [&](int j, int u, int b, bool first) {
    const uint32_t v = at + ((L::V + j % L::NS * L::KV_BYTES) >> 4);
    constexpr int n = L::H / 16;  // products of 16 tokens in a half
#pragma unroll
    for (int h = 0; h < L::NH; ++h) {
      warp_wait(bar + kPFull + b * L::NH + h, (j / L::kAhead) & 1, abort);
      fence_after();
      if (leader && !*abort) {
#pragma unroll
        for (int c = h * n; c < (h + 1) * n; ++c)
          mma_ts(tbase + L::O(u), tbase + L::S(b) + 8 * c, v0 | (v + c * 16), idO, c > 0 || !first);
      }
      commit(kPVDone + u * L::NH + h);
    }
  };
  auto wait_k = [&](int j) {
    warp_wait(bar + kKFull + j % L::NS, (j / L::NS) & 1, abort);
    fence_after();
  };
  auto wait_v = [&](int j) {
    warp_wait(bar + kVFull + j % L::NS, (j / L::NS) & 1, abort);
    fence_after();
  };
  for (int j = 0; j < L::kAhead && j < it.nt; ++j) {
    wait_k(j);
#pragma unroll
    for (int u = 0; u < L::kUnits; ++u) scores(j, u, L::kAhead * u + j);
    commit(kKEmpty + j);
  }
#pragma unroll 1
  for (int j = 0; j < it.nt; ++j) {
    const int next = j + L::kAhead;
    wait_v(j);
#pragma unroll
    for (int u = 0; u < L::kUnits; ++u) {
      const int b = L::kAhead * u + j % L::kAhead;
      values(j, MODE == kQ8TwoStreams ? b : u, b, MODE == kQ8TwoStreams ? j < 2 : j == 0);
      if (next < it.nt) {
        if (u == 0) wait_k(next);
        scores(next, u, b);
      }
    }
    if (leader) mbar_arrive(bar + kScEmpty + (j & (kScaleSlots - 1)));
    commit(kVEmpty + j % L::NS);
    if (next < it.nt) commit(kKEmpty + next % L::NS);
  }
  commit(kDone);
  if (leader) mbar_drain(bar + kDone, 0);
}

// --------------------------------------------------------------------- softmax

// 2^x on the FMA pipe, of arguments limited to [-kCubicTop, kCubicTop]: a masked score counts as
// the lower end, and one far above the reference must come out large, for the reference to be
// moved, and not run over into the sign.  The saturation of the multiply-add that yields
// y = (x / kCubicTop + 1) / 2 does both (minimum and maximum as instructions: a 2048-token
// chunk at 16K 970 us against 960; d = 64 434 against 425).
constexpr float kCubicTop = 126.0f;
__device__ __forceinline__ float saturated(float a, float b, float c) {
  float d;
  asm("fma.rn.sat.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// With x = n + r, n the nearest integer (by the adder: 1.5 2^23 + x), 2^r is the cubic that
// minimises the relative error on |r| <= 1/2 (7.5e-5, by exchange; a weight is rounded to
// 2^-11 anyway) and n is added to the exponent.
__device__ __forceinline__ float2 ex2_cubic(float2 y) {
  constexpr float kMagic = 12582912.0f, c0 = 0.99992806f, c1 = 0.69326097f, c2 = 0.24261113f, c3 = 0.05517167f;
  const float2 span = make_float2(2.0f * kCubicTop, 2.0f * kCubicTop), from = make_float2(kMagic - kCubicTop, kMagic - kCubicTop);
  const float2 t = fma2(y, span, from);
  const float2 r = fma2(y, span, sub2(from, t));
  float2 p = fma2(r, make_float2(c3, c3), make_float2(c2, c2));
  p = fma2(p, r, make_float2(c1, c1));
  p = fma2(p, r, make_float2(c0, c0));
  return make_float2(__uint_as_float(__float_as_uint(p.x) + (__float_as_uint(t.x) << 23)),
                     __uint_as_float(__float_as_uint(p.y) + (__float_as_uint(t.y) << 23)));
}

// A half tile of H tokens of one row: its scores in registers, and for each 16 tokens
// {s_k, log2(s_v / ref), ref / s_v} in shared memory.  What else a thread keeps is little
// enough for 128 registers: anything spilled here costs an L2 access per tile, since the
// operands leave L1 next to nothing.
template <int H>
struct Half {
  uint32_t s[H / 32][32];

  __device__ __forceinline__ void load(uint32_t col) {
#pragma unroll
    for (int c = 0; c < H / 32; ++c) tld_x32(col + 32 * c, s[c]);
    wait_ld();
#pragma unroll
    for (int c = 0; c < H / 32; ++c) tie32(s[c]);
  }
  __device__ __forceinline__ float at(int i) const { return __uint_as_float(s[i / 32][i % 32]); }
  // A factor of 0 (a block of zeros, whose scores are 0 with any factor) must not let
  // masked scores through.
  static __device__ __forceinline__ float factor(float s_k, float crow) { return fmaxf(s_k * crow, 1e-30f); }

  // the row sees only the first `left` tokens
  __device__ __forceinline__ void mask(int left) {
#pragma unroll
    for (int i = 0; i < H; ++i)
      if (i >= left) s[i / 32][i % 32] = __float_as_uint(kMasked);
  }

  // The largest weight's logarithm before the reference is taken off: with the blocks' V
  // scales, so that weights keep their bits where a row sees only blocks far below ref.
  __device__ __forceinline__ float max(const float4* sc, float crow) const {
    float mx = -INFINITY;
#pragma unroll
    for (int g = 0; g < H / 16; ++g) {
      float top = at(16 * g);
#pragma unroll
      for (int i = 16 * g + 1; i < 16 * g + 16; ++i) top = fmaxf(top, at(i));
      mx = fmaxf(mx, fmaf(top, factor(sc[g].x, crow), sc[g].y));
    }
    return mx;
  }

  // The weights 2^(x + log2(s_v / ref) - m), into tensor memory over scores already read.
  // Returns the sum of 2^(x - m); top is the largest sum of 16 weights.
  __device__ __forceinline__ float weights(uint32_t col, const float4* sc, float crow, float m, float& top) const {
    float l = 0.0f;
    top = 0.0f;
    float4 k = sc[0];
#pragma unroll
    for (int g = 0; g < H / 16; ++g) {
      const float4 now = k;
      if (g + 1 < H / 16) k = sc[g + 1];
      const float f = factor(now.x, crow), off = now.y - m;
      const float f_y = f * (0.5f / kCubicTop), off_y = fmaf(off, 0.5f / kCubicTop, 0.5f);
      float2 x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float s0 = at(16 * g + 2 * i), s1 = at(16 * g + 2 * i + 1);
        if (i * kCubic / 8 != (i + 1) * kCubic / 8)
          x[i] = make_float2(saturated(s0, f_y, off_y), saturated(s1, f_y, off_y));
        else
          x[i] = fma2(make_float2(s0, s1), make_float2(f, f), make_float2(off, off));
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        x[i] = i * kCubic / 8 != (i + 1) * kCubic / 8 ? ex2_cubic(x[i]) : make_float2(ex2(x[i].x), ex2(x[i].y));
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = f16x2(x[i].x, x[i].y);
      tst_x8_quiet(col + 8 * g, w);
      const float2 s2 = add2(add2(add2(x[0], x[1]), add2(x[2], x[3])), add2(add2(x[4], x[5]), add2(x[6], x[7])));
      const float sum = s2.x + s2.y;
      top = fmaxf(top, sum);
      l = fmaf(sum, now.z, l);
    }
    return l;
  }
};

template <typename F, int D, int MODE>
__device__ __forceinline__ void softmax_role(const Q8AttendArgs& a, int begin, int stop, int nt, const Q8Seq& seq,
                                             unsigned char* smem, uint64_t* bar, volatile int* abort,
                                             uint32_t tbase, float ref) {
  using L = Layout<D, MODE>;
  constexpr int T = L::T;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, u = warp >> 2, quarter = warp & 3;
  const int local = ((MODE == kQ8TwoRows ? 128 * u : 0) + 32 * quarter + lane) ^ L::kRowFlip;
  int limit = INT_MAX;  // (of a row of no query)
  bool live = false;
  {
    const Item it(a, blockIdx.x);
    const int i = it.token(local);
    live = it.row0 + local < it.rows && i < seq.q_len;
    if (live) limit = seq.limit(i);
  }
  const bool warp_live = __any_sync(0xffffffffu, live);
  const int open = __reduce_min_sync(0xffffffffu, limit);  // tokens below are seen by the whole warp
  const float crow = reinterpret_cast<const float*>(smem + L::CROW)[local];
  const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
  float m = -INFINITY, l = 0.0f;
  // this warp's tiles: all of them, or every second
  constexpr int step = MODE == kQ8TwoStreams ? 2 : 1;
  const int ou = MODE == kQ8OneStream ? 0 : u;
  int n = 0;  // tiles done
  for (int j = MODE == kQ8TwoStreams ? u : 0; j < nt; j += step, ++n) {
    const int sb = (MODE == kQ8TwoRows ? L::kAhead * u : 0) + j % L::kAhead;
    const uint32_t s_col = tbase + lanes + L::S(sb);
    warp_wait(bar + kScFull + (j & (kScaleSlots - 1)), (j / kScaleSlots) & 1, abort);
    const float4* sc = reinterpret_cast<const float4*>(smem + L::SCALES) + (j & (kScaleSlots - 1)) * (T / 16);
    warp_wait(bar + kSFull + sb, (j / L::kAhead) & 1, abort);
    fence_after();
    // 64 tokens are a step of the online softmax: that many scores fit in registers, and the
    // product of one half of a tile of 128 starts while the other's weights are computed.  The weights are
    // computed with the reference as it is; if 16 of them sum to more than kTopSum
    // (f16 would overflow soon) it is moved and they are computed again, so that no maximum
    // has to be taken otherwise.
#pragma unroll 1
    for (int h = 0; h < L::NH; ++h) {
      if (warp_live) {
        constexpr int H = L::H;
        Half<H> x;
        const float4* sch = sc + h * (H / 16);
        const int tok0 = begin + j * T + h * H;
        const int left = min(limit, stop) - tok0;  // tokens of this half that the row sees
        x.load(s_col + h * H);
        if (tok0 + H > min(open, stop)) x.mask(left);
        const uint32_t p_col = s_col + h * (H / 2);
        float top, sum = x.weights(p_col, sch, crow, m == -INFINITY ? 0.0f : m, top);
        const bool move = top > kTopSum || m == -INFINITY;
        if (__any_sync(0xffffffffu, move)) {
          const float mn = move && left > 0 ? fmaxf(m, x.max(sch, crow) - kShift) : m;  // m is held 2^kShift low
          const float alpha = mn == m ? 1.0f : exp2f(m - mn);
          m = mn;
          l *= alpha;
          if (n + h > 0) {  // once O is up to date
            // (the scores at hand came after all but the last tile's product)
            if (n > 0) warp_wait(bar + kPVDone + (ou + 1) * L::NH - 1, (n - 1) & 1, abort);
            if (h > 0) warp_wait(bar + kPVDone + ou * L::NH, n & 1, abort);
            fence_after();
            rescale<D>(tbase + lanes + L::O(ou), alpha);
          }
          wait_st();
          sum = x.weights(p_col, sch, crow, m == -INFINITY ? 0.0f : m, top);
        }
        l += sum;
        wait_st();
        fence_before();
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(bar + kPFull + sb * L::NH + h);
    }
  }
  if (nt > 0) warp_wait(bar + kDone, 0, abort);
  fence_after();
  if (!warp_live) return;
  const bool none = n == 0 || (m == -INFINITY && l == l);  // (masked weights of the cubic are 2^-126, not 0)
  if (none) l = 0.0f;
  // where the row goes, worked out anew rather than kept in registers through the loop
  int id;
  asm volatile("mov.u32 %0, %%ctaid.x;" : "=r"(id));
  const Item it(a, id);
  const int64_t orow = it.out_row(a, local);
  const bool split = it.split;
  if (*abort) l = __int_as_float(0x7fc00000);
  const int e = sum_exponent(l);
  const float down = pow2i(-e);
  m += (float)e;
  l *= down;
  float f = split ? down : down / l;
  if (__any_sync(0xffffffffu, f * ref < 0x1p-100f)) {  // O by parts, where the product might lose bits
    rescale<D>(tbase + lanes + L::O(ou), f);
    wait_st();
    f = 1.0f;
  }
  f *= ref;
  float* part = it.part(a, local, MODE == kQ8TwoStreams ? u : 0);
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
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  Item it(a, blockIdx.x);
  const Q8Seq seq(a, it.b);
  q8_write_flags(a);
  const int first_i = it.row0 / it.G;
  const int q_last = min(min(it.rows - 1, it.row0 + a.plan.row_tile - 1) / it.G, seq.q_len - 1);
  const int stop_all = q_last < first_i ? 0 : seq.limit(q_last);
  it.begin = it.chunk_id * it.chunk;
  it.stop = it.split ? it.begin + min(stop_all - it.begin, it.chunk) : stop_all;
  it.nt = max(0, (it.stop - it.begin + L::T - 1) / L::T);
  // nothing to do (rows that see no token get zeros here, or from the merge)
  if (!it.any || q_last < first_i || (it.nt == 0 && it.split)) return;

  if (warp == kScaleWarp && lane == 0)
    for (int j = 0; j < kPrefetch; ++j) prefetch_tile<D, MODE>(a, it, j);
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar + kKFull + i, kConvertWarps);
      mbar_init(bar + kKEmpty + i, 1);
      mbar_init(bar + kVFull + i, kConvertWarps);
      mbar_init(bar + kVEmpty + i, 1);
      mbar_init(bar + kSFull + i, 1);
      mbar_init(bar + kPFull + i, 4);
      mbar_init(bar + kPVDone + i, 1);
    }
#pragma unroll
    for (int i = 0; i < kScaleSlots; ++i) {
      mbar_init(bar + kScFull + i, 1);
      mbar_init(bar + kScEmpty + i, 1);
    }
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
  constexpr int R = 7;                  // rows of a warp whose loads are in flight together
#pragma unroll 1
  for (int r0 = warp; r0 < L::QT * 128; r0 += R * kWarps) {
    uint2 v[R][W];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int r = r0 + k * kWarps;
      const bool live = r < L::QT * 128 && it.row0 + r < it.rows && it.token(r) < seq.q_len;
      const uint16_t* q = static_cast<const uint16_t*>(a.q) + it.out_row(a, r) * D;
#pragma unroll
      for (int w = 0; w < W; ++w)
        v[k][w] = live && lane + 32 * w < D / 4 ? *reinterpret_cast<const uint2*>(q + 4 * (lane + 32 * w))
                                                : make_uint2(0u, 0u);
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int r = r0 + k * kWarps;
      if (r >= L::QT * 128) break;
      float x[W][4], big = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        x[w][0] = __uint_as_float(v[k][w].x << 16);
        x[w][1] = __uint_as_float(v[k][w].x & 0xffff0000u);
        x[w][2] = __uint_as_float(v[k][w].y << 16);
        x[w][3] = __uint_as_float(v[k][w].y & 0xffff0000u);
#pragma unroll
        for (int e = 0; e < 4; ++e) big = fmaxf(big, fabsf(x[w][e]));
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
      const int e = query_exponent(big);
      const float up = pow2i(e);
      unsigned char* dst = smem + L::Q + (r >> 7) * L::Q_BYTES + ((r ^ L::kRowFlip) & 127) * 16;
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
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tbase = static_cast<uint32_t>(misc[0]);
  float ref = 0.0f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) ref = fmaxf(ref, warp_max[w]);

  if (warp >= kSoftmaxWarps)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  else
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
  if (warp < kSoftmaxWarps) {
    if (MODE != kQ8OneStream || warp < 4)
      softmax_role<F, D, MODE>(a, it.begin, it.stop, it.nt, seq, smem, bar, abort, tbase, ref);
  } else if (warp < kMmaWarp) {
    const int tid = threadIdx.x - 32 * kSoftmaxWarps;
    const bool is_v = tid >= kConvertThreads;
    convert_role<F, D, MODE>(a, it, smem, bar, abort, is_v, is_v ? tid - kConvertThreads : tid);
  } else if (warp == kScaleWarp) {
    scale_role<D, MODE>(a, it, smem, bar, abort, ref, lane);
  } else {
    if (it.nt > 0) mma_role<D, MODE>(it, smem, bar, abort, __shfl_sync(0xffffffffu, tbase, 0));
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
  tc_kernel<F, D, MODE><<<(unsigned)a.plan.items(), kThreads, bytes, stream>>>(a);
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

int q8_tc_tile_tokens(int d, Q8Mode mode) { return tile_tokens(d, mode); }

cudaError_t launch_q8_tc(const Q8AttendArgs& a, cudaStream_t stream) {
  return a.c.e4m3 ? launch_format<E4m3>(a, stream) : launch_format<Int8>(a, stream);
}

}  // namespace tq
