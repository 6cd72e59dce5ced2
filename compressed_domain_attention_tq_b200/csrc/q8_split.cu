// q8_split.cu -- attention over the 8-bit block-scaled cache for few query rows
// per kv head (decode, drafted tokens), and for fp32 outputs of any length.
//
// Rows.  The query rows of a kv head are its n tokens x G query heads, row
// r = i G + g.  A work item is (sequence, kv head, tile of 8 NT rows, chunk of
// the context); a CTA of four warps takes one, its warps every fourth step of
// 16 tokens.  16 tokens never cross a block, so a step has one scale of K and
// one of V.
//
// A step is two products on the warp-level tensor cores (m16n8k16, f16 in,
// fp32 sums), both with the cache as the 16-row operand:
//   S (16 tokens x 8 rows) = K codes (16 x d) . Q^T,
//   O (16 dims x 8 rows)  += V codes^T (16 dims x 16 tokens) . W.
// The summed index may be permuted as long as both operands agree, so a lane
// takes 16 contiguous bytes of a row wherever the fragment wants four pairs.
// A warp copies its own steps into a ring of its own in shared memory
// (cp.async), two steps ahead of the one it computes: no barrier is on the way,
// and the copies cost no registers.  Loads straight into the lanes' registers,
// one step ahead, waited for HBM in every step (side by side: 128K, 64/8 heads, d 128
// 62 us against 60; d 256, 64K, 4 sequences 408 against 356).
//
// Precision: codes are exact in f16.  Each query row is scaled by a power of
// two and split into f16 hi + lo (22 bits; bf16 queries have no lo part), the
// weights W = 2^(x - m) s_v / 2^E likewise, so a product costs two instructions and
// keeps ~2^-22.  x = S s_k scale log2(e); E is the exponent of the largest V scale so
// far; m is a row's reference, moved only when a W comes near 2^15.  It is taken from
// x and s_v together, so the tokens that make up the output have their bits, whether
// by their weight or by their values: with m from x alone the weights of a block of V
// 1e5 times the others' and 14 nats below them came near f16's smallest number.  When
// E grows m falls with it, and O stays as it is.  Sums of weights and O are fp32.
//
// Bound: HBM for decode (one pass over the codes).  Measured (int8, bf16 queries, captured
// calls repeated on one input): d 256, 64K x 4 sequences, 32/16 heads 359 us, 91% of the
// measured copy rate; d 128, 32K x 8 sequences, 64/8 heads 109 us, 75%; 128K of one
// sequence 62 us, 66% (e4m3 59), about 15 us of it launches, the first step's latency and
// the merge.  Tiles of 16 rows
// (NT = 2) convert a code once for two products; they are taken when a kv head
// has more than 8 rows.
#include <limits.h>
#include <math.h>

#include "q8_common.cuh"
#include "q8_internal.h"

namespace tq {
namespace {

using namespace q8;

constexpr int kWarps = 4, kThreads = 32 * kWarps, kStep = 16;
constexpr float kTau = 7.0f;    // how far (log2) a weight may exceed the reference
constexpr float kShift = 7.0f;  // weights are kept 2^kShift larger: W < 2^(kTau + kShift + 1)
// V scales count as no further than 2^kSpan apart in m, so that sums of 2^(x - m) stay in
// fp32's range (2^(kTau + kShift + kSpan) a token); those of blocks of zeros, which add to the
// sum of weights alone, as 2^-kZeroSpan of the largest
constexpr int kSpan = 90, kZeroSpan = 45, kNoScale = -1000;

// Byte offsets in a row of d codes.  K: word w (0 .. d/16 - 1) of lane t of 4;
// V: word w (0 .. d/32 - 1) of lane g of 8.  Whole 16-byte loads where d allows.
template <int D>
__device__ __forceinline__ int k_offset(int w, int t) {
  constexpr int full = D / 64 * 4;
  return w < full ? 64 * (w >> 2) + 16 * t + 4 * (w & 3) : 16 * full + 8 * t + 4 * (w - full);
}
template <int D>
__device__ __forceinline__ int v_offset(int w, int g) {
  if constexpr (D >= 128) return 128 * (w >> 2) + 16 * g + 4 * (w & 3);
  return w < 2 ? 8 * g + 4 * w : 64 + 4 * g;  // 64, 96
}

// A warp's ring of steps in shared memory: 16 rows of K, 16 of V, their two scales.
// 16-byte chunks are placed so that the fragment loads of eight lanes (K: two rows, four
// chunks; V: four rows, two chunks) meet no bank twice.
template <int D, int NT = 1>
struct Ring {
  // as many steps as leave room for the CTAs that the registers allow (resident())
  static constexpr int kRows = kStep * D, kBytes = 2 * kRows + 16, kSlots = D == 64 ? 4 : D == 256 && NT == 2 ? 2 : 3;
  // A step's rows are contiguous in the cache; lane l copies its chunks 32 i + l, i < D / 32.
  // Where they go: 512 i behind chunk l's place, for V with the bits of the row that change
  // with i folded in.
  static __host__ __device__ constexpr int v_flip(int i) { return D == 256 ? 32 * i & 96 : D == 128 ? 64 * i & 64 : 0; }
  static __device__ __forceinline__ int k_chunk(int row, int ch) { return D >= 128 ? ch ^ ((row & 1) << 2) : ch; }
  static __device__ __forceinline__ int v_chunk(int row, int ch) {
    return D >= 128 ? ch ^ (row & 6) : D == 64 ? ch ^ (row & 2) : ch;
  }
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

template <int N>
__device__ __forceinline__ void ld(uint32_t* r, const unsigned char* p) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    r[0] = v.x, r[1] = v.y;
  } else {
    r[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// K words of token row g (or g + 8) of lane t; V words of token row 2t (+ 1, 8, 9) of lane g
template <int D>
__device__ __forceinline__ void load_k(uint32_t (&r)[D / 16], const unsigned char* row, int g, int t) {
#pragma unroll
  for (int w = 0; w + 4 <= D / 16; w += 4) ld<4>(r + w, row + 16 * Ring<D>::k_chunk(g, 4 * (w >> 2) + t));
  if constexpr (D % 64) ld<2>(r + D / 64 * 4, row + k_offset<D>(D / 64 * 4, t));
}
template <int D>
__device__ __forceinline__ void load_v(uint32_t (&r)[D / 32], const unsigned char* row, int g, int t) {
  if constexpr (D >= 128) {
#pragma unroll
    for (int w = 0; w < D / 32; w += 4) ld<4>(r + w, row + 16 * Ring<D>::v_chunk(2 * t, 8 * (w >> 2) + g));
  } else {
    ld<2>(r, row + 16 * Ring<D>::v_chunk(2 * t, g >> 1) + 8 * (g & 1));
    if constexpr (D == 96) ld<1>(r + 2, row + v_offset<D>(2, g));
  }
}

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// f16 hi and lo parts of a pair of fp32
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = tc::f16x2(x, y);
  const float2 h = f16x2_to_f32(hi);
  lo = tc::f16x2(x - h.x, y - h.y);
}

template <int D, int NT, bool LO>
struct Smem {
  // query fragments: hi pair 0, hi pair 1, and lo pair 0, lo pair 1 where queries have a lo part
  uint2 q[NT][D / 16][LO ? 2 : 1][32];
  float crow[8 * NT];               // scale of a row's sums: attn_scale log2(e) 2^-e
  float m[kWarps][8 * NT], l[kWarps][8 * NT];
  union {
    alignas(16) unsigned char ring[kWarps][Ring<D, NT>::kSlots][Ring<D, NT>::kBytes];
    float acc[kWarps][8][D + 4];    // a row tile's sums of each warp (rows padded against bank conflicts)
  };
};

// One query element in fp32.
__device__ __forceinline__ float q_elem(const Q8AttendArgs& a, int64_t row, int x) {
  const int64_t at = row * a.c.d + x;
  return a.q_bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.q)[at] << 16)
                  : static_cast<const float*>(a.q)[at];
}

// CTAs per SM that the registers of a variant allow (accumulators, a step's codes and the
// queries' row state).
constexpr int resident(int d, int nt) { return d == 256 ? 2 : d == 128 ? 5 - nt : nt == 1 ? 5 : 4; }

template <typename F, int D, int NT, bool LO>
__global__ void __launch_bounds__(kThreads, resident(D, NT)) split_kernel(Q8AttendArgs a) {
  extern __shared__ __align__(16) unsigned char raw[];
  Smem<D, NT, LO>& sm = *reinterpret_cast<Smem<D, NT, LO>*>(raw);
  constexpr int KW = D / 16, VW = D / 32, MT = D / 16;
  using R = Ring<D, NT>;
  const Q8Cache& c = a.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const Q8Item it(a, blockIdx.x);
  const int bh = it.bh, b = it.b, hk = it.hk, G = it.G, rows = it.rows, row0 = it.row0;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // a decode step's append comes first
  const Q8Seq seq(a, b);
  q8_write_flags(a);
  if (!it.any) return;

  const int last_i = min(rows - 1, row0 + 8 * NT - 1) / G;  // the tile's last and first query token
  const int first_i = row0 / G;
  const int q_last = min(last_i, seq.q_len - 1);
  const int stop_all = q_last < first_i ? 0 : seq.limit(q_last);  // rows any of the tile's queries sees
  const int begin = it.chunk_id * it.chunk;
  const int stop = it.split ? begin + min(stop_all - begin, it.chunk) : stop_all;
  if (begin >= stop && it.split) return;

  const uint8_t* kc = c.k_codes + (int64_t)bh * c.capacity * D;
  const uint8_t* vc = c.v_codes + (int64_t)bh * c.capacity * D;
  const float* ksc = c.k_scales + (int64_t)bh * c.n_blocks();
  const float* vsc = c.v_scales + (int64_t)bh * c.n_blocks();
  const int shift = 31 - __clz(c.block);

  // step `tok` into slot `slot` (rows behind the last one repeat it, so what a lane multiplies
  // is always cache content); an empty group where there is none
  const uint32_t ring = tc::smem_u32(sm.ring[warp]);
  const int row_l = lane / (D / 16), ch_l = lane % (D / 16);
  const uint32_t k_at = row_l * D + 16 * R::k_chunk(row_l, ch_l), v_at = row_l * D + 16 * R::v_chunk(row_l, ch_l);
  auto fetch = [&](int tok, int slot) {
    const uint32_t dst = ring + slot * R::kBytes;
    if (tok + kStep <= stop) {
      const int64_t src = (int64_t)tok * D + 16 * lane;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        copy16(dst + k_at + 512 * i, kc + src + 512 * i);
        copy16(dst + R::kRows + (v_at ^ R::v_flip(i)) + 512 * i, vc + src + 512 * i);
      }
    } else if (tok < stop) {
#pragma unroll 1
      for (int id = lane; id < D; id += 32) {
        const int row = id / (D / 16), ch = id % (D / 16);
        const int64_t src = (int64_t)min(tok + row, stop - 1) * D + 16 * ch;
        copy16(dst + row * D + 16 * R::k_chunk(row, ch), kc + src);
        copy16(dst + R::kRows + row * D + 16 * R::v_chunk(row, ch), vc + src);
      }
    }
    if (tok < stop && lane < 2) copy4(dst + 2 * R::kRows + 4 * lane, (lane ? vsc : ksc) + (tok >> shift));
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int tok = begin + kStep * warp, slot = 0;
#pragma unroll
  for (int i = 0; i + 1 < R::kSlots; ++i) fetch(tok + i * kStep * kWarps, i);  // while the queries are prepared

  // -- query fragments, each row scaled so that its largest element is in [2^13, 2^14)
  for (int r = warp; r < 8 * NT; r += kWarps) {
    const int i = (row0 + r) / G;
    const bool live = row0 + r < rows && i < seq.q_len;
    const int64_t qrow = ((int64_t)b * a.Hq + hk * G + (row0 + r) % G) * a.n + i;
    float top = 0.0f;
    if (live)
      for (int x = lane; x < D; x += 32) top = fmaxf(top, fabsf(q_elem(a, qrow, x)));
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const int e = query_exponent(top);
    const float up = tc::pow2i(e);
    const int nt = r >> 3, rg = r & 7;
    for (int p = lane; p < KW * 4; p += 32) {  // (word, lane of 4)
      const int w = p >> 2, tt = p & 3, off = k_offset<D>(w, tt);
      float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (live) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          x[k] = q_elem(a, qrow, off + F::place(0, k)) * up;
          x[2 + k] = q_elem(a, qrow, off + F::place(1, k)) * up;
        }
      }
      uint4 f;
      split2(x[0], x[1], f.x, f.z);
      split2(x[2], x[3], f.y, f.w);
      sm.q[nt][w][0][rg * 4 + tt] = make_uint2(f.x, f.y);
      if constexpr (LO) sm.q[nt][w][1][rg * 4 + tt] = make_uint2(f.z, f.w);
    }
    if (lane == 0) sm.crow[r] = a.attn_scale * kLog2e * tc::pow2i(-e);
  }
  __syncthreads();

  // -- this lane's rows of the S and O fragments: 8 nt + 2t, 8 nt + 2t + 1
  float crow[NT][2], m[NT][2], l[NT][2];
  int limit[NT][2];
  int open = stop;  // tokens below this are seen by every row of the tile
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int r = 8 * nt + 2 * t + k, i = (row0 + r) / G;
      crow[nt][k] = sm.crow[r];
      limit[nt][k] = row0 + r < rows && i < seq.q_len ? seq.limit(i) : INT_MAX;  // rows of no query: ignored
      open = min(open, limit[nt][k]);
      m[nt][k] = -INFINITY;
      l[nt][k] = 0.0f;
    }
  open = __reduce_min_sync(0xffffffffu, open);
  float acc[NT][MT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[nt][i][j] = 0.0f;
  int ref = kNoScale, span = 0;  // E, and how far below it V scales have been

  for (; tok < stop; tok += kStep * kWarps) {
    asm volatile("cp.async.wait_group %0;" ::"n"(R::kSlots - 2) : "memory");
    __syncwarp();  // everyone's copies of this step have landed, and the last step's slot is read
    {
      const int last = slot == 0 ? R::kSlots - 1 : slot - 1;
      fetch(tok + (R::kSlots - 1) * kStep * kWarps, last);
    }
    const unsigned char* now = sm.ring[warp][slot];
    slot = slot + 1 == R::kSlots ? 0 : slot + 1;
    const float ks_now = reinterpret_cast<const float*>(now + 2 * R::kRows)[0];
    const float vs = reinterpret_cast<const float*>(now + 2 * R::kRows)[1];
    float s[NT][2][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[nt][0][j] = s[nt][1][j] = 0.0f;
    uint32_t kr[2][KW];
    load_k<D>(kr[0], now + g * D, g, t);
    load_k<D>(kr[1], now + (g + 8) * D, g, t);
#pragma unroll
    for (int w = 0; w < KW; ++w) {
      uint32_t f[4];
      F::cvt_word(kr[0][w], f[0], f[2]);
      F::cvt_word(kr[1][w], f[1], f[3]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint2 hi = sm.q[nt][w][0][lane];
        mma(s[nt][0], f, hi.x, hi.y);
        if constexpr (LO) {
          const uint2 lo = sm.q[nt][w][1][lane];
          mma(s[nt][1], f, lo.x, lo.y);
        }
      }
    }

    const bool some = vs != 0.0f;  // (warp-uniform, as all of this)
    const int ve = max(-126, min(126, (int)(__float_as_uint(vs) >> 23) - 127));
    if (some && ve > ref) {
      const int low = ref == kNoScale ? span : min(ve - ref, kSpan - span);
      const float up = tc::pow2i(low), down = tc::pow2i(max(low - (ve - ref), -126));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          m[nt][k] -= (float)low;
          l[nt][k] *= up;
        }
        if (down != 1.0f)
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[nt][i][j] *= down;
      }
      if (ref != kNoScale) span += low;
      ref = ve;
    }
    const int gap = some ? min(ref - ve, kSpan) : kZeroSpan;
    span = max(span, gap);
    const float ratio = some ? vs * tc::pow2i(-ref) : 0.0f, below = ref == kNoScale ? 0.0f : -(float)gap;
    uint32_t whi[NT][2], wlo[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = (LO ? s[nt][0][j] + s[nt][1][j] : s[nt][0][j]) * (ks_now * crow[nt][j & 1]);
      if (tok + kStep > open) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (tok + g + 8 * (j >> 1) >= limit[nt][j & 1]) x[j] = -INFINITY;
      }
      const float top0 = fmaxf(x[0], x[2]) + below, top1 = fmaxf(x[1], x[3]) + below;
      const bool move = top0 > m[nt][0] + (kTau + kShift) || top1 > m[nt][1] + (kTau + kShift);
      if (__any_sync(0xffffffffu, move)) {
        float top[2] = {top0, top1};
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          top[0] = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], o));
          top[1] = fmaxf(top[1], __shfl_xor_sync(0xffffffffu, top[1], o));
        }
        float alpha[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // m is held 2^kShift low
          const float mn = fmaxf(m[nt][k], top[k] - kShift);
          alpha[k] = mn == m[nt][k] ? 1.0f : exp2f(m[nt][k] - mn);
          m[nt][k] = mn;
          l[nt][k] *= alpha[k];
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[nt][i][j] *= alpha[j & 1];
      }
      float p[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float mm = m[nt][j & 1] == -INFINITY ? 0.0f : m[nt][j & 1];
        p[j] = tc::ex2(x[j] - mm);
        l[nt][j & 1] += p[j];
        p[j] *= ratio;
      }
      uint32_t h0, l0, h1, l1;
      split2(p[0], p[1], h0, l0);
      split2(p[2], p[3], h1, l1);
      whi[nt][0] = transpose8(h0);
      whi[nt][1] = transpose8(h1);
      wlo[nt][0] = transpose8(l0);
      wlo[nt][1] = transpose8(l1);
    }
    uint32_t vr[4][VW];
#pragma unroll
    for (int j = 0; j < 4; ++j) load_v<D>(vr[j], now + R::kRows + (2 * t + (j & 1) + 8 * (j >> 1)) * D, g, t);
#pragma unroll
    for (int w = 0; w < VW; ++w) {
      uint32_t f01[4], f23[4];  // bytes 0..3 for tokens (2t, 2t+1) and (2t+8, 2t+9)
      F::cvt_two(vr[0][w], vr[1][w], f01);
      F::cvt_two(vr[2][w], vr[3][w], f23);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t f[4] = {f01[2 * h], f01[2 * h + 1], f23[2 * h], f23[2 * h + 1]};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          // a step's sum of its own, added with rounding to nearest: the tensor cores cut
          // off below the accumulator's last bit, which over hundreds of steps (d = 256 at
          // 64K) was the largest error of all
          float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          mma(o, f, wlo[nt][0], wlo[nt][1]);
          mma(o, f, whi[nt][0], whi[nt][1]);
          float(&sum)[4] = acc[nt][2 * w + h];
          const float2 s0 = add2(make_float2(sum[0], sum[1]), make_float2(o[0], o[1]));
          const float2 s1 = add2(make_float2(sum[2], sum[3]), make_float2(o[2], o[3]));
          sum[0] = s0.x, sum[1] = s0.y, sum[2] = s1.x, sum[3] = s1.y;
        }
      }
    }
  }
  __syncthreads();  // (the sums take the place of the rings)

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the merge starts and waits for this grid

  // -- join the warps: sums over the lanes of a row, then over the warps
  const float unit = ref == kNoScale ? 0.0f : tc::pow2i(ref);
  float down[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l[nt][k] += __shfl_xor_sync(0xffffffffu, l[nt][k], o);
      const int e = sum_exponent(l[nt][k]);
      down[nt][k] = tc::pow2i(-e);
      if (g == 0) {
        sm.m[warp][8 * nt + 2 * t + k] = m[nt][k] + (float)e;
        sm.l[warp][8 * nt + 2 * t + k] = l[nt][k] * down[nt][k];
      }
    }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    if (nt > 0) __syncthreads();
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int byte = 2 * i + (j >> 1);  // byte of this lane's part of a V row
        sm.acc[warp][2 * t + (j & 1)][v_offset<D>(byte >> 2, g) + (byte & 3)] = acc[nt][i][j] * down[nt][j & 1] * unit;
      }
    __syncthreads();
    for (int p = threadIdx.x; p < 8 * (D / 4); p += kThreads) {
      const int rr = p / (D / 4), x = p % (D / 4) * 4, r = 8 * nt + rr;
      const int i = (row0 + r) / G;
      if (row0 + r >= rows || i >= seq.q_len) continue;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm.m[w][r]);
      const float base = M == -INFINITY ? 0.0f : M;
      float L = 0.0f;
      float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = exp2f(sm.m[w][r] - base);
        const float4 v = *reinterpret_cast<const float4*>(&sm.acc[w][rr][x]);
        L = fmaf(f, sm.l[w][r], L);
        o.x = fmaf(f, v.x, o.x);
        o.y = fmaf(f, v.y, o.y);
        o.z = fmaf(f, v.z, o.z);
        o.w = fmaf(f, v.w, o.w);
      }
      if (it.split) {
        float* part = it.part(a, r, 0);
        *reinterpret_cast<float4*>(part + x) = o;
        if (x == 0) *reinterpret_cast<float2*>(part + D) = make_float2(M, L);
        continue;
      }
      const int64_t orow = it.out_row(a, r);
      const bool none = M == -INFINITY && L == 0.0f;  // no row seen
      const float inv = none ? 0.0f : 1.0f / L;
      o = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
      if (a.out_bf16)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + orow * D + x) =
            make_uint2(bf16x2(o.x, o.y), bf16x2(o.z, o.w));
      else
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + orow * D + x) = o;
      if (a.lse != nullptr && x == 0) *reinterpret_cast<float2*>(a.lse + orow * 2) = make_float2(M, L);
    }
  }
}

// Joins the partials of each row of the split units: with M = max m_c, o = sum
// 2^(m_c - M) acc_c / sum 2^(m_c - M) l_c.  W warps take a row, warp w its partials w,
// w + W, ... with a lane on every fourth output element; their sums meet in shared memory.
// With up to eight partials a row a warp of its own takes it (many rows); else 8 warps, and
// with more than 64 partials (decode of few rows) 32, so that a warp has few rounds of four
// independent loads.  The launch is the
// first kernel's programmatic dependent, so its start overlaps that one's tail.
template <int D, int W>
__global__ void __launch_bounds__(W == 1 ? 256 : 32 * W) merge_q8_kernel(Q8AttendArgs a) {
  constexpr int P = (D + 127) / 128;  // pieces of 128 elements
  constexpr int kMergeWarps = W == 1 ? 8 : W;
  __shared__ float4 sums[kMergeWarps][P][32];
  __shared__ float2 state[kMergeWarps];
  const int lane = threadIdx.x & 31, team = (threadIdx.x >> 5) / W, warp = (threadIdx.x >> 5) % W;
  const int64_t id = (int64_t)blockIdx.x * (kMergeWarps / W) + team;
  Q8Item it;
  const int unit = a.plan.whole + (int)min(id / a.plan.merge_rows, (int64_t)(a.plan.units - a.plan.whole - 1));
  it.place_unit(a, unit);
  it.first_item(a, unit);
  const int r = (int)(id % a.plan.merge_rows), i = it.token(r);
  const Q8Seq seq(a, it.b);
  const bool live = id < (int64_t)(a.plan.units - a.plan.whole) * a.plan.merge_rows && it.row0 + r < it.rows && i < seq.q_len;
  const int nc = live ? (seq.limit(i) + it.chunk - 1) / it.chunk * a.plan.parts : 0;
  const int64_t step = Q8Item::part_step(a);
  const float* part = it.part(a, r, 0);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float M = -INFINITY, L = 0.0f;  // of this warp's chunks
  float4 o[P];
#pragma unroll
  for (int p = 0; p < P; ++p) o[p] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  constexpr int U = 4;
  for (int k0 = warp; k0 < nc; k0 += U * W) {
    float2 ml[U];
    float4 v[U][P];
    float top = M;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * W;
      const float* pk = part + k * step;
      ml[u] = k < nc ? *reinterpret_cast<const float2*>(pk + D) : make_float2(-INFINITY, 0.0f);
#pragma unroll
      for (int p = 0; p < P; ++p)
        v[u][p] = k < nc && 128 * p + 4 * lane < D ? *reinterpret_cast<const float4*>(pk + 128 * p + 4 * lane)
                                                   : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) top = fmaxf(top, ml[u].x);
    const float base = top == -INFINITY ? 0.0f : top;
    const float keep = exp2f(M - base);
    M = top;
    L *= keep;
#pragma unroll
    for (int p = 0; p < P; ++p) o[p] = make_float4(o[p].x * keep, o[p].y * keep, o[p].z * keep, o[p].w * keep);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float f = exp2f(ml[u].x - base);
      L = fmaf(f, ml[u].y, L);
#pragma unroll
      for (int p = 0; p < P; ++p) {
        o[p].x = fmaf(f, v[u][p].x, o[p].x);
        o[p].y = fmaf(f, v[u][p].y, o[p].y);
        o[p].z = fmaf(f, v[u][p].z, o[p].z);
        o[p].w = fmaf(f, v[u][p].w, o[p].w);
      }
    }
  }
#pragma unroll
  for (int p = 0; p < P; ++p) sums[team * W + warp][p][lane] = o[p];
  if (lane == 0) state[team * W + warp] = make_float2(M, L);
  if constexpr (W > 1)
    __syncthreads();
  else
    __syncwarp();
  // the team's threads, one per four output elements
  const int at = threadIdx.x - 32 * W * team;
  if (!live) return;
  M = -INFINITY;
#pragma unroll
  for (int w = 0; w < W; ++w) M = fmaxf(M, state[team * W + w].x);
  const float base = M == -INFINITY ? 0.0f : M;
  const int64_t orow = it.out_row(a, r);
#pragma unroll
  for (int x4 = at; x4 < D / 4; x4 += 32 * W) {
    L = 0.0f;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = exp2f(state[team * W + w].x - base);
      const float4 s = sums[team * W + w][x4 >> 5][x4 & 31];
      L = fmaf(f, state[team * W + w].y, L);
      v.x = fmaf(f, s.x, v.x);
      v.y = fmaf(f, s.y, v.y);
      v.z = fmaf(f, s.z, v.z);
      v.w = fmaf(f, s.w, v.w);
    }
    const float inv = nc == 0 ? 0.0f : 1.0f / L;
    v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
    if (a.out_bf16)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + orow * D + 4 * x4) =
          make_uint2(bf16x2(v.x, v.y), bf16x2(v.z, v.w));
    else
      *reinterpret_cast<float4*>(static_cast<float*>(a.out) + orow * D + 4 * x4) = v;
    if (a.lse != nullptr && x4 == 0) *reinterpret_cast<float2*>(a.lse + orow * 2) = make_float2(M, L);
  }
}

template <typename F, int D, int NT, bool LO>
cudaError_t launch_one(const Q8AttendArgs& a, cudaStream_t stream) {
  static SmemLimitSet done;
  constexpr int bytes = sizeof(Smem<D, NT, LO>);
  const cudaError_t e = ensure_smem_limit(split_kernel<F, D, NT, LO>, bytes, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.plan.items());
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, split_kernel<F, D, NT, LO>, a);
}

template <typename F, int D>
cudaError_t launch_width(const Q8AttendArgs& a, cudaStream_t stream) {
  if (a.q_bf16)
    return a.plan.row_tile == 16 ? launch_one<F, D, 2, false>(a, stream) : launch_one<F, D, 1, false>(a, stream);
  return a.plan.row_tile == 16 ? launch_one<F, D, 2, true>(a, stream) : launch_one<F, D, 1, true>(a, stream);
}

template <typename F>
cudaError_t launch_format(const Q8AttendArgs& a, cudaStream_t stream) {
  switch (a.c.d) {
    case 64: return launch_width<F, 64>(a, stream);
    case 96: return launch_width<F, 96>(a, stream);
    case 128: return launch_width<F, 128>(a, stream);
    default: return launch_width<F, 256>(a, stream);
  }
}

}  // namespace

int q8_split_per_sm(int d, int row_tile) { return resident(d, row_tile / 8); }

cudaError_t launch_q8_split(const Q8AttendArgs& a, cudaStream_t stream) {
  return a.c.e4m3 ? launch_format<E4m3>(a, stream) : launch_format<Int8>(a, stream);
}

template <int D>
static cudaError_t merge_rows(const Q8AttendArgs& a, cudaStream_t stream) {
  const int W = a.plan.row_parts <= 8 ? 1 : a.plan.row_parts <= 64 ? 8 : 32, per_cta = W == 1 ? 8 : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.plan.split_rows() + per_cta - 1) / per_cta));
  cfg.blockDim = dim3(W == 1 ? 256 : 32 * W);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (W == 1) return cudaLaunchKernelEx(&cfg, merge_q8_kernel<D, 1>, a);
  if (W == 8) return cudaLaunchKernelEx(&cfg, merge_q8_kernel<D, 8>, a);
  return cudaLaunchKernelEx(&cfg, merge_q8_kernel<D, 32>, a);
}

cudaError_t launch_q8_merge(const Q8AttendArgs& a, cudaStream_t stream) {
  switch (a.c.d) {
    case 64: return merge_rows<64>(a, stream);
    case 96: return merge_rows<96>(a, stream);
    case 128: return merge_rows<128>(a, stream);
    default: return merge_rows<256>(a, stream);
  }
}

}  // namespace tq
