// q8_append.cu -- writing tokens into the 8-bit block-scaled cache, and
// reading a range of it back.
//
// Writing.  One team of threads owns one block of one kv head's K or V, so the block's
// new scale and every code that changes with it are decided in one place:
//   a     = max finite |x| over the block's new rows,  s_new = fl32(a / Q)
//   s     = max(s_old, s_new) if rows of the block before the first new one are
//           kept, else s_new
//   code  = R(fl32(x / s)) (R: nearest, halves to even; NaN -> 0, ends saturate)
//   kept rows, only when s > s_old:  code' = R(fl32(fl32(code s_old) / s))
// The new rows stay in registers between the maximum and the division, so HBM
// sees each input once and each code once.  A thread holds four pieces of
// eight elements (one 16-byte load of bf16, one 8-byte store), six at d = 96, which
// makes a team of 32 to 1024 threads; small teams share a CTA of 256.  Bound: HBM
// for fp32 inputs, nearly the instructions for bf16 (the exact division is five
// packed operations a pair, half of it all).
//
// Measured (captured calls repeated on one input): fp32 to e4m3, 4 x 16 heads x 4096 x 256,
// 109 us (6.1 TB/s of input and codes); bf16 to int8, 8 heads x 128K x 128, 176 us
// (4.6 TB/s); to e4m3 174 us.
//
// Reading is a stream of 8-byte (bf16) or 4-byte (fp32) code loads with one
// 16-byte store each.  Bound: HBM (8 heads x 128K x 128 to bf16 127 us, 6.3 TB/s).
#include "q8_common.cuh"
#include "q8_internal.h"

namespace tq {
namespace {

using namespace q8;


template <bool BF16>
struct Piece {
  uint4 w[BF16 ? 1 : 2];
  __device__ __forceinline__ void load(const void* base, int64_t elem) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(base) +
                                                    elem * (BF16 ? 2 : 4));
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); ++i)
      asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                   : "l"(p + i));
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); ++i) w[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void values(float2 (&x)[4]) const {
    if constexpr (BF16) {
      const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
    } else {
      const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
    }
  }
  // signs of elements 4 half .. 4 half + 3 in the top bits of the bytes
  __device__ __forceinline__ uint32_t signs(int half) const {
    if constexpr (BF16) {
      return (half ? tc::prmt(w[0].z, w[0].w, 0x7531) : tc::prmt(w[0].x, w[0].y, 0x7531)) & 0x80808080u;
    } else {
      const uint4 u = w[half];
      return tc::prmt(tc::prmt(u.x, u.y, 0x0073), tc::prmt(u.z, u.w, 0x0073), 0x5410) & 0x80808080u;
    }
  }
  // Running maximum of the bits of |x|: two 16-bit lanes for bf16, one word for fp32.
  __device__ __forceinline__ void max_bits(uint32_t& top) const {
    if constexpr (BF16) {
      const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) asm("max.u16x2 %0, %0, %1;" : "+r"(top) : "r"(u[i] & 0x7fff7fffu));
    } else {
      const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
      for (int i = 0; i < 8; i += 2) top = __vimax3_u32(top, u[i] & 0x7fffffffu, u[i + 1] & 0x7fffffffu);
    }
  }
};

// Maximum over the `threads` threads (whole warps) of one block's team; smem[32] is the
// CTA's, and each team has a barrier of its own.
__device__ __forceinline__ uint32_t team_max(uint32_t v, uint32_t* smem, int threads, int team) {
  v = __reduce_max_sync(0xffffffffu, v);
  const int warps = threads >> 5, lane = threadIdx.x & 31;
  if (warps == 1) return v;
  if (lane == 0) smem[threadIdx.x >> 5] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(threads) : "memory");
  v = lane < warps ? smem[team * warps + lane] : 0u;
  return __reduce_max_sync(0xffffffffu, v);
}

// x / d for x, d < 2^31 by the upper half of x ceil(2^64 / d) (the error, below x d / 2^64,
// does not reach the next integer); integer division took a third of a team's instructions.
struct Quotient {
  uint64_t m;
  explicit Quotient(unsigned d) : m(~0ull / d + 1) {}  // 0 for d = 1
  __device__ __forceinline__ unsigned of(unsigned x) const { return m ? (unsigned)__umul64hi(x, m) : x; }
};

struct Teams {
  int touched;   // blocks of one sequence's window
  int shift;     // log2 of a team's threads
  unsigned units;
  Quotient per_head, per_sequence;
};

template <typename F, bool BF16, int kPieces>
__global__ void __launch_bounds__(1024, BF16 ? 1 : 0) append_kernel(Q8WriteArgs a, Teams teams) {
  __shared__ uint32_t red[2][32];
  const Q8Cache& c = a.c;
  const int threads = 1 << teams.shift, team = threadIdx.x >> teams.shift, tid = threadIdx.x & (threads - 1);
  const unsigned id = blockIdx.x * (blockDim.x >> teams.shift) + team;
  if (id >= teams.units) return;
  const bool is_v = id & 1;
  const int bh = teams.per_head.of(id >> 1);
  const int j = (id >> 1) - bh * teams.touched;  // block of this sequence's window
  const int b = teams.per_sequence.of(bh);
  const int block_shift = 31 - __clz(c.block);
  int pos = a.pos[b], valid = a.n_valid ? a.n_valid[b] : a.n;
  if (a.pos_is_ctx) pos = min(pos, a.max_ctx) - 1;
  if (pos < 0 || valid <= 0) return;
  valid = min(valid, a.n);
  const int64_t first = (int64_t)((pos >> block_shift) + j) << block_shift;  // the block's first row
  const int64_t stop = min((int64_t)pos + valid, c.capacity);
  if (first >= stop) return;  // (the differences below then fit in 32 bits, wherever pos is)
  const int new0 = (int)max((int64_t)0, pos - first);           // new rows [new0, new1) of the block
  const int new1 = (int)min((int64_t)c.block, stop - first);
  if (new0 >= new1) return;

  const int per_row = c.d >> 3;
  const void* in = is_v ? a.v : a.k;
  uint8_t* codes = (is_v ? c.v_codes : c.k_codes) + ((int64_t)bh * c.capacity + first) * c.d;
  float* scale = (is_v ? c.v_scales : c.k_scales) + (int64_t)bh * ((c.capacity + c.block - 1) >> block_shift) + (first >> block_shift);
  // element of the input that corresponds to the block's row 0
  const int64_t in0 = ((int64_t)bh * a.n + (first - pos)) * c.d;
  const float s_old = new0 > 0 ? *scale : 0.0f;

  Piece<BF16> x[kPieces];
  uint32_t top = 0;  // bits of the largest |x|: above 0x7f800000 for NaN
  const int lo = new0 * per_row, hi = new1 * per_row;
  const bool whole = lo == 0 && hi == kPieces * threads;  // (no piece to leave out)
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int p = tid + i * threads;
    if (whole || (p >= lo && p < hi))
      x[i].load(in, in0 + (int64_t)p * 8);
    else
      x[i].zero();
  }
#pragma unroll
  for (int i = 0; i < kPieces; ++i) x[i].max_bits(top);
  if constexpr (BF16) top = max(top << 16, top & 0xffff0000u);
  top = team_max(top, red[0], threads, team);
  const bool finite = top < 0x7f800000u;
  if (!finite) {  // infinities and NaN do not set the scale
    top = 0;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      float2 v[4];
      x[i].values(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t u = __float_as_uint(e & 1 ? v[e >> 1].y : v[e >> 1].x) & 0x7fffffffu;
        if (u < 0x7f800000u) top = max(top, u);
      }
    }
    top = team_max(top, red[1], threads, team);
  }
  const float s = fmaxf(s_old, __fdiv_rn(__uint_as_float(top), F::kMax));
  const Divider div = Divider::by(s);

  if (finite && div.fast) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int p = tid + i * threads;
      float2 v[4];
      x[i].values(v);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = div.quick(v[e]);
      uint2 code = make_uint2(F::codes4(v[0], v[1]), F::codes4(v[2], v[3]));
      if constexpr (F::kSignedZero) {  // the division's residual steps turn -0 into +0
        code.x |= x[i].signs(0);
        code.y |= x[i].signs(1);
      }
      if (whole || (p >= lo && p < hi)) *reinterpret_cast<uint2*>(codes + (int64_t)p * 8) = code;
    }
  } else {
#pragma unroll 1
    for (int i = 0; i < kPieces; ++i) {
      const int p = tid + i * threads;
      if (p < lo || p >= hi) continue;
      Piece<BF16> again;  // re-read: a block with such values is rare
      again.load(in, in0 + (int64_t)p * 8);
      float2 v[4];
      again.values(v);
      uint32_t w[2] = {0, 0};
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e >> 2] |= F::code(div.any(e & 1 ? v[e >> 1].y : v[e >> 1].x)) << (8 * (e & 3));
      *reinterpret_cast<uint2*>(codes + (int64_t)p * 8) = make_uint2(w[0], w[1]);
    }
  }
  if (new0 > 0 && s > s_old) {  // the kept rows' codes move to the larger scale
    for (int p = tid; p < lo; p += threads) {
      uint2* at = reinterpret_cast<uint2*>(codes + (int64_t)p * 8);
      const uint2 old = *at;
      uint32_t w[2] = {0, 0};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        w[e >> 2] |= F::code(div.any(F::value(e < 4 ? old.x : old.y, e & 3) * s_old)) << (8 * (e & 3));
      *at = make_uint2(w[0], w[1]);
    }
  }
  if (tid == 0) *scale = s;
}

// -------------------------------------------------------------------- reading

constexpr int kReadThreads = 256, kReadPieces = 4;

// A piece is what one 16-byte store holds: 8 bf16 or 4 fp32 values.
template <typename F, bool BF16>
__global__ void __launch_bounds__(kReadThreads) read_kernel(Q8ReadArgs a, int row_tiles, int tile_rows,
                                                              unsigned row_magic, int block_shift) {
  const Q8Cache& c = a.c;
  const bool is_v = blockIdx.x & 1;
  const unsigned unit = blockIdx.x >> 1;
  const int tile = unit % row_tiles, bh = unit / row_tiles, b = bh / c.Hkv;
  const int pos = a.pos ? a.pos[b] : 0;
  const int row0 = tile * tile_rows, all = min(tile_rows, a.n - row0);
  int64_t rows = min(a.n_valid ? a.n_valid[b] : a.n, a.n);
  rows = min(min(rows, c.capacity - pos) - row0, (int64_t)all);
  if (rows <= 0 || pos < 0) rows = 0;
  constexpr int E = BF16 ? 8 : 4;
  const int per_row = c.d / E, pieces = (int)rows * per_row;
  const uint8_t* codes = (is_v ? c.v_codes : c.k_codes) + ((int64_t)bh * c.capacity + pos + row0) * c.d;
  const float* scales = (is_v ? c.v_scales : c.k_scales) + (int64_t)bh * c.n_blocks();
  unsigned char* out = static_cast<unsigned char*>(is_v ? a.v : a.k) +
                       ((int64_t)bh * a.n + row0) * c.d * (BF16 ? 2 : 4);
  const int first = pos + row0;
  if (a.fill)  // rows outside the cache or behind the last are zeros
    for (int p = pieces + threadIdx.x; p < all * per_row; p += kReadThreads)
      __stcs(reinterpret_cast<uint4*>(out) + p, make_uint4(0, 0, 0, 0));
  for (int p0 = threadIdx.x; p0 < pieces; p0 += kReadThreads * kReadPieces) {
    uint32_t w[kReadPieces][2];
    float s[kReadPieces];
#pragma unroll
    for (int i = 0; i < kReadPieces; ++i) {
      const int p = p0 + i * kReadThreads;
      if (p >= pieces) continue;
      s[i] = scales[(first + (int)__umulhi(p, row_magic)) >> block_shift];
      if constexpr (BF16) {
        const uint2 v = __ldcs(reinterpret_cast<const uint2*>(codes) + p);
        w[i][0] = v.x;
        w[i][1] = v.y;
      } else {
        w[i][0] = __ldcs(reinterpret_cast<const uint32_t*>(codes) + p);
      }
    }
#pragma unroll
    for (int i = 0; i < kReadPieces; ++i) {
      const int p = p0 + i * kReadThreads;
      if (p >= pieces) continue;
      uint4 o;
      if constexpr (BF16) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = s[i] * F::value(w[i][e >> 2], e & 3);
        o = make_uint4(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]), bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
      } else {
        uint32_t x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = __float_as_uint(s[i] * F::value(w[i][0], e));
        o = make_uint4(x[0], x[1], x[2], x[3]);
      }
      __stcs(reinterpret_cast<uint4*>(out) + p, o);
    }
  }
}

}  // namespace

template <int kPieces>
static cudaError_t write_blocks(const Q8WriteArgs& a, int touched, unsigned units, cudaStream_t stream) {
  const int threads = a.c.block * a.c.d / (8 * kPieces), cta = threads > 256 ? threads : 256;
  const Teams teams = {touched, 31 - __builtin_clz((unsigned)threads), units, Quotient(touched), Quotient(a.c.Hkv)};
  const unsigned per_cta = cta / threads;
  auto* kernel = a.c.e4m3 ? (a.bf16 ? append_kernel<E4m3, true, kPieces> : append_kernel<E4m3, false, kPieces>)
                          : (a.bf16 ? append_kernel<Int8, true, kPieces> : append_kernel<Int8, false, kPieces>);
  kernel<<<(units + per_cta - 1) / per_cta, cta, 0, stream>>>(a, teams);
  return cudaGetLastError();
}

cudaError_t launch_q8_append(const Q8WriteArgs& a, cudaStream_t stream) {
  const int touched = (a.n + a.c.block - 2) / a.c.block + 1;  // most blocks n rows can lie in
  const unsigned units = 2u * a.c.B * a.c.Hkv * touched;
  return a.c.d == 96 ? write_blocks<6>(a, touched, units, stream) : write_blocks<4>(a, touched, units, stream);
}

cudaError_t launch_q8_read(const Q8ReadArgs& a, cudaStream_t stream) {
  const int elems = a.bf16 ? 8 : 4;
  int tile_rows = kReadThreads * kReadPieces * elems / a.c.d;
  if (tile_rows > a.n) tile_rows = a.n;
  const int row_tiles = (a.n + tile_rows - 1) / tile_rows;
  const unsigned grid = 2u * a.c.B * a.c.Hkv * row_tiles;
  auto* kernel = a.c.e4m3 ? (a.bf16 ? read_kernel<E4m3, true> : read_kernel<E4m3, false>)
                          : (a.bf16 ? read_kernel<Int8, true> : read_kernel<Int8, false>);
  const unsigned per_row = a.c.d / elems;
  const unsigned row_magic = (unsigned)(((1ull << 32) + per_row - 1) / per_row);  // p / per_row for p < 2^16
  kernel<<<grid, kReadThreads, 0, stream>>>(a, row_tiles, tile_rows, row_magic,
                                            31 - __builtin_clz((unsigned)a.c.block));
  return cudaGetLastError();
}

}  // namespace tq
