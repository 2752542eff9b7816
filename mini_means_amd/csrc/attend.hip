// Attention over packed sequences, forward and backward (bf16 and fp16).
//
// For a query row i of a sequence (lq queries, lk keys) and the keys j it sees, all of
// them or (causal) those with j <= i + lk - lq:
//   s = scale q k^T, o = sum exp(s - m) v / l, m the largest s, l = sum exp(s - m)
// in one pass over the keys with a running maximum and sum. Backward, with
// P = exp(s - lse), lse = m + log l, D = rowsum(dO o):
//   dV = P^T dO, dS = P (dO V^T - D), dQ = scale dS K, dK = scale dS^T Q,
// as two kernels, one that owns query rows (dQ) and one that owns key rows (dK, dV,
// summed over the query heads of a group in order): seven products instead of the
// five that atomic sums of dQ would leave, but the same bits each time.
//
// Bound by the matrix unit and, as much, by the vector instructions beside it (143 for a
// wave's 32 x 64 scores, whose 32 products take 1088 cycles). All products
// are 32 x 32 x 16 MFMAs laid out so that nothing crosses lanes between them: with A
// the tile's rows and B a wave's own 32 rows (kept in registers), a lane holds 16 of
// 32 results of one own row, and these are the B operand of the next product when
// its sum index is counted in the order in which they stand. Its A operand is the
// tile transposed, which ds_read_b64_tr_b16 reads from the same LDS rows. Two workgroups of
// four waves share a CU: one wave's products run beside the other's exponentials.
// Measured, 32 query and 8 key-value heads of 128 in bf16, causal: 16384 tokens 2.12 to 2.22
// ms (990 to 1040 TFLOP/s; the library's product of 8192 a side 1223); seven sequences of
// up to 4000 tokens 0.38 ms, dQ 0.52, dK and dV 0.73 and 0.04 for their sums (fp16 0.40, 0.57,
// 0.79, 0.04). 33 sequences of up to 500 tokens, 16
// heads of 64 in fp16, not causal: 33 us.
#include <type_traits>

#include "block.hpp"
#include "kernels.hpp"

namespace emk {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kTile = 64;  // rows of a tile in LDS
constexpr int kZeroGroups = 32;
constexpr float kLog2e = 1.4426950408889634f;

template <bool F16>
using Half8 = std::conditional_t<F16, f16x8, bf16x8>;

template <bool F16>
__device__ __forceinline__ f32x16 product(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// The place of a row's 16-byte chunks: XOR with a number of the row. LDS has 16 times 16
// bytes in its banks, so that is what the 16 rows (of one chunk) that a phase of a row
// read takes, and the four rows of four chunks of a transposed read, have to differ in.
// Rows of 64 and 96 values start at two and four different places already. (Against
// three bits of the row in any order, row reads took 1.5 times as long.)
template <int W>
__device__ __forceinline__ int swizzle(int row) {
  if constexpr (W == 64)
    return ((row >> 1) & 1) << 2 | ((row >> 2) & 3);
  else if constexpr (W == 96)
    return (row >> 2) & 3;
  else
    return (row & 3) << 2 | ((row >> 2) & 3);
}

// Rows row0 .. row0 + R - 1 of a head into LDS, past `last` that row again (so that what
// is masked is a row of this sequence, never another's). Chunks past width are not
// written: they hold the zeros that the workgroup began with. A lane's offsets in a
// whole tile are the same for each tile (`at`), beside a uniform address.
template <int W, int NW, int R = kTile>
struct TileLoads {
  static constexpr int CPR = W / 8, ALL = CPR * R / 64, N = (ALL + NW - 1) / NW;
  // the rows of a lane's loads are a multiple of 16 apart, so its chunk is the same
  static constexpr bool kEven = NW * 64 % CPR == 0;
  static constexpr int kStep = NW * 64 / CPR, M = kEven ? 1 : N;
  uint32_t at[M];
  int row[M];  // -1: not this lane's
  __device__ __forceinline__ void init(int64_t rs, int width, int wave, int lane) {
#pragma unroll
    for (int i = 0; i < M; ++i) {
      const int c = (i * NW + wave) * 64 + lane, r = c / CPR;
      const int chunk = (c - r * CPR) ^ swizzle<W>(r);
      row[i] = chunk * 8 < width && (ALL % NW == 0 || i * NW + wave < ALL) ? r : -1;
      at[i] = (uint32_t)(r * (int)rs + chunk * 8) * 2;
    }
  }
  __device__ __forceinline__ void load(const uint16_t* base, int64_t rs, int row0, int last,
                                       uint8_t* lds, int wave) const {
    const uint16_t* from = base + row0 * rs;
    const bool whole = row0 + R - 1 <= last;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int q = kEven ? 0 : i, more = kEven ? i * kStep : 0;
      const uint16_t* src = from + more * rs;
      uint32_t off = at[q];
      if (!whole) {  // from the tile's first row, so that no offset is negative
        src = from;
        off += (uint32_t)((more - max(row0 + more + row[q] - last, 0)) * (int)rs) * 2;
      }
      if (row[q] >= 0) lds_load16_from(src, off, lds + (i * NW + wave) * 1024);
    }
  }
};

// Operands read from a tile in LDS. A lane's addresses in one buffer, kept in
// registers: everything else is an immediate offset. rows(i, r0): A operand of rows r0 +
// lane % 32, values 16 i + 8 h + {0..7}. columns(dt, r0): of the tile transposed, values
// 32 dt + lane % 32 of the 16 rows from r0 on, in the order r0 + 4 h + {0..3},
// r0 + 8 + 4 h + {0..3} for lane half h. (r0 a multiple of 16.)
template <int W>
struct TileReads {
  typedef __attribute__((address_space(3))) const u32x4* quad_at;
  typedef __attribute__((address_space(3))) s16x4* tr_at;
  uint32_t row[W / 16], col[W / 32], col8[W / 32];  // col8: eight rows on
  __device__ __forceinline__ void init(const uint8_t* lds, int lane) {
    const uint32_t at = (uint32_t)(uintptr_t)(lds_ptr_t)(lds);
    const int r = lane & 31, half = lane >> 5;
#pragma unroll
    for (int i = 0; i < W / 16; ++i) row[i] = at + r * W * 2 + (((2 * i + half) ^ swizzle<W>(r)) << 4);
    const int c = 4 * half + ((lane & 15) >> 2);
#pragma unroll
    for (int dt = 0; dt < W / 32; ++dt) {
      const int chunk = 4 * dt + ((lane >> 4) & 1) * 2 + ((lane >> 1) & 1);
      col[dt] = at + c * W * 2 + ((chunk ^ swizzle<W>(c)) << 4) + (lane & 1) * 8;
      col8[dt] = at + (c + 8) * W * 2 + ((chunk ^ swizzle<W>(c + 8)) << 4) + (lane & 1) * 8;
    }
  }
  __device__ __forceinline__ void move(uint32_t by) {
#pragma unroll
    for (int i = 0; i < W / 16; ++i) row[i] += by;
#pragma unroll
    for (int dt = 0; dt < W / 32; ++dt) {
      col[dt] += by;
      col8[dt] += by;
    }
  }
  __device__ __forceinline__ u32x4 rows(int i, int r0, int tile = 0) const {
    return *(quad_at)(uintptr_t)(row[i] + r0 * (W * 2) + tile);
  }
  __device__ __forceinline__ u32x4 columns(int dt, int r0, int tile = 0) const {
    const uint32_t off = r0 * (W * 2) + tile;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((tr_at)(uintptr_t)(col[dt] + off));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((tr_at)(uintptr_t)(col8[dt] + off));
    const u32x2 a = __builtin_bit_cast(u32x2, lo), b = __builtin_bit_cast(u32x2, hi);
    return u32x4{a[0], a[1], b[0], b[1]};
  }
};

// A wave's own rows as B operands: row `row` of a head (any valid one for lanes past
// the last), values 16 ks + 8 h + {0..7}; zeros past width.
template <int W>
__device__ __forceinline__ void own_frags(const uint16_t* p, int width, int half,
                                          u32x4 (&f)[W / 16]) {
#pragma unroll
  for (int ks = 0; ks < W / 16; ++ks) {
    const int c = 16 * ks + 8 * half;
    f[ks] = c < width ? *reinterpret_cast<const u32x4*>(p + c) : u32x4{0u, 0u, 0u, 0u};
  }
}

// Results of 8 sum indices, in order, as a B operand.
template <bool F16>
__device__ __forceinline__ u32x4 packed(const f32x16& s, int r) {
  constexpr int OT = F16 ? 4 : 1;
  return u32x4{pack2<OT>(s[r], s[r + 1]), pack2<OT>(s[r + 2], s[r + 3]),
               pack2<OT>(s[r + 4], s[r + 5]), pack2<OT>(s[r + 6], s[r + 7])};
}

__device__ __forceinline__ float half_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

__device__ __forceinline__ float half_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// acc (values 8 (r / 4) + 4 h + r % 4 of 32, of row lane % 32) times f to 16-bit rows:
// the lane halves trade their runs of four, so that a lane stores 16 bytes. rest: what
// the rounding took away, rounded to 16 bits itself, or NULL.
template <bool F16, int W>
__device__ __forceinline__ void store_rows(const f32x16 (&acc)[W / 32], float f, uint16_t* row,
                                           uint16_t* rest, int width, int half, bool on) {
  constexpr int OT = F16 ? 4 : 1;
  auto put = [&](uint16_t* to, int c, const uint32_t(&a)[2], const uint32_t(&b)[2]) {
    const auto x = __builtin_amdgcn_permlane32_swap(a[0], b[0], false, false);
    const auto y = __builtin_amdgcn_permlane32_swap(a[1], b[1], false, false);
    if (on && c < width) *reinterpret_cast<u32x4*>(to + c) = u32x4{x[0], y[0], x[1], y[1]};
  };
  auto left = [&](float x, float y, uint32_t w) {
    return pack2<OT>(x - half_to_f32((uint16_t)w, F16), y - half_to_f32((uint16_t)(w >> 16), F16));
  };
#pragma unroll
  for (int dt = 0; dt < W / 32; ++dt)
#pragma unroll
    for (int g = 0; g < 4; g += 2) {
      uint32_t a[2], b[2];
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = acc[dt][4 * g + i] * f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        a[i] = pack2<OT>(x[2 * i], x[2 * i + 1]);
        b[i] = pack2<OT>(x[4 + 2 * i], x[5 + 2 * i]);
      }
      const int c = dt * 32 + (g + half) * 8;
      put(row, c, a, b);
      if (rest) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          a[i] = left(x[2 * i], x[2 * i + 1], a[i]);
          b[i] = left(x[4 + 2 * i], x[5 + 2 * i], b[i]);
        }
        put(rest, c, a, b);
      }
    }
}

// Rows of a sequence in the packed order, cut to what the tensors hold whatever
// `starts` says.
struct Span {
  int first, len;
};

__device__ __forceinline__ Span span_of(const int32_t* starts, int s, int64_t n) {
  const int a = max(0, min(starts[s], (int)n)), b = max(a, min(starts[s + 1], (int)n));
  return {a, b - a};
}

// Tiles of `rows` rows: sequence s has those from starts[s] / rows + s on, enough for
// any alignment, so that a tile finds its sequence without the host knowing lengths.
struct Place {
  int seq, row0;  // first row of the tile in its sequence
};

__device__ __forceinline__ Place place_of(const int32_t* starts, int seqs, int64_t n, int rows,
                                          int64_t tile) {
  const int lane = threadIdx.x & 63;
  auto first_tile = [&](int s) { return (int64_t)(max(0, min(starts[s], (int)n)) / rows) + s; };
  // the last sequence whose first tile is not after this one, 64 of them looked at in one
  // read: a search by halves would be a chain of ten reads for 1000 sequences
  int lo = 0, len = seqs;
  while (len > 1) {
    const int step = (len + 63) / 64, s = lane * step;
    const int i = max(__popcll(__ballot(s < len && first_tile(lo + min(s, len - 1)) <= tile)) - 1, 0);
    lo += i * step;
    len = min(step, len - i * step);
  }
  const int64_t j = tile - first_tile(lo);
  return {lo, j < 0 || j * rows > 0x7FFFFFFF ? 0x7FFFFFFF : (int)(j * rows)};
}

// Rows of out (rows x d) that no sequence has become zeros.
__device__ __forceinline__ void zero_outside(const int32_t* starts, int seqs, int64_t n, int64_t d,
                                             uint16_t* out, int64_t wg, int threads) {
  const int64_t first = max(0, min(starts[0], (int)n)), last = max(0, min(starts[seqs], (int)n));
  const int64_t step = (int64_t)kZeroGroups * threads * 8;
  for (int64_t i = (wg * threads + threadIdx.x) * 8; i < first * d; i += step)
    *reinterpret_cast<u32x4*>(out + i) = u32x4{0u, 0u, 0u, 0u};
  for (int64_t i = last * d + (wg * threads + threadIdx.x) * 8; i < n * d; i += step)
    *reinterpret_cast<u32x4*>(out + i) = u32x4{0u, 0u, 0u, 0u};
}

// Workgroup b as (tile, head): the heads of a tile follow each other, and where eight
// divides them, those of one XCD (every eighth workgroup) are neighbours, which share
// a key-value head's rows in its L2.
__device__ __forceinline__ int head_of(int64_t b, int heads) {
  const int i = (int)(b % heads);
  return heads % 8 ? i : (i % 8) * (heads / 8) + i / 8;
}

template <int W>
__device__ __forceinline__ void clear_lds(uint8_t* lds, int bytes, int width, int threads) {
  if (width == W) return;
  for (int i = threadIdx.x * 16; i < bytes; i += threads * 16)
    *reinterpret_cast<u32x4*>(lds + i) = u32x4{0u, 0u, 0u, 0u};
  __syncthreads();
}

// V rows that a query does not see must not show in it, but 0 x infinity is NaN. Where a
// first pass gave no numbers, the tiles that the workgroup's rows see in part are therefore
// done with infinities and NaN taken out, and odd_values adds those that a row sees.
template <bool F16>
__device__ __forceinline__ u32x4 numbers_of(u32x4 v) {
  constexpr uint32_t E = F16 ? 0x7C00u : 0x7F80u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((v[i] & E) == E) v[i] &= 0xFFFF0000u;
    if ((v[i] >> 16 & E) == E) v[i] &= 0x0000FFFFu;
  }
  return v;
}

// Infinities and NaN of the keys [k0, k1) that the lane's row sees (keys below `sees`),
// read once more; acc as store_rows has it.
template <bool F16, int W>
__device__ __forceinline__ void odd_values(const uint16_t* v, int64_t rs, int k0, int k1, int sees,
                                           int width, int half, f32x16 (&acc)[W / 32]) {
#pragma unroll 1
  for (int k = k0; k < k1; ++k)
#pragma unroll
    for (int dt = 0; dt < W / 32; ++dt)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int c = dt * 32 + 8 * g + 4 * half;
        if (c >= width || k >= sees) continue;
        const u32x2 w = *reinterpret_cast<const u32x2*>(v + k * rs + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = half_to_f32((uint16_t)(w[i >> 1] >> (16 * (i & 1))), F16);
          if (!(fabsf(x) < INFINITY)) acc[dt][4 * g + i] += x;
        }
      }
}

// A workgroup owns NW waves x 32 query rows of one head and goes over its keys in tiles
// of 64, double buffered, the next tile's direct loads beside this tile's products; one
// barrier per tile.
template <bool F16, int W, int NW>
__global__ __launch_bounds__(NW * 64, 2) void attend_kernel(Attend a, int64_t wg0, int64_t tiles) {
  constexpr int ROWS = NW * 32;
  constexpr int TB = kTile * W * 2;  // bytes of a tile
  __shared__ __align__(1024) uint8_t lds[4 * TB];
  const int64_t b = wg0 + blockIdx.x;
  if (b >= tiles * a.hq) {
    zero_outside(a.starts, a.seqs, a.n, (int64_t)a.hq * a.width, static_cast<uint16_t*>(a.o),
                 b - tiles * a.hq, NW * 64);
    return;
  }
  // causal: later rows see more keys, so the longest workgroups of a sequence come first (the
  // sequences themselves in packed order, from the last)
  const Place at = place_of(a.starts, a.seqs, a.n, ROWS, tiles - 1 - b / a.hq);
  const Span sq = span_of(a.starts, at.seq, a.n), sk = span_of(a.k_starts, at.seq, a.nk);
  if (at.row0 >= sq.len) return;
  const int head = head_of(b, a.hq), kvh = head / (a.hq / a.hk);
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);  // uniform to the compiler too
  const int shift = sk.len - sq.len;
  const uint16_t* kp = static_cast<const uint16_t*>(a.k) + sk.first * a.k_rs + kvh * a.k_hs;
  const uint16_t* vp = static_cast<const uint16_t*>(a.v) + sk.first * a.v_rs + kvh * a.v_hs;
  clear_lds<W>(lds, 4 * TB, a.width, NW * 64);

  const int row0 = at.row0 + wave * 32;
  const int row = row0 + (lane & 31), r0 = min(row, sq.len - 1);  // a lane's query row
  const int sees = max(a.causal ? min(r0 + shift + 1, sk.len) : sk.len, 0);  // and its keys
  u32x4 qf[W / 16];
  own_frags<W>(static_cast<const uint16_t*>(a.q) + (sq.first + r0) * a.q_rs + head * a.q_hs,
               a.width, half, qf);
  // scores times a positive number keep their order, and -infinity (masked) its value
  if (a.scale <= 0.0f)
#pragma unroll
    for (int ks = 0; ks < W / 16; ++ks)
      qf[ks] = a.scale == 0.0f ? u32x4{0u, 0u, 0u, 0u} : qf[ks] ^ 0x80008000u;
  const float c2 = a.scale == 0.0f ? 1.0f : fabsf(a.scale) * kLog2e;
  // fp16: weights stand times 2^9 beside the values, which leaves a row's largest (2^6 at most
  // where its maximum is not followed) in range, and whole digits to those under it by 2^-23;
  // without it many weights under 2^-14 lost theirs together (e^-15: 2.5% of their sum)
  constexpr float kLift = F16 ? 9.0f : 0.0f;
  const int keys = max(a.causal ? min(min(at.row0 + ROWS, sq.len) + shift, sk.len) : sk.len, 0);
  const int n_tiles = (keys + kTile - 1) / kTile;
  TileLoads<W, NW> k_loads, v_loads;
  k_loads.init(a.k_rs, a.width, wave, lane);
  v_loads.init(a.v_rs, a.width, wave, lane);
  // keys below: seen by every row of the workgroup; by every and by any row of the wave
  const int by_all = max(a.causal ? min(at.row0 + shift + 1, sk.len) : sk.len, 0) / kTile * kTile;
  const int least = a.causal ? min(row0 + shift + 1, sk.len) : sk.len;
  const int most = row0 >= sq.len ? 0 : a.causal ? min(row0 + 32 + shift, sk.len) : sk.len;

  TileReads<W> reads;
  f32x16 acc[W / 32];
  float m, l;
  for (int careful = 0;; careful = 1) {
    reads.init(lds, lane);
    m = -INFINITY;
    l = 0.0f;
#pragma unroll
    for (int dt = 0; dt < W / 32; ++dt)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[dt][r] = 0.0f;
    if (n_tiles > 0) {
      k_loads.load(kp, a.k_rs, 0, sk.len - 1, lds, wave);
      v_loads.load(vp, a.v_rs, 0, sk.len - 1, lds + TB, wave);
    }
    for (int j = 0; j < n_tiles; ++j) {
      EMK_WAIT_VMCNT(0);
      lds_barrier();  // tile j is whole, and tile j - 1 has been read
      uint8_t* now = lds + (j & 1) * 2 * TB;
      if (j + 1 < n_tiles) {
        uint8_t* next = lds + ((j + 1) & 1) * 2 * TB;
        k_loads.load(kp, a.k_rs, (j + 1) * kTile, sk.len - 1, next, wave);
        v_loads.load(vp, a.v_rs, (j + 1) * kTile, sk.len - 1, next + TB, wave);
      }
      const int k0 = j * kTile;
      if (careful && k0 >= by_all) {
        for (int i = threadIdx.x * 16; i < TB; i += NW * 64 * 16) {
          u32x4* v = reinterpret_cast<u32x4*>(now + TB + i);
          *v = numbers_of<F16>(*v);
        }
        lds_barrier();
      }
      if (j > 0) reads.move(j & 1 ? 2 * TB : -2 * TB);
      if (k0 >= most) continue;
      const bool part = k0 + kTile > least;
      // operands are read four products ahead (the barriers keep the order: left to
      // itself the compiler reads each right before its product)
      constexpr int N = W / 8, kAhead = 4;
      u32x4 f[kAhead];
      f32x16 s[2];
      auto key = [&](int i) { return reads.rows(i % (W / 16), i / (W / 16) * 32); };
#pragma unroll
      for (int i = 0; i < kAhead; ++i) f[i] = key(i);
#pragma unroll
      for (int r = 0; r < 16; ++r) s[0][r] = s[1][r] = 0.0f;
      __builtin_amdgcn_s_setprio(1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        f32x16& to = s[i / (W / 16)];
        to = product<F16>(f[i % kAhead], qf[i % (W / 16)], to);
        if (i + kAhead < N) f[i % kAhead] = key(i + kAhead);
        __builtin_amdgcn_sched_barrier(0);
      }
      __builtin_amdgcn_s_setprio(0);
      if (part) {
        asm volatile("");  // a branch: whole tiles are most
#pragma unroll
        for (int kt = 0; kt < 2; ++kt)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (k0 + kt * 32 + (r >> 2) * 8 + 4 * half + (r & 3) >= sees) s[kt][r] = -INFINITY;
      }
      float top = s[0][0];
#pragma unroll
      for (int r = 1; r < 32; ++r) top = fmaxf(top, s[r >> 4][r & 15]);
      top = half_max(top);
      // a row's maximum is followed only when it grows by a factor of 2^6 of the weights:
      // what matters is that they stay in range
      const bool up = (top - m) * c2 > 6.0f;
      if (__any(up)) {
        const float f = up ? __builtin_amdgcn_exp2f((m - top) * c2) : 1.0f;
        m = up ? top : m;
        l *= f;
#pragma unroll
        for (int dt = 0; dt < W / 32; ++dt)
#pragma unroll
          for (int r = 0; r < 16; ++r) acc[dt][r] *= f;
      }
      const float ref = (m == -INFINITY ? 0.0f : m) * c2 - kLift;
      auto value = [&](int i) { return reads.columns(i % (W / 32), 16 * (i / (W / 32)), TB); };
#pragma unroll
      for (int i = 0; i < kAhead; ++i) f[i] = value(i);
      __builtin_amdgcn_sched_barrier(0);
      u32x4 p[4];
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) {
        float sum = 0.0f;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          s[kt][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kt][r], c2, -ref));
          sum += s[kt][r];
        }
        l += sum;
        p[2 * kt] = packed<F16>(s[kt], 0);
        p[2 * kt + 1] = packed<F16>(s[kt], 8);
      }
      __builtin_amdgcn_s_setprio(1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int dt = i % (W / 32);
        acc[dt] = product<F16>(f[i % kAhead], p[i / (W / 32)], acc[dt]);
        if (i + kAhead < N) f[i % kAhead] = value(i + kAhead);
        __builtin_amdgcn_sched_barrier(0);
      }
      __builtin_amdgcn_s_setprio(0);
    }
    if (careful) {
      odd_values<F16, W>(vp, a.v_rs, by_all, keys, sees, a.width, half, acc);
      break;
    }
    // no numbers though the scores were: look again, rows that see part of a tile apart
    float z = 0.0f;
#pragma unroll
    for (int dt = 0; dt < W / 32; ++dt)
#pragma unroll
      for (int r = 0; r < 16; ++r) z += acc[dt][r] * 0.0f;
    if (!__syncthreads_or(z != 0.0f && l == l)) break;
  }
  const float sum = half_sum(l);
  const bool on = row < sq.len;
  if (a.lse && half == 0 && on)
    a.lse[(int64_t)head * a.n + sq.first + row] =
        sum == 0.0f ? INFINITY : (m == -INFINITY ? 0.0f : m * c2) + (__builtin_amdgcn_logf(sum) - kLift);
  const int64_t to = ((int64_t)(sq.first + r0) * a.hq + head) * a.width;
  store_rows<F16, W>(acc, sum == 0.0f ? 0.0f : 1.0f / sum, static_cast<uint16_t*>(a.o) + to,
                     a.rest ? static_cast<uint16_t*>(a.rest) + to : nullptr, a.width, half, on);
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------

// fp16 holds 2^-24 to 65504, while dS may be anything: where a product's sum runs over them, it
// is kept times a power of two that the result's own row makes (a query of dQ, a key of dK),
// so that nothing else in the call costs its digits. The number starts at 2^80 (|dO V^T - D|
// is under 2^41 for fp16 data) and falls when the row's largest leaves fp16's safe range,
// to 2^11: what is added is off by half a unit of its own or by 2^-36 of the largest. A number
// for the whole call, made by a pass over dO and V, lost a sequence's digits to large values of
// others and of rows outside all sequences, and took longer (seven sequences of up to 4000 tokens,
// 32 / 8 heads of 128, the whole step 1848 us against 1753).
constexpr float kFirstLift = 0x1p80f, kTopDs = 0x1p15f;

// ds (times the row's number) made to fit: true where acc, and the number, have to be
// multiplied by `by`. Both halves of a row have the same one, as they share acc's columns.
__device__ __forceinline__ bool outgrown(const f32x16& ds, float& by) {
  float top = 0.0f;
#pragma unroll
  for (int r = 0; r < 16; ++r) top = fmaxf(top, fabsf(ds[r]));
  top = half_max(top);
  const bool up = top > kTopDs;
  // 2^(11 - exponent of top); an infinity counts as 2^128
  by = up ? __uint_as_float((127 + 11 + 127 - (__float_as_uint(top) >> 23)) << 23) : 1.0f;
  return __any(up);
}

// dQ: a workgroup owns 128 query rows of a head; P^T and dS^T of a tile of 64 keys have
// a lane's query row as column. D of the rows is made here and left for the other
// kernel.
template <bool F16, int W>
__global__ __launch_bounds__(256, 2) void query_grad_kernel(Attend a, int64_t wg0, int64_t tiles) {
  constexpr int NW = 4, ROWS = NW * 32, TB = kTile * W * 2;
  __shared__ __align__(1024) uint8_t lds[4 * TB];
  const int64_t b = wg0 + blockIdx.x;
  if (b >= tiles * a.hq) {
    zero_outside(a.starts, a.seqs, a.n, (int64_t)a.hq * a.width, static_cast<uint16_t*>(a.dq),
                 b - tiles * a.hq, NW * 64);
    return;
  }
  const Place at = place_of(a.starts, a.seqs, a.n, ROWS, tiles - 1 - b / a.hq);
  const Span sq = span_of(a.starts, at.seq, a.n), sk = span_of(a.k_starts, at.seq, a.nk);
  if (at.row0 >= sq.len) return;
  const int head = head_of(b, a.hq), kvh = head / (a.hq / a.hk);
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);  // uniform to the compiler too
  const int shift = sk.len - sq.len;
  const uint16_t* kp = static_cast<const uint16_t*>(a.k) + sk.first * a.k_rs + kvh * a.k_hs;
  const uint16_t* vp = static_cast<const uint16_t*>(a.v) + sk.first * a.v_rs + kvh * a.v_hs;
  clear_lds<W>(lds, 4 * TB, a.width, NW * 64);

  const int row = at.row0 + wave * 32 + (lane & 31), r0 = min(row, sq.len - 1);
  const int sees = max(a.causal ? min(r0 + shift + 1, sk.len) : sk.len, 0);
  const int64_t full = sq.first + r0;
  u32x4 qf[W / 16], gf[W / 16];
  own_frags<W>(static_cast<const uint16_t*>(a.q) + full * a.q_rs + head * a.q_hs, a.width, half, qf);
  own_frags<W>(static_cast<const uint16_t*>(a.dout) + full * a.do_rs + head * a.do_hs, a.width, half, gf);
  float d = 0.0f;
  {
    // o as it was before its rounding to 16 bits: the rounding would stand in D, which all
    // of a row's dS share, and grow the error of dQ and dK by 8% (measured on causal rows)
    u32x4 of[W / 16], rf[W / 16];
    const int64_t o = (full * a.hq + head) * a.width;
    own_frags<W>(static_cast<const uint16_t*>(a.o) + o, a.width, half, of);
    own_frags<W>(static_cast<const uint16_t*>(a.rest) + o, a.width, half, rf);
    auto number = [](const u32x4& w, int i) {
      return half_to_f32((uint16_t)(w[i >> 1] >> (16 * (i & 1))), F16);
    };
#pragma unroll
    for (int ks = 0; ks < W / 16; ++ks)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        d += (number(of[ks], i) + number(rf[ks], i)) * number(gf[ks], i);
  }
  d = half_sum(d);
  const float lse = a.lse[(int64_t)head * a.n + full];
  if (half == 0 && row < sq.len) a.delta[(int64_t)head * a.n + full] = d;
  float factor = F16 ? kFirstLift : 1.0f;
  d *= factor;
  const float c2 = a.scale * kLog2e;
  const int keys = max(a.causal ? min(min(at.row0 + ROWS, sq.len) + shift, sk.len) : sk.len, 0);
  const int n_tiles = (keys + kTile - 1) / kTile;
  f32x16 acc[W / 32];
#pragma unroll
  for (int dt = 0; dt < W / 32; ++dt)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[dt][r] = 0.0f;
  TileLoads<W, NW> k_loads, v_loads;
  k_loads.init(a.k_rs, a.width, wave, lane);
  v_loads.init(a.v_rs, a.width, wave, lane);
  TileReads<W> reads;
  reads.init(lds, lane);
  if (n_tiles > 0) {
    k_loads.load(kp, a.k_rs, 0, sk.len - 1, lds, wave);
    v_loads.load(vp, a.v_rs, 0, sk.len - 1, lds + TB, wave);
  }
  for (int j = 0; j < n_tiles; ++j) {
    EMK_WAIT_VMCNT(0);
    lds_barrier();
    if (j + 1 < n_tiles) {
      uint8_t* next = lds + ((j + 1) & 1) * 2 * TB;
      k_loads.load(kp, a.k_rs, (j + 1) * kTile, sk.len - 1, next, wave);
      v_loads.load(vp, a.v_rs, (j + 1) * kTile, sk.len - 1, next + TB, wave);
    }
    const int k0 = j * kTile, w0 = at.row0 + wave * 32;
    if (j > 0) reads.move(j & 1 ? 2 * TB : -2 * TB);
    if (k0 >= (a.causal ? min(w0 + 32 + shift, sk.len) : sk.len) || w0 >= sq.len) continue;
    const bool part = k0 + kTile > (a.causal ? min(w0 + shift + 1, sk.len) : sk.len);
    constexpr int N = W / 16, kAhead = 4, kTurn = N % kAhead;
#pragma unroll
    for (int kt = 0; kt < 2; ++kt) {
      u32x4 f[kAhead];
      f32x16 s, dp;
#pragma unroll
      for (int r = 0; r < 16; ++r) s[r] = dp[r] = 0.0f;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) f[i] = reads.rows(i, kt * 32);
      __builtin_amdgcn_s_setprio(1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        s = product<F16>(f[i % kAhead], qf[i], s);
        f[i % kAhead] = i + kAhead < N ? reads.rows(i + kAhead, kt * 32)
                                       : reads.rows(i + kAhead - N, kt * 32, TB);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        dp = product<F16>(f[(i + kTurn) % kAhead], gf[i], dp);
        if (i + kAhead < N) f[(i + kTurn) % kAhead] = reads.rows(i + kAhead, kt * 32, TB);
        __builtin_amdgcn_sched_barrier(0);
      }
      auto column = [&](int i) { return reads.columns(i % (W / 32), kt * 32 + 16 * (i / (W / 32))); };
#pragma unroll
      for (int i = 0; i < kAhead; ++i) f[i] = column(i);
      __builtin_amdgcn_s_setprio(0);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], c2, -lse));
        dp[r] = p * __builtin_fmaf(dp[r], factor, -d);
      }
      if (part) {
        asm volatile("");  // a branch: whole tiles are most
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (k0 + kt * 32 + (r >> 2) * 8 + 4 * half + (r & 3) >= sees) dp[r] = 0.0f;
      }
      if constexpr (F16) {
        float by;
        if (outgrown(dp, by)) {
          factor *= by;
          d *= by;
#pragma unroll
          for (int r = 0; r < 16; ++r) dp[r] *= by;
#pragma unroll
          for (int dt = 0; dt < W / 32; ++dt)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[dt][r] *= by;
        }
      }
      // dS (and P of dV) rounded to the inputs' type, as large an error as the result's own
      // rounding and independent of it; two terms would take a product more
      const u32x4 ds[2] = {packed<F16>(dp, 0), packed<F16>(dp, 8)};
      __builtin_amdgcn_s_setprio(1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int dt = i % (W / 32);
        acc[dt] = product<F16>(f[i % kAhead], ds[i / (W / 32)], acc[dt]);
        if (i + kAhead < N) f[i % kAhead] = column(i + kAhead);
        __builtin_amdgcn_sched_barrier(0);
      }
      __builtin_amdgcn_s_setprio(0);
    }
  }
  store_rows<F16, W>(acc, a.scale / factor,
                     static_cast<uint16_t*>(a.dq) + (full * a.hq + head) * a.width, nullptr, a.width,
                     half, row < sq.len);
}

// dK and dV: a workgroup owns 128 key rows of a key-value head and goes over the
// queries that see them, head by head of the group, in tiles of 32; P and dS of a tile
// have a lane's key row as column. K stays in registers and V in LDS, which leaves room
// for two waves on a SIMD (both in registers and one wave: 1.56 against 0.88 ms, seven
// sequences of up to 4000 tokens, 32 / 8 heads of 128).
// Where that leaves CUs idle, `cuts` workgroups share the list of a key tile's (head, query
// tile) pairs and leave fp32 sums, which key_sum_kernel adds in order.
template <bool F16, int W>
__global__ __launch_bounds__(256, 2) void key_grad_kernel(Attend a, int64_t wg0, int64_t tiles,
                                                          int cuts) {
  constexpr int NW = 4, ROWS = NW * 32, R = 32;
  constexpr int QB = R * W * 2, VB = ROWS * W * 2;  // bytes: of a tile of Q or dO, of V
  // fp16: P for dV times 2^14, in range as P <= 1; whole digits down to 2^-28, a step of 2^-38 below
  constexpr float kLift = F16 ? 14.0f : 0.0f;
  __shared__ __align__(1024) uint8_t lds[4 * QB + VB];
  __shared__ float lse[2][R], delta[2][R];
  const int64_t all = wg0 + blockIdx.x, b = all / cuts;
  const int cut = (int)(all - b * cuts);
  if (b >= tiles * a.hk) {
    if (b - tiles * a.hk >= kZeroGroups || cut) return;
    zero_outside(a.k_starts, a.seqs, a.nk, (int64_t)a.hk * a.width, static_cast<uint16_t*>(a.dk),
                 b - tiles * a.hk, NW * 64);
    zero_outside(a.k_starts, a.seqs, a.nk, (int64_t)a.hk * a.width, static_cast<uint16_t*>(a.dv),
                 b - tiles * a.hk, NW * 64);
    return;
  }
  const Place at = place_of(a.k_starts, a.seqs, a.nk, ROWS, b / a.hk);
  const Span sq = span_of(a.starts, at.seq, a.n), sk = span_of(a.k_starts, at.seq, a.nk);
  if (at.row0 >= sk.len) return;
  const int kvh = head_of(b, a.hk), group = a.hq / a.hk;
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);  // uniform to the compiler too
  const int shift = sk.len - sq.len;
  clear_lds<W>(lds, 4 * QB + VB, a.width, NW * 64);

  const int w0 = at.row0 + wave * 32, key = w0 + (lane & 31);
  const int64_t full = sk.first + min(key, sk.len - 1);
  u32x4 kf[W / 16];
  own_frags<W>(static_cast<const uint16_t*>(a.k) + full * a.k_rs + kvh * a.k_hs, a.width, half, kf);
  // query rows that see the workgroup's first key
  const int first = a.causal ? max(at.row0 - shift, 0) / R * R : 0;
  const int per = sq.len > first ? (sq.len - first + R - 1) / R : 0;
  // this workgroup's part of the list
  const int64_t listed = (int64_t)per * group;
  const int from = (int)(listed * cut / cuts), n_tiles = (int)(listed * (cut + 1) / cuts) - from;
  if (n_tiles > 0) {  // waited for before the first tile: no load outlives the workgroup
    TileLoads<W, NW> loads;
    loads.init(a.v_rs, a.width, wave, lane);
    const uint16_t* vp = static_cast<const uint16_t*>(a.v) + sk.first * a.v_rs + kvh * a.v_hs;
    loads.load(vp, a.v_rs, at.row0, sk.len - 1, lds + 4 * QB, wave);
    loads.load(vp, a.v_rs, min(at.row0 + kTile, sk.len - 1), sk.len - 1, lds + 4 * QB + VB / 2, wave);
  }
  // fp16: dS is 2^14 P times (dP - D) times `factor`
  constexpr float kUnlift = F16 ? 0x1p-14f : 1.0f;
  float factor = F16 ? kFirstLift * kUnlift : 1.0f;
  const float c2 = a.scale * kLog2e;
  f32x16 dk[W / 32], dv[W / 32];
#pragma unroll
  for (int dt = 0; dt < W / 32; ++dt)
#pragma unroll
    for (int r = 0; r < 16; ++r) dk[dt][r] = dv[dt][r] = 0.0f;
  TileLoads<W, NW, R> q_loads, g_loads;
  q_loads.init(a.q_rs, a.width, wave, lane);
  g_loads.init(a.do_rs, a.width, wave, lane);
  // the next tile to be fetched
  int head = kvh * group + (per ? from / per : 0), q0 = first + (per ? from % per : 0) * R;
  int at_q = q0;
  auto fetch = [&](int j) {
    uint8_t* to = lds + (j & 1) * 2 * QB;
    q_loads.load(static_cast<const uint16_t*>(a.q) + sq.first * a.q_rs + head * a.q_hs, a.q_rs, q0,
                 sq.len - 1, to, wave);
    g_loads.load(static_cast<const uint16_t*>(a.dout) + sq.first * a.do_rs + head * a.do_hs,
                 a.do_rs, q0, sq.len - 1, to + QB, wave);
    if (wave < 2 && lane < R) {
      const float* from = (wave ? a.delta : a.lse) + (int64_t)head * a.n + sq.first;
      lds_load4(from + min(q0 + lane, sq.len - 1), wave ? &delta[j & 1][0] : &lse[j & 1][0]);
    }
    q0 += R;
    if (q0 >= sq.len) {
      q0 = first;
      ++head;
    }
  };
  TileReads<W> reads;
  reads.init(lds, lane);
  const uint32_t v_rows = 4 * QB + wave * 32 * W * 2;  // of the wave's V beside the tile's rows
  if (n_tiles > 0) fetch(0);
  for (int j = 0; j < n_tiles; ++j, at_q = at_q + R >= sq.len ? first : at_q + R) {
    EMK_WAIT_VMCNT(0);
    lds_barrier();
    if (j + 1 < n_tiles) fetch(j + 1);
    if (j > 0) reads.move(j & 1 ? 2 * QB : -2 * QB);
    if (w0 >= sk.len) continue;
    if (a.causal && at_q + R - 1 + shift < w0) continue;  // no row sees the wave's first key
    const bool part = at_q + R > sq.len || (a.causal && at_q + shift < w0 + 31);
    const uint32_t v_at = v_rows - (j & 1) * 2 * QB;
    constexpr int N = W / 16, kAhead = 4;
    u32x4 f[kAhead];
    f32x16 s, dp;
#pragma unroll
    for (int r = 0; r < 16; ++r) s[r] = dp[r] = 0.0f;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) f[i] = reads.rows(i, 0);
    __builtin_amdgcn_s_setprio(1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      s = product<F16>(f[i % kAhead], kf[i], s);
      f[i % kAhead] = i + kAhead < N ? reads.rows(i + kAhead, 0) : reads.rows(i + kAhead - N, 0, QB);
      __builtin_amdgcn_sched_barrier(0);
    }
    // (W 96 leaves the first fragments of dO in another place)
    constexpr int kTurn = N % kAhead;
    u32x4 v[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) v[i] = reads.rows(i, 0, v_at);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      dp = product<F16>(f[(i + kTurn) % kAhead], v[i % kAhead], dp);
      if (i + kAhead < N) {
        f[(i + kTurn) % kAhead] = reads.rows(i + kAhead, 0, QB);
        v[i % kAhead] = reads.rows(i + kAhead, 0, v_at);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    auto column = [&](int i) {  // of dO, then of Q
      const int k = i % N;
      return reads.columns(k % (W / 32), 16 * (k / (W / 32)), i < N ? QB : 0);
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) f[i] = column(i);
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int r0 = 8 * g + 4 * half;
      const f32x4 e = *reinterpret_cast<const f32x4*>(&lse[j & 1][r0]);
      const f32x4 d = *reinterpret_cast<const f32x4*>(&delta[j & 1][r0]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 4 * g + i;
        s[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], c2, kLift - e[i]));
        dp[r] = s[r] * __builtin_fmaf(dp[r], factor, -d[i] * factor);
      }
    }
    if (part) {
      asm volatile("");  // a branch: whole tiles are most
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int q = at_q + 8 * (r >> 2) + 4 * half + (r & 3);
        if (q >= sq.len || (a.causal && q + shift < key)) s[r] = dp[r] = 0.0f;
      }
    }
    if constexpr (F16) {
      float by;
      if (outgrown(dp, by)) {
        factor *= by;
#pragma unroll
        for (int r = 0; r < 16; ++r) dp[r] *= by;
#pragma unroll
        for (int dt = 0; dt < W / 32; ++dt)
#pragma unroll
          for (int r = 0; r < 16; ++r) dk[dt][r] *= by;
      }
    }
    const u32x4 p[2] = {packed<F16>(s, 0), packed<F16>(s, 8)};
    const u32x4 ds[2] = {packed<F16>(dp, 0), packed<F16>(dp, 8)};
    __builtin_amdgcn_s_setprio(1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < 2 * N; ++i) {
      const int k = i % N, dt = k % (W / 32), h = k / (W / 32);
      if (i < N)
        dv[dt] = product<F16>(f[i % kAhead], p[h], dv[dt]);
      else
        dk[dt] = product<F16>(f[i % kAhead], ds[h], dk[dt]);
      if (i + kAhead < 2 * N) f[i % kAhead] = column(i + kAhead);
      __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_setprio(0);
  }
  const int64_t to = (full * a.hk + kvh) * a.width;
  const float back = a.scale / factor * kUnlift;
  if (cuts > 1) {
    if (key >= sk.len) return;
    const int64_t size = a.nk * a.hk * a.width;
    float* part = a.part + cut * 2 * size + to;
#pragma unroll
    for (int dt = 0; dt < W / 32; ++dt)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int c = dt * 32 + 8 * g + 4 * half;
        if (c >= a.width) continue;
        f32x4 x, y;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] = dk[dt][4 * g + i] * back;
          y[i] = dv[dt][4 * g + i] * kUnlift;
        }
        *reinterpret_cast<f32x4*>(part + c) = x;
        *reinterpret_cast<f32x4*>(part + size + c) = y;
      }
    return;
  }
  store_rows<F16, W>(dk, back, static_cast<uint16_t*>(a.dk) + to, nullptr, a.width,
                     half, key < sk.len);
  store_rows<F16, W>(dv, kUnlift, static_cast<uint16_t*>(a.dv) + to, nullptr, a.width, half,
                     key < sk.len);
}

// The sums that several workgroups left, added in order and rounded: rows of sequences, of
// which none lies before the first start or behind the last.
template <bool F16>
__global__ __launch_bounds__(256) void key_sum_kernel(Attend a, int cuts) {
  constexpr int OT = F16 ? 4 : 1;
  const int64_t d = (int64_t)a.hk * a.width, size = a.nk * d;
  const int64_t first = max(0, min(a.k_starts[0], (int)a.nk)) * d;
  const int64_t last = max(0, min(a.k_starts[a.seqs], (int)a.nk)) * d;
  for (int64_t i = first + ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < last;
       i += (int64_t)gridDim.x * 1024) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int c = 0; c < cuts; ++c)
        v += *reinterpret_cast<const f32x4*>(a.part + (2 * c + s) * size + i);
      *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(s ? a.dv : a.dk) + i) =
          u32x2{pack2<OT>(v[0], v[1]), pack2<OT>(v[2], v[3])};
    }
  }
}

template <typename GO>
hipError_t in_launches(int64_t wgs, GO go) {
  for (int64_t wg0 = 0; wg0 < wgs; wg0 += kMaxGroups) {
    go(wg0, (unsigned)(wgs - wg0 < kMaxGroups ? wgs - wg0 : kMaxGroups));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <bool F16, int W>
hipError_t forward_t(const Attend& a, hipStream_t st) {
  constexpr int NW = 4;
  const int64_t tiles = a.seqs ? a.n / (NW * 32) + a.seqs : 0;
  return in_launches(tiles * a.hq + kZeroGroups, [&](int64_t wg0, unsigned grid) {
    attend_kernel<F16, W, NW><<<grid, NW * 64, 0, st>>>(a, wg0, tiles);
  });
}

// Workgroups that share a key tile: two per CU fit, and a tile's list may be long. Measured:
// one sequence of 3800 tokens, 16 / 4 heads of 128 (120 tiles), the step 845 us with one
// each, 443 with four, 408 with eight; seven sequences of up to 4000, 32 / 8 heads (568
// tiles), dK and dV 877 us with one each, 765 and 42 for the sums with two.
int cuts_of(int64_t nk, int64_t seqs, int hk) {
  const int64_t wgs = (nk / 128 + seqs) * hk;
  if (wgs < 1 || wgs >= 1024) return 1;
  const int64_t cuts = (1024 + wgs - 1) / wgs;
  return (int)(cuts > 8 ? 8 : cuts);
}

template <bool F16, int W>
hipError_t backward_t(const Attend& a, hipStream_t st) {
  const int64_t q_tiles = a.seqs ? a.n / 128 + a.seqs : 0, k_tiles = a.seqs ? a.nk / 128 + a.seqs : 0;
  hipError_t e = in_launches(q_tiles * a.hq + kZeroGroups, [&](int64_t wg0, unsigned grid) {
    query_grad_kernel<F16, W><<<grid, 256, 0, st>>>(a, wg0, q_tiles);
  });
  if (e != hipSuccess) return e;
  const int cuts = cuts_of(a.nk, a.seqs, a.hk);
  e = in_launches((k_tiles * a.hk + kZeroGroups) * cuts, [&](int64_t wg0, unsigned grid) {
    key_grad_kernel<F16, W><<<grid, 256, 0, st>>>(a, wg0, k_tiles, cuts);
  });
  if (e != hipSuccess || cuts == 1) return e;
  const int64_t quads = a.nk * a.hk * a.width / 4;
  key_sum_kernel<F16><<<(unsigned)(quads / 256 + 1 < 2048 ? quads / 256 + 1 : 2048), 256, 0, st>>>(a, cuts);
  return hipGetLastError();
}

template <typename GO>
hipError_t by_type(const Attend& a, GO go) {
  auto width = [&](auto f16) {
    if (a.width <= 64) return go(f16, std::integral_constant<int, 64>());
    if (a.width <= 96) return go(f16, std::integral_constant<int, 96>());
    return go(f16, std::integral_constant<int, 128>());
  };
  return a.dt == 4 ? width(std::true_type()) : width(std::false_type());
}

}  // namespace

size_t attend_work(int64_t n, int64_t nk, int hq, int hk, int width, int64_t seqs) {
  const int cuts = cuts_of(nk, seqs, hk);
  return (cuts > 1 ? (size_t)cuts * 2 * nk * hk * width * 4 : 0) + (size_t)n * hq * 4;
}

hipError_t launch_attend(const Attend& a, hipStream_t st) {
  return by_type(a, [&](auto f16, auto w) {
    return forward_t<decltype(f16)::value, decltype(w)::value>(a, st);
  });
}

hipError_t launch_attend_back(Attend a, void* work, hipStream_t st) {
  a.part = static_cast<float*>(work);
  const int cuts = cuts_of(a.nk, a.seqs, a.hk);
  a.delta = a.part + (cuts > 1 ? (int64_t)cuts * 2 * a.nk * a.hk * a.width : 0);
  return by_type(a, [&](auto f16, auto w) {
    return backward_t<decltype(f16)::value, decltype(w)::value>(a, st);
  });
}

}  // namespace emk
