// 8-bit codes with one power-of-two scale for each block of values: encoding
// (along rows, along columns, in 128 x 128 tiles) and a store of such codes
// written and read row by row.
//
// The scale of a block with largest finite magnitude a is s = 2^e, the
// smallest power of two with a <= L s (L = 448 for E4M3, 127 for int8; e in
// [-127, 127]; s = 1 where a = 0), kept as the byte e + 127 (E8M0; byte 255
// stands for NaN and is never written). A code is the nearest representable
// value of x / s (exact but for results that E4M3 rounds to zero anyway), ties
// to even; infinities saturate, NaN becomes the E4M3 NaN or int8 0.
//
// All kernels here move bytes: a few VALU operations per value, bound by HBM
// at large sizes (a 1 GiB copy reaches 5.2 TB/s on this card) and by the launch
// at small ones (3.5-4 us in a graph, of which the kernel is a third).
#include <type_traits>

#include "block.hpp"
#include "kernels.hpp"

namespace emk {

namespace {

// Store the first cnt <= 8 code bytes of w.
__device__ __forceinline__ void store_codes(uint8_t* p, u32x2 w, int cnt) {
  if (cnt >= 8) {
    store_any(p, w);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < cnt) p[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
}

// ---------------------------------------------------------------------------
// Rows with a scale per block along the row. A group of G lanes, eight values
// each, takes one block of one row (G = the power of two that covers the
// block, 16 for 128): the block's maximum stays in the group, and each byte is
// read once and written once. With SLOTS the row goes to row slots[row] of the
// output (skipped where that lies outside [0, cap)).
//
// The value (h, c) of row r sits at r * rs + h * hs + c, c < width: heads of a
// fused projection, or one head of width d for plain rows. Blocks never
// straddle heads (the host checks it).
//
// Measured: 32768 rows of 16 heads of 128, bf16, to random slots 43.6 us (4.6
// TB/s: each row lands in a 2 KB run of its own); 33 rows 4 us.
// ---------------------------------------------------------------------------
struct RowsIn {
  const void* X;
  int64_t rs, hs;
  int width;
};

// A workgroup takes (256 / G) U consecutive blocks, a group every 256 / G'th of
// them, all U loaded before the first is encoded. U = 2 at large sizes (16384 x
// 4096 bf16: 36.4 us, 5.5 TB/s; U = 1 38.9, 4 40.9, 8 47.0), U = 1 where that
// would leave CUs without a workgroup.
__device__ __forceinline__ uint32_t quotient(uint32_t a, uint32_t div, uint32_t inv) {
  return inv ? __umulhi(a, inv) : a / div;  // inv = 2^32 / div rounded up, or 0
}

uint32_t inverse(uint64_t div, uint64_t most) {  // exact for dividends up to most; 0: divide
  return div > 1 && most * div < (1ull << 32) ? (uint32_t)((1ull << 32) / div + 1) : 0;
}

template <int DT, bool I8, int G, int SLOTS, int U>
__global__ __launch_bounds__(256) void encode_rows_kernel(RowsIn in, int64_t wg0, int64_t n, int d,
                                                          int block, uint32_t nb, uint32_t nb_inv,
                                                          const void* __restrict__ slots,
                                                          int64_t cap,
                                                          uint8_t* __restrict__ codes,
                                                          int64_t ldc,
                                                          uint8_t* __restrict__ scales,
                                                          int64_t lds) {
  constexpr int kGroups = 256 / G;
  const int64_t first = (wg0 + blockIdx.x) * (kGroups * U);
  const int64_t row0 = first / nb;
  const uint32_t skip = (uint32_t)(first - row0 * nb) + threadIdx.x / G;
  const int sub = threadIdx.x & (G - 1);
  float v[U][8];
  int64_t to[U];
  int cnt[U], c0[U], blk[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t j = skip + kGroups * u;
    const uint32_t r = quotient(j, nb, nb_inv);
    const int64_t row = row0 + r;
    blk[u] = (int)(j - r * nb);
    to[u] = row < n ? row : -1;
    if constexpr (SLOTS != 0) {
      if (row < n) {
        to[u] = SLOTS == 8 ? static_cast<const int64_t*>(slots)[row]
                           : (int64_t) static_cast<const int32_t*>(slots)[row];
        if (to[u] >= cap) to[u] = -1;
      }
    }
    c0[u] = blk[u] * block + 8 * sub;  // first column of the lane
    cnt[u] = 8 * sub < block ? min(8, min(d, (blk[u] + 1) * block) - c0[u]) : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[u][i] = 0.0f;
    if (cnt[u] > 0 && row < n) {
      int64_t at = row * in.rs + c0[u];
      if (in.width != d) {
        const int h = c0[u] / in.width;
        at += h * (in.hs - in.width);
      }
      load8<DT>(in.X, at, cnt[u], v[u]);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint32_t m = group_max<G>(amax8(v[u]));
    const bool odd = m >= kInfBits;
    if (odd) m = group_max<G>(amax8_finite(v[u]));
    const uint32_t byte = scale_byte<I8>(m);
    if (to[u] < 0) continue;
    if (cnt[u] > 0)
      store_codes(codes + to[u] * ldc + c0[u], codes8<I8>(v[u], inv_scale(byte), odd), cnt[u]);
    if (sub == 0) scales[to[u] * lds + blk[u]] = (uint8_t)byte;
  }
}

// ---------------------------------------------------------------------------
// One 128 x 128 tile per workgroup, read once for both orders: codes of the
// rows and the codes of the columns, transposed. Thread t holds PR rows from
// PR (t / 16) on (PR = 8, or 4 for fp32) and columns 8 (t % 16) .. + 8, so a
// row's maximum is a reduction over 16 lanes, a column's one over the thread's
// rows, four lane groups and the waves, and a column's codes of a thread are
// PR consecutive bytes of the transposed output. TILES: one scale for the tile,
// and both orders hold the same codes.
// ---------------------------------------------------------------------------
// Magnitudes are compared as the bits of the number type (16-bit types two at
// a time, in packed registers that also hold the values until they are used).
//
// Measured: 16384 x 4096 bf16 both orders 56 us (4.8 TB/s), tiles 47 us (5.7);
// fp32 both 80 us (5.1); 777 x 768 fp32 7.3 us, where 42 tiles do not fill the
// card: a column's block is 128 rows, so the tile cannot be smaller.
constexpr int kT = 128;
constexpr int kTPitch = kT + 8;  // bytes per transposed row in LDS: 8-byte aligned

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

struct MaxU16x2 {
  __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                  __builtin_bit_cast(u16x2, b)));
  }
};

// A thread's patch of PR x 8 values: 8 rows, or 4 for fp32 (its values would
// take 64 registers, and the rest did not fit beside them). Keys are magnitude
// bits: one per word for fp32, two per word for the 16-bit types.
template <int DT>
struct Patch {
  static constexpr int PR = DT == 0 ? 4 : 8;
  static constexpr int kThreads = 16 * kT / PR;
  static constexpr int kWaves = kThreads / 64;
  static constexpr int W = DT == 0 ? 8 : 4;  // words of a row
  static constexpr uint32_t kAbs = DT == 0 ? 0x7FFFFFFFu : 0x7FFF7FFFu;
  static constexpr uint32_t kInf = DT == 0 ? kInfBits : DT == 1 ? 0x7F80u : 0x7C00u;
  uint32_t w[PR][W];

  __device__ __forceinline__ static uint32_t kmax(uint32_t a, uint32_t b) {
    if constexpr (DT == 0)
      return max(a, b);
    else
      return MaxU16x2()(a, b);
  }
  __device__ __forceinline__ static uint32_t finite(uint32_t k) {  // non-finite keys as 0
    if constexpr (DT == 0) return k < kInf ? k : 0u;
    const uint32_t lo = k & 0xFFFFu, hi = k >> 16;
    return (lo < kInf ? lo : 0u) | (hi < kInf ? hi << 16 : 0u);
  }
  __device__ __forceinline__ static uint32_t widest(uint32_t k) {  // of a word's keys
    if constexpr (DT == 0) return k;
    return max(k & 0xFFFFu, k >> 16);
  }
  __device__ __forceinline__ static uint32_t key(uint32_t k, int i) {  // of value i of two
    if constexpr (DT == 0) return k;
    return i ? k >> 16 : k & 0xFFFFu;
  }
  __device__ __forceinline__ static uint32_t bits(uint32_t key) {  // key as fp32 bits
    if constexpr (DT == 0) return key;
    return __float_as_uint(half_to_f32((uint16_t)key, DT == 4));
  }
  __device__ __forceinline__ float at(int p, int i) const {
    if constexpr (DT == 0) return __uint_as_float(w[p][i]);
    if constexpr (DT == 1)
      return __uint_as_float(i & 1 ? w[p][i >> 1] & 0xFFFF0000u : w[p][i >> 1] << 16);
    return f16_to_f32((uint16_t)(w[p][i >> 1] >> (16 * (i & 1))));
  }
  // row p from memory: the cnt <= 8 values from base[at0] on, zeros after them
  __device__ __forceinline__ void load(int p, const void* base, int64_t at0, int cnt) {
#pragma unroll
    for (int q = 0; q < W; ++q) w[p][q] = 0u;
    if (cnt >= 8) {
      const char* v = static_cast<const char*>(base) + at0 * (DT == 0 ? 4 : 2);
#pragma unroll
      for (int h = 0; h < W / 4; ++h) {
        const u32x4 x = load_any<u32x4>(v + 16 * h);
#pragma unroll
        for (int q = 0; q < 4; ++q) w[p][4 * h + q] = x[q];
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < cnt) {
        if constexpr (DT == 0)
          w[p][i] = static_cast<const uint32_t*>(base)[at0 + i];
        else
          w[p][i >> 1] |= (uint32_t) static_cast<const uint16_t*>(base)[at0 + i] << (16 * (i & 1));
      }
  }
  // Keeps the compiler from holding unpacked values across this point: 64
  // registers more, which would spill.
  __device__ __forceinline__ void forget() {
#pragma unroll
    for (int p = 0; p < PR; ++p)
#pragma unroll
      for (int q = 0; q < W; ++q) asm volatile("" : "+v"(w[p][q]));
  }
  template <bool FINITE>
  __device__ __forceinline__ uint32_t row_key(int p) const {
    uint32_t m = 0;
#pragma unroll
    for (int q = 0; q < W; ++q) m = kmax(m, FINITE ? finite(w[p][q] & kAbs) : w[p][q] & kAbs);
    return widest(m);
  }
  template <bool FINITE>
  __device__ __forceinline__ uint32_t col_key(int q) const {  // of word q's column(s)
    uint32_t m = 0;
#pragma unroll
    for (int p = 0; p < PR; ++p) m = kmax(m, FINITE ? finite(w[p][q] & kAbs) : w[p][q] & kAbs);
    return m;
  }
  __device__ __forceinline__ u32x2 row_codes(int p, float inv, bool odd) const {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = at(p, i);
    return codes8<false>(y, inv, odd);
  }
  // codes of column i to p[0 .. PR)
  __device__ __forceinline__ void col_codes(int i, float inv, bool odd, uint8_t* p) const {
    const uint32_t lo = codes4<false>(at(0, i), at(1, i), at(2, i), at(3, i), inv, odd);
    if constexpr (PR == 8)
      *reinterpret_cast<u32x2*>(p) =
          u32x2{lo, codes4<false>(at(4, i), at(5, i), at(6, i), at(7, i), inv, odd)};
    else
      *reinterpret_cast<uint32_t*>(p) = lo;
  }
};

template <int DT, bool TILES>
__global__ __launch_bounds__(Patch<DT>::kThreads) void encode_tile_kernel(
    const void* __restrict__ X, int64_t ldx, int64_t n, int d, uint8_t* __restrict__ codes,
    int64_t ldc, uint8_t* __restrict__ scales, int64_t lds, uint8_t* __restrict__ codes_t,
    int64_t ldct, uint8_t* __restrict__ scales_t, int64_t ldst) {
  using P = Patch<DT>;
  constexpr int PR = P::PR;
  constexpr int CW = P::W * 16;  // key words of a tile's columns
  __shared__ __attribute__((aligned(16))) uint8_t tr[kT * kTPitch];
  __shared__ uint32_t kmax[P::kWaves][CW];
  __shared__ uint32_t tmax[2][P::kWaves];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int rg = t >> 4, cg = t & 15;
  const int64_t r0 = (int64_t)blockIdx.y * kT;
  const int c0 = blockIdx.x * kT;
  const int rows = (int)min((int64_t)kT, n - r0), cols = min(kT, d - c0);
  const int ccnt = min(8, cols - 8 * cg);  // columns of this thread (may be <= 0)

  P x;
#pragma unroll
  for (int p = 0; p < PR; ++p) {
    const int r = PR * rg + p;
    x.load(p, X, (r0 + min(r, rows - 1)) * ldx + c0 + 8 * cg, r < rows ? ccnt : 0);
  }

  if constexpr (TILES) {
    uint32_t m = 0;
#pragma unroll
    for (int p = 0; p < PR; ++p) m = max(m, x.template row_key<false>(p));
    m = group_max<64>(m);
    if (lane == 0) tmax[0][wave] = m;
    __syncthreads();
#pragma unroll
    for (int v = 0; v < P::kWaves; ++v) m = max(m, tmax[0][v]);
    const bool odd = m >= P::kInf;
    if (odd) {  // the same answer in every thread of the workgroup
      m = 0;
#pragma unroll
      for (int p = 0; p < PR; ++p) m = max(m, x.template row_key<true>(p));
      m = group_max<64>(m);
      if (lane == 0) tmax[1][wave] = m;
      __syncthreads();
#pragma unroll
      for (int v = 0; v < P::kWaves; ++v) m = max(m, tmax[1][v]);
    }
    const uint32_t byte = scale_byte<false>(P::bits(m));
    const float inv = inv_scale(byte);
    if (t == 0) {
      if (codes) scales[(int64_t)blockIdx.y * lds + blockIdx.x] = (uint8_t)byte;
      if (codes_t) scales_t[(int64_t)blockIdx.x * ldst + blockIdx.y] = (uint8_t)byte;
    }
    if (codes) {
#pragma unroll
      for (int p = 0; p < PR; ++p)
        if (PR * rg + p < rows && ccnt > 0)
          store_codes(codes + (r0 + PR * rg + p) * ldc + c0 + 8 * cg, x.row_codes(p, inv, odd), ccnt);
    }
    if (!codes_t) return;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x.col_codes(i, inv, odd, &tr[(8 * cg + i) * kTPitch + PR * rg]);
  } else {
    // columns: the thread's rows, the four row groups of the wave, the waves.
    // A column that holds a non-finite value takes its finite maximum in a
    // second round.
    uint32_t ck[P::W];
    auto columns = [&](auto fin) {
#pragma unroll
      for (int q = 0; q < P::W; ++q) {
        uint32_t m = x.template col_key<decltype(fin)::value>(q);
        auto mx = [](uint32_t a, uint32_t b) { return P::kmax(a, b); };
        m = max_xor32(max_xor16(m, mx), mx);
        if (lane < 16) kmax[wave][P::W * cg + q] = m;
      }
      __syncthreads();
#pragma unroll
      for (int q = 0; q < P::W; ++q) {
        const int c = P::W * cg + q;
        uint32_t m = kmax[0][c];
#pragma unroll
        for (int v = 1; v < P::kWaves; ++v) m = P::kmax(m, kmax[v][c]);
        ck[q] = m;
      }
    };
    columns(std::false_type());
    bool odd = false;
#pragma unroll
    for (int q = 0; q < P::W; ++q) odd |= P::widest(ck[q]) >= P::kInf;
    odd = __syncthreads_or(odd);
    if (odd) columns(std::true_type());
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t byte = scale_byte<false>(
          P::bits(DT == 0 ? ck[i] : P::key(ck[DT == 0 ? i : i >> 1], i & 1)));
      x.col_codes(i, inv_scale(byte), odd, &tr[(8 * cg + i) * kTPitch + PR * rg]);
      if (rg == 0 && i < ccnt)
        scales_t[(int64_t)(c0 + 8 * cg + i) * ldst + blockIdx.y] = (uint8_t)byte;
    }
    x.forget();
    if (codes) {
#pragma unroll
      for (int p = 0; p < PR; ++p) {
        uint32_t m = group_max<16>(x.template row_key<false>(p));
        const bool bad = m >= P::kInf;
        if (bad) m = group_max<16>(x.template row_key<true>(p));
        const uint32_t byte = scale_byte<false>(P::bits(m));
        const int r = PR * rg + p;
        if (r < rows) {
          if (ccnt > 0)
            store_codes(codes + (r0 + r) * ldc + c0 + 8 * cg, x.row_codes(p, inv_scale(byte), bad),
                        ccnt);
          if (cg == 0) scales[(r0 + r) * lds + blockIdx.x] = (uint8_t)byte;
        }
      }
    }
  }
  __syncthreads();
  // transposed rows: 8 lanes write the 128 bytes of one column
#pragma unroll
  for (int q = 0; q < kT * 8 / P::kThreads; ++q) {
    const int f = q * P::kThreads + t;
    const int c = f >> 3, ch = f & 7;
    if (c >= cols) break;
    const u32x2 lo = *reinterpret_cast<const u32x2*>(&tr[c * kTPitch + 16 * ch]);
    const u32x2 hi = *reinterpret_cast<const u32x2*>(&tr[c * kTPitch + 16 * ch + 8]);
    uint8_t* p = codes_t + (int64_t)(c0 + c) * ldct + r0 + 16 * ch;
    const int cnt = rows - 16 * ch;
    if (cnt >= 16) {
      store_any(p, u32x4{lo[0], lo[1], hi[0], hi[1]});
    } else {
      store_codes(p, lo, cnt);
      store_codes(p + 8, hi, cnt - 8);
    }
  }
}

// ---------------------------------------------------------------------------
// Reading rows back: out = code * 2^e, rounded once to the output type. A lane
// makes 16 bytes of output, so a wave's stores are whole 1 KB runs.
// ---------------------------------------------------------------------------
template <bool I8>
__device__ __forceinline__ void values4(uint32_t w, float s, float (&y)[4]) {
  if constexpr (I8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = (float)(int8_t)(w >> (8 * i)) * s;
  } else {
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
    const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    y[0] = a[0] * s;
    y[1] = a[1] * s;
    y[2] = b[0] * s;
    y[3] = b[1] * s;
  }
}

// Where the rows come from: slots (one per row), or a page table.
struct RowsFrom {
  const void* slots;      // PAGES false: n entries of 4 or 8 bytes
  int slot_bytes;
  const int32_t* table;   // PAGES true: seqs x table_ld page ids
  int64_t table_ld;
  int table_pages;        // entries of a table row
  const int32_t* starts;  // seqs + 1: first packed row of each sequence
  int seqs;
  int page;               // rows per page
};

template <bool PAGES>
__device__ __forceinline__ int64_t source_row(const RowsFrom& f, int64_t row, int64_t cap) {
  if constexpr (!PAGES) {
    const int64_t s = f.slot_bytes == 8 ? static_cast<const int64_t*>(f.slots)[row]
                                        : (int64_t) static_cast<const int32_t*>(f.slots)[row];
    return s >= 0 && s < cap ? s : -1;
  } else {
    // the last sequence that starts at or before the row (empty ones share
    // their start with the next, which comes after them)
    int lo = 0, hi = f.seqs;  // starts[lo] <= row < starts[hi], if the row is in a sequence
    if (row < (int64_t)f.starts[0] || row >= (int64_t)f.starts[hi]) return -1;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((int64_t)f.starts[mid] <= row)
        lo = mid;
      else
        hi = mid;
    }
    const int64_t pos = row - f.starts[lo];
    const int64_t pi = pos / f.page;
    if (pi >= f.table_pages) return -1;
    const int64_t pg = f.table[(int64_t)lo * f.table_ld + pi];
    const int64_t s = pg * f.page + (pos - pi * f.page);
    return pg >= 0 && s < cap ? s : -1;
  }
}

// A workgroup takes R rows: their places are found first, one thread per row
// (a page table costs a chain of dependent reads, paid once per R rows), then
// the threads go over the rows' pieces of E values, E = 4 (fp32 out) or 8
// (16-bit out; block borders are at multiples of 16). Only a row's last piece
// may be short. Rows outside the store are zeros. Measured: 65536 random rows of
// 768 to fp32 41 us (6.1 TB/s, most of it written); 33 sequences of up to 4000
// rows of 2048 to bf16 through pages of 16 rows 64.5 us (6.3 TB/s; 191
// with the place found by every thread, one piece in flight and plain stores).
// The quotients by the pieces per row and by the block are products by `inv` =
// 2^32 / divisor, rounded up (exact while dividend x divisor < 2^32, which the
// host checks).
constexpr int kReadRows = 64;  // R at most

// The first cnt values of a piece of output, stored past the caches: most of the
// time of large reads is the writing (figures above, timed without a reader; what
// the next call gains from a small result in the caches was not measured).
__device__ __forceinline__ void store_out(float* o, f32x4 v, int cnt) {
  typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
  if (cnt >= 4) {
    __builtin_nontemporal_store(v, reinterpret_cast<f32x4_any*>(o));
    return;
  }
#pragma unroll
  for (int q = 0; q < 3; ++q)
    if (q < cnt) o[q] = v[q];
}

__device__ __forceinline__ void store_out(uint16_t* o, u32x4 v, int cnt) {
  typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
  if (cnt >= 8) {
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any*>(o));
    return;
  }
#pragma unroll
  for (int q = 0; q < 7; ++q)
    if (q < cnt) o[q] = (uint16_t)(v[q >> 1] >> (16 * (q & 1)));
}

struct Divisors {
  uint32_t per, per_inv, block, block_inv;
};

template <int OT, bool I8, bool PAGES>
__global__ __launch_bounds__(256) void decode_rows_kernel(const uint8_t* __restrict__ codes,
                                                          const uint8_t* __restrict__ scales,
                                                          int64_t cap, int d, int nb,
                                                          RowsFrom from, int64_t wg0, int64_t n,
                                                          int R, Divisors dv,
                                                          void* __restrict__ out, int64_t ldo) {
  constexpr int E = OT == 0 ? 4 : 8;
  constexpr int U = 4;  // pieces in flight per thread
  __shared__ int64_t place[kReadRows];
  const int64_t row0 = (wg0 + blockIdx.x) * R;
  const int rows = (int)min((int64_t)R, n - row0);
  if ((int)threadIdx.x < rows)
    place[threadIdx.x] = source_row<PAGES>(from, row0 + threadIdx.x, cap);
  __syncthreads();
  const uint32_t items = (uint32_t)rows * dv.per;
  for (uint32_t i0 = threadIdx.x; i0 < items; i0 += 256 * U) {
    u32x2 w[U];
    uint32_t sb[U];
    int r[U], c[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t i = i0 + 256 * u;
      w[u] = u32x2{0u, 0u};
      sb[u] = 0;
      if (i < items) {
        r[u] = (int)quotient(i, dv.per, dv.per_inv);
        c[u] = (int)(i - r[u] * dv.per) * E;
        const int64_t src = place[r[u]];
        if (src >= 0) {
          const uint8_t* p = codes + src * d + c[u];
          const int cnt = d - c[u];
          if (cnt >= E) {
            if constexpr (E == 8)
              w[u] = load_any<u32x2>(p);
            else
              w[u][0] = load_any<uint32_t>(p);
          } else {
#pragma unroll
            for (int q = 0; q < E - 1; ++q)
              if (q < cnt) w[u][q >> 2] |= (uint32_t)p[q] << (8 * (q & 3));
          }
          sb[u] = scales[src * nb + quotient(c[u], dv.block, dv.block_inv)];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + 256 * u >= items) break;
      float y[E];
      const float s = scale_value(sb[u]);
#pragma unroll
      for (int q = 0; q < E; q += 4) {
        float z[4];
        values4<I8>(w[u][q >> 2], s, z);
#pragma unroll
        for (int e = 0; e < 4; ++e) y[q + e] = z[e];
      }
      const int64_t at = (row0 + r[u]) * ldo + c[u];
      const int cnt = d - c[u];
      if constexpr (OT == 0) {
        store_out(static_cast<float*>(out) + at, f32x4{y[0], y[1], y[2], y[3]}, cnt);
      } else {
        store_out(static_cast<uint16_t*>(out) + at,
                  u32x4{pack2<OT>(y[0], y[1]), pack2<OT>(y[2], y[3]), pack2<OT>(y[4], y[5]),
                        pack2<OT>(y[6], y[7])}, cnt);
      }
    }
  }
}

// go(first workgroup, workgroups) for each launch that `wgs` workgroups take.
template <typename GO>
hipError_t in_launches(int64_t wgs, GO go) {
  for (int64_t wg0 = 0; wg0 < wgs; wg0 += kMaxGroups) {
    go(wg0, (unsigned)(wgs - wg0 < kMaxGroups ? wgs - wg0 : kMaxGroups));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT, bool I8, int G, int U>
hipError_t encode_rows_u(const EncodeRows& a, hipStream_t st) {
  const int64_t nb = (a.d + a.block - 1) / a.block;
  constexpr int64_t per = 256 / G * U;
  const int64_t wgs = (a.n * nb + per - 1) / per;
  const RowsIn in{a.X, a.rs, a.hs, a.width};
  const uint32_t inv = inverse(nb, nb + per);
  return in_launches(wgs, [&](int64_t wg0, unsigned grid) {
#define EMK_GO(S)                                                                                 \
  encode_rows_kernel<DT, I8, G, S, U><<<grid, 256, 0, st>>>(in, wg0, a.n, a.d, a.block,           \
                                                            (uint32_t)nb, inv, a.slots, a.cap,    \
                                                            a.codes, a.ldc, a.scales, a.lds)
    if (!a.slots)
      EMK_GO(0);
    else if (a.slot_bytes == 8)
      EMK_GO(8);
    else
      EMK_GO(4);
#undef EMK_GO
  });
}

template <int DT, bool I8, int G>
hipError_t encode_rows_g(const EncodeRows& a, hipStream_t st) {
  const int64_t groups = a.n * ((a.d + a.block - 1) / a.block);
  if (groups * G >= 4 * 256 * 1024) return encode_rows_u<DT, I8, G, 2>(a, st);
  return encode_rows_u<DT, I8, G, 1>(a, st);
}

template <int DT, bool I8>
hipError_t encode_rows_t(const EncodeRows& a, hipStream_t st) {
  if (a.block <= 16) return encode_rows_g<DT, I8, 2>(a, st);
  if (a.block <= 32) return encode_rows_g<DT, I8, 4>(a, st);
  if (a.block <= 64) return encode_rows_g<DT, I8, 8>(a, st);
  if (a.block <= 128) return encode_rows_g<DT, I8, 16>(a, st);
  return encode_rows_g<DT, I8, 32>(a, st);
}

template <int DT>
hipError_t encode_tile_t(const EncodeTiles& a, hipStream_t st) {
  const int64_t gx = (a.d + kT - 1) / kT, gy = (a.n + kT - 1) / kT;
  // rows in launches of at most 65535 tiles (the grid's y limit)
  for (int64_t y0 = 0; y0 < gy; y0 += 65535) {
    const unsigned ny = (unsigned)(gy - y0 < 65535 ? gy - y0 : 65535);
    const hipError_t e = in_launches(gx, [&](int64_t x0, unsigned nx) {
      const dim3 grid(nx, ny), wg(Patch<DT>::kThreads);
      const int64_t r = y0 * kT, c = x0 * kT, size = DT == 0 ? 4 : 2;
      const void* X = static_cast<const char*>(a.X) + (r * a.ldx + c) * size;
      uint8_t* codes = a.codes ? a.codes + r * a.ldc + c : nullptr;
      uint8_t* scales = a.scales ? a.scales + (a.tiles ? y0 : r) * a.lds + x0 : nullptr;
      uint8_t* ct = a.codes_t ? a.codes_t + c * a.ldct + r : nullptr;
      uint8_t* stt = a.scales_t ? a.scales_t + (a.tiles ? x0 : c) * a.ldst + y0 : nullptr;
      const int d = a.d - (int)c;
      if (a.tiles)
        encode_tile_kernel<DT, true><<<grid, wg, 0, st>>>(X, a.ldx, a.n - r, d, codes, a.ldc, scales,
                                                          a.lds, ct, a.ldct, stt, a.ldst);
      else
        encode_tile_kernel<DT, false><<<grid, wg, 0, st>>>(X, a.ldx, a.n - r, d, codes, a.ldc,
                                                           scales, a.lds, ct, a.ldct, stt, a.ldst);
    });
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int OT, bool I8>
hipError_t decode_rows_t(const DecodeRows& a, hipStream_t st) {
  constexpr int E = OT == 0 ? 4 : 8;
  const int nb = (a.d + a.block - 1) / a.block;
  const uint32_t per = (uint32_t)((a.d + E - 1) / E);
  // rows per workgroup: about 4096 pieces, fewer where that leaves CUs idle
  int64_t R = 4096 / per;
  if (R > a.n / 2048) R = a.n / 2048;
  R = R < 1 ? 1 : R > kReadRows ? kReadRows : R;
  const Divisors dv{per, inverse(per, (uint64_t)R * per), (uint32_t)a.block,
                    inverse(a.block, a.d)};
  const RowsFrom f{a.slots, a.slot_bytes, a.table, a.table_ld, a.table_pages, a.starts, a.seqs,
                   a.page};
  return in_launches((a.n + R - 1) / R, [&](int64_t wg0, unsigned grid) {
    if (a.slots)
      decode_rows_kernel<OT, I8, false><<<grid, 256, 0, st>>>(a.codes, a.scales, a.cap, a.d, nb, f,
                                                              wg0, a.n, (int)R, dv, a.out, a.ldo);
    else
      decode_rows_kernel<OT, I8, true><<<grid, 256, 0, st>>>(a.codes, a.scales, a.cap, a.d, nb, f,
                                                             wg0, a.n, (int)R, dv, a.out, a.ldo);
  });
}

}  // namespace

hipError_t launch_encode_rows(const EncodeRows& a, hipStream_t st) {
  if (a.n <= 0) return hipSuccess;
#define EMK_DT(DT) return a.i8 ? encode_rows_t<DT, true>(a, st) : encode_rows_t<DT, false>(a, st)
  switch (a.dt) {
    case 0: EMK_DT(0);
    case 1: EMK_DT(1);
    case 4: EMK_DT(4);
  }
#undef EMK_DT
  return hipErrorInvalidValue;
}

hipError_t launch_encode_tiles(const EncodeTiles& a, hipStream_t st) {
  if (a.n <= 0) return hipSuccess;
  switch (a.dt) {
    case 0: return encode_tile_t<0>(a, st);
    case 1: return encode_tile_t<1>(a, st);
    case 4: return encode_tile_t<4>(a, st);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_decode_rows(const DecodeRows& a, hipStream_t st) {
  if (a.n <= 0) return hipSuccess;
#define EMK_OT(OT) return a.i8 ? decode_rows_t<OT, true>(a, st) : decode_rows_t<OT, false>(a, st)
  switch (a.ot) {
    case 0: EMK_OT(0);
    case 1: EMK_OT(1);
    case 4: EMK_OT(4);
  }
#undef EMK_OT
  return hipErrorInvalidValue;
}

}  // namespace emk
