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
// at large sizes and by the launch at small ones.
#include "block.hpp"
#include "kernels.hpp"

namespace emk {

namespace {

// Store up to eight code bytes; wide when `vec` (8-byte aligned and whole).
__device__ __forceinline__ void store_codes(uint8_t* p, u32x2 w, int cnt, bool vec) {
  if (vec && cnt >= 8) {
    *reinterpret_cast<u32x2*>(p) = w;
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
// ---------------------------------------------------------------------------
struct RowsIn {
  const void* X;
  int64_t rs, hs;
  int width;
};

template <int DT, bool I8, int G, bool VEC, int SLOTS>  // SLOTS 0 none, 4 int32, 8 int64
__global__ __launch_bounds__(256) void encode_rows_kernel(RowsIn in, int64_t n, int d, int block,
                                                          int nb, const void* __restrict__ slots,
                                                          int64_t cap,
                                                          uint8_t* __restrict__ codes,
                                                          int64_t ldc,
                                                          uint8_t* __restrict__ scales,
                                                          int64_t lds, bool vec_out) {
  const int64_t item = ((int64_t)blockIdx.x * 256 + threadIdx.x) / G;
  if (item >= n * nb) return;  // whole groups leave together
  const int64_t row = item / nb;
  const int b = (int)(item - row * nb);
  const int sub = threadIdx.x & (G - 1);
  int64_t to = row;
  if constexpr (SLOTS != 0) {
    to = SLOTS == 8 ? static_cast<const int64_t*>(slots)[row]
                    : (int64_t) static_cast<const int32_t*>(slots)[row];
    if (to < 0 || to >= cap) return;
  }
  const int c0 = b * block + 8 * sub;  // first column of the lane
  const int end = min(d, (b + 1) * block);
  const int cnt = 8 * sub < block ? min(8, end - c0) : 0;
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  if (cnt > 0) {
    const int h = c0 / in.width;
    const int64_t at = row * in.rs + h * in.hs + (c0 - h * in.width);
    if (VEC && cnt == 8)
      load8<DT, true>(in.X, at, 8, v);
    else
      load8<DT, false>(in.X, at, cnt, v);
  }
  uint32_t m = group_max<G>(amax8(v));
  const bool odd = m >= kInfBits;
  if (odd) m = group_max<G>(amax8_finite(v));
  const uint32_t byte = scale_byte<I8>(m);
  if (cnt > 0) store_codes(codes + to * ldc + c0, codes8<I8>(v, inv_scale(byte), odd), cnt, vec_out);
  if (sub == 0) scales[to * lds + b] = (uint8_t)byte;
}

// ---------------------------------------------------------------------------
// One 128 x 128 tile per workgroup, read once for both orders: codes of the
// rows and the codes of the columns, transposed. Thread t holds rows
// 8 (t / 16) .. + 8 and columns 8 (t % 16) .. + 8, so a row's maximum is a
// reduction over 16 lanes, a column's one over the thread's rows, four lane
// groups and four waves, and a column's eight codes of a thread are eight
// consecutive bytes of the transposed output. TILES: one scale for the tile,
// and both orders hold the same codes.
// ---------------------------------------------------------------------------
constexpr int kT = 128;
constexpr int kTPitch = kT + 8;  // bytes per transposed row in LDS: 8-byte aligned

template <int DT, bool TILES, bool VEC>
__global__ __launch_bounds__(256) void encode_tile_kernel(
    const void* __restrict__ X, int64_t ldx, int64_t n, int d, uint8_t* __restrict__ codes,
    int64_t ldc, uint8_t* __restrict__ scales, int64_t lds, uint8_t* __restrict__ codes_t,
    int64_t ldct, uint8_t* __restrict__ scales_t, int64_t ldst, bool vec_out, bool vec_t) {
  __shared__ __attribute__((aligned(16))) uint8_t tr[kT * kTPitch];
  __shared__ uint32_t cmax[4][kT];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int rg = t >> 4, cg = t & 15;
  const int64_t r0 = (int64_t)blockIdx.y * kT;
  const int c0 = blockIdx.x * kT;
  const int rows = (int)min((int64_t)kT, n - r0), cols = min(kT, d - c0);
  const int ccnt = min(8, cols - 8 * cg);  // columns of this thread (may be <= 0)

  float v[8][8];
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int r = 8 * rg + p;
    if (r < rows && ccnt > 0) {
      const int64_t at = (r0 + r) * ldx + c0 + 8 * cg;
      if (VEC && ccnt == 8)
        load8<DT, true>(X, at, 8, v[p]);
      else
        load8<DT, false>(X, at, ccnt, v[p]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[p][i] = 0.0f;
    }
  }

  if constexpr (TILES) {
    uint32_t m = 0;
#pragma unroll
    for (int p = 0; p < 8; ++p) m = max(m, amax8(v[p]));
    m = group_max<64>(m);
    if (lane == 0) cmax[0][wave] = m;
    __syncthreads();
    m = max(max(cmax[0][0], cmax[0][1]), max(cmax[0][2], cmax[0][3]));
    const bool odd = m >= kInfBits;
    if (odd) {  // the same answer in every thread of the workgroup
      m = 0;
#pragma unroll
      for (int p = 0; p < 8; ++p) m = max(m, amax8_finite(v[p]));
      m = group_max<64>(m);
      if (lane == 0) cmax[1][wave] = m;
      __syncthreads();
      m = max(max(cmax[1][0], cmax[1][1]), max(cmax[1][2], cmax[1][3]));
    }
    const uint32_t byte = scale_byte<false>(m);
    const float inv = inv_scale(byte);
    uint32_t w[8][2];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const u32x2 q = codes8<false>(v[p], inv, odd);
      w[p][0] = q[0];
      w[p][1] = q[1];
      if (codes && 8 * rg + p < rows && ccnt > 0)
        store_codes(codes + (r0 + 8 * rg + p) * ldc + c0 + 8 * cg, q, ccnt, vec_out);
    }
    if (t == 0) {
      if (codes) scales[(int64_t)blockIdx.y * lds + blockIdx.x] = (uint8_t)byte;
      if (codes_t) scales_t[(int64_t)blockIdx.x * ldst + blockIdx.y] = (uint8_t)byte;
    }
    if (!codes_t) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      u32x2 q = {0u, 0u};
#pragma unroll
      for (int p = 0; p < 8; ++p)
        q[p >> 2] |= ((w[p][i >> 2] >> (8 * (i & 3))) & 0xFFu) << (8 * (p & 3));
      *reinterpret_cast<u32x2*>(&tr[(8 * cg + i) * kTPitch + 8 * rg]) = q;
    }
  } else {
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      if (!codes) break;
      uint32_t m = group_max<16>(amax8(v[p]));
      const bool odd = m >= kInfBits;
      if (odd) m = group_max<16>(amax8_finite(v[p]));
      const uint32_t byte = scale_byte<false>(m);
      const int r = 8 * rg + p;
      if (r < rows) {
        if (ccnt > 0)
          store_codes(codes + (r0 + r) * ldc + c0 + 8 * cg,
                      codes8<false>(v[p], inv_scale(byte), odd), ccnt, vec_out);
        if (cg == 0) scales[(r0 + r) * lds + blockIdx.x] = (uint8_t)byte;
      }
    }
    // columns: the thread's rows, the four row groups of the wave, the waves.
    // Column maxima in LDS carry the non-finite mark; a column that has one
    // takes its finite maximum in a second round.
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t m = 0;
#pragma unroll
      for (int p = 0; p < 8; ++p) m = max(m, abs_bits(v[p][i]));
      m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
      m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
      if (lane < 16) cmax[wave][8 * cg + i] = m;
    }
    __syncthreads();
    uint32_t cm[8];
    bool any = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = 8 * cg + i;
      cm[i] = max(max(cmax[0][c], cmax[1][c]), max(cmax[2][c], cmax[3][c]));
      any |= cm[i] >= kInfBits;
    }
    uint32_t fm[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) fm[i] = cm[i];
    if (__syncthreads_or(any)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t m = 0;
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          const uint32_t b = abs_bits(v[p][i]);
          m = max(m, b < kInfBits ? b : 0u);
        }
        m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
        m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
        if (lane < 16) cmax[wave][8 * cg + i] = m;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = 8 * cg + i;
        fm[i] = max(max(cmax[0][c], cmax[1][c]), max(cmax[2][c], cmax[3][c]));
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t byte = scale_byte<false>(fm[i]);
      float y[8];
#pragma unroll
      for (int p = 0; p < 8; ++p) y[p] = v[p][i];
      *reinterpret_cast<u32x2*>(&tr[(8 * cg + i) * kTPitch + 8 * rg]) =
          codes8<false>(y, inv_scale(byte), cm[i] >= kInfBits);
      if (rg == 0 && i < ccnt) scales_t[(int64_t)(c0 + 8 * cg + i) * ldst + blockIdx.y] = (uint8_t)byte;
    }
  }
  __syncthreads();
  // transposed rows: 8 lanes write the 128 bytes of one column
#pragma unroll
  for (int q = 0; q < kT * 8 / 256; ++q) {
    const int f = q * 256 + t;
    const int c = f >> 3, ch = f & 7;
    if (c >= cols) break;
    const u32x2 lo = *reinterpret_cast<const u32x2*>(&tr[c * kTPitch + 16 * ch]);
    const u32x2 hi = *reinterpret_cast<const u32x2*>(&tr[c * kTPitch + 16 * ch + 8]);
    uint8_t* p = codes_t + (int64_t)(c0 + c) * ldct + r0 + 16 * ch;
    const int cnt = rows - 16 * ch;
    if (vec_t && cnt >= 16) {
      *reinterpret_cast<u32x4*>(p) = u32x4{lo[0], lo[1], hi[0], hi[1]};
    } else {
      store_codes(p, lo, cnt, false);
      store_codes(p + 8, hi, cnt - 8, false);
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
// (16-bit out). VEC: pieces are whole and aligned (d a multiple of E, no block
// border inside a piece). Rows outside the store are zeros. The quotients by
// the pieces per row and by the block are products by `inv` = 2^32 / divisor,
// rounded up (exact while dividend x divisor < 2^32, which the host checks).
constexpr int kReadRows = 64;  // R at most

__device__ __forceinline__ uint32_t quotient(uint32_t a, uint32_t div, uint32_t inv) {
  return inv ? __umulhi(a, inv) : a / div;
}

struct Divisors {
  uint32_t per, per_inv, block, block_inv;
};

template <int OT, bool I8, bool VEC, bool PAGES>
__global__ __launch_bounds__(256) void decode_rows_kernel(const uint8_t* __restrict__ codes,
                                                          const uint8_t* __restrict__ scales,
                                                          int64_t cap, int d, int nb,
                                                          RowsFrom from, int64_t n, int R,
                                                          Divisors dv, void* __restrict__ out,
                                                          int64_t ldo) {
  constexpr int E = OT == 0 ? 4 : 8;
  constexpr int U = VEC ? 4 : 1;  // pieces in flight per thread
  __shared__ int64_t place[kReadRows];
  const int64_t row0 = (int64_t)blockIdx.x * R;
  const int rows = (int)min((int64_t)R, n - row0);
  if ((int)threadIdx.x < rows)
    place[threadIdx.x] = source_row<PAGES>(from, row0 + threadIdx.x, cap);
  __syncthreads();
  const uint32_t items = (uint32_t)rows * dv.per;
  for (uint32_t i0 = threadIdx.x; i0 < items; i0 += 256 * U) {
    u32x2 w[U];
    uint32_t sb[U];
    int r[U], c[U];
    bool in[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t i = i0 + 256 * u;
      w[u] = u32x2{0u, 0u};
      sb[u] = 0;
      in[u] = false;
      if (i < items) {
        r[u] = (int)quotient(i, dv.per, dv.per_inv);
        c[u] = (int)(i - r[u] * dv.per) * E;
        const int64_t src = place[r[u]];
        in[u] = src >= 0;
        if (VEC && in[u]) {
          const uint8_t* p = codes + src * d + c[u];
          w[u][0] = *reinterpret_cast<const uint32_t*>(p);
          if constexpr (E == 8) w[u][1] = *reinterpret_cast<const uint32_t*>(p + 4);
          sb[u] = scales[src * nb + quotient(c[u], dv.block, dv.block_inv)];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + 256 * u >= items) break;
      float y[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) y[q] = 0.0f;
      const int cnt = min(E, d - c[u]);
      if constexpr (VEC) {
        if (in[u]) {
          const float s = scale_value(sb[u]);
          float z[4];
#pragma unroll
          for (int q = 0; q < E; q += 4) {
            values4<I8>(w[u][q >> 2], s, z);
#pragma unroll
            for (int e = 0; e < 4; ++e) y[q + e] = z[e];
          }
        }
      } else if (in[u]) {
        const int64_t src = place[r[u]];
#pragma unroll
        for (int q = 0; q < E; ++q)
          if (q < cnt) {
            float z[4];
            values4<I8>(codes[src * d + c[u] + q],
                        scale_value(scales[src * nb + quotient(c[u] + q, dv.block, dv.block_inv)]),
                        z);
            y[q] = z[0];
          }
      }
      const int64_t at = (row0 + r[u]) * ldo + c[u];
      if constexpr (OT == 0) {
        float* o = static_cast<float*>(out) + at;
        if constexpr (VEC) {
          __builtin_nontemporal_store(f32x4{y[0], y[1], y[2], y[3]}, reinterpret_cast<f32x4*>(o));
        } else {
#pragma unroll
          for (int q = 0; q < E; ++q)
            if (q < cnt) o[q] = y[q];
        }
      } else {
        uint16_t* o = static_cast<uint16_t*>(out) + at;
        if constexpr (VEC) {
          __builtin_nontemporal_store(u32x4{pack2<OT>(y[0], y[1]), pack2<OT>(y[2], y[3]),
                                            pack2<OT>(y[4], y[5]), pack2<OT>(y[6], y[7])},
                                      reinterpret_cast<u32x4*>(o));
        } else {
#pragma unroll
          for (int q = 0; q < E; ++q)
            if (q < cnt) o[q] = (uint16_t)pack2<OT>(y[q], 0.0f);
        }
      }
    }
  }
}

template <int DT, bool I8, int G>
hipError_t encode_rows_g(const EncodeRows& a, bool vec, bool vec_out, hipStream_t st) {
  const int nb = (a.d + a.block - 1) / a.block;
  const int64_t groups = a.n * nb;
  const int64_t blocks = (groups * G + 255) / 256;
  if (blocks > INT32_MAX) return hipErrorInvalidValue;
  const dim3 grid((unsigned)blocks), wg(256);
  const RowsIn in{a.X, a.rs, a.hs, a.width};
#define EMK_GO(V, S)                                                                          \
  encode_rows_kernel<DT, I8, G, V, S><<<grid, wg, 0, st>>>(in, a.n, a.d, a.block, nb, a.slots, \
                                                           a.cap, a.codes, a.ldc, a.scales,   \
                                                           a.lds, vec_out)
  if (!a.slots) {
    if (vec) EMK_GO(true, 0);
    else EMK_GO(false, 0);
  } else if (a.slot_bytes == 8) {
    if (vec) EMK_GO(true, 8);
    else EMK_GO(false, 8);
  } else {
    if (vec) EMK_GO(true, 4);
    else EMK_GO(false, 4);
  }
#undef EMK_GO
  return hipGetLastError();
}

template <int DT, bool I8>
hipError_t encode_rows_t(const EncodeRows& a, hipStream_t st) {
  const int64_t unit = DT == 0 ? 4 : 8;  // elements of 16 bytes
  const bool vec = (uintptr_t)a.X % 16 == 0 && a.rs % unit == 0 &&
                   (a.width == a.d || (a.hs % unit == 0 && a.width % 8 == 0));
  const bool vec_out = (uintptr_t)a.codes % 8 == 0 && a.ldc % 8 == 0;
  if (a.block <= 16) return encode_rows_g<DT, I8, 2>(a, vec, vec_out, st);
  if (a.block <= 32) return encode_rows_g<DT, I8, 4>(a, vec, vec_out, st);
  if (a.block <= 64) return encode_rows_g<DT, I8, 8>(a, vec, vec_out, st);
  if (a.block <= 128) return encode_rows_g<DT, I8, 16>(a, vec, vec_out, st);
  return encode_rows_g<DT, I8, 32>(a, vec, vec_out, st);
}

template <int DT>
hipError_t encode_tile_t(const EncodeTiles& a, hipStream_t st) {
  const int64_t gx = (a.d + kT - 1) / kT, gy = (a.n + kT - 1) / kT;
  const int64_t unit = DT == 0 ? 4 : 8;
  const bool vec = (uintptr_t)a.X % 16 == 0 && a.ldx % unit == 0;
  const bool vec_out = (uintptr_t)a.codes % 8 == 0 && a.ldc % 8 == 0;
  const bool vec_t = (uintptr_t)a.codes_t % 16 == 0 && a.ldct % 16 == 0;
  // rows in launches of at most 65535 tiles (the grid's y limit)
  for (int64_t y0 = 0; y0 < gy; y0 += 65535) {
    const int64_t ny = gy - y0 < 65535 ? gy - y0 : 65535;
    const dim3 grid((unsigned)gx, (unsigned)ny), wg(256);
    const int64_t r = y0 * kT, size = DT == 0 ? 4 : 2;
    const void* X = static_cast<const char*>(a.X) + r * a.ldx * size;
    uint8_t* codes = a.codes ? a.codes + r * a.ldc : nullptr;
    uint8_t* scales = a.scales ? a.scales + (a.tiles ? y0 : r) * a.lds : nullptr;
    uint8_t* ct = a.codes_t ? a.codes_t + r : nullptr;
    uint8_t* stt = a.scales_t ? a.scales_t + y0 : nullptr;
#define EMK_GO(T, V)                                                                         \
  encode_tile_kernel<DT, T, V><<<grid, wg, 0, st>>>(X, a.ldx, a.n - r, a.d, codes, a.ldc,     \
                                                    scales, a.lds, ct, a.ldct, stt, a.ldst,  \
                                                    vec_out, vec_t)
    if (a.tiles) {
      if (vec) EMK_GO(true, true);
      else EMK_GO(true, false);
    } else {
      if (vec) EMK_GO(false, true);
      else EMK_GO(false, false);
    }
#undef EMK_GO
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

uint32_t inverse(uint64_t div, uint64_t most) {  // 0: divide
  return div > 1 && most * div < (1ull << 32) ? (uint32_t)((1ull << 32) / div + 1) : 0;
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
  const int64_t blocks = (a.n + R - 1) / R;
  if (blocks > INT32_MAX) return hipErrorInvalidValue;
  const Divisors dv{per, inverse(per, (uint64_t)R * per), (uint32_t)a.block,
                    inverse(a.block, a.d)};
  const bool vec = a.d % E == 0 && (uintptr_t)a.codes % 4 == 0 && (uintptr_t)a.out % 16 == 0 &&
                   a.ldo % E == 0;
  const dim3 grid((unsigned)blocks), wg(256);
  const RowsFrom f{a.slots, a.slot_bytes, a.table, a.table_ld, a.table_pages, a.starts, a.seqs,
                   a.page};
#define EMK_GO(V, P)                                                                       \
  decode_rows_kernel<OT, I8, V, P><<<grid, wg, 0, st>>>(a.codes, a.scales, a.cap, a.d, nb, f, \
                                                        a.n, (int)R, dv, a.out, a.ldo)
  if (a.slots) {
    if (vec) EMK_GO(true, false);
    else EMK_GO(false, false);
  } else {
    if (vec) EMK_GO(true, true);
    else EMK_GO(false, true);
  }
#undef EMK_GO
  return hipGetLastError();
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
