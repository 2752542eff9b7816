// Attention of one new token per sequence over a paged store of 8-bit codes.
//
// For query head h and the keys k_p, values v_p of its key-value head at the places
// p of the sequence: s_p = scale q.k_p, out = sum exp(s_p - m) v_p / sum exp(s_p - m),
// m the largest. One pass over the codes with a running maximum and sum; the
// sequence is cut into parts that are joined afterwards (m = max m_i, parts weighed
// by exp(m_i - m)), as a few sequences would leave most of the card idle.
//
// Bound by HBM: the codes are read once. So that decoding them and the products
// take less than the reads, both products are on the matrix unit in bf16, where a
// code times its scale is exact, and nothing passes through LDS on the way: a wave
// takes 32 places; S^T = K q^T leaves lane (h, g) the scores of places 4 g + i of
// head h, which is what the product with the values reads as its operand if its
// places are counted in that order. Queries are sums of one, two and three bf16 terms for bf16,
// fp16 and fp32 (8, 16 and 24 bits); softmax weights of two (three for fp32), as one would
// round them to 8 bits where values cancel (products more on a matrix unit that is 8% busy:
// 1% of the time).
//
// Measured, 32 query and 8 key-value heads of 128, E4M3, bf16: one sequence of 131072 places
// 51 us and 8 for the join (5.3 TB/s; a large copy 5.0), 64 sequences of up to 8192 124 and
// 6 (4.4 TB/s), 16 of up to 4000 with weights 24 and 5. With each load in a branch of its
// own, and none a round ahead, the first took 127 us.
#include <type_traits>

#include "block.hpp"
#include "kernels.hpp"

namespace emk {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kPlaces = 32;      // of a wave at a time
constexpr int kWaves = 4;
constexpr int kHeads = 16;       // query heads of a workgroup (of one key-value head)
constexpr int kMaxPart = 2048;   // places of a workgroup at most
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float xor_max(float v) {
  uint32_t b = __float_as_uint(v);
  auto mx = [](uint32_t x, uint32_t y) {
    return __float_as_uint(fmaxf(__uint_as_float(x), __uint_as_float(y)));
  };
  b = max_xor16(b, mx);
  return __uint_as_float(max_xor32(b, mx));
}

__device__ __forceinline__ float xor_sum(float v) {
  uint32_t b = __float_as_uint(v);
  auto add = [](uint32_t x, uint32_t y) {
    return __float_as_uint(__uint_as_float(x) + __uint_as_float(y));
  };
  b = max_xor16(b, add);
  return __uint_as_float(max_xor32(b, add));
}

// Four codes as bf16 values. int8: a byte with its sign bit turned over, u = code + 128, in
// the last bits of 2^23 is 2^23 + u, from which 2^23 + 128 is taken: two instructions at
// full rate, where the conversion of an integer is slower (64 sequences of up to 8192 249 us with it, 152 without).
template <bool I8>
__device__ __forceinline__ u32x2 values_of(uint32_t w, float s) {
  if constexpr (I8) {
    const uint32_t u = w ^ 0x80808080u;
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      y[i] = (__uint_as_float(__builtin_amdgcn_perm(0x4B000000u, u, 0x070C0C00u | i)) - 8388736.0f) * s;
    return u32x2{pack2<1>(y[0], y[1]), pack2<1>(y[2], y[3])};
  } else {
    return u32x2{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, true))};
  }
}

// x as NT bf16 terms whose sum is x to 8 NT bits.
template <int NT>
__device__ __forceinline__ void terms_of(const float (&x)[8], bf16x8 (&t)[NT]) {
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack2<1>(r[2 * i], r[2 * i + 1]);
    t[n] = __builtin_bit_cast(bf16x8, w);
    if (n + 1 < NT) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float hi = __uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
        r[i] = abs_bits(hi) < kInfBits ? r[i] - hi : 0.0f;  // no inf - inf
      }
    }
  }
}

struct Split {
  CacheAttend a;
  int64_t wg0;
  int group;        // query heads per key-value head
  int tiles;        // of kHeads query heads
  int part;         // places of a workgroup, a multiple of kWaves * kPlaces
  int parts;        // of a sequence
  int nb;           // scales of a row
  float* sums;      // seqs x hq x parts x width: unnormalised results (parts > 1)
  f32x2* tops;      // seqs x hq x parts: (largest, sum), scores in units of log 2
  float* scores;    // seqs x hq x (parts * part) (weights asked for)
};

__device__ __forceinline__ int length_of(const CacheAttend& a, int seq) {
  const int64_t cap = (int64_t)a.table_pages * a.page, len = a.lengths[seq];
  return (int)(len < 0 ? 0 : len > cap ? cap : len);
}

template <int DT>
__device__ __forceinline__ void store_number(void* out, int64_t at, float v) {
  if constexpr (DT == 0)
    static_cast<float*>(out)[at] = v;
  else
    static_cast<uint16_t*>(out)[at] = to_half_rne(v, DT == 4);
}

// What a wave has in flight of 32 places: their codes and, where a head has more than
// one scale, the scales' bytes. Lane l = 16 g + n. Keys: of place 16 u + n the 16 codes
// from 64 j + 16 g on. Values: of places 4 g + i and 16 + 4 g + i the VD codes from n VD on.
template <int W, bool ONE>
struct Places {
  static constexpr int KJ = W / 64, VD = W / 16;
  u32x4 k[2][KJ];
  u32x2 v[8];
  uint32_t ks[ONE ? 1 : 2][KJ], vs[ONE ? 1 : 8];
};

// W: width rounded up to 64 or 128. ONE: a head lies in one block, so that its scale is a
// factor of the score and of the softmax weight (and the store has under 2^32 rows); else
// every 16 codes have a scale of their own. Three workgroups on a CU (168 registers) where that
// holds what is in flight, else two, as spilling in the loop costs more than the third gives: heads of
// 128, 64 sequences of up to 8192, two against three: bf16 queries over int8 142 us against 162,
// fp16 over E4M3 133 / 159, over int8 145 / 217, fp32 134 / 205 and 150 / 297. bf16 over E4M3 fits (162).
template <int DT, bool I8, int W, bool SCORES, bool ONE>
__global__ __launch_bounds__(256, ONE && (W == 64 || (DT == 1 && !I8)) ? 3 : 2) void split_kernel(Split s) {
  // bf16 terms of a query's values and of a softmax weight
  constexpr int NT = DT == 1 ? 1 : DT == 4 ? 2 : 3, NP = DT == 0 ? 3 : 2;
  constexpr int KJ = W / 64, VD = W / 16;
  typedef std::conditional_t<ONE, uint32_t, int64_t> At;
  const CacheAttend& a = s.a;
  // per place: its row of the store (general: -1 outside the store), and for ONE both scales, the keys' times scale log2 e; the values' is 0 where there is no place.
  // Afterwards the waves' results.
  constexpr int kRoom = kMaxPart * (ONE ? 12 : 8), kJoin = kWaves * kHeads * (W + 4) * 4;
  __shared__ __align__(16) uint8_t room[kRoom > kJoin ? kRoom : kJoin];
  At* const rows = reinterpret_cast<At*>(room);
  float* const k_scale = reinterpret_cast<float*>(room + kMaxPart * 4);
  float* const v_scale = reinterpret_cast<float*>(room + kMaxPart * 8);
  float(*const join)[kHeads][W + 4] = reinterpret_cast<float(*)[kHeads][W + 4]>(room);
  __shared__ float top[kWaves][kHeads], sum[kWaves][kHeads];
  __shared__ int holes;
  // eight parts beside each other, one per XCD, whose heads follow each other there:
  // the heads of a row share its lines in that XCD's L2
  const int hh = a.hk * s.tiles;
  const int64_t b = s.wg0 + blockIdx.x;
  const int64_t unit = b / (8 * hh) * 8 + b % 8;
  if (unit >= (int64_t)a.seqs * s.parts) return;
  const int head = (int)(b / 8 % hh), kvh = head / s.tiles, q0 = head % s.tiles * kHeads;
  const int seq = (int)(unit % a.seqs), part = (int)(unit / a.seqs);
  const int len = length_of(a, seq), p0 = part * s.part;
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int heads = min(s.group - q0, kHeads);
  const int hq0 = kvh * s.group + q0;
  if (p0 >= len) {
    if (s.parts == 1)
      for (int i = threadIdx.x; i < heads * a.width; i += 256)
        store_number<DT>(a.out, ((int64_t)seq * a.hq + hq0) * a.width + i, 0.0f);
    return;
  }
  const int cnt = min(s.part, len - p0);
  const uint32_t d = (uint32_t)a.hk * a.width;
  const int col = kvh * a.width;
  const float c2 = a.scale * kLog2e;
  if (threadIdx.x == 0) holes = 0;
  __syncthreads();
  // behind the last place the first one's row again (never a row that the sequence does
  // not have)
  const int whole = (cnt + kPlaces - 1) / kPlaces * kPlaces;
  // four of a thread at a time: each is a chain of reads (table, scales)
  constexpr int kDeep = 4;
  for (int i0 = threadIdx.x; i0 < whole; i0 += 256 * kDeep) {
    int64_t page[kDeep];
    int in_page[kDeep];
#pragma unroll
    for (int e = 0; e < kDeep; ++e) {
      const int i = i0 + 256 * e, p = p0 + (i < cnt ? i : 0), pi = p / a.page;
      page[e] = a.table[seq * a.table_ld + pi];
      in_page[e] = p - pi * a.page;
    }
    uint32_t ks[kDeep], vs[kDeep];
    int64_t row[kDeep];
#pragma unroll
    for (int e = 0; e < kDeep; ++e) {
      row[e] = page[e] * a.page + in_page[e];
      if (page[e] < 0 || row[e] >= a.rows) row[e] = -1;
      if constexpr (ONE) {
        const int64_t at = max(row[e], (int64_t)0) * s.nb + col / a.block;
        ks[e] = a.k.scales[at];
        vs[e] = a.v.scales[at];
      }
    }
#pragma unroll
    for (int e = 0; e < kDeep; ++e) {
      const int i = i0 + 256 * e;
      if (i >= whole) break;
      if (row[e] < 0) holes = 1;
      if constexpr (ONE) {
        rows[i] = (uint32_t)max(row[e], (int64_t)0);
        k_scale[i] = scale_value(ks[e]) * c2;
        v_scale[i] = row[e] >= 0 && i < cnt ? scale_value(vs[e]) : 0.0f;
      } else {
        rows[i] = row[e];
      }
    }
  }
  bf16x8 qf[2 * KJ][NT];
#pragma unroll
  for (int m = 0; m < 2 * KJ; ++m) {
    const int c = (m >> 1) * 64 + g * 16 + (m & 1) * 8;
    float x[8] = {};
    if (n < heads && c < a.width)
      load8<DT>(a.q, seq * a.q_rs + (hq0 + n) * a.q_hs + c, 8, x);
    terms_of<NT>(x, qf[m]);
  }
  __syncthreads();
  const bool gaps = holes != 0;
  // Lanes past the width read codes of the same row again: the query has zeros there, and
  // their values go nowhere.
  uint32_t kc[KJ], kb[KJ];
#pragma unroll
  for (int j = 0; j < KJ; ++j) {
    kc[j] = col + min(j * 64 + g * 16, a.width - 16);
    kb[j] = kc[j] / a.block;
  }
  const uint32_t vc = col + min(n * VD, a.width - VD), vb = vc / a.block;

  auto fetch = [&](int t, Places<W, ONE>& x) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      At row = rows[t + 16 * u + n];
      if (!ONE) row = max(row, (At)0);
#pragma unroll
      for (int j = 0; j < KJ; ++j) {
        x.k[u][j] = load_any<u32x4>(a.k.codes + (uint64_t)row * d + kc[j]);
        if constexpr (!ONE) x.ks[u][j] = a.k.scales[row * s.nb + kb[j]];
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      At row = rows[t + 16 * (e >> 2) + 4 * g + (e & 3)];
      if (!ONE) row = max(row, (At)0);
      const uint8_t* p = a.v.codes + (uint64_t)row * d + vc;
      if constexpr (VD == 8)
        x.v[e] = load_any<u32x2>(p);
      else
        x.v[e][0] = load_any<uint32_t>(p);
      if constexpr (!ONE) x.vs[e] = a.v.scales[row * s.nb + vb];
    }
  };

  f32x4 acc[VD];
#pragma unroll
  for (int j = 0; j < VD; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  float m = -INFINITY, l = 0.0f;
  auto take = [&](int t, Places<W, ONE>& x) {
    // scores: st[u][i] of place t + 16 u + 4 g + i
    f32x4 st[2], fv[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      st[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < KJ; ++j) {
        const float f = ONE ? 1.0f : scale_value(x.ks[ONE ? 0 : u][j]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const u32x2 lo = values_of<I8>(x.k[u][j][2 * h], f), hi = values_of<I8>(x.k[u][j][2 * h + 1], f);
          const bf16x8 kf = __builtin_bit_cast(bf16x8, u32x4{lo[0], lo[1], hi[0], hi[1]});
#pragma unroll
          for (int e = NT - 1; e >= 0; --e)
            st[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[2 * j + h][e], st[u], 0, 0, 0);
        }
      }
      if constexpr (ONE) {
        st[u] *= *reinterpret_cast<const f32x4*>(&k_scale[t + 16 * u + 4 * g]);
        fv[u] = *reinterpret_cast<const f32x4*>(&v_scale[t + 16 * u + 4 * g]);
      } else {
        st[u] *= c2;
      }
    }
    if (gaps || t + kPlaces > cnt) {
      asm volatile("");  // a branch: most parts are whole
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int p = t + 16 * (e >> 2) + 4 * g + (e & 3);
        bool out;
        if constexpr (ONE)
          out = fv[e >> 2][e & 3] == 0.0f;
        else
          out = p >= cnt || rows[p] < 0;
        if (out) {
          st[e >> 2][e & 3] = -INFINITY;
          if (gaps) {  // some row of the store, which may hold NaN
            x.v[e] = u32x2{0u, 0u};
            if constexpr (!ONE) x.vs[e] = 127;
          }
        }
      }
    }
    float top_now = -INFINITY;
#pragma unroll
    for (int e = 0; e < 8; ++e) top_now = fmaxf(top_now, st[e >> 2][e & 3]);
    if constexpr (SCORES) {
      if (n < heads) {
        const int64_t at = ((int64_t)seq * a.hq + hq0 + n) * s.parts * s.part + p0 + t + 4 * g;
        store_any(s.scores + at, st[0]);
        store_any(s.scores + at + 16, st[1]);
      }
    }
    const float m_new = fmaxf(m, xor_max(top_now));
    const float ref = m_new == -INFINITY ? 0.0f : m_new;
    if (__any(m_new != m)) {
      const float f = __builtin_amdgcn_exp2f(m - ref);
      l *= f;
#pragma unroll
      for (int j = 0; j < VD; ++j) acc[j] *= f;
      m = m_new;
    }
    float p[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      p[e] = __builtin_amdgcn_exp2f(st[e >> 2][e & 3] - ref);
      l += p[e];
      if constexpr (ONE) p[e] *= fv[e >> 2][e & 3];
    }
    bf16x8 pf[NP];
    terms_of<NP>(p, pf);
    u32x4 y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float f = ONE ? 1.0f : scale_value(x.vs[ONE ? 0 : e]);
      const u32x2 lo = values_of<I8>(x.v[e][0], f);
      const u32x2 hi = VD == 8 ? values_of<I8>(x.v[e][1], f) : u32x2{0u, 0u};
      y[e] = u32x4{lo[0], lo[1], hi[0], hi[1]};
    }
#pragma unroll
    for (int j = 0; j < VD; ++j) {
      u32x4 w;  // value j of the eight places
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = __builtin_amdgcn_perm(y[2 * e + 1][j >> 1], y[2 * e][j >> 1],
                                     j & 1 ? 0x07060302u : 0x05040100u);
      const bf16x8 vf = __builtin_bit_cast(bf16x8, w);
#pragma unroll
      for (int e = NP - 1; e >= 0; --e)
        acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pf[e], acc[j], 0, 0, 0);
    }
  };
  // the next places' codes are on their way while these are worked on
  {
    constexpr int kStep = kWaves * kPlaces;
    Places<W, ONE> x, y;
    int t = wave * kPlaces;
    if (t < whole) fetch(t, x);
    while (t < whole) {
      if (t + kStep < whole) fetch(t + kStep, y);
      take(t, x);
      t += kStep;
      if (t >= whole) break;
      if (t + kStep < whole) fetch(t + kStep, x);
      take(t, y);
      t += kStep;
    }
  }
  // the waves' parts joined: acc[j][i] is value VD (4 g + i) + j of head n
  l = xor_sum(l);
  if (g == 0) {
    top[wave][n] = m;
    sum[wave][n] = l;
  }
  __syncthreads();
  float all = -INFINITY;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) all = fmaxf(all, top[w][n]);
  const float f = __builtin_amdgcn_exp2f(m - (all == -INFINITY ? 0.0f : all));
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < VD; j += 4)
      *reinterpret_cast<f32x4*>(&join[wave][n][VD * (4 * g + i) + j]) =
          f32x4{acc[j][i] * f, acc[j + 1][i] * f, acc[j + 2][i] * f, acc[j + 3][i] * f};
  __syncthreads();
  const int h = threadIdx.x >> 4, c0 = (threadIdx.x & 15) * VD;
  if (h >= heads) return;
  float mh = -INFINITY, lh = 0.0f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) mh = fmaxf(mh, top[w][h]);
#pragma unroll
  for (int w = 0; w < kWaves; ++w)
    lh += sum[w][h] * __builtin_amdgcn_exp2f(top[w][h] - (mh == -INFINITY ? 0.0f : mh));
  const int64_t at = (int64_t)seq * a.hq + hq0 + h;
  if ((SCORES || s.parts > 1) && c0 == 0) s.tops[at * s.parts + part] = f32x2{mh, lh};
  if (c0 >= a.width) return;
  const float inv = s.parts > 1 ? 1.0f : lh == 0.0f ? 0.0f : 1.0f / lh;
#pragma unroll
  for (int j = 0; j < VD; ++j) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += join[w][h][c0 + j];
    v = lh == 0.0f ? 0.0f : v * inv;
    if (s.parts > 1)
      s.sums[(at * s.parts + part) * a.width + c0 + j] = v;
    else
      store_number<DT>(a.out, at * a.width + c0 + j, v);
  }
}

__device__ __forceinline__ float guarded(float m) { return m == -INFINITY ? 0.0f : m; }

// Workgroups below seqs * hq: the parts of one head of one sequence joined. The
// others (weights asked for): the attention weights of 256 places, summed over the heads,
// from the scores that split_kernel left.
constexpr int kJoinHeads = 1024;

template <int DT, int LANES>
__global__ __launch_bounds__(256) void join_kernel(Split s, int64_t joins) {
  const CacheAttend& a = s.a;
  __shared__ f32x2 ml[kJoinHeads];
  __shared__ f32x4 acc[4][LANES];
  __shared__ float tmp[8];
  const int64_t b = s.wg0 + blockIdx.x;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  if (b < joins) {
    const int seq = (int)(b / a.hq);
    const int used = (length_of(a, seq) + s.part - 1) / s.part;
    const f32x2* tops = s.tops + b * s.parts;
    float m = -INFINITY;
    for (int i = threadIdx.x; i < used; i += 256) m = fmaxf(m, tops[i][0]);
    m = wave_max(m);
    if (lane == 0) tmp[wave] = m;
    __syncthreads();
    m = guarded(fmaxf(fmaxf(tmp[0], tmp[1]), fmaxf(tmp[2], tmp[3])));
    // LANES lanes of four values each, the others over the parts
    const int c = blockIdx.y * (LANES * 4) + (threadIdx.x % LANES) * 4, i0 = threadIdx.x / LANES;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    float l = 0.0f;
    for (int i = i0; i < used; i += 256 / LANES) {
      const f32x2 t = tops[i];
      if (t[1] == 0.0f) continue;  // a part of gaps
      const float f = __builtin_amdgcn_exp2f(t[0] - m);
      l += t[1] * f;
      if (c < a.width) v += *reinterpret_cast<const f32x4*>(s.sums + (b * s.parts + i) * a.width + c) * f;
    }
#pragma unroll
    for (int off = LANES; off < 64; off <<= 1) {
      l += __shfl_xor(l, off, kWave);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += __shfl_xor(v[i], off, kWave);
    }
    if (lane < LANES) acc[wave][lane] = v;
    if (lane == 0) tmp[4 + wave] = l;
    __syncthreads();
    if (threadIdx.x >= LANES || c >= a.width) return;
    const float sum = tmp[4] + tmp[5] + tmp[6] + tmp[7];
    v = acc[0][lane] + acc[1][lane] + acc[2][lane] + acc[3][lane];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      store_number<DT>(a.out, b * a.width + c + i, sum == 0.0f ? 0.0f : v[i] / sum);
    return;
  }
  if (blockIdx.y) return;
  const int64_t unit = b - joins;
  const int seq = (int)(unit % a.seqs), p0 = (int)(unit / a.seqs) * 256;
  const int len = length_of(a, seq);
  if (p0 >= len) return;
  const int used = (len + s.part - 1) / s.part;
  // eight lanes a head: its largest score and one over its sum
  for (int h = threadIdx.x >> 3; h - (int)(threadIdx.x >> 3) < a.hq; h += 32) {
    const f32x2* tops = s.tops + ((int64_t)seq * a.hq + min(h, a.hq - 1)) * s.parts;
    float m = -INFINITY, l = 0.0f;
    for (int i = lane & 7; i < used; i += 8) m = fmaxf(m, tops[i][0]);
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, kWave));
    m = guarded(m);
    for (int i = lane & 7; i < used; i += 8) {
      const f32x2 t = tops[i];
      if (t[1] != 0.0f) l += t[1] * __builtin_amdgcn_exp2f(t[0] - m);
    }
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) l += __shfl_xor(l, off, kWave);
    if ((lane & 7) == 0 && h < a.hq) ml[h] = f32x2{m, l == 0.0f ? 0.0f : 1.0f / l};
  }
  __syncthreads();
  const int p = p0 + threadIdx.x;
  if (p >= len) return;
  const int64_t ld = (int64_t)s.parts * s.part;
  const float* sc = s.scores + (int64_t)seq * a.hq * ld + p;
  float v = 0.0f;
#pragma unroll 8
  for (int h = 0; h < a.hq; ++h) v += __builtin_amdgcn_exp2f(sc[h * ld] - ml[h][0]) * ml[h][1];
  a.weights[seq * a.weights_ld + p] += v;
}

// Places of a workgroup: at most 4096 workgroups (where sequences reach the table's
// width), and 512 places unless that leaves fewer than 1024, as a workgroup's first reads
// are a chain (lengths, table, scales) of about 3 us. Measured: one sequence of 131072
// places, 8 key-value heads: 256 places 62 us, 512 50, 1024 50; 64 sequences of up to
// 8192: 1024 places 123 us, 2048 129. Up to 512 places are one part: a join's launch
// costs more than the other waves save.
int part_of(int seqs, int hk, int tiles, int64_t places) {
  if (places <= 512) return 512;
  int part = kWaves * kPlaces;
  auto groups = [&] { return (int64_t)seqs * hk * tiles * ((places + part - 1) / part); };
  while (part < kMaxPart && groups() > (part < 512 ? 1024 : 4096)) part *= 2;
  return part;
}

struct Room {
  size_t sums, tops, scores, all;
};

Room room_of(int64_t seqs, int64_t hq, int64_t width, int64_t parts, int64_t part, bool weights) {
  Room r = {0, 0, 0, 0};
  auto take = [&](size_t n) {
    const size_t at = r.all;
    r.all += (n + 255) / 256 * 256;
    return at;
  };
  if (parts > 1) r.sums = take((size_t)(seqs * hq * parts * width) * 4);
  if (parts > 1 || weights) r.tops = take((size_t)(seqs * hq * parts) * 8);
  if (weights) r.scores = take((size_t)(seqs * hq * parts * part) * 4);
  return r;
}

template <int DT, bool I8, int W>
hipError_t split_t(Split& s, int64_t wgs, bool weights, hipStream_t st) {
  // a head in one block, whichever: block a multiple of width, or width itself
  const bool one = s.a.block % s.a.width == 0 && s.a.rows < ((int64_t)1 << 32);
  for (int64_t wg0 = 0; wg0 < wgs; wg0 += kMaxGroups) {
    const unsigned grid = (unsigned)(wgs - wg0 < kMaxGroups ? wgs - wg0 : kMaxGroups);
    s.wg0 = wg0;
    if (weights && one)
      split_kernel<DT, I8, W, true, true><<<grid, 256, 0, st>>>(s);
    else if (weights)
      split_kernel<DT, I8, W, true, false><<<grid, 256, 0, st>>>(s);
    else if (one)
      split_kernel<DT, I8, W, false, true><<<grid, 256, 0, st>>>(s);
    else
      split_kernel<DT, I8, W, false, false><<<grid, 256, 0, st>>>(s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT>
hipError_t cache_attend_t(const CacheAttend& a, hipStream_t st) {
  const int group = a.hq / a.hk, tiles = (group + kHeads - 1) / kHeads;
  const int64_t places = (int64_t)a.table_pages * a.page;
  const int part = part_of(a.seqs, a.hk, tiles, places);
  const int64_t parts = places < 1 ? 1 : (places + part - 1) / part;
  const bool weights = a.weights != nullptr;
  const Room r = room_of(a.seqs, a.hq, a.width, parts, part, weights);
  uint8_t* work = static_cast<uint8_t*>(a.work);
  Split s{a, 0, group, tiles, part, (int)parts, (int)(((int64_t)a.hk * a.width + a.block - 1) / a.block),
          reinterpret_cast<float*>(work + r.sums), reinterpret_cast<f32x2*>(work + r.tops),
          reinterpret_cast<float*>(work + r.scores)};
  const int64_t wgs = (a.seqs * parts + 7) / 8 * 8 * a.hk * tiles;
  hipError_t e;
  if (a.width <= 64)
    e = a.i8 ? split_t<DT, true, 64>(s, wgs, weights, st) : split_t<DT, false, 64>(s, wgs, weights, st);
  else
    e = a.i8 ? split_t<DT, true, 128>(s, wgs, weights, st) : split_t<DT, false, 128>(s, wgs, weights, st);
  if (e != hipSuccess || (parts == 1 && !weights)) return e;
  const int64_t joins = parts > 1 ? (int64_t)a.seqs * a.hq : 0;
  const int64_t more = joins + (weights ? a.seqs * ((places + 255) / 256) : 0);
  for (int64_t wg0 = 0; wg0 < more; wg0 += kMaxGroups) {
    s.wg0 = wg0;
    const unsigned grid = (unsigned)(more - wg0 < kMaxGroups ? more - wg0 : kMaxGroups);
    if (parts > 16)
      join_kernel<DT, 8><<<dim3(grid, (a.width + 31) / 32), 256, 0, st>>>(s, joins);
    else
      join_kernel<DT, 32><<<grid, 256, 0, st>>>(s, joins);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

size_t cache_attend_work(int seqs, int hq, int hk, int width, int64_t places, bool weights) {
  const int tiles = (hq / hk + kHeads - 1) / kHeads;
  const int part = part_of(seqs, hk, tiles, places);
  const int64_t parts = places < 1 ? 1 : (places + part - 1) / part;
  return room_of(seqs, hq, width, parts, part, weights).all;
}

hipError_t launch_cache_attend(const CacheAttend& a, hipStream_t st) {
  switch (a.dt) {
    case 0: return cache_attend_t<0>(a, st);
    case 1: return cache_attend_t<1>(a, st);
    case 4: return cache_attend_t<4>(a, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace emk
