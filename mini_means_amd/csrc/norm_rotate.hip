// Queries and keys normed per head and turned by their positions, in one pass.
//
// For a head x of w values with weights g: y = g x r, r = 1 / sqrt(mean x^2 + eps);
// then the pairs (c, c + half), c < half, are turned by positions[t] freqs[c],
// and the values from 2 half on stay as they are. With the gradient dy of the result
// and u = dy turned back: dx = r (g u) - x r^3 mean(g u x), dg = sum of u x r over
// tokens and heads.
//
// Bound by HBM: each value is read and written once, with about ten operations. A
// workgroup takes whole tokens, so that an angle is made once for all heads. Measured:
// 16384 tokens of 40 heads of 128 in bf16 66 us (5.1 TB/s; 82 with a lane's 32 weights read
// one by one), 5 tokens 5 us; 4099 tokens of 16 heads of 96 in fp32 13 us, their gradients
// 17 and 4 us.
#include <type_traits>

#include "block.hpp"
#include "kernels.hpp"

namespace emk {
namespace {

// The pairs of a head are cut into chunks of E; chunk j holds the values
// [lo, lo + E) and [hi, hi + E), so that a lane has both of each pair and nothing
// crosses lanes but the sum of squares. What is not turned is cut the same way
// (its first half against its second).
struct Chunk {
  int lo, hi, pair;  // pair: first index into the angles; -1 not turned
};

template <int E>
__device__ __forceinline__ Chunk chunk_of(int j, int half, int width) {
  const int p = j * E;
  if (p < half) return {p, p + half, p};
  const int at = half + p;  // 2 half + (p - half)
  return {at, at + (width - 2 * half) / 2, -1};
}

// E values as they lie in memory (16 bytes, or 8 of a 16-bit type), and as numbers.
template <int DT, int E>
using Run = std::conditional_t<DT == 0 || E == 8, u32x4, u32x2>;

template <int DT, int E>
__device__ __forceinline__ Run<DT, E> load_run(const void* base, int64_t at) {
  return load_any<Run<DT, E>>(static_cast<const uint8_t*>(base) + at * (DT == 0 ? 4 : 2));
}

template <int DT, int E>
__device__ __forceinline__ void numbers_of(const Run<DT, E>& w, float (&v)[E]) {
#pragma unroll
  for (int i = 0; i < E; ++i)
    v[i] = DT == 0 ? __uint_as_float(w[i])
                   : half_to_f32((uint16_t)(w[i >> 1] >> (16 * (i & 1))), DT == 4);
}

template <int DT, int E>
__device__ __forceinline__ void store_run(void* base, int64_t at, const float (&v)[E]) {
  if constexpr (DT == 0) {
    float* p = static_cast<float*>(base) + at;
#pragma unroll
    for (int i = 0; i < E; i += 4) store_any(p + i, f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]});
  } else {
    uint16_t* p = static_cast<uint16_t*>(base) + at;
    if constexpr (E == 8)
      store_any(p, u32x4{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]),
                         pack2<DT>(v[6], v[7])});
    else
      store_any(p, u32x2{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])});
  }
}

// A lane's weights of both sides: E values at lo, then E at hi.
template <int DT, int E>
__device__ __forceinline__ void weights_of(const NormRotate& a, const Chunk& c, float (&g)[2][2 * E]) {
  Run<DT, E> w[2][2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const void* p = s ? a.gk : a.gq;
    w[s][0] = load_run<DT, E>(p, c.lo);
    w[s][1] = load_run<DT, E>(p, c.hi);
  }
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    float x[E], y[E];
    numbers_of<DT, E>(w[s][0], x);
    numbers_of<DT, E>(w[s][1], y);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      g[s][i] = x[i];
      g[s][E + i] = y[i];
    }
  }
}

template <int E>
__device__ __forceinline__ void all_weights(const NormRotate& a, const Chunk& c, float (&g)[2][2 * E]) {
  if (a.gdt == 0) {
    if constexpr (E == 4) {
      weights_of<0, 4>(a, c, g);
    } else {  // in two halves of 16 bytes
      float x[2][8], y[2][8];
      weights_of<0, 4>(a, c, x);
      weights_of<0, 4>(a, {c.lo + 4, c.hi + 4, 0}, y);
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          g[s][i] = x[s][i];
          g[s][4 + i] = y[s][i];
          g[s][8 + i] = x[s][4 + i];
          g[s][12 + i] = y[s][4 + i];
        }
    }
  } else if (a.gdt == 1) {
    weights_of<1, E>(a, c, g);
  } else {
    weights_of<4, E>(a, c, g);
  }
}

// Sum over the L consecutive lanes of a head.
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int off = L / 2; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
  return v;
}

// cos and sin of positions x freqs. The product and its reduction to [-pi, pi]
// are in 64 bits: in 32, an angle of 10^6 would be off by 0.06.
__device__ __forceinline__ f32x2 turn_of(double position, double freq) {
  constexpr double kTurns = 0.15915494309189533577, k2Pi = 6.283185307179586232,
                   k2PiRest = 2.4492935982947063545e-16;
  const double a = position * freq;
  const double n = __builtin_rint(a * kTurns);
  const float r = (float)__builtin_fma(-n, k2PiRest, __builtin_fma(-n, k2Pi, a));
  float s, c;
  sincosf(r, &s, &c);
  return f32x2{c, s};
}

__device__ __forceinline__ double position_of(const NormRotate& a, int64_t t) {
  return a.pos_bytes == 8 ? (double)static_cast<const int64_t*>(a.positions)[t]
                          : (double)static_cast<const int32_t*>(a.positions)[t];
}

constexpr int kMaxTokens = 4;   // tokens of a workgroup at a time
constexpr int kMaxHalf = 128;   // width at most 256

// The angles of the workgroup's tokens, one per thread and turn: cos at [2 i], sin
// at [2 i + 1] of pair i of each token.
__device__ __forceinline__ void turns_of(const NormRotate& a, int64_t t0, int tokens,
                                         f32x2 (&turn)[kMaxTokens * kMaxHalf]) {
  for (int i = threadIdx.x; i < tokens * a.half; i += 256) {
    const int t = i / a.half;
    turn[i] = turn_of(position_of(a, t0 + t), a.freqs[i - t * a.half]);
  }
}

struct Head {
  const void* x;
  int64_t at;
  int64_t to;
  bool key;
};

// Head h of token t (queries first): where it is read and written.
__device__ __forceinline__ Head head_of(const NormRotate& a, int64_t t, int h) {
  if (h < a.hq) return {a.q, t * a.q_rs + h * a.q_hs, (t * a.hq + h) * (int64_t)a.width, false};
  h -= a.hq;
  return {a.k, t * a.k_rs + h * a.k_hs, (t * a.hk + h) * (int64_t)a.width, true};
}

// A workgroup takes T tokens: their angles first, one per thread, then all heads,
// L lanes each; a lane's chunk, and with it its weights, stays the same.
template <int DT, int E, int L>
__global__ __launch_bounds__(256) void norm_rotate_kernel(NormRotate a, int64_t wg0, int T) {
  __shared__ f32x2 turn[kMaxTokens * kMaxHalf];
  const int64_t t0 = (wg0 + blockIdx.x) * T;
  const int tokens = (int)min((int64_t)T, a.n - t0);
  const int j = threadIdx.x % L, heads = a.hq + a.hk;
  const bool on = j * E * 2 < a.width;
  const Chunk c = chunk_of<E>(on ? j : 0, a.half, a.width);
  float g[2][2 * E];
  all_weights<E>(a, c, g);
  // a lane's next head is on its way while this one is worked on, and the first while the
  // angles are made; past the last it is the last again (a whole wave takes part in the
  // sums), and lanes past the width have the first chunk
  const int items = tokens * heads, first = threadIdx.x / L;
  auto head = [&](int i, int& t) {
    const int it = min(i, items - 1);
    t = it / heads;
    return head_of(a, t0 + t, it - t * heads);
  };
  int t, next_t;
  Head hd, next = head(first, next_t);
  Run<DT, E> lo = load_run<DT, E>(next.x, next.at + c.lo), hi = load_run<DT, E>(next.x, next.at + c.hi);
  turns_of(a, t0, tokens, turn);
  __syncthreads();
  const float inv = 1.0f / (float)a.width;
  for (int i = first; i - first < items; i += 256 / L) {
    const bool live = i < items;
    float x[E], y[E];
    numbers_of<DT, E>(lo, x);
    numbers_of<DT, E>(hi, y);
    if (!on) {
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = y[e] = 0.0f;
    }
    hd = next;
    t = next_t;
    next = head(i + 256 / L, next_t);
    lo = load_run<DT, E>(next.x, next.at + c.lo);
    hi = load_run<DT, E>(next.x, next.at + c.hi);
    float sq = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) sq += x[e] * x[e] + y[e] * y[e];
    const float r = 1.0f / sqrtf(lanes_sum<L>(sq) * inv + a.eps);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      x[e] = x[e] * r * (hd.key ? g[1][e] : g[0][e]);
      y[e] = y[e] * r * (hd.key ? g[1][E + e] : g[0][E + e]);
    }
    if (c.pair >= 0) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const f32x2 w = turn[t * a.half + c.pair + e];
        const float lo = x[e] * w[0] - y[e] * w[1];
        y[e] = y[e] * w[0] + x[e] * w[1];
        x[e] = lo;
      }
    }
    if (on && live) {
      void* to = hd.key ? a.ko : a.qo;
      store_run<DT, E>(to, hd.to + c.lo, x);
      store_run<DT, E>(to, hd.to + c.hi, y);
    }
  }
}

// The gradients: the workgroup goes over tokens a.groups x T apart and keeps its
// lanes' sums for the weights in registers; they are joined in LDS and written to
// `part` (groups x 2 x width, fp32), which weight_sum_kernel adds in one order.
template <int DT, int E, int L>
__global__ __launch_bounds__(256) void norm_rotate_back_kernel(NormRotate a, int T) {
  __shared__ f32x2 turn[kMaxTokens * kMaxHalf];
  __shared__ float sum[256 / L][2 * E * L];
  const int j = threadIdx.x % L, heads = a.hq + a.hk;
  const bool on = j * E * 2 < a.width;
  const Chunk c = chunk_of<E>(on ? j : 0, a.half, a.width);
  float g[2][2 * E], dg[2][2 * E];
  all_weights<E>(a, c, g);
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int i = 0; i < 2 * E; ++i) dg[s][i] = 0.0f;
  const float inv = 1.0f / (float)a.width;
  for (int64_t t0 = (int64_t)blockIdx.x * T; t0 < a.n; t0 += (int64_t)gridDim.x * T) {
    const int tokens = (int)min((int64_t)T, a.n - t0);
    __syncthreads();  // the last round's angles have been read
    turns_of(a, t0, tokens, turn);
    __syncthreads();
    const int items = tokens * heads;
    for (int i = threadIdx.x / L; i - (int)(threadIdx.x / L) < items; i += 256 / L) {
      const bool live = i < items;
      const int it = live ? i : items - 1;
      const int t = it / heads, h = it - t * heads;
      const Head hd = head_of(a, t0 + t, h);
      const void* dy = hd.key ? a.dk : a.dq;
      const int64_t dat = hd.key ? (t0 + t) * a.dk_rs + (h - a.hq) * a.dk_hs
                                 : (t0 + t) * a.dq_rs + h * a.dq_hs;
      float x[E], y[E], u[E], v[E];
      {
        const Run<DT, E> xr = load_run<DT, E>(hd.x, hd.at + c.lo), yr = load_run<DT, E>(hd.x, hd.at + c.hi),
                         ur = load_run<DT, E>(dy, dat + c.lo), vr = load_run<DT, E>(dy, dat + c.hi);
        numbers_of<DT, E>(xr, x);
        numbers_of<DT, E>(yr, y);
        numbers_of<DT, E>(ur, u);
        numbers_of<DT, E>(vr, v);
      }
      if (!on || !live) {
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = y[e] = u[e] = v[e] = 0.0f;
      }
      if (c.pair >= 0) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const f32x2 w = turn[t * a.half + c.pair + e];
          const float lo = u[e] * w[0] + v[e] * w[1];
          v[e] = v[e] * w[0] - u[e] * w[1];
          u[e] = lo;
        }
      }
      float sq = 0.0f, in = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        sq += x[e] * x[e] + y[e] * y[e];
        in += u[e] * (hd.key ? g[1][e] : g[0][e]) * x[e] +
              v[e] * (hd.key ? g[1][E + e] : g[0][E + e]) * y[e];
      }
      const float r = 1.0f / sqrtf(lanes_sum<L>(sq) * inv + a.eps);
      const float f = lanes_sum<L>(in) * inv * r * r * r;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float xr = x[e] * r * u[e], yr = y[e] * r * v[e];
        dg[0][e] += hd.key ? 0.0f : xr;
        dg[0][E + e] += hd.key ? 0.0f : yr;
        dg[1][e] += hd.key ? xr : 0.0f;
        dg[1][E + e] += hd.key ? yr : 0.0f;
        u[e] = u[e] * (hd.key ? g[1][e] : g[0][e]) * r - x[e] * f;
        v[e] = v[e] * (hd.key ? g[1][E + e] : g[0][E + e]) * r - y[e] * f;
      }
      if (on && live) {
        void* to = hd.key ? a.ko : a.qo;
        store_run<DT, E>(to, hd.to + c.lo, u);
        store_run<DT, E>(to, hd.to + c.hi, v);
      }
    }
  }
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < E; ++e) {
      sum[threadIdx.x / L][2 * E * j + e] = dg[s][e];
      sum[threadIdx.x / L][2 * E * j + E + e] = dg[s][E + e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * E * L; i += 256) {
      const int cj = i / (2 * E), e = i - cj * 2 * E;
      if (cj * E * 2 >= a.width) continue;
      float v = 0.0f;
      for (int q = 0; q < 256 / L; ++q) v += sum[q][i];
      const Chunk cc = chunk_of<E>(cj, a.half, a.width);
      a.part[((int64_t)blockIdx.x * 2 + s) * a.width + (e < E ? cc.lo + e : cc.hi + e - E)] = v;
    }
  }
}

// dg[side][c] = sum of the workgroups' parts, in 64 bits and in one order.
__global__ __launch_bounds__(256) void weight_sum_kernel(const float* part, int groups, int width,
                                                         int gdt, void* dgq, void* dgk) {
  __shared__ double tmp[4];
  const int s = blockIdx.x / width, c = blockIdx.x - s * width;
  double v = 0.0;
  for (int i = threadIdx.x; i < groups; i += 256) v += (double)part[((int64_t)i * 2 + s) * width + c];
  v = block_sum<double, 256>(v, tmp);
  if (threadIdx.x == 0) {
    void* to = s ? dgk : dgq;
    if (gdt == 0)
      static_cast<float*>(to)[c] = (float)v;
    else
      static_cast<uint16_t*>(to)[c] = to_half_rne((float)v, gdt == 4);
  }
}

// go(E, L) for the head's width: E pairs per lane, as wide as the cuts at half and
// in the rest allow (fp32 4: 16 bytes), L lanes.
template <int DT, typename GO>
hipError_t by_width(const NormRotate& a, GO go) {
  const bool eight = DT != 0 && a.half % 8 == 0 && (a.width - 2 * a.half) % 16 == 0;
  const int chunks = a.width / 2 / (eight ? 8 : 4);
#define EMK_GO(E, L)                                                                \
  if (chunks <= L) {                                                                \
    go(std::integral_constant<int, E>(), std::integral_constant<int, L>());         \
    return hipGetLastError();                                                       \
  }
  if constexpr (DT != 0) {
    if (eight) {
      EMK_GO(8, 4) EMK_GO(8, 8) EMK_GO(8, 16)
      return hipErrorInvalidValue;
    }
  }
  EMK_GO(4, 4) EMK_GO(4, 8) EMK_GO(4, 16) EMK_GO(4, 32)
#undef EMK_GO
  return hipErrorInvalidValue;
}

template <int DT>
hipError_t forward_t(const NormRotate& a, hipStream_t st) {
  // one token per workgroup until there are enough to fill the card
  const int T = a.n >= 4096 ? kMaxTokens : 1;
  const int64_t wgs = (a.n + T - 1) / T;
  for (int64_t wg0 = 0; wg0 < wgs; wg0 += kMaxGroups) {
    const unsigned grid = (unsigned)(wgs - wg0 < kMaxGroups ? wgs - wg0 : kMaxGroups);
    const hipError_t e = by_width<DT>(a, [&](auto E, auto L) {
      norm_rotate_kernel<DT, decltype(E)::value, decltype(L)::value><<<grid, 256, 0, st>>>(a, wg0, T);
    });
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT>
hipError_t backward_t(const NormRotate& a, hipStream_t st) {
  const int groups = norm_rotate_groups(a.n);
  const int T = a.n >= 4096 ? kMaxTokens : 1;
  const hipError_t e = by_width<DT>(a, [&](auto E, auto L) {
    norm_rotate_back_kernel<DT, decltype(E)::value, decltype(L)::value><<<groups, 256, 0, st>>>(a, T);
  });
  if (e != hipSuccess) return e;
  weight_sum_kernel<<<2 * a.width, 256, 0, st>>>(a.part, groups, a.width, a.gdt, a.dgq, a.dgk);
  return hipGetLastError();
}

}  // namespace

int norm_rotate_groups(int64_t n) { return (int)(n < 1 ? 1 : n < 1024 ? n : 1024); }

hipError_t launch_norm_rotate(const NormRotate& a, hipStream_t st) {
  if (a.n <= 0) return hipSuccess;
  switch (a.dt) {
    case 0: return forward_t<0>(a, st);
    case 1: return forward_t<1>(a, st);
    case 4: return forward_t<4>(a, st);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_norm_rotate_back(const NormRotate& a, hipStream_t st) {
  switch (a.dt) {
    case 0: return backward_t<0>(a, st);
    case 1: return backward_t<1>(a, st);
    case 4: return backward_t<4>(a, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace emk
