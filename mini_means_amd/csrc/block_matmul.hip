// Matrix product of E4M3 codes with one power-of-two scale for each 128
// values: out[m][n] = sum_k a[m][k] 2^ea b[n][k] 2^eb, both matrices with k
// along their rows, fp32 sums.
//
// gfx950's scaled MFMA (v_mfma_scale_f32_16x16x128_f8f6f4) takes one E8M0
// scale byte for each row and 32 values of k of either operand. A block of
// 128 is one such instruction with the row's byte in all four lane groups, so
// the scales cost no arithmetic at all: the sums stay in the accumulator from
// the first k to the last.
//
// The FP8 unit adds a row's 128 products in groups of eight consecutive codes,
// each group aligned to its largest product with 14 bits kept below it; only
// the groups and the accumulator add in fp32 (measured: a term of 2^3 beside
// one of 2^16 survives, 2^2 does not; on normal data the sums are off by 1.5e-5
// of their norm). Beside the rounding of a bf16 or fp16 result (1.7e-3, 2e-4)
// that is nothing, so those results take the FP8 unit. An fp32 result takes
// the bf16 unit instead, at half the rate: every E4M3 value times its scale is
// a bf16 value (v_cvt_scalef32_pk_bf16_fp8 makes two at a time), products are
// then exact and sums fp32 throughout.
//
// Operands: lane l holds, for row l % 16, two 16-byte pieces of its 128 codes
// (the same two for both matrices, so their order along k does not matter).
// The first operand is B's rows (n), the second A's (m): the result then has
// n = 4 (l / 16) + v, v < 4, and m = l % 16 in lane l, four consecutive
// values of an output row.
#include "kernels.hpp"

namespace emk {

namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr int kStep = 128;  // codes of k per MFMA, and per scale

__device__ __forceinline__ i32x8 join(u32x4 lo, u32x4 hi) {
  return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
               (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// 16 codes at p, of which the first cnt exist (the rest read as zeros);
// wide when vec (p 16-byte aligned) and whole.
__device__ __forceinline__ u32x4 load16(const uint8_t* p, int cnt, bool vec) {
  if (vec && cnt >= 16) return *reinterpret_cast<const u32x4*>(p);
  u32x4 w = {0u, 0u, 0u, 0u};
  if (cnt <= 0) return w;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i < cnt) w[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
  return w;
}

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// One lane's 32 codes of a k-step as an MFMA operand, with its scale byte: as
// they are for the FP8 unit, decoded for the bf16 unit.
//
// bf16 unit: the scale is folded into the decoded values as long as it is
// within 2^+-kFold, so that every value is a normal bf16 number and every
// product one of fp32's range; what is left of a scale beyond (`rest`, 0 in
// all ordinary data) is applied to the step's sums.
constexpr int kFold = 50;
constexpr int kRestNaN = 1 << 20;  // the scale byte 255

template <bool F8>
struct Operand;

template <>
struct Operand<true> {
  i32x8 v;
  uint32_t scale;
  __device__ __forceinline__ void set(u32x4 lo, u32x4 hi, uint32_t byte) {
    v = join(lo, hi);
    scale = byte;
  }
};

template <>
struct Operand<false> {
  bf16x8 v[4];
  int rest;
  __device__ __forceinline__ void set(u32x4 lo, u32x4 hi, uint32_t byte) {
    const int e = (int)byte - 127;
    const int f = max(-kFold, min(kFold, e));
    rest = byte == 255u ? kRestNaN : e - f;
    const float s = __uint_as_float((uint32_t)(f + 127) << 23);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t w0 = q < 2 ? lo[2 * q] : hi[2 * q - 4];
      const uint32_t w1 = q < 2 ? lo[2 * q + 1] : hi[2 * q - 3];
      const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s, false);
      const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, s, true);
      const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s, false);
      const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, s, true);
      v[q] = bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
    }
  }
};

__device__ __forceinline__ f32x4 step(const Operand<true>& bn, const Operand<true>& am, f32x4 c) {
  // formats 0, 0: E4M3 operands; byte 0 of each scale register
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(bn.v, am.v, c, 0, 0, 0, (int)bn.scale, 0,
                                                          (int)am.scale);
}

__device__ __forceinline__ f32x4 step(const Operand<false>& bn, const Operand<false>& am, f32x4 c) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bn.v[q], am.v[q], c, 0, 0, 0);
  return c;
}

// c += one k-step of a 16 x 16 tile. `extreme` (the same in all lanes): some
// row of the operands has a rest.
__device__ __forceinline__ f32x4 add_step(const Operand<true>& bn, const Operand<true>& am,
                                          f32x4 c, bool) {
  return step(bn, am, c);
}

__device__ __forceinline__ f32x4 add_step(const Operand<false>& bn, const Operand<false>& am,
                                          f32x4 c, bool extreme) {
  if (!extreme) return step(bn, am, c);
  const f32x4 t = step(bn, am, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int r = am.rest + __shfl(bn.rest, 4 * (lane >> 4) + v, 64);  // row n = 4 (l / 16) + v
    c[v] += r >= kRestNaN ? __builtin_nanf("") : __builtin_ldexpf(t[v], r);
  }
  return c;
}

template <int N>
__device__ __forceinline__ bool any_rest(const Operand<true> (&)[N]) {
  return false;
}

template <int N>
__device__ __forceinline__ bool any_rest(const Operand<false> (&o)[N]) {
  int r = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) r |= o[i].rest;
  return __any(r != 0);
}

template <int OT>  // 1 bf16, 4 fp16
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (OT == 1)
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
  else
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), f16x2));
}

// Four consecutive values of an output row, of which the first cnt exist;
// wide when vec (the row's values are aligned to four) and whole.
template <int OT>
__device__ __forceinline__ void store4(void* out, int64_t at, f32x4 y, int cnt, bool vec) {
  if constexpr (OT == 0) {
    float* o = static_cast<float*>(out) + at;
    if (vec && cnt >= 4) {
      *reinterpret_cast<f32x4*>(o) = y;
      return;
    }
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (v < cnt) o[v] = y[v];
  } else {
    uint16_t* o = static_cast<uint16_t*>(out) + at;
    const u32x2 w = {pack2<OT>(y[0], y[1]), pack2<OT>(y[2], y[3])};
    if (vec && cnt >= 4) {
      *reinterpret_cast<u32x2*>(o) = w;
      return;
    }
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (v < cnt) o[v] = (uint16_t)(w[v >> 1] >> (16 * (v & 1)));
  }
}

// ---------------------------------------------------------------------------
// Any alignment, any row pitch: 64 x 64 tiles, one k-step of both matrices at
// a time through registers into LDS. Chunk c of row r sits at c ^ (r % 8), so
// the eight rows that an operand read touches in one pass of the LDS fall on
// distinct banks.
// ---------------------------------------------------------------------------
constexpr int kAT = 64;

template <int OT>
__global__ __launch_bounds__(256) void product_any_kernel(BlockProduct p, bool vec_a, bool vec_b,
                                                          bool vec_o, unsigned tiles_n) {
  __shared__ __attribute__((aligned(16))) uint8_t la[kAT * kStep], lb[kAT * kStep];
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int64_t m0 = (int64_t)(blockIdx.x / tiles_n) * kAT;
  const int64_t n0 = (int64_t)(blockIdx.x % tiles_n) * kAT;
  const int r = t >> 2, q = 2 * (t & 3);  // this thread's row and first of two chunks
  const int64_t am = min(m0 + r, p.m - 1), bn = min(n0 + r, p.n - 1);
  const uint8_t* ap = p.A + am * p.lda + 16 * q;
  const uint8_t* bp = p.B + bn * p.ldb + 16 * q;
  const int col = lane & 15, grp = lane >> 4;
  const int wm = 32 * (wave & 1), wn = 32 * (wave >> 1);
  const uint8_t *sa[2], *sb[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    sa[i] = p.As + min(m0 + wm + 16 * i + col, p.m - 1) * p.ldas;
    const int64_t nn = min(n0 + wn + 16 * i + col, p.n - 1);
    sb[i] = p.Bs + (p.b_tiles ? nn / kStep : nn) * p.ldbs;
  }
  f32x4 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const int steps = (p.k + kStep - 1) / kStep;
  for (int s = 0; s < steps; ++s) {
    const int left = p.k - s * kStep - 16 * q;
    const u32x4 a0 = load16(ap + (int64_t)s * kStep, left, vec_a);
    const u32x4 a1 = load16(ap + (int64_t)s * kStep + 16, left - 16, vec_a);
    const u32x4 b0 = load16(bp + (int64_t)s * kStep, left, vec_b);
    const u32x4 b1 = load16(bp + (int64_t)s * kStep + 16, left - 16, vec_b);
    __syncthreads();
    *reinterpret_cast<u32x4*>(&la[r * kStep + 16 * (q ^ (r & 7))]) = a0;
    *reinterpret_cast<u32x4*>(&la[r * kStep + 16 * ((q + 1) ^ (r & 7))]) = a1;
    *reinterpret_cast<u32x4*>(&lb[r * kStep + 16 * (q ^ (r & 7))]) = b0;
    *reinterpret_cast<u32x4*>(&lb[r * kStep + 16 * ((q + 1) ^ (r & 7))]) = b1;
    __syncthreads();
    Operand<OT != 0> fa[2], fb[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int ra = wm + 16 * i + col, rb = wn + 16 * i + col, x = col & 7;
      fa[i].set(*reinterpret_cast<const u32x4*>(&la[ra * kStep + 16 * (grp ^ x)]),
                *reinterpret_cast<const u32x4*>(&la[ra * kStep + 16 * ((grp + 4) ^ x)]), sa[i][s]);
      fb[i].set(*reinterpret_cast<const u32x4*>(&lb[rb * kStep + 16 * (grp ^ x)]),
                *reinterpret_cast<const u32x4*>(&lb[rb * kStep + 16 * ((grp + 4) ^ x)]), sb[i][s]);
    }
    const bool extreme = any_rest(fa) || any_rest(fb);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = add_step(fb[j], fa[i], acc[i][j], extreme);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t m = m0 + wm + 16 * i + col;
    if (m >= p.m) continue;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t n = n0 + wn + 16 * j + 4 * grp;
      store4<OT>(p.out, m * p.ldo + n, acc[i][j], (int)min((int64_t)4, p.n - n), vec_o);
    }
  }
}

template <int OT>
hipError_t product_t(const BlockProduct& p, hipStream_t st) {
  const bool vec_a = (uintptr_t)p.A % 16 == 0 && p.lda % 16 == 0;
  const bool vec_b = (uintptr_t)p.B % 16 == 0 && p.ldb % 16 == 0;
  const bool vec_o = (uintptr_t)p.out % (OT == 0 ? 16 : 8) == 0 && p.ldo % 4 == 0;
  const int64_t tm = (p.m + kAT - 1) / kAT, tn = (p.n + kAT - 1) / kAT;
  if (tm * tn > INT32_MAX) return hipErrorInvalidValue;
  product_any_kernel<OT><<<(unsigned)(tm * tn), 256, 0, st>>>(p, vec_a, vec_b, vec_o, (unsigned)tn);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_block_product(const BlockProduct& p, hipStream_t st) {
  if (p.m <= 0 || p.n <= 0) return hipSuccess;
  switch (p.ot) {
    case 0: return product_t<0>(p, st);
    case 1: return product_t<1>(p, st);
    case 4: return product_t<4>(p, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace emk
