// Rows of small accumulated weight dropped from paged stores.
//
// Of a sequence of more than `keep` rows stay the last `recent` and, of those before
// them, the keep - recent of largest weight (of equal ones the first). They move to
// the sequence's first places in their order, in place.
//
// Bound by HBM and by latency: a workgroup per sequence finds the threshold digit by
// digit (the weights stay in L2) and lists the moves; then workgroups of a sequence and
// 128 bytes of a row each go along the list. Measured, 16 sequences of up to 8192 rows cut to
// 2048, two stores of 1024 codes a row: 20 us for the lists (latency: a workgroup each),
// 18 us for the rows (5.9 TB/s; 110 us with 128 rows in flight per workgroup, not 512).
#include <type_traits>

#include "block.hpp"
#include "kernels.hpp"

namespace emk {
namespace {

constexpr int kSelect = 1024;

struct Move {
  int64_t from, to;
};

struct Moves {
  Move* list;    // seqs x keep (none where every row stays); from or to < 0: a page outside the store
  int32_t* span; // seqs x 2: [first rank that moves, ranks)
};

// Order of weights as unsigned numbers; NaN as -infinity, -0 as 0.
__device__ __forceinline__ uint32_t order_of(float w) {
  const uint32_t b = __float_as_uint(w != w ? -INFINITY : w + 0.0f);
  return b >> 31 ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ int64_t place_of(const CacheEvict& a, int seq, int p) {
  const int64_t page = a.table[seq * a.table_ld + p / a.page];
  const int64_t row = page * a.page + p % a.page;
  return page >= 0 && row < a.rows ? row : -1;
}

// The threshold in three digits of 11, 11 and 10 bits from the top: the first has the
// exponent and two more bits, as counts of an exponent alone would all meet in a few
// words of LDS. Then each wave takes a run of places: counts first, ranks after.
__global__ __launch_bounds__(kSelect) void select_kernel(CacheEvict a, Moves mv) {
  constexpr int kBins = 2048, kWaves = kSelect / 64, kDeep = 8;
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t tmp[kWaves];
  __shared__ uint32_t above[kWaves], equal[kWaves];
  __shared__ uint32_t found[2];  // digit, how many of it are still wanted
  const int seq = blockIdx.x, t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int64_t cap = (int64_t)a.table_pages * a.page;
  const int64_t given = a.lengths[seq];
  const int len = (int)(given < 0 ? 0 : given > cap ? cap : given);
  const float* w = a.weights + seq * a.weights_ld;
  float* new_w = a.new_weights + seq * cap;
  int32_t* kept = a.kept + (int64_t)seq * a.keep;
  const int old = max(len - a.recent, 0);  // the rows that compete
  uint32_t want = len > a.keep ? (uint32_t)(a.keep - a.recent) : (uint32_t)old;
  uint32_t edge = 0;  // stay: order > edge, and of those equal to it the first `want`
  if (len > a.keep) {
    uint32_t known = 0;
    for (int d = 0; d < 3 && want > 0; ++d) {
      const int shift = d == 0 ? 21 : d == 1 ? 10 : 0;
      const uint32_t mask = d == 2 ? 1023u : 2047u;
      hist[t] = hist[kSelect + t] = 0;
      __syncthreads();
      for (int64_t p0 = t; p0 < old; p0 += kSelect * kDeep) {
        uint32_t o[kDeep];
#pragma unroll
        for (int e = 0; e < kDeep; ++e) {
          const int64_t p = p0 + e * kSelect;
          o[e] = p < old ? order_of(w[p]) : 0u;
        }
#pragma unroll
        for (int e = 0; e < kDeep; ++e)
          if (p0 + e * kSelect < old && (o[e] & known) == edge) atomicAdd(&hist[o[e] >> shift & mask], 1u);
      }
      __syncthreads();
      // thread t has bins 2047 - 2 t and 2046 - 2 t
      const uint32_t c0 = hist[kBins - 1 - 2 * t], c1 = hist[kBins - 2 - 2 * t];
      const uint32_t before = block_incl_scan<uint32_t, kSelect>(c0 + c1, tmp) - c0 - c1;
      if (before < want && before + c0 + c1 >= want) {
        const int i = before + c0 < want;
        found[0] = kBins - 1 - 2 * t - i;
        found[1] = want - before - (i ? c0 : 0u);
      }
      __syncthreads();
      edge |= found[0] << shift;
      known |= mask << shift;
      want = found[1];
      __syncthreads();
    }
    if (want == 0) edge = 0xFFFFFFFFu;  // keep == recent: no other stays
  }
  const int run = (int)(((int64_t)old + kSelect - 1) / kSelect * 64);  // a wave's places
  const int64_t from = (int64_t)wave * run, to = min(from + run, (int64_t)old);
  uint32_t gts = 0, eqs = 0;
  for (int64_t p0 = from; p0 < to; p0 += 64 * kDeep) {
    uint32_t o[kDeep];
#pragma unroll
    for (int e = 0; e < kDeep; ++e) {
      const int64_t p = p0 + e * 64 + lane;
      o[e] = p < to ? order_of(w[p]) : 0u;
    }
#pragma unroll
    for (int e = 0; e < kDeep; ++e) {
      const bool in = p0 + e * 64 + lane < to;
      gts += __popcll(__ballot(in && o[e] > edge));
      eqs += __popcll(__ballot(in && o[e] == edge));
    }
  }
  if (lane == 0) {
    above[wave] = gts;
    equal[wave] = eqs;
  }
  __syncthreads();
  uint32_t g0 = 0, e0 = 0, all_g = 0, all_e = 0;
  for (int i = 0; i < kWaves; ++i) {
    if (i < wave) {
      g0 += above[i];
      e0 += equal[i];
    }
    all_g += above[i];
    all_e += equal[i];
  }
  const uint64_t below = ((uint64_t)1 << lane) - 1;
  for (int64_t p0 = from; p0 < to; p0 += 64 * kDeep) {
    float v[kDeep];
#pragma unroll
    for (int e = 0; e < kDeep; ++e) {
      const int64_t p = p0 + e * 64 + lane;
      v[e] = p < to ? w[p] : 0.0f;
    }
#pragma unroll
    for (int e = 0; e < kDeep; ++e) {
      const int64_t p = p0 + e * 64 + lane;
      const uint32_t o = order_of(v[e]);
      const bool gt = p < to && o > edge, eq = p < to && o == edge;
      const uint64_t bg = __ballot(gt), be = __ballot(eq);
      const uint32_t ge = e0 + __popcll(be & below);
      if (gt || (eq && ge < want)) {
        const uint32_t r = g0 + __popcll(bg & below) + min(ge, want);
        kept[r] = (int)p;
        new_w[r] = v[e];
      }
      g0 += __popcll(bg);
      e0 += __popcll(be);
    }
  }
  const int stay = (int)(all_g + min(all_e, want)), count = stay + len - old;
  for (int p = old + t; p < len; p += kSelect) {
    kept[stay + p - old] = p;
    new_w[stay + p - old] = w[p];
  }
  for (int64_t r = (int64_t)count + t; r < a.keep; r += kSelect) kept[r] = -1;
  for (int64_t r = (int64_t)count + t; r < cap; r += kSelect) new_w[r] = 0.0f;
  if (t == 0) {
    found[0] = (uint32_t)count;
    a.new_lengths[seq] = count;
  }
  __threadfence_block();
  __syncthreads();
  // the moves; ranks are in order, so those before the first gap stay where they are
  for (int64_t r = t; r < count; r += kSelect) {
    const int p = kept[r];
    if (p != r) {
      if (r == 0 || kept[r - 1] == r - 1) found[0] = (uint32_t)r;
      mv.list[(int64_t)seq * a.keep + r] = Move{place_of(a, seq, p), place_of(a, seq, (int)r)};
    }
  }
  __syncthreads();
  if (t == 0) {
    mv.span[2 * seq] = (int32_t)found[0];
    mv.span[2 * seq + 1] = count;
  }
}

constexpr int kSlice = 128;  // bytes of a row that a workgroup moves
constexpr int kMovers = 1024;
constexpr int kDeep = 4;     // rows in flight per thread and round

struct Slices {
  uint8_t* plane[CacheEvict::kPlanes];
  int64_t row_bytes[CacheEvict::kPlanes];
  int unit[CacheEvict::kPlanes];   // bytes of a lane: 16, 8, 4 or 1
  int lanes[CacheEvict::kPlanes];  // log 2 of the lanes of a row
  int first[CacheEvict::kPlanes];  // first slice of the plane
  int planes, slices;
};

// A row's place is never before its rank, so what one round overwrites are sources of that
// round or of an earlier one: a round is stored once every lane holds its rows of it. The
// next round's rows are fetched before that, and the list's entries another round ahead,
// as a row's address comes from one.
template <typename V>
__device__ __forceinline__ void move_rows(uint8_t* plane, int64_t row_bytes, int64_t off,
                                          int lanes, const Move* list, int first, int count) {
  const int rpt = kMovers >> lanes;  // rows of the workgroup at once
  const int round = rpt * kDeep, row = threadIdx.x >> lanes;
  const int64_t at = off + (int64_t)(threadIdx.x & ((1 << lanes) - 1)) * sizeof(V);
  const bool on = at < row_bytes;
  using Held = std::conditional_t<sizeof(V) == 1, uint32_t, V>;  // in whole registers
  Held held[2][kDeep] = {};
  int64_t to[2][kDeep];
  Move mv[kDeep];
  auto entries = [&](uint32_t r0) {
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const uint32_t r = r0 + u * rpt + row;  // up to three rounds past count
      mv[u] = r < (uint32_t)count ? list[r] : Move{-1, -1};
    }
  };
  auto fetch = [&](Held(&v)[kDeep], int64_t(&dst)[kDeep]) {
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const bool go = on && mv[u].from >= 0 && mv[u].to >= 0;
      dst[u] = go ? mv[u].to * row_bytes + at : -1;
      if (go) v[u] = load_any<V>(plane + mv[u].from * row_bytes + at);
    }
  };
  auto put = [&](Held(&v)[kDeep], int64_t(&dst)[kDeep]) {
#pragma unroll
    for (int u = 0; u < kDeep; ++u)
      if (dst[u] >= 0) store_any(plane + dst[u], (V)v[u]);
  };
  // the loads themselves have ended, not their issue alone
  auto arrived = [](Held(&v)[kDeep]) {
#pragma unroll
    for (int u = 0; u < kDeep; ++u) asm volatile("" : "+v"(v[u])::"memory");
  };
  entries(first);
  fetch(held[0], to[0]);
  entries(first + round);
  for (uint32_t r0 = first; r0 < (uint32_t)count; r0 += 2 * round) {
    arrived(held[0]);
    __syncthreads();
    fetch(held[1], to[1]);
    entries(r0 + 2 * round);
    put(held[0], to[0]);
    arrived(held[1]);
    __syncthreads();
    fetch(held[0], to[0]);
    entries(r0 + 3 * round);
    put(held[1], to[1]);
  }
}

__global__ __launch_bounds__(kMovers) void move_kernel(Slices s, Moves mv, int keep) {
  const int seq = blockIdx.x / s.slices, slice = blockIdx.x % s.slices;
  const int first = mv.span[2 * seq], count = mv.span[2 * seq + 1];
  if (first >= count) return;
  int p = 0;
  while (p + 1 < s.planes && slice >= s.first[p + 1]) ++p;
  const int64_t off = (int64_t)(slice - s.first[p]) * kSlice;
  const Move* list = mv.list + (int64_t)seq * keep;
  uint8_t* plane = s.plane[p];
  const int64_t len = s.row_bytes[p];
  switch (s.unit[p]) {
    case 16: return move_rows<u32x4>(plane, len, off, s.lanes[p], list, first, count);
    case 8: return move_rows<u32x2>(plane, len, off, s.lanes[p], list, first, count);
    case 4: return move_rows<uint32_t>(plane, len, off, s.lanes[p], list, first, count);
    default: return move_rows<uint8_t>(plane, len, off, s.lanes[p], list, first, count);
  }
}

// A table that holds no more than keep rows has none to move, however large keep is.
size_t list_bytes(int seqs, int keep, int64_t places) {
  return keep >= places ? 0 : ((size_t)seqs * keep * sizeof(Move) + 255) / 256 * 256;
}

}  // namespace

size_t cache_evict_work(int seqs, int keep, int64_t places) {
  return list_bytes(seqs, keep, places) + (size_t)seqs * 8;
}

hipError_t launch_cache_evict(const CacheEvict& a, hipStream_t st) {
  if (a.seqs <= 0) return hipSuccess;
  uint8_t* work = static_cast<uint8_t*>(a.work);
  const int64_t places = (int64_t)a.table_pages * a.page;
  const Moves mv{reinterpret_cast<Move*>(work),
                 reinterpret_cast<int32_t*>(work + list_bytes(a.seqs, a.keep, places))};
  select_kernel<<<a.seqs, kSelect, 0, st>>>(a, mv);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.keep >= places) return e;
  Slices s{};
  for (int p = 0; p < a.planes; ++p) {
    s.plane[p] = a.plane[p];
    s.row_bytes[p] = a.row_bytes[p];
    const uint64_t bits = (uint64_t)a.row_bytes[p] | (uint64_t)(uintptr_t)a.plane[p];
    s.unit[p] = bits % 16 == 0 ? 16 : bits % 8 == 0 ? 8 : bits % 4 == 0 ? 4 : 1;
    const int64_t of_row = (a.row_bytes[p] < kSlice ? a.row_bytes[p] : kSlice) / s.unit[p];
    while (((int64_t)1 << s.lanes[p]) < of_row) ++s.lanes[p];
    s.first[p] = s.slices;
    s.slices += (int)((a.row_bytes[p] + kSlice - 1) / kSlice);
  }
  s.planes = a.planes;
  move_kernel<<<(unsigned)a.seqs * s.slices, kMovers, 0, st>>>(s, mv, a.keep);
  return hipGetLastError();
}

}  // namespace emk
