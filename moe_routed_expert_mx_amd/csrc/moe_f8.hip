// moe_f8.hip -- MI355X (gfx950) kernels of the layer in block-scaled FP8: routes sorted by expert, the
// product of e4m3 matrices with a scale for each block of 128, and the same product grouped by
// expert, behind the C ABI of include/moe_mx.h.
#include <algorithm>
#include <cstring>
#include <type_traits>

#include "dense_common.h"

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));

// --------------------------------------------------------------------- lists
// A stable counting sort: counts of each wave's share of the routes, their prefix over the waves (and
// over the workgroups before), then each wave places its routes in order.  Up to 8192 routes one
// workgroup does it; beyond that a first launch counts, the second places.
constexpr int kListWaves = 16, kListThreads = 64 * kListWaves, kListOne = 8192;

struct ListArgs {
  const int32_t* ids;
  int32_t *offsets, *pairs;
  uint32_t* counts;  // [workgroups][E], of the first launch
  uint32_t R, E, share;  // routes a wave (a multiple of 64)
};

__device__ __forceinline__ void count_ids(const ListArgs& a, uint32_t first, uint32_t last, uint32_t* counts, int lane) {
  for (uint32_t i = first + lane; i < last; i += 64) {
    const uint32_t id = static_cast<uint32_t>(a.ids[i]);
    if (id < a.E) atomicAdd(counts + id, 1u);
  }
}

__global__ __launch_bounds__(kListThreads) void lists_count_kernel(ListArgs a) {
  extern __shared__ uint32_t list_lds[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (uint32_t e = threadIdx.x; e < a.E; e += kListThreads) list_lds[e] = 0;
  __syncthreads();
  const uint64_t begin = (static_cast<uint64_t>(blockIdx.x) * kListWaves + wave) * a.share;
  const uint32_t first = static_cast<uint32_t>(begin < a.R ? begin : a.R), last = a.R - first < a.share ? a.R : first + a.share;
  count_ids(a, first, last, list_lds, lane);
  __syncthreads();
  for (uint32_t e = threadIdx.x; e < a.E; e += kListThreads) a.counts[static_cast<uint64_t>(blockIdx.x) * a.E + e] = list_lds[e];
}

// Placing.  E <= kListThreads: thread e adds up expert e.
__global__ __launch_bounds__(kListThreads) void lists_place_kernel(ListArgs a) {
  extern __shared__ uint32_t list_lds[];  // [waves][E]: counts, then where the wave's next route goes; sums
  uint32_t* const sums = list_lds + kListWaves * a.E;
  uint32_t* const joined = sums + kListWaves;  // [2][E]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t e = threadIdx.x;
  for (uint32_t i = threadIdx.x; i < kListWaves * a.E; i += kListThreads) list_lds[i] = 0;
  for (uint32_t i = threadIdx.x; i < 2 * a.E; i += kListThreads) joined[i] = 0;
  __syncthreads();
  const uint64_t begin = (static_cast<uint64_t>(blockIdx.x) * kListWaves + wave) * a.share;
  const uint32_t first = static_cast<uint32_t>(begin < a.R ? begin : a.R), last = a.R - first < a.share ? a.R : first + a.share;
  // routes of each expert in all, and in the workgroups before this one: all threads share the counts out
  if (gridDim.x > 1) {
    const uint32_t parts = kListThreads / a.E, part = e / a.E, mine = e % a.E;
    if (part < parts) {
      uint32_t all = 0, before = 0;
      for (uint32_t g0 = part; g0 < gridDim.x; g0 += 16 * parts) {  // (from other XCDs: far away, so many at once)
        uint32_t c[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const uint32_t g = g0 + k * parts;
          c[k] = g < gridDim.x ? a.counts[static_cast<uint64_t>(g) * a.E + mine] : 0;
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          all += c[k];
          before += g0 + k * parts < blockIdx.x ? c[k] : 0;
        }
      }
      atomicAdd(joined + mine, all);
      atomicAdd(joined + a.E + mine, before);
    }
  }
  // the wave's first 512 ids stay in registers (all of them up to 2^21 routes), E for those left out
  constexpr int kHeld = 8;
  uint32_t held[kHeld];
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const uint32_t i = first + k * 64 + lane;
    held[k] = i < last ? static_cast<uint32_t>(a.ids[i]) : a.E;
  }
#pragma unroll
  for (int k = 0; k < kHeld; ++k)
    if (held[k] < a.E) atomicAdd(list_lds + wave * a.E + held[k], 1u);
  if (last - first > kHeld * 64) count_ids(a, first + kHeld * 64, last, list_lds + wave * a.E, lane);
  __syncthreads();
  uint32_t all = 0, before = 0;
  if (e < a.E) {
    if (gridDim.x > 1) {
      all = joined[e];
      before = joined[a.E + e];
    } else {
#pragma unroll
      for (int w = 0; w < kListWaves; ++w) all += list_lds[w * a.E + e];
    }
  }
  // where expert e begins: the sum of `all` over the threads before
  uint32_t begins = all;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const uint32_t o = __shfl_up(begins, d);
    if (lane >= d) begins += o;
  }
  if (lane == 63) sums[wave] = begins;
  __syncthreads();
  begins -= all;
  uint32_t total = 0;
#pragma unroll
  for (int w = 0; w < kListWaves; ++w) {
    begins += w < wave ? sums[w] : 0;
    total += sums[w];
  }
  if (e < a.E) {
    if (blockIdx.x == 0) a.offsets[e] = static_cast<int32_t>(begins);
    uint32_t next = begins + before;
#pragma unroll
    for (int w = 0; w < kListWaves; ++w) {
      const uint32_t c = list_lds[w * a.E + e];
      list_lds[w * a.E + e] = next;
      next += c;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[a.E] = static_cast<int32_t>(total);
  __syncthreads();
  uint32_t* const next = list_lds + wave * a.E;
  const int bits = 32 - __builtin_clz(a.E);  // ids and E itself, which stands for those left out
  auto place = [&](uint32_t i, uint32_t id) {
    id = id < a.E ? id : a.E;
    uint64_t same = ~0ull;  // lanes with this lane's id
    for (int b = 0; b < bits; ++b) {
      const bool set = id >> b & 1;
      const uint64_t m = __ballot(set);
      same &= set ? m : ~m;
    }
    const uint32_t rank = static_cast<uint32_t>(__popcll(same & ((1ull << lane) - 1)));
    uint32_t at = 0;
    if (id < a.E) at = next[id];
    wave_sync();
    if (id < a.E) {
      a.pairs[at + rank] = static_cast<int32_t>(i);
      if (rank == 0) next[id] = at + static_cast<uint32_t>(__popcll(same));
    }
    wave_sync();
  };
#pragma unroll
  for (int k = 0; k < kHeld; ++k)
    if (first + k * 64 < last) place(first + k * 64 + lane, held[k]);
  for (uint32_t i0 = first + kHeld * 64; i0 < last; i0 += 64) place(i0 + lane, i0 + lane < last ? static_cast<uint32_t>(a.ids[i0 + lane]) : a.E);
  // behind the last list; each workgroup its share of the places
  const uint32_t span = kListWaves * a.share;
  const uint64_t p0 = static_cast<uint64_t>(blockIdx.x) * span;
  for (uint64_t p = p0 + threadIdx.x; p < p0 + span && p < a.R; p += kListThreads)
    if (p >= total) a.pairs[p] = -1;
}

// ------------------------------------------------------------------- product
struct F8Args {
  const uint8_t *a, *w;
  const float *sa, *sw, *bias;
  const void* add;
  void* out;
  const int32_t *offsets, *pairs;  // grouped
  int64_t lda, ldw, ldwe, ldsa, ldo, ldadd, a_rows, out_rows;
  int32_t M, N, K, E, gather, scatter;
};

// A run of up to BM rows that share a weight.
struct Unit {
  int e, first, rows;
};
// Sum over the lanes up to this one.
__device__ __forceinline__ int scan64(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // from the lane 1, 2, 4, 8 before, within 16
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // lanes 15 and 47 to the 16 behind each
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // lane 31 to the upper half
  return v;
}
// Unit `u` of a grouped product, by the prefix of the experts' unit counts; all lanes of a wave together.
// false: there are not as many.
template <int BM>
__device__ __forceinline__ bool find_unit(const F8Args& a, uint32_t u, Unit& unit) {
  const int lane = threadIdx.x & 63;
  for (int e0 = 0; e0 < a.E; e0 += 256) {
    int b[5], n[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      const int e = e0 + lane * 4 + i, v = a.offsets[e < a.E ? e : a.E];
      b[i] = v < 0 ? 0 : v > a.M ? a.M : v;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      n[i] = b[i + 1] > b[i] ? b[i + 1] - b[i] : 0;
      sum += static_cast<int>((static_cast<uint32_t>(n[i]) + BM - 1) / BM);
    }
    const int upto = scan64(sum);
    const uint32_t all = static_cast<uint32_t>(__builtin_amdgcn_readlane(upto, 63));
    if (u < all) {
      uint32_t in = u - static_cast<uint32_t>(upto - sum);
      const uint64_t here = __ballot(u >= static_cast<uint32_t>(upto - sum) && u < static_cast<uint32_t>(upto));
      int e = 0, first = 0, rows = 0;
      bool found = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t c = (static_cast<uint32_t>(n[i]) + BM - 1) / BM;
        if (!found && in < c) {
          found = true;
          e = e0 + lane * 4 + i;
          first = b[i] + static_cast<int>(in) * BM;
          rows = n[i] - static_cast<int>(in) * BM;
        }
        in -= c;
      }
      const int l = static_cast<int>(__builtin_ctzll(here));
      unit.e = __builtin_amdgcn_readlane(e, l);
      unit.first = __builtin_amdgcn_readlane(first, l);
      rows = __builtin_amdgcn_readlane(rows, l);
      unit.rows = rows < BM ? rows : BM;
      return true;
    }
    u -= all;
  }
  return false;
}

// Units there are.
template <int BM>
__device__ __forceinline__ uint32_t count_units(const F8Args& a) {
  const int lane = threadIdx.x & 63;
  uint32_t all = 0;
  for (int e0 = 0; e0 < a.E; e0 += 256) {
    int b[5], sum = 0;
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      const int e = e0 + lane * 4 + i, v = a.offsets[e < a.E ? e : a.E];
      b[i] = v < 0 ? 0 : v > a.M ? a.M : v;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      sum += b[i + 1] > b[i] ? static_cast<int>((static_cast<uint32_t>(b[i + 1] - b[i]) + BM - 1) / BM) : 0;
    all += static_cast<uint32_t>(__builtin_amdgcn_readlane(scan64(sum), 63));
  }
  return all;
}

// Row of a, and of out, of place i of the lists (-1: none).
__device__ __forceinline__ int64_t row_of_a(const F8Args& a, int i) {
  if (!a.gather) return i;
  const int p = a.pairs[i];
  const int64_t r = p < 0 ? -1 : static_cast<uint32_t>(p) / static_cast<uint32_t>(a.gather);
  return r < a.a_rows ? r : -1;
}
__device__ __forceinline__ int64_t row_of_out(const F8Args& a, int i) {
  if (!a.pairs) return i;
  const int p = a.pairs[i];
  if (p < 0 || (a.gather && static_cast<uint32_t>(p) / static_cast<uint32_t>(a.gather) >= a.a_rows)) return -1;
  if (!a.scatter) return i;
  return p < a.out_rows ? p : -1;
}

// A block's sum for a 16 x 16 tile, w's rows times a's.  The FP8 matrix cores add eight neighbouring
// products at a time with 13 bits behind the largest of them, the rest cut off (measured: a product 2^-13 of
// the largest counts, one of 2^-14 does not, unless they are in different eights): some 1.5e-5 of
// the sum.  An output of 16 bits that is final does not show it (2^-9 and 2^-12 of it on average).  FP32 outputs do, and so
// does a hidden that is quantized again: where 1.5e-5 turns its rounding to BF16 next to the middle of two codes, a value
// changes by 2^-4 (the experts' error against 64 bits grew from 0.0017 to 0.0020).  EXACT, for FP32 outputs and where the
// caller asks: the codes become BF16, exactly, and the BF16 cores add them with FP32's bits at half the rate.
template <bool EXACT>
struct Operand {
  using T = v8i;
  static __device__ __forceinline__ T make(v4i lo, v4i hi) { return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7); }
  static __device__ __forceinline__ v4f product(const T& w, const T& a) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, v4f{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
  }
};
template <>
struct Operand<true> {
  struct T {
    v8bf q[4];
  };
  static __device__ __forceinline__ T make(v4i lo, v4i hi) {
    T r;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t c = static_cast<uint32_t>(i < 4 ? lo[i] : hi[i - 4]);
      const auto x = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, false), y = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, true);
      r.q[i / 2][i % 2 * 4] = x[0];
      r.q[i / 2][i % 2 * 4 + 1] = x[1];
      r.q[i / 2][i % 2 * 4 + 2] = y[0];
      r.q[i / 2][i % 2 * 4 + 3] = y[1];
    }
    return r;
  }
  static __device__ __forceinline__ v4f product(const T& w, const T& a) {
    v4f d = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.q[i], a.q[i], d, 0, 0, 0);
    return d;
  }
};

// ------------------------------------------------------------ product: few rows
// The weight is read once, so its bytes bound the product.  WK of a workgroup's WV waves share 16 RT weight
// rows (SwiGLU: 16 gate rows and their 16 up rows) and 16 TT rows of a, and split K in blocks of 128.  A wave loads a block's rows eight lanes to a row, some blocks ahead, and turns them into operands
// through LDS of its own; a block's sum is scaled and added in FP32.
// Lane l's operand holds parts l / 16 and 4 + l / 16 of its row's eight: any order of k within the block
// will do that both sides have, and this one meets all banks of LDS.  The 16 experts of one token (gate and up rows of 384
// x 3584, 44 MB) take 14 us, 3.1 TB/s, exact sums or not, their second product 8 us (22 MB).
template <int OUT, bool SWIGLU, bool GROUPED, bool EXACT, int RT, int TT, int WV, int WK>
__global__ __launch_bounds__(64 * WV) void f8_stream_kernel(F8Args a, uint32_t nx) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  constexpr int COLS = SWIGLU ? 16 : 16 * RT, NL = 2 * (RT + TT), NS = SWIGLU ? 2 : 1;
  constexpr int kRegs = (2048 / WV - 4 * RT * TT - (EXACT ? 18 : 12) * (RT + TT) - 48) / (NL * 4 + TT + NS);
  constexpr int U = kRegs > 6 ? 6 : kRegs < 2 ? 2 : kRegs;  // blocks in flight
  static_assert(!SWIGLU || RT == 2, "a gate and an up tile");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int WN = WV / WK;  // groups of waves, along the weight rows
  const int H = SWIGLU ? a.N / 2 : a.N, wg0 = blockIdx.x % nx * (COLS * WN), n0 = wg0 + wave / WK * COLS;
  const int blocks = (a.K + 127) / 128, per = (blocks + WK - 1) / WK, c0 = wave % WK * per;
  const int n = blocks - c0 < per ? (blocks > c0 ? blocks - c0 : 0) : per;
  Unit unit;
  if constexpr (GROUPED) {
    if (!find_unit<16 * TT>(a, blockIdx.x / nx, unit)) return;
  } else {
    unit.e = 0;
    unit.first = blockIdx.x / nx * (16 * TT);
    unit.rows = a.M - unit.first < 16 * TT ? a.M - unit.first : 16 * TT;
  }
  // load i brings rows 8 i .. 8 i + 7 of the wave's tile: weight rows first, then rows of a
  const int part = lane & 7;
  const uint8_t* rows[NL];
  const float* scale[TT + NS];
  const uint8_t* const w = a.w + unit.e * a.ldwe;
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int r = i * 8 + (lane >> 3);
    if (i < 2 * RT) {
      const int c = n0 + (SWIGLU ? r & 15 : r);
      rows[i] = w + ((c < H ? c : H - 1) + (SWIGLU ? static_cast<int64_t>(r >> 4) * H : 0)) * a.ldw;
    } else {
      const int m = r - 16 * RT;
      const int64_t at = GROUPED ? row_of_a(a, unit.first + (m < unit.rows ? m : unit.rows - 1))
                                 : unit.first + (m < unit.rows ? m : unit.rows - 1);
      rows[i] = a.a + (at < 0 ? 0 : at) * a.lda;
    }
  }
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    const int m = j * 16 + (lane & 15);
    const int64_t at = GROUPED ? row_of_a(a, unit.first + (m < unit.rows ? m : unit.rows - 1))
                               : unit.first + (m < unit.rows ? m : unit.rows - 1);
    scale[j] = a.sa + (at < 0 ? 0 : at) * a.ldsa;
  }
  const int halves = SWIGLU ? 2 : 1, nb = (H + 127) / 128;  // blocks of weight rows in each
#pragma unroll
  for (int h = 0; h < NS; ++h) scale[TT + h] = a.sw + ((static_cast<int64_t>(unit.e) * halves + h) * nb + (n0 < H ? n0 / 128 : nb - 1)) * blocks;
  v4i held[U][NL];
  float held_scale[U][TT + NS];
  // 16 bytes lie wholly inside the row or wholly behind it; those behind are read from the row's last 16, and
  // the weight's set to zero when used
  auto load = [&](int u, int c) {
    const int k = (c0 + c) * 128 + part * 16;
#pragma unroll
    for (int i = 0; i < NL; ++i) held[u][i] = *reinterpret_cast<const v4i*>(rows[i] + (k < a.K ? k : a.K - 16));
#pragma unroll
    for (int i = 0; i < TT + NS; ++i) held_scale[u][i] = scale[i][c0 + c];
  };
  unsigned char* const own = smem + wave * (NL * 1024);
  auto place = [](int r, int c) { return r * 128 + (c ^ ((r >> 1) & 7)) * 16; };
  v4f acc[RT][TT] = {};
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (u < n) load(u, u);
  compiler_fence();
  for (int c = 0; c < n; c += U) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c + u < n) {
        const bool behind = (c0 + c + u) * 128 + part * 16 >= a.K;
        float s[TT + NS];
#pragma unroll
        for (int i = 0; i < NL; ++i)
          *reinterpret_cast<v4i*>(own + place(i * 8 + (lane >> 3), part)) = i < 2 * RT && behind ? v4i{0, 0, 0, 0} : held[u][i];
#pragma unroll
        for (int i = 0; i < TT + NS; ++i) s[i] = held_scale[u][i];
        if (c + u + U < n) load(u, c + u + U);
        wave_sync();
        using Op = Operand<EXACT>;
        typename Op::T fw[RT], fa[TT];
        auto operand = [&](int tile) {
          return Op::make(*reinterpret_cast<const v4i*>(own + place(tile * 16 + (lane & 15), lane >> 4)),
                          *reinterpret_cast<const v4i*>(own + place(tile * 16 + (lane & 15), 4 + (lane >> 4))));
        };
#pragma unroll
        for (int i = 0; i < RT; ++i) fw[i] = operand(i);
#pragma unroll
        for (int j = 0; j < TT; ++j) fa[j] = operand(RT + j);
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
          for (int j = 0; j < TT; ++j) {
            const v4f d = Op::product(fw[i], fa[j]);
            const float f = s[j] * s[TT + (SWIGLU ? i : 0)];
#pragma unroll
            for (int x = 0; x < 4; ++x) acc[i][j][x] = __builtin_fmaf(d[x], f, acc[i][j][x]);
          }
        wave_sync();
      }
  }
  // [wave][row of a][weight row], padded by four words a row
  constexpr int kRow = 16 * RT + 4, kTile = 16 * TT * kRow;
  float* const sums = reinterpret_cast<float*>(smem);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < TT; ++j)
      *reinterpret_cast<v4f*>(sums + wave * kTile + (j * 16 + (lane & 15)) * kRow + i * 16 + (lane >> 4) * 4) = acc[i][j];
  __syncthreads();
  using T = typename Elem<OUT>::T;
  constexpr int ALL = COLS * WN;
  for (int o = threadIdx.x; o < ALL * 16 * TT; o += 64 * WV) {
    const int r = o / ALL, c = wg0 + o % ALL;
    if (r >= unit.rows || c >= H) continue;
    const int64_t m = GROUPED ? row_of_out(a, unit.first + r) : unit.first + r;
    if (GROUPED && m < 0) continue;
    const float* p = sums + o % ALL / COLS * (WK * kTile) + r * kRow + o % COLS;
    float y = 0.0f, up = 0.0f;
#pragma unroll
    for (int v = 0; v < WK; ++v) {
      y += p[v * kTile];
      if (SWIGLU) up += p[v * kTile + 16];
    }
    if (a.bias) y += a.bias[c];
    if (SWIGLU) y = silu(y) * (a.bias ? up + a.bias[H + c] : up);
    if (a.add) y += to_f32<OUT>(static_cast<const T*>(a.add)[m * a.ldadd + c]);
    static_cast<T*>(a.out)[m * a.ldo + c] = from_f32<OUT>(y);
  }
}

// Eight values to 16-byte aligned memory.
template <int OUT>
__device__ __forceinline__ void store8(typename Elem<OUT>::T* p, const float (&y)[8]) {
  if constexpr (OUT == MOE_F32) {
    __builtin_memcpy(__builtin_assume_aligned(p, 16), y, 32);
  } else {
    typedef std::conditional_t<OUT == MOE_BF16, __bf16, _Float16> E;
    typedef E v8 __attribute__((ext_vector_type(8)));
    v8 v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = static_cast<E>(y[e]);
    *reinterpret_cast<v8*>(__builtin_assume_aligned(p, 16)) = v;
  }
}

// ----------------------------------------------------------- product: many rows
__device__ __forceinline__ void dma4s(v4i rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {  // 4 bytes a lane
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
               : "m0", "memory");
}

// Workgroup tile of BM rows of a x BN weight rows, WM x WN waves, each with TM x TN tiles of 16 x 16.  K goes
// through LDS in stages of one block, NS deep, by LDS DMA; with the stage come the scales of a's rows, while those of
// the weight's blocks lie in LDS from the start.  A row's 16-byte parts lie permuted by its index (as in
// the int8 product's tiles).  A wave holds its 64 weight rows for a whole block and takes its rows of a 16 at a
// time; as the last of them leaves the weight's registers the next block's rows follow.
//   8192 x 8192 x 8192 with tiles of 256 x 256: 508 us, 2.16 PFLOP/s (a library product without block scales 411).
// The DMA bounds it, 64 KB for 2048 cycles of products: without it 394 us, from L2-hot lines 450; the scaled sums take 36
// us, the products alone 292.  8192 x 7168 x 3584, SwiGLU: 217 us, 1.94 PFLOP/s, in four rounds of which the last is half
// empty.  Stages of 128 x 256 tiles fit three deep, but move 1.5 times the bytes (8192 x 8192 x 8192 607 us).
template <int BM, int BN, int WM, int WN, int NS, int OUT, bool SWIGLU, bool GROUPED, bool EXACT>
__global__ __launch_bounds__(64 * WM * WN, 1) void f8_tile_kernel(F8Args a, uint32_t nm, uint32_t nn, uint32_t per_xcd) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  constexpr int NW = WM * WN, kRows = (BM + BN) * 128, kStage = kRows + BM * 4;
  constexpr int RA = BM / 8 / NW, RW = BN / 8 / NW, kIssue = RA + RW + 1;  // DMAs of a wave: 8 rows each, and scales
  constexpr int TM = BM / WM / 16, TN = BN / WN / 16, kWaveRows = BN / WN;
  constexpr int NB = SWIGLU ? 2 : BN > 128 ? BN / 128 : 1;  // scale blocks of the weight
  static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0 && BM / 64 <= NW && TN % 2 == 0 && TM % 2 == 0 && kWaveRows == 64, "whole DMAs, whole blocks");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int H = SWIGLU ? a.N / 2 : a.N, KB = (a.K + 127) / 128, KBP = (KB + 63) / 64 * 64;
  constexpr int kLag = 2;     // a product is scaled and added behind the second one after it
  constexpr int kSpread = 4;  // a stage's DMAs go out in the first quarter of the time that they have
  constexpr int kCols = SWIGLU ? BN / 2 : BN;
  // each XCD (workgroups go round the eight) takes a contiguous range of tiles: what runs at once on an XCD
  // shares operands in its L2
  Unit unit;
  int n0;
  if constexpr (GROUPED) {
    const uint32_t units = count_units<BM>(a);  // (lists that overlap could have more than the grid was made for)
    const uint32_t tiles = (units < nm ? units : nm) * nn, per = (tiles + 7) / 8, tile = blockIdx.x % 8 * per + blockIdx.x / 8;
    if (blockIdx.x / 8 >= per || tile >= tiles || !find_unit<BM>(a, tile / nn, unit)) return;
    n0 = static_cast<int>(tile % nn) * kCols;
  } else {
    const uint32_t tile = blockIdx.x % 8 * per_xcd + blockIdx.x / 8;
    if (blockIdx.x / 8 >= per_xcd || tile >= nm * nn) return;
    const uint32_t band = tile / (8 * nn), left = nm - band * 8, height = left < 8 ? left : 8, in = tile - band * 8 * nn;
    unit.e = 0;
    unit.first = static_cast<int>(band * 8 + in % height) * BM;
    unit.rows = a.M - unit.first < BM ? a.M - unit.first : BM;
    n0 = static_cast<int>(in / height) * kCols;
  }
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) void*)smem));
  constexpr int kDummy = NS * kStage, kMap = kDummy + 256, kScales = kMap + BM * 4;
  int* const out_row = reinterpret_cast<int*>(smem + kMap);

  for (int r = threadIdx.x; r < BM; r += 64 * NW)
    out_row[r] = r >= unit.rows ? -1 : GROUPED ? static_cast<int>(row_of_out(a, unit.first + r)) : unit.first + r;
  auto place = [](int r, int c) { return c ^ ((r >> 1) & 7); };
  // what this lane moves: a part of row lane / 8 of its wave's blocks of 8 rows
  const bool gather = GROUPED && a.gather;
  const uint64_t base = gather ? 0 : static_cast<uint64_t>(unit.first);
  const uint32_t extent_rows = gather ? static_cast<uint32_t>(a.a_rows) : static_cast<uint32_t>(unit.rows);
  auto row_in = [&](int r) -> uint32_t {  // row r of the tile, counted from the base; behind the last: none
    if (r >= unit.rows) return ~0u;
    if (!gather) return static_cast<uint32_t>(r);
    return static_cast<uint32_t>(row_of_a(a, unit.first + r));
  };
  const v4i ra = make_rsrc(a.a + base * a.lda, static_cast<uint32_t>((extent_rows - 1) * a.lda + a.K));
  const v4i rs = make_rsrc(a.sa + base * a.ldsa, static_cast<uint32_t>(((extent_rows - 1) * a.ldsa + KB) * 4));
  // Of 32 columns, the one in row r of their two tiles: a lane's four rows of one tile and of the other are
  // neighbours.  (column_of(8 b + r) = column_of(8 b) + column_of(r) for r < 8.)
  auto column_of = [](int r) { return ((r >> 2) & 3) * 8 + (r >> 4) * 4 + (r & 3); };
  // parts of row r lie in the order place() gives, so that DMAs of even and of odd blocks of 8 rows differ: by 64 in k
  const int kpart = ((lane & 7) ^ (lane >> 4)) * 16;
  auto part_of = [&](int block) { return kpart ^ (block & 1) * 64; };
  uint32_t va[GROUPED ? RA : 2], vw[2], vs;
  if constexpr (GROUPED) {
#pragma unroll
    for (int i = 0; i < RA; ++i) {
      const uint32_t at = row_in((wave * RA + i) * 8 + (lane >> 3));
      va[i] = at != ~0u ? at * static_cast<uint32_t>(a.lda) + part_of(wave * RA + i) : kOutside;
    }
  } else {
    // (rows behind the last lie behind the extent)
#pragma unroll
    for (int i = 0; i < 2; ++i) va[i] = (lane >> 3) * static_cast<uint32_t>(a.lda) + part_of(wave * RA + i);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) vw[i] = column_of(lane >> 3) * static_cast<uint32_t>(a.ldw) + part_of(wave * RW + i);
  {
    const uint32_t at = wave < BM / 64 ? row_in(wave * 64 + lane) : ~0u;
    vs = at != ~0u ? at * static_cast<uint32_t>(a.ldsa) * 4u : kOutside;
  }
  const int nrows = H - n0 < kCols ? H - n0 : kCols;
  const uint8_t* const w = a.w + unit.e * a.ldwe + static_cast<int64_t>(n0) * a.ldw;
  const v4i rw = make_rsrc(w, static_cast<uint32_t>((nrows - 1) * a.ldw + a.K));
  const v4i ru = SWIGLU ? make_rsrc(w + static_cast<int64_t>(H) * a.ldw, static_cast<uint32_t>((nrows - 1) * a.ldw + a.K)) : rw;
  // What stage s adds to the offsets of even and of odd blocks: parts behind K, and whole stages behind it, are
  // outside, which makes them zeros (with no scalar offset then: nothing says that the bounds check's difference does
  // not wrap).
  struct Stage {
    uint32_t out[2], soff, scale;
    bool in;
  };
  auto stage = [&](int s) {
    const int left = a.K - s * 128;
    Stage r;
    r.in = left > 0;
    r.soff = r.in ? s * 128 : 0;
    r.scale = r.in ? s * 4 : 0;
    r.out[0] = kpart < left ? 0 : kOutside;
    r.out[1] = (kpart ^ 64) < left ? 0 : kOutside;
    return r;
  };
  // DMA d of this wave for a stage into the LDS at buf
  auto issue = [&](const Stage& s, int buf, int d) {
    if (d < RA) {
      const int block = wave * RA + d;
      uint32_t v;
      if constexpr (GROUPED) v = va[d];
      else v = va[d & 1] + static_cast<uint32_t>(block * 8) * static_cast<uint32_t>(a.lda);
      dma16(ra, v | s.out[block & 1], s.soff, lds0 + buf + block * 1024);
    } else if (d < RA + RW) {
      // SwiGLU: a wave's gate rows, then its up rows
      const int block = wave * RW + d - RA, slot = block * 8, half = SWIGLU ? slot / (kWaveRows / 2) & 1 : 0;
      const int row = (SWIGLU ? slot / kWaveRows * (kWaveRows / 2) + slot % (kWaveRows / 2) : slot) / 32 * 32 + column_of(slot % 32);
      const uint32_t v = vw[(d - RA) & 1] + static_cast<uint32_t>(row) * static_cast<uint32_t>(a.ldw);
      dma16(half ? ru : rw, v | s.out[block & 1], s.soff, lds0 + buf + BM * 128 + block * 1024);
    } else {
      dma4s(rs, s.in ? vs : kOutside, s.scale, lds0 + (wave < BM / 64 ? buf + kRows + wave * 256 : kDummy));
    }
  };

  using T = typename Elem<OUT>::T;
  const int wm = wave % WM * (BM / WM), wn = wave / WM * kWaveRows;
  using Op = Operand<EXACT>;
  const int la0 = (lane & 15) * 128 + place(lane & 15, lane >> 4) * 16, la1 = (lane & 15) * 128 + place(lane & 15, 4 + (lane >> 4)) * 16;
  auto operand = [&](int at) {
    return Op::make(*reinterpret_cast<const v4i*>(smem + at + la0), *reinterpret_cast<const v4i*>(smem + at + la1));
  };
  v4f acc[TN][TM] = {};
  // The weight rows of a block are held, and replaced by the next block's as the last tile leaves them; a's come 16 at
  // a time, a tile ahead.
  typename Op::T fa[2], fw[TN];
  float sa[2], sw[2];
  const float* const wscale = reinterpret_cast<const float*>(smem + kScales) + (SWIGLU ? 0 : wn / 128 * KBP);
  auto read_a = [&](int buf, int j) {
    fa[j & 1] = operand(buf + (wm + j * 16) * 128);
    sa[j & 1] = *reinterpret_cast<const float*>(smem + buf + kRows + (wm + j * 16 + (lane & 15)) * 4);
  };
  auto read_w = [&](int buf, int i) { fw[i] = operand(buf + (BM + wn + i * 16) * 128); };
  auto read_sw = [&](int s) {  // of the gate rows, and of the up rows
    s = s < KB ? s : KB - 1;
    sw[0] = wscale[s];
    if (SWIGLU) sw[1] = wscale[KBP + s];
  };
  // the weight's scales first
  {
    const int halves = SWIGLU ? 2 : 1, nb = (H + 127) / 128;
    for (int d = wave; d < NB * KBP / 64; d += NW) {
      const int h = d / (KBP / 64), k = d % (KBP / 64) * 64, block = n0 / 128 + (SWIGLU ? 0 : h);
      const int64_t row = (static_cast<int64_t>(unit.e) * halves + (SWIGLU ? h : 0)) * nb + (block < nb ? block : nb - 1);
      dma4(make_rsrc(a.sw + row * KB, static_cast<uint32_t>(KB) * 4u), k + lane < KB ? (k + lane) * 4u : kOutside,
           lds0 + kScales + (h * KBP + k) * 4);
    }
  }
  // a stage's DMAs are issued one by one behind the products that follow its buffer's release
  constexpr int kAll = TN * TM, kFree = (TM - 1) * TN;  // products of a block; those before the release
  auto slot = [](int q) { return q * kSpread * kIssue / kAll < kIssue ? q * kSpread * kIssue / kAll : kIssue; };
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const Stage st = stage(s);
#pragma unroll
    for (int d = 0; d < (s < NS - 1 ? kIssue : slot(kAll - kFree)); ++d) issue(st, s * kStage, d);
  }
  wait_vm<kIssue*(NS - 2) + slot(kAll - kFree)>();
  __builtin_amdgcn_s_barrier();
  compiler_fence();
#pragma unroll
  for (int i = 0; i < TN; ++i) read_w(0, i);
  read_sw(0);
  read_a(0, 0);
  int prev = (NS - 1) * kStage, cur = 0;  // LDS offsets of stages s - 1 and s
  for (int s = 0; s < KB; ++s) {
    const int next = cur + kStage == NS * kStage ? 0 : cur + kStage;
    Stage st = stage(s + NS - 1);
    v4f d[kLag + 1];
    float f[2], g[2];  // of the tile before and of this one
    auto add = [&](int m) {  // product m of the block
      const int j = m / TN, i = m % TN;
      const float x = SWIGLU && i >= TN / 2 ? g[j & 1] : f[j & 1];
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(d[m % (kLag + 1)][e], x, acc[i][j][e]);
    };
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      f[j & 1] = sa[j & 1] * sw[0];
      if (SWIGLU) g[j & 1] = sa[j & 1] * sw[1];
      if (j == TM - 1) {
        // this stage is read out (but for what the products to come hold) and the next has landed, for every wave
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        wait_vm<kIssue*(NS - 2)>();
        __builtin_amdgcn_s_barrier();
        compiler_fence();
        __builtin_amdgcn_sched_barrier(0);
        st = stage(s + NS);
        read_sw(s + 1);
        read_a(next, 0);
      } else {
        read_a(cur, j + 1);
      }
#pragma unroll
      for (int i = 0; i < TN; ++i) {
        const int m = j * TN + i, q = (m - kFree + kAll) % kAll;
        d[m % (kLag + 1)] = Op::product(fw[i], fa[j & 1]);
        __builtin_amdgcn_sched_barrier(0);
        if (j == TM - 1) read_w(next, i);
        if (m >= kLag) add(m - kLag);
#pragma unroll
        for (int x = slot(q); x < slot(q + 1); ++x) issue(st, m >= kFree ? cur : prev, x);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int m = kAll - kLag; m < kAll; ++m) add(m);
    prev = cur;
    cur = next;
    compiler_fence();
  }
  // A lane has eight neighbouring columns of each of its TM rows (column_of), 32 of a wave's columns at a time: 16
  // bytes straight to memory.  (By way of LDS, a whole row's 128 bytes at a time, the instructions took longer:
  // 16384 x 3584 x 384 68 us.)
  constexpr int kOut = SWIGLU ? kWaveRows / 2 : kWaveRows;
  const int nw0 = n0 + (SWIGLU ? wn / 2 : wn);
  const bool vec = (reinterpret_cast<uintptr_t>(a.out) | (a.ldo * sizeof(T))) % 16 == 0 &&
                   (!a.add || (reinterpret_cast<uintptr_t>(a.add) | (a.ldadd * sizeof(T))) % 16 == 0);
#pragma unroll
  for (int p = 0; p < kOut / 32; ++p) {
    const int col = nw0 + p * 32 + (lane >> 4) * 8;
    if (col >= H) continue;
    float b[8] = {}, bu[8] = {};
    if (a.bias) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        b[e] = col + e < H ? a.bias[col + e] : 0.0f;
        if (SWIGLU) bu[e] = col + e < H ? a.bias[H + col + e] : 0.0f;
      }
    }
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      const int64_t m = out_row[wm + j * 16 + (lane & 15)];
      if (m < 0) continue;
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[e] = acc[2 * p + e / 4][j][e % 4] + b[e];
        if (SWIGLU) y[e] = silu(y[e]) * (acc[TN / 2 + 2 * p + e / 4][j][e % 4] + bu[e]);
      }
      T* const out = static_cast<T*>(a.out) + m * a.ldo + col;
      const T* const add = static_cast<const T*>(a.add) + m * a.ldadd + col;
      if (vec && col + 8 <= H) {
        if (a.add) {
          T v[8];
          __builtin_memcpy(v, __builtin_assume_aligned(add, 16), sizeof(v));
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] += to_f32<OUT>(v[e]);
        }
        store8<OUT>(out, y);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (col + e < H) out[e] = from_f32<OUT>(a.add ? y[e] + to_f32<OUT>(add[e]) : y[e]);
      }
    }
  }
  wait_vm<0>();  // (the last stages' DMAs, zeros, have to land before the LDS is another workgroup's)
}

// ---------------------------------------------------------------------- host
template <int OUT, bool SWIGLU, bool GROUPED, bool EXACT, int RT, int TT, int WV, int WK = WV>
int launch_stream(const F8Args& a, hipStream_t st) {
  static std::atomic<uint64_t> done{0};
  constexpr size_t lds = WV * std::max(2048 * (RT + TT), 64 * TT * (16 * RT + 4));
  static_assert(lds <= 160 * 1024, "LDS of a CU");
  if (!allow_lds(f8_stream_kernel<OUT, SWIGLU, GROUPED, EXACT, RT, TT, WV, WK>, lds, done)) return hip_failed();
  const int64_t cols = SWIGLU ? a.N / 2 : a.N, per = (SWIGLU ? 16 : 16 * RT) * (WV / WK), nx = (cols + per - 1) / per;
  constexpr int BM = 16 * TT;
  // grouped: the experts' last runs may be short
  const int64_t units = GROUPED ? (a.M + static_cast<int64_t>(std::min(a.E, a.M)) * (BM - 1)) / BM : (a.M + BM - 1) / BM;
  if (nx * units * (64 * WV) >> 32) return MOE_EINVAL;  // (threads of a launch)
  return launch(f8_stream_kernel<OUT, SWIGLU, GROUPED, EXACT, RT, TT, WV, WK>, static_cast<uint32_t>(nx * units), 64 * WV, lds, st, a,
                static_cast<uint32_t>(nx));
}

template <int BM, int BN, int WM, int WN, int NS, int OUT, bool SWIGLU, bool GROUPED, bool EXACT>
int launch_tile(const F8Args& a, hipStream_t st) {
  static std::atomic<uint64_t> done{0};
  constexpr int NB = SWIGLU ? 2 : BN > 128 ? BN / 128 : 1;
  constexpr size_t fixed = NS * ((BM + BN) * 128 + BM * 4) + 256 + BM * 4, most = fixed + NB * 512 * 4;  // K <= 65536
  static_assert(most <= 160 * 1024, "LDS of a CU");
  if (!allow_lds(f8_tile_kernel<BM, BN, WM, WN, NS, OUT, SWIGLU, GROUPED, EXACT>, most, done)) return hip_failed();
  const size_t lds = fixed + NB * static_cast<size_t>((a.K + 8191) / 8192 * 64) * 4;
  const int64_t bn = SWIGLU ? BN / 2 : BN, nn = ((SWIGLU ? a.N / 2 : a.N) + bn - 1) / bn;
  const int64_t nm = GROUPED ? (a.M + static_cast<int64_t>(std::min(a.E, a.M)) * (BM - 1)) / BM : (a.M + BM - 1) / BM;
  const int64_t groups = (nm * nn + 7) / 8 * 8;
  if (groups * (64 * WM * WN) >> 32) return MOE_EINVAL;  // (threads of a launch)
  const uint32_t per = static_cast<uint32_t>(groups / 8);
  return launch(f8_tile_kernel<BM, BN, WM, WN, NS, OUT, SWIGLU, GROUPED, EXACT>, per * 8, 64 * WM * WN, lds, st, a, static_cast<uint32_t>(nm),
                static_cast<uint32_t>(nn), per);
}

template <int OUT, bool SWIGLU, bool GROUPED, bool EXACT>
int launch_product(const F8Args& a, hipStream_t st) {
  constexpr int R1 = SWIGLU ? 2 : 1;
  const int64_t rows = GROUPED ? (a.M + std::min(a.E, a.M) - 1) / std::min(a.E, a.M) : a.M;  // that share a weight
  const int64_t cols = SWIGLU ? a.N / 2 : a.N;
  auto tiles = [&](int bm, int bn) {
    const int64_t b = SWIGLU ? bn / 2 : bn;
    // (grouped: as if the experts had equal shares)
    return (GROUPED ? std::min(a.E, a.M) * ((rows + bm - 1) / bm) : (a.M + bm - 1) / bm) * ((cols + b - 1) / b);
  };
  const int64_t n0 = tiles(64, 128), met = GROUPED ? std::min(a.E, a.M) : 1;
  const bool shallow = a.K <= 1024;  // few blocks of K: nothing to split among waves, little to keep in flight
  // The streaming kernel where the smallest tiles leave CUs idle, or hardly any row shares a weight.  Experts of 3584 x
  // 384 (160, 16 a token) took, us: both products of one token 12 and 6 with it, 19 and 7 with tiles; of 8 tokens 58 and
  // 27, 41 and 29; of 50 tokens 115 and 49, 79 and 47.
  if (shallow && rows <= 4 && met * (a.N / 32) >= 1024) return launch_stream<OUT, SWIGLU, GROUPED, EXACT, 2, 1, 4, 1>(a, st);
  if (rows <= 64 && n0 < 256) {
    if (rows <= 16) {
      if constexpr (GROUPED) return launch_stream<OUT, SWIGLU, true, EXACT, 2, 1, 8, 4>(a, st);
      else return launch_stream<OUT, SWIGLU, false, EXACT, R1, 1, SWIGLU && EXACT ? 8 : 16>(a, st);
    }
    if constexpr (!EXACT)  // (four row tiles of BF16 operands do not fit the registers)
      if (rows > 32) return launch_stream<OUT, SWIGLU, GROUPED, false, 2, 4, 8>(a, st);
    return launch_stream<OUT, SWIGLU, GROUPED, EXACT, R1, 2, 8>(a, st);
  }
  // Rounds of tiles over 256 CUs, weighed with a round's time at K = 4096 (us): large tiles move fewer bytes for each
  // product, small ones fill the CUs.  The order holds for short K too (experts' second product, K = 384, 16 a token, with
  // 64 x 128, 128 x 128, 128 x 256, 256 x 256, us: 512 tokens 74, 114, 88, 99; 2048 232, 236, 182, 159; 8192 745, 748, 629, 555).  Two or three of the smallest fit a CU.  Exact sums take some 1.56 times as long with
  // each of the first three (8192 x 7168 x 3584, SwiGLU: 365 to 376 us, against 217 with tiles of 256 x 256, whose BF16
  // operands do not fit the registers; 128 x 128 454).
  const int64_t c0 = n0 <= 256 ? 20 : (n0 + 511) / 512 * 25, c1 = (tiles(128, 128) + 255) / 256 * 24,
                c2 = (tiles(128, 256) + 255) / 256 * 39, c3 = (tiles(256, 256) + 255) / 256 * 65;
  if (std::min(c0, c1) <= (EXACT ? c2 : std::min(c2, c3))) {
    if (c0 < c1) {
      // two stages: three workgroups a CU (50 tokens' second product 47 us, against 53 with three stages and two
      // workgroups; their first one 94 against 79, 8 tokens' first one, 540 tiles, 41 against 48).  Exact sums have
      // registers for two workgroups only (that one 72 us with two stages, 68 with three)
      if constexpr (!EXACT)
        if (shallow || (n0 > 512 && n0 <= 768)) return launch_tile<64, 128, 2, 2, 2, OUT, SWIGLU, GROUPED, false>(a, st);
      return launch_tile<64, 128, 2, 2, 3, OUT, SWIGLU, GROUPED, EXACT>(a, st);
    }
    return launch_tile<128, 128, 4, 2, 4, OUT, SWIGLU, GROUPED, EXACT>(a, st);
  }
  if constexpr (!EXACT)
    if (c2 >= c3) return launch_tile<256, 256, 2, 4, 2, OUT, SWIGLU, GROUPED, false>(a, st);
  return launch_tile<128, 256, 2, 4, 3, OUT, SWIGLU, GROUPED, EXACT>(a, st);
}
template <int OUT, bool SWIGLU, bool GROUPED>
int launch_product(const F8Args& a, bool exact, hipStream_t st) {
  if constexpr (OUT != MOE_F32)
    if (!exact) return launch_product<OUT, SWIGLU, GROUPED, false>(a, st);
  return launch_product<OUT, SWIGLU, GROUPED, true>(a, st);
}
template <bool GROUPED>
int launch_product(const F8Args& a, int32_t out_type, bool swiglu, bool exact, hipStream_t st) {
  auto to = [&](auto act) {
    constexpr bool SWIGLU = decltype(act)::value;
    if (out_type == MOE_F32) return launch_product<MOE_F32, SWIGLU, GROUPED>(a, true, st);
    if (out_type == MOE_F16) return launch_product<MOE_F16, SWIGLU, GROUPED>(a, exact, st);
    return launch_product<MOE_BF16, SWIGLU, GROUPED>(a, exact, st);
  };
  return swiglu ? to(std::true_type()) : to(std::false_type());
}

constexpr int64_t kMaxLd = 1 << 22, kMaxRoutes = 1 << 26;
uint32_t list_groups(int64_t R) {  // workgroups: 4096 routes each, 256 at most
  return static_cast<uint32_t>(R <= kListOne ? 1 : std::min<int64_t>((R + 4095) / 4096, 256));
}
bool product_ok(const void* a, int64_t lda, const float* sa, int64_t ldsa, const void* w, int64_t ldw, const float* sw, int32_t N,
                int32_t K, int32_t act, int32_t exact, const void* out, int32_t out_type, int64_t ldo) {
  return a && sa && w && sw && out && type_ok(out_type) && N >= 1 && N <= 1 << 20 && K >= 16 && K <= 65536 && lda >= K && ldw >= K &&
         lda < kMaxLd && ldw < kMaxLd && ldsa < kMaxLd / 4 && ldsa >= (K + 127) / 128 && act >= 0 && act <= 1 && exact >= 0 && exact <= 1 &&
         !(act == 1 && N % 2) && ldo >= (act == 1 ? N / 2 : N) &&
         (reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(w) | lda | ldw | static_cast<uintptr_t>(K)) % 16 == 0;
}

}  // namespace

extern "C" {

size_t moe_lists_ws_bytes(int64_t R, int32_t E) {
  if (R < 1 || R > kMaxRoutes || E < 1 || E > 1024 || R <= kListOne) return 0;
  return static_cast<size_t>(list_groups(R)) * E * 4;
}

int moe_lists(const int32_t* ids, int64_t R, int32_t E, int32_t* offsets, int32_t* pairs, void* ws, size_t ws_bytes, void* stream) {
  if (!ids || !offsets || !pairs || R < 1 || R > kMaxRoutes || E < 1 || E > 1024) return MOE_EINVAL;
  const size_t need = moe_lists_ws_bytes(R, E);
  if (need && (!ws || reinterpret_cast<uintptr_t>(ws) % 4)) return MOE_EINVAL;
  if (ws_bytes < need) return MOE_ENOSPACE;
  const uint32_t groups = list_groups(R);
  const int64_t waves = static_cast<int64_t>(groups) * kListWaves, share = ((R + waves - 1) / waves + 63) / 64 * 64;
  const ListArgs a = {ids, offsets, pairs, static_cast<uint32_t*>(ws), static_cast<uint32_t>(R), static_cast<uint32_t>(E),
                      static_cast<uint32_t>(share)};
  hipStream_t st = as_stream(stream);
  static std::atomic<uint64_t> done{0};
  const size_t lds = (static_cast<size_t>(kListWaves) * (E + 1) + 2 * E) * 4;
  if (lds > 65536 && !allow_lds(lists_place_kernel, (static_cast<size_t>(kListWaves) * 1025 + 2048) * 4, done)) return hip_failed();
  if (groups > 1) {
    const int r = launch(lists_count_kernel, groups, kListThreads, E * 4, st, a);
    if (r != MOE_OK) return r;
  }
  return launch(lists_place_kernel, groups, kListThreads, lds, st, a);
}

int moe_linear_f8(const uint8_t* a, int64_t lda, const float* sa, int64_t ldsa, const uint8_t* w, int64_t ldw, const float* sw,
                  int32_t M, int32_t N, int32_t K, const moe_linear_opts_t* opts, void* out, int32_t out_type, int64_t ldo,
                  void* stream) {
  moe_linear_opts_t o;
  std::memset(&o, 0, sizeof(o));
  if (opts) o = *opts;
  if (!product_ok(a, lda, sa, ldsa, w, ldw, sw, N, K, o.act, o.exact, out, out_type, ldo) || M < 1 || M > kMaxRows ||
      static_cast<int64_t>(M) * N > 1LL << 34 || (o.add_dev && o.ldadd < (o.act == 1 ? N / 2 : N)))
    return MOE_EINVAL;
  F8Args r = {a, w, sa, sw, o.bias_dev, o.add_dev, out, nullptr, nullptr, lda, ldw, 0, ldsa, ldo, o.ldadd, M, M, M, N, K, 1, 0, 0};
  return launch_product<false>(r, out_type, o.act == 1, o.exact == 1, as_stream(stream));
}

int moe_grouped_f8(const uint8_t* a, int64_t lda, const float* sa, int64_t ldsa, int64_t a_rows, const uint8_t* w, int64_t ldw,
                   int64_t ldwe, const float* sw, const int32_t* offsets, int64_t R, int32_t E, int32_t N, int32_t K,
                   const moe_grouped_opts_t* opts, void* out, int32_t out_type, int64_t ldo, int64_t out_rows, void* stream) {
  moe_grouped_opts_t o;
  std::memset(&o, 0, sizeof(o));
  if (opts) o = *opts;
  if (!product_ok(a, lda, sa, ldsa, w, ldw, sw, N, K, o.act, o.exact, out, out_type, ldo) || !offsets || R < 1 || R > kMaxRoutes || E < 1 ||
      E > 1024 || R * N > 1LL << 40 || o.gather < 0 || o.scatter < 0 || o.scatter > 1 ||
      ldwe < (static_cast<int64_t>(N) - 1) * ldw + K || ldwe % 16 || a_rows < 1 || out_rows < 1)
    return MOE_EINVAL;
  if (o.gather || o.scatter ? !o.pairs_dev : o.pairs_dev != nullptr) return MOE_EINVAL;
  if (o.gather ? a_rows > 1LL << 26 || a_rows * lda >= 1LL << 31 || a_rows * ldsa >= 1LL << 29 : a_rows < R) return MOE_EINVAL;
  if (!o.scatter && out_rows < R) return MOE_EINVAL;
  F8Args r = {a,    w,    sa,  sw,      nullptr, nullptr, out,      offsets,
              o.pairs_dev, lda, ldw,    ldwe,    ldsa,    ldo,      0,       a_rows, out_rows, static_cast<int32_t>(R), N, K, E, o.gather, o.scatter};
  return launch_product<true>(r, out_type, o.act == 1, o.exact == 1, as_stream(stream));
}

}  // extern "C"
