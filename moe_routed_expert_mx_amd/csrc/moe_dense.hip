// moe_dense.hip -- MI355X (gfx950) kernels of the dense side of a routed-experts layer: the
// router in front of the experts (product and top-k choice) and the int8 products of a
// shared expert beside them, behind the C ABI of include/moe_mx.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "moe_mx.h"

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

__device__ __forceinline__ void compiler_fence() { asm volatile("" ::: "memory"); }

// ------------------------------------------------------------------ elements
__device__ __forceinline__ float bf16_to_f32(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }
__device__ __forceinline__ float f16_to_f32(uint16_t b) {
  _Float16 h;
  __builtin_memcpy(&h, &b, 2);
  return static_cast<float>(h);
}
// binary32 -> bf16, round to nearest even; NaN stays NaN.
__device__ __forceinline__ uint16_t f32_to_bf16(float f) {
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return static_cast<uint16_t>((u >> 16) | 0x40u);
  return static_cast<uint16_t>((u + 0x7fffu + ((u >> 16) & 1u)) >> 16);
}
__device__ __forceinline__ uint16_t f32_to_f16(float f) {
  const _Float16 h = static_cast<_Float16>(f);
  uint16_t b;
  __builtin_memcpy(&b, &h, 2);
  return b;
}

template <int TYPE>
struct Elem {
  using T = uint16_t;
};
template <>
struct Elem<MOE_F32> {
  using T = float;
};
template <int TYPE>
__device__ __forceinline__ float to_f32(typename Elem<TYPE>::T v) {
  if constexpr (TYPE == MOE_F32) return v;
  else if constexpr (TYPE == MOE_F16) return f16_to_f32(v);
  else return bf16_to_f32(v);
}
template <int TYPE>
__device__ __forceinline__ typename Elem<TYPE>::T from_f32(float v) {
  if constexpr (TYPE == MOE_F32) return v;
  else if constexpr (TYPE == MOE_F16) return f32_to_f16(v);
  else return f32_to_bf16(v);
}

constexpr size_t elem_size(int type) { return type == MOE_F32 ? 4 : 2; }

// --------------------------------------------------------------------- route
struct RouteArgs {
  const void* logits;
  int64_t ldl;
  int32_t B, E, topk, sigmoid, groups, kept, sums, renorm;
  float scale;
  const float* bias;
  int32_t* ids;
  float* weights;
};

// Order between the lanes of one wave through LDS.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}
template <int N>
__device__ __forceinline__ uint32_t rotate_row(uint32_t v) {  // among 16 lanes
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x120 + N, 0xf, 0xf, false));
}
template <int LPT>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  auto up = [&](uint32_t o) { v = o > v ? o : v; };
  up(rotate_row<8>(v));
  up(rotate_row<4>(v));
  up(rotate_row<2>(v));
  up(rotate_row<1>(v));
  if constexpr (LPT == 64) {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 64; i += 16) {
      const uint32_t o = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), i));
      r = o > r ? o : r;
    }
    return r;
  }
  return v;
}
template <int LPT>
__device__ __forceinline__ double lanes_sum(double v) {
  auto add = [&](auto turn) {
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v));
    const uint64_t o = static_cast<uint64_t>(turn(static_cast<uint32_t>(u >> 32))) << 32 | turn(static_cast<uint32_t>(u));
    v += __longlong_as_double(static_cast<int64_t>(o));
  };
  add([](uint32_t w) { return rotate_row<8>(w); });
  add([](uint32_t w) { return rotate_row<4>(w); });
  add([](uint32_t w) { return rotate_row<2>(w); });
  add([](uint32_t w) { return rotate_row<1>(w); });
  if constexpr (LPT == 64) {
    double r = 0.0;
#pragma unroll
    for (int i = 0; i < 64; i += 16) {
      const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v));
      const uint32_t hi = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(u >> 32), i));
      const uint32_t lo = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(u), i));
      r += __longlong_as_double(static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo));
    }
    return r;
  }
  return v;
}
// Bits of a number as an unsigned word that orders as the number does.
__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t u = __float_as_uint(f);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u ^ (u >> 31 ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint64_t ordered(double f) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(f));
  return u ^ (static_cast<uint64_t>(static_cast<int64_t>(u) >> 63) | 0x8000000000000000ull);
}
// exp within about a step: 2^n exp(r), |r| <= ln(2) / 2, exp(r) by its series to r^13 / 13!
// (the next term is below 2^-57).
__device__ __forceinline__ double exp_f64(double x) {
  x = __builtin_fmin(__builtin_fmax(x, -800.0), 800.0);
  const double n = __builtin_rint(x * 1.4426950408889634);
  double r = __builtin_fma(n, -2977044471.0 / 4294967296.0, x);  // ln 2 cut at 2^-32: n times it is exact
  r = __builtin_fma(n, -1.9082149292705877e-10, r);  // and the rest
  double p = 1.0 / 6227020800.0;
  p = __builtin_fma(p, r, 1.0 / 479001600.0);
  p = __builtin_fma(p, r, 1.0 / 39916800.0);
  p = __builtin_fma(p, r, 1.0 / 3628800.0);
  p = __builtin_fma(p, r, 1.0 / 362880.0);
  p = __builtin_fma(p, r, 1.0 / 40320.0);
  p = __builtin_fma(p, r, 1.0 / 5040.0);
  p = __builtin_fma(p, r, 1.0 / 720.0);
  p = __builtin_fma(p, r, 1.0 / 120.0);
  p = __builtin_fma(p, r, 1.0 / 24.0);
  p = __builtin_fma(p, r, 1.0 / 6.0);
  p = __builtin_fma(p, r, 0.5);
  p = __builtin_fma(p, r, 1.0);
  p = __builtin_fma(p, r, 1.0);
  return __builtin_ldexp(p, static_cast<int>(n));
}

// LPT lanes per token, lane l of them holding experts l, l + LPT, ..., NV of them at most.  Each
// lane sorts its choices (stably, so that equal ones stay in index order) into LDS; then the
// lanes' heads compete topk times: the largest upper word by rotations among the lanes, and
// only where several lanes share it the lower word and the index.  For many tokens vector
// instructions bound it (463 a token with 160 experts in 10 groups, top 16: 20.4 us for 16384
// tokens), and in part LDS: the ranking of groups reads runs of experts that lie on the same banks
// (69 % of the LDS cycles are conflicts).  The choice in FP64 is a small part of the instructions: a
// contest in FP32 first, FP64 only for waves whose result it cannot tell, was no faster (16384
// tokens with bias and groups 23 us against 20.7) and much slower for few tokens, whose slowest
// wave counts.
template <int TYPE, int LPT, int NV>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs a) {
  constexpr int TPW = 64 / LPT;
  __shared__ uint64_t lds_key[4][NV + 1][64];  // behind a lane's last choice, one that never wins
  __shared__ uint16_t lds_id[4][NV + 1][64];
  __shared__ uint16_t lds_out[4][TPW][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = lane % LPT, sub = lane / LPT;
  const int64_t tok = (static_cast<int64_t>(blockIdx.x) * 4 + wave) * TPW + sub, t = tok < a.B ? tok : a.B - 1;
  const float kMasked = -__builtin_huge_valf();
  // a masked expert's choice: below every other, FP32 or the sum of two; -inf: not there at all
  const double kNone = -1e300;
  const typename Elem<TYPE>::T* const row = static_cast<const typename Elem<TYPE>::T*>(a.logits) + t * a.ldl;
  auto logit_at = [&](int e) {
    const float v = to_f32<TYPE>(row[e]);
    return v == v ? v : kMasked;
  };
  // the selected experts' logits: few tokens wait less for LDS, many take less of it
  constexpr bool kKeep = LPT == 64;
  __shared__ float lds_logit[kKeep ? 4 : 1][kKeep ? NV : 1][64];
  float x[NV], bias[NV], m = kMasked;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = l + LPT * j;
    x[j] = e < a.E ? logit_at(e) : kMasked;
    bias[j] = a.bias && e < a.E ? a.bias[e] : 0.0f;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if constexpr (kKeep) lds_logit[wave][j][lane] = x[j];
    m = fmaxf(m, x[j]);
  }
  m = unordered(lanes_max<LPT>(ordered(m)));
  auto score_of = [&](float v) -> double {  // softmax: without the common denominator
    if (v == kMasked) return 0.0;
    if (a.sigmoid) return 1.0 / (1.0 + exp_f64(-static_cast<double>(v)));
    return v == m ? 1.0 : exp_f64(static_cast<double>(v) - static_cast<double>(m));
  };
  const bool scored = a.bias || (a.groups && a.sums);  // else the choice is the logit
  const int size = a.groups ? a.E / a.groups : 1;
  const uint32_t per = (1u << 22) / static_cast<uint32_t>(size) + 1;  // e / size = e * per >> 22, as e * size < 2^22

  // kept groups of this token, from the experts' values vals[0 .. E) in LDS
  auto keep_groups = [&](double* vals) -> uint64_t {
    double v1 = kNone, v2 = kNone;
    wave_sync();
    if (l < a.groups)
#pragma unroll 8
      for (int i = 0; i < size; ++i) {
        const double v = vals[l * size + i];
        v2 = v > v1 ? v1 : v > v2 ? v : v2;
        v1 = v > v1 ? v : v1;
      }
    const double r = a.sums && v2 != kNone ? v1 + v2 : v1;
    wave_sync();
    if (l < a.groups) vals[l] = r;
    wave_sync();
    int before = 0;
#pragma unroll 4
    for (int g = 0; g < a.groups; ++g) {
      const double o = vals[g];
      before += o > r || (o == r && g < l);
    }
    wave_sync();
    return __ballot(l < a.groups && before < a.kept) >> (LPT == 64 ? 0 : sub * LPT);
  };

  double c[NV], inv = 1.0;  // scores
  if (scored) {
#pragma unroll
    for (int j = 0; j < NV; ++j) c[j] = score_of(x[j]);
  }
  if (!a.sigmoid && (a.bias || !a.renorm)) {
    double d = 0.0;
#pragma unroll
    for (int j = 0; j < NV; ++j) d += scored ? c[j] : score_of(x[j]);
    d = lanes_sum<LPT>(d);
    inv = d > 0.0 ? 1.0 / d : 1.0;  // 0: every expert masked
  }
  double choice[NV];
  double* const vals = reinterpret_cast<double*>(lds_key[wave]) + sub * a.E;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = l + LPT * j;
    double v = x[j];
    if (a.bias) v = c[j] * inv + static_cast<double>(bias[j]);
    if (x[j] == kMasked || !(v > kNone)) v = kNone;
    if (a.groups && e < a.E) vals[e] = scored && !a.bias && v != kNone ? c[j] : v;
    choice[j] = e < a.E ? v : -__builtin_huge_val();
  }
  if (a.groups) {
    const uint64_t kept = keep_groups(vals);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e = l + LPT * j;
      if (e < a.E && !((kept >> (static_cast<uint32_t>(e) * per >> 22)) & 1)) choice[j] = -__builtin_huge_val();
    }
  }
  uint32_t id[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) id[j] = l + LPT * j;
#pragma unroll
  for (int round = 0; round < NV; ++round)
#pragma unroll
    for (int j = round & 1; j + 1 < NV; j += 2) {
      const bool swap = choice[j] < choice[j + 1];  // neighbours only: equal ones keep their order
      const double c0 = choice[j], c1 = choice[j + 1];
      const uint32_t i0 = id[j], i1 = id[j + 1];
      choice[j] = swap ? c1 : c0;
      choice[j + 1] = swap ? c0 : c1;
      id[j] = swap ? i1 : i0;
      id[j + 1] = swap ? i0 : i1;
    }
  uint64_t key[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) key[j] = ordered(choice[j] + 0.0);  // one zero
  constexpr bool kShort = NV <= 4;  // stays in registers
  if constexpr (!kShort) {
#pragma unroll
    for (int j = 1; j < NV; ++j) {
      lds_key[wave][j][lane] = key[j];
      lds_id[wave][j][lane] = static_cast<uint16_t>(id[j]);
    }
    lds_key[wave][NV][lane] = 0;
    lds_id[wave][NV][lane] = 0;
  }
  uint64_t head = key[0];
  uint32_t head_id = id[0];
  int next = 1;
  for (int k = 0; k < a.topk; ++k) {
    const uint32_t hi = static_cast<uint32_t>(head >> 32), lo = static_cast<uint32_t>(head);
    bool win = hi == lanes_max<LPT>(hi);
    // (the maxima are taken by all lanes, outside any condition on `win`)
    if (__popcll(__ballot(win)) != TPW) {
      const uint32_t top = lanes_max<LPT>(win ? lo : 0u);
      win &= lo == top;
      if (__popcll(__ballot(win)) != TPW) {
        const uint32_t first = lanes_max<LPT>(win ? ~head_id : 0u);
        win &= ~head_id == first;
      }
    }
    if (win) {
      lds_out[wave][sub][k] = static_cast<uint16_t>(head_id);
      if constexpr (kShort) {
        head = key[1];
        head_id = id[1];
#pragma unroll
        for (int j = 1; j < NV; ++j) {
          key[j] = j + 1 < NV ? key[j + 1] : 0;
          id[j] = j + 1 < NV ? id[j + 1] : 0;
        }
      } else {
        head = lds_key[wave][next][lane];
        head_id = lds_id[wave][next][lane];
        ++next;
      }
    }
  }
  wave_sync();
  constexpr int KP = 64 / LPT;  // selected experts per lane
  double w[KP], total = 0.0;
#pragma unroll
  for (int i = 0; i < KP; ++i) {
    const int k = l + LPT * i;
    w[i] = 0.0;
    if (k < a.topk) {
      const int e = lds_out[wave][sub][k];
      if constexpr (kKeep) w[i] = score_of(lds_logit[wave][e / LPT][e % LPT]);
      else w[i] = score_of(logit_at(e));
      if (tok < a.B) a.ids[t * a.topk + k] = e;
    }
    total += w[i];
  }
  if (a.renorm) {
    total = lanes_sum<LPT>(total);
    inv = total > 0.0 ? 1.0 / total : 0.0;
  }
#pragma unroll
  for (int i = 0; i < KP; ++i) {
    const int k = l + LPT * i;
    if (k < a.topk && tok < a.B) a.weights[t * a.topk + k] = static_cast<float>(w[i] * inv * static_cast<double>(a.scale));
  }
}

// --------------------------------------------------------------------- quant
// code = x * 127 / amax, half to even, exactly.
//
// The quick way adds 1.5 * 2^23 to x * inv in one rounding, inv = 127 / amax rounded up by a step or
// two: the sum's low byte is the code, unless the exact quotient is (16-bit types) or may be
// (FP32) a half.
//   BF16, FP16: with significands of at most 11 bits, X and A, x / amax = X / (A 2^j).  A quotient q that
// is no half lies |254 X - (2 k + 1) A 2^j| / (A 2^(j + 1)) from k + 1/2, the numerator being 1 or
// more: q / (254 X), above q 2^-19 (closest: A = 2033, X = 2025, j = 0).  inv's error moves q by
// q 2^-22 at most.  A half, (2 k + 1) amax = 254 x, needs 127 to divide amax's significand, or
// 2 k + 1 = 127, x = amax / 2, code 64: inv being high, that one comes out right.
//   FP32: within 2^-14 of a half, the exact way decides.
// Rows with an amax that 127 divides (16-bit types), or below 2^-100, go the exact way: by the
// remainder x * 127 - r * amax in FP64, x and amax first scaled by a power of two.
struct QuantScale {
  int exp;
  float amax, inv;  // scaled; 127 / amax
};
__device__ __forceinline__ int quant_exact(float x, const QuantScale& q) {
  const float xs = __builtin_ldexpf(x, -q.exp);  // exact but for values whose code is 0
  const double n = static_cast<double>(xs) * 127.0, amax = static_cast<double>(q.amax);
  const float r0 = __builtin_rintf(xs * q.inv);
  const double d = 2.0 * __builtin_fma(-static_cast<double>(r0), amax, n), far = __builtin_fabs(d);
  const int r = static_cast<int>(r0);
  return far > amax || (far == amax && (r & 1)) ? r + (d > 0.0 ? 1 : -1) : r;
}

// W waves per token, which they hold in registers: NV 16-byte pieces a lane (NV 0: any length,
// the row is read twice).  One pass over the data: bytes bound it (8192 x 3584 BF16: 88 MB, 17 us
// at a copy's rate), so an element may cost few instructions: four, with the quick way (15 made
// it 23.5 us).
template <int TYPE, int W, int NV>
__global__ __launch_bounds__(256) void quant_kernel(const void* x, int64_t ldx, int32_t M, int32_t K,
                                                    int8_t* codes, int64_t ldc, float* scales) {
  using T = typename Elem<TYPE>::T;
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  constexpr int VE = 16 / sizeof(T), HELD = NV ? NV : 1;
  constexpr float kMagic = 12582912.0f;
  __shared__ uint32_t part[4];
  const int lane = threadIdx.x % (64 * W), wave = threadIdx.x >> 6;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (4 / W) + threadIdx.x / (64 * W);
  if (W == 1 && row >= M) return;
  const T* p = static_cast<const T*>(x) + row * ldx;
  int8_t* q = codes + row * ldc;
  const int pieces = (K + VE - 1) / VE;
  struct Piece {
    uint32_t w[4];
    __device__ __forceinline__ float at(int e) const {
      if constexpr (TYPE == MOE_F32) return __uint_as_float(w[e]);
      else return to_f32<TYPE>(static_cast<uint16_t>(e & 1 ? w[e >> 1] >> 16 : w[e >> 1]));
    }
  };
  auto load = [&](int i) {  // any alignment; zeros behind K
    Piece r;
    if ((i + 1) * VE <= K) {
      __builtin_memcpy(&r, p + i * VE, 16);
    } else {
      T v[VE];
#pragma unroll
      for (int e = 0; e < VE; ++e) v[e] = i * VE + e < K ? p[i * VE + e] : T(0);
      __builtin_memcpy(&r, v, 16);
    }
    return r;
  };
  // magnitudes order as their bits, infinity and NaN above all
  uint32_t top = 0;
  u16x2 top2 = {0, 0};
  auto raise = [&](const Piece& r) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (TYPE == MOE_F32) {
        const uint32_t b = r.w[i] & 0x7fffffffu;
        top = b > top ? b : top;
      } else {
        u16x2 b;
        const uint32_t u = r.w[i] & 0x7fff7fffu;
        __builtin_memcpy(&b, &u, 4);
        top2 = __builtin_elementwise_max(top2, b);
      }
    }
  };
  Piece held[HELD];
  if constexpr (NV > 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = lane + 64 * W * j;
      if (i < pieces) held[j] = load(i);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (lane + 64 * W * j < pieces) raise(held[j]);
  } else {
    for (int i = lane; i < pieces; i += 64 * W) raise(load(i));
  }
  if constexpr (TYPE != MOE_F32) top = top2[0] > top2[1] ? top2[0] : top2[1];
  top = lanes_max<64>(top);
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) part[wave] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) top = part[i] > top ? part[i] : top;
  }
  float amax;
  if constexpr (TYPE == MOE_F32) amax = __uint_as_float(top);
  else amax = to_f32<TYPE>(static_cast<uint16_t>(top));
  const bool finite = (__float_as_uint(amax) & 0x7fffffffu) < 0x7f800000u, some = top != 0 && finite;
  const uint32_t significand = (__float_as_uint(amax) & 0x7fffffu) | 0x800000u;
  const bool quick = some && amax >= 0x1p-100f && (TYPE == MOE_F32 || significand % 127 != 0);
  QuantScale s = {0, 1.0f, 0.0f};
  if (some && (!quick || TYPE == MOE_F32)) {
    s.exp = __builtin_amdgcn_frexp_expf(amax) - 1;
    s.amax = __builtin_ldexpf(amax, -s.exp);
    s.inv = 127.0f / s.amax;
  }
  const float inv = quick ? __uint_as_float(__float_as_uint(127.0f / amax) + 1) : 0.0f;
  auto store = [&](int i, const Piece& r) {
    uint32_t c[VE / 4] = {};
    bool redo = some && !quick;
    if (quick) {
#pragma unroll
      for (int g = 0; g < VE / 4; ++g) {
        uint32_t b[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float v = r.at(4 * g + e), y = __builtin_fmaf(v, inv, kMagic);
          b[e] = __float_as_uint(y);
          if constexpr (TYPE == MOE_F32)
            redo |= __builtin_fabsf(__builtin_fmaf(v, inv, kMagic - y)) >= 0.5f - 0x1p-14f;
        }
        const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400), hi = __builtin_amdgcn_perm(b[3], b[2], 0x0c0c0400);
        c[g] = lo | hi << 16;
      }
    }
    if (redo) {
#pragma unroll
      for (int g = 0; g < VE / 4; ++g) {
        c[g] = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) c[g] |= static_cast<uint32_t>(quant_exact(r.at(4 * g + e), s) & 255) << (8 * e);
      }
    }
    if ((i + 1) * VE <= K) {
      __builtin_memcpy(q + i * VE, c, VE);
    } else {
#pragma unroll
      for (int e = 0; e < VE; ++e)
        if (i * VE + e < K) q[i * VE + e] = static_cast<int8_t>(c[e / 4] >> (8 * (e & 3)));
    }
  };
  if constexpr (NV > 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = lane + 64 * W * j;
      if (i < pieces) store(i, held[j]);
    }
  } else {
    for (int i = lane; i < pieces; i += 64 * W) store(i, load(i));
  }
  if (lane == 0) scales[row] = finite ? amax / 127.0f : __builtin_nanf("");
}

// ---------------------------------------------------------------------- gate
// Packed router weight: [E/16][D/32][plane] runs of the 16x16x32 MFMA's operand, 1 KB each: lane
// l holds expert l % 16, features 8 * (l / 16) .. + 7 of the step.  An FP32 weight is cut into its
// upper, middle and lower eight significant bits, each a BF16 exactly, whose three planes' products
// are summed: the BF16 rate is sixteen times the FP32 one.  Cutting in the kernel instead (4 bytes
// a weight instead of 6) took 44 vector instructions to a tile's 12 MFMAs and longer in all
// (8192 tokens: 35 us against 31).
template <int WTYPE>
__global__ __launch_bounds__(256) void gate_pack_kernel(const typename Elem<WTYPE>::T* w, int32_t E, int32_t D,
                                                        uint16_t* packed) {
  constexpr int P = WTYPE == MOE_F32 ? 3 : 1;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int steps = D / 32;
  const int64_t n = static_cast<int64_t>((E + 15) / 16) * steps * 64;
  if (i >= n) return;
  const int lane = static_cast<int>(i & 63);
  const int64_t run = i >> 6;
  const int s = static_cast<int>(run % steps);
  const int e = static_cast<int>(run / steps) * 16 + (lane & 15);
  const int k = s * 32 + (lane >> 4) * 8;
  for (int j = 0; j < 8; ++j) {
    float v = e < E ? to_f32<WTYPE>(w[static_cast<int64_t>(e) * D + k + j]) : 0.0f;
    for (int p = 0; p < P; ++p) {
      const uint32_t b = __float_as_uint(v);
      const bool finite = (b & 0x7fffffffu) < 0x7f800000u;
      uint16_t h = static_cast<uint16_t>(b >> 16);  // cut off towards zero; the rest is exact
      if (!finite && (b & 0x7fffffu)) h |= 0x40;
      packed[(run * P + p) * 512 + lane * 8 + j] = h;
      v = finite ? v - bf16_to_f32(h) : 0.0f;
    }
  }
}

struct GateArgs {
  const uint16_t* x;
  int64_t ldx;
  const void* packed;
  int32_t B, E, D;
  float* logits;
  int64_t ldl;
};

// A workgroup's tile is 16 TT tokens x 16 ET experts; its WV waves take a share of the features
// each and add their FP32 tiles through LDS in wave order.  The packed weight comes straight into
// registers.  x is loaded eight lanes to a row, 64 features at a time, and turned into operands
// through LDS of the wave's own: read in the operand's layout, every lane at a row of its own,
// it took four times the L1's time and set the pace (8192 tokens, FP32 weight: 40 us).
template <int P, int TT, int ET, int WV>
__global__ __launch_bounds__(64 * WV) void gate_kernel(GateArgs a, uint32_t cols, uint32_t rows) {
  extern __shared__ __attribute__((aligned(16))) float gate_lds[];
  constexpr int kOut = 256 * TT * ET;  // outputs of the tile
  // in flight, as far as the registers of a wave go: UX blocks of 64 features of x, which comes
  // from HBM, and UW steps of 32 of the weight, which L2 holds
  constexpr int kRegs = 2048 / WV - 4 * TT * ET - (WV == 4 ? 192 : 64);
  constexpr int fit = (kRegs - 16 * TT) / (4 * P * ET), UW = fit >= 8 ? 8 : fit >= 4 ? 4 : 2;
  constexpr int UX = kRegs - UW * 4 * P * ET >= 32 * TT ? 4 : 2, UN = UX > UW / 2 ? UX : UW / 2;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // the tiles of one token range run on one XCD (workgroups go round the eight), so that its L2
  // serves x to all of them
  const uint32_t span = 8 * cols, row = blockIdx.x / span * 8 + blockIdx.x % 8, col = blockIdx.x % span / 8;
  if (row >= rows) return;
  const int64_t t0 = static_cast<int64_t>(row) * (16 * TT);
  // blocks of 64 features, shared out evenly
  const int tiles = (a.E + 15) / 16, steps = a.D / 32, blocks = steps / 2;
  const int b0 = wave * blocks / WV, n = (wave + 1) * blocks / WV - b0;
  const uint16_t* xp[2 * TT];
  const v8bf* wp[ET];
#pragma unroll
  for (int i = 0; i < 2 * TT; ++i) {
    const int64_t t = t0 + i * 8 + (lane >> 3);
    xp[i] = a.x + (t < a.B ? t : a.B - 1) * a.ldx + b0 * 64 + (lane & 7) * 8;
  }
#pragma unroll
  for (int i = 0; i < ET; ++i) {
    const int et = static_cast<int>(col) * ET + i;
    wp[i] = static_cast<const v8bf*>(a.packed) +
            (static_cast<int64_t>(et < tiles ? et : tiles - 1) * steps + b0 * 2) * (64 * P) + lane;
  }
  v4f acc[TT][ET] = {};
  v4i xb[UX][2 * TT];
  v8bf wb[UW][ET][P];
  auto load_x = [&](int u, int s) {
#pragma unroll
    for (int i = 0; i < 2 * TT; ++i) xb[u][i] = *reinterpret_cast<const v4i*>(xp[i] + s * 64);
  };
  auto load_w = [&](int u, int k) {
#pragma unroll
    for (int i = 0; i < ET; ++i)
#pragma unroll
      for (int p = 0; p < P; ++p) wb[u][i][p] = wp[i][(k * P + p) * 64];
  };
  unsigned char* const own = reinterpret_cast<unsigned char*>(gate_lds) + wave * (TT * 2048);
  auto place = [](int r, int c) { return r * 128 + (c ^ ((r >> 1) & 7)) * 16; };
#pragma unroll
  for (int u = 0; u < UX; ++u)
    if (u < n) load_x(u, u);
#pragma unroll
  for (int u = 0; u < UW; ++u)
    if (u < 2 * n) load_w(u, u);
  compiler_fence();  // the loads stay where they are written, ahead of their use
  for (int s0 = 0; s0 < n; s0 += UN) {
#pragma unroll
    for (int v = 0; v < UN; ++v) {
      const int s = s0 + v;
      if (s < n) {
#pragma unroll
        for (int i = 0; i < 2 * TT; ++i)
          *reinterpret_cast<v4i*>(own + place(i * 8 + (lane >> 3), lane & 7)) = xb[v % UX][i];
        if (s + UX < n) load_x(v % UX, s + UX);
        wave_sync();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int u = (2 * v + h) % UW;
          v8bf x[TT];
#pragma unroll
          for (int j = 0; j < TT; ++j)
            x[j] = *reinterpret_cast<const v8bf*>(own + place(j * 16 + (lane & 15), h * 4 + (lane >> 4)));
#pragma unroll
          for (int p = 0; p < P; ++p)
#pragma unroll
            for (int i = 0; i < ET; ++i)
#pragma unroll
              for (int j = 0; j < TT; ++j)
                acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[u][i][p], x[j], acc[j][i], 0, 0, 0);
          if (2 * s + h + UW < 2 * n) load_w(u, 2 * s + h + UW);
          compiler_fence();
        }
        wave_sync();
      }
    }
  }
  __syncthreads();
  // [wave][token][expert], padded by a word a row
  constexpr int kRow = 16 * ET + 4;
#pragma unroll
  for (int j = 0; j < TT; ++j)
#pragma unroll
    for (int i = 0; i < ET; ++i)
      *reinterpret_cast<v4f*>(gate_lds + (wave * 16 * TT + j * 16 + (lane & 15)) * kRow + i * 16 + (lane >> 4) * 4) =
          acc[j][i];
  __syncthreads();
  const bool vec = (reinterpret_cast<uintptr_t>(a.logits) | (a.ldl * 4)) % 16 == 0;
#pragma unroll
  for (int o = threadIdx.x; o < kOut / 4; o += 64 * WV) {
    const int tok = o / (4 * ET), e = o % (4 * ET) * 4;
    v4f v = *reinterpret_cast<const v4f*>(gate_lds + tok * kRow + e);
#pragma unroll
    for (int w = 1; w < WV; ++w) v += *reinterpret_cast<const v4f*>(gate_lds + (w * 16 * TT + tok) * kRow + e);
    const int64_t t = t0 + tok;
    const int ge = static_cast<int>(col) * 16 * ET + e;
    if (t >= a.B) continue;
    float* out = a.logits + t * a.ldl + ge;
    if (vec && ge + 4 <= a.E) {
      *reinterpret_cast<v4f*>(out) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (ge + i < a.E) out[i] = v[i];
    }
  }
}

// -------------------------------------------------------------------- linear
struct LinearArgs {
  const int8_t* a;
  const int8_t* w;
  const float* sa;
  const float* sw;
  const float* bias;
  const void* add;
  void* out;
  int64_t lda, ldw, ldo, ldadd;
  int32_t M, N, K;
};

// 16 bytes from any address, as the aligned words they lie in: loads that straddle words are
// several times slower than aligned ones (64 x 4096 x 4095: 47 us against 15).  `whole`: all 16 bytes
// belong to the row; else words from `end` on are zero.  Every word read holds a byte of the row.
struct Words {
  v4i v;
  int x;
};
__device__ __forceinline__ Words words16(const int8_t* p, bool whole, const int8_t* end) {
  typedef int v4i_word __attribute__((ext_vector_type(4), aligned(4)));
  const uintptr_t b = reinterpret_cast<uintptr_t>(p) & ~static_cast<uintptr_t>(3);
  Words r = {{0, 0, 0, 0}, 0};
  if (whole) {
    r.v = *reinterpret_cast<const v4i_word*>(b);
    r.x = *reinterpret_cast<const int*>((reinterpret_cast<uintptr_t>(p) + 15) & ~static_cast<uintptr_t>(3));
  } else {
    const uintptr_t e = reinterpret_cast<uintptr_t>(end);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (b + 4 * i < e) r.v[i] = *reinterpret_cast<const int*>(b + 4 * i);
    if (b + 16 < e) r.x = *reinterpret_cast<const int*>(b + 16);
  }
  return r;
}
// The 16 bytes, `skip` bytes into their words; only the first n of them unless WHOLE.
template <bool WHOLE>
__device__ __forceinline__ v4i bytes16(const Words& r, uint32_t skip, int n = 16) {
  v4i o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t hi = static_cast<uint32_t>(i < 3 ? r.v[i + 1] : r.x);
    uint32_t w = __builtin_amdgcn_alignbyte(hi, static_cast<uint32_t>(r.v[i]), skip);
    if (!WHOLE) w &= n >= 4 * i + 4 ? ~0u : n <= 4 * i ? 0u : (1u << (8 * (n - 4 * i))) - 1;
    o[i] = static_cast<int>(w);
  }
  return o;
}
__device__ __forceinline__ uint32_t skip_of(const int8_t* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 3);
}
// g / (1 + exp(-g)) with the hardware's exp2 and reciprocal (an ulp each).
__device__ __forceinline__ float silu(float g) { return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)); }

// ------------------------------------------------- linear: up to 64 tokens
// The weight is read once, so its bytes bound the product.  A workgroup takes 16 RT weight rows
// (SwiGLU: 16 gate rows and their 16 up rows) and 16 TT tokens; its WV waves split K in pieces of
// 128 bytes.  A wave loads a piece's rows eight lanes to a row (lanes that each read a row of
// their own, as the operand's layout would have it, get a quarter of the L1's rate), some pieces ahead, and
// turns them into operands through LDS of its own, so that no wave waits for another before
// the 32-bit sums are added.
template <int OUT, bool SWIGLU, bool ALIGNED, int RT, int TT, int WV>
__global__ __launch_bounds__(64 * WV) void linear_stream_kernel(LinearArgs a, uint32_t nx) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  constexpr int COLS = SWIGLU ? 16 : 16 * RT, NL = 2 * (RT + TT);  // columns of out; loads of a piece
  constexpr int kRegs = (2048 / WV - 4 * RT * TT - 8 * (RT + TT) - 40) / (NL * (ALIGNED ? 4 : 5));
  constexpr int U = kRegs > 6 ? 6 : kRegs < 2 ? 2 : kRegs;         // pieces in flight
  static_assert(!SWIGLU || RT == 2, "a gate and an up tile");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int H = SWIGLU ? a.N / 2 : a.N, n0 = blockIdx.x % nx * COLS, m0 = blockIdx.x / nx * (16 * TT);
  const int pieces = (a.K + 127) / 128, per = (pieces + WV - 1) / WV, c0 = wave * per;
  const int n = pieces - c0 < per ? (pieces > c0 ? pieces - c0 : 0) : per;
  // load i brings rows 8 i .. 8 i + 7 of the wave's tile: weight rows first, then tokens
  const int part = lane & 7;
  const int8_t* rows[NL];
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int r = i * 8 + (lane >> 3);
    if (i < 2 * RT) {
      const int c = n0 + (SWIGLU ? r & 15 : r);
      rows[i] = a.w + ((c < H ? c : H - 1) + (SWIGLU ? static_cast<int64_t>(r >> 4) * H : 0)) * a.ldw;
    } else {
      const int m = m0 + r - 16 * RT;
      rows[i] = a.a + static_cast<int64_t>(m < a.M ? m : a.M - 1) * a.lda;
    }
  }
  using Held = std::conditional_t<ALIGNED, v4i, Words>;
  Held held[U][NL];
  // aligned: 16 bytes lie wholly inside the row or wholly behind it; those behind are read from
  // the row's last 16 and set to zero when used
  auto load = [&](int u, int c) {
    const int k = (c0 + c) * 128 + part * 16;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      if constexpr (ALIGNED) held[u][i] = *reinterpret_cast<const v4i*>(rows[i] + (k < a.K ? k : a.K - 16));
      else held[u][i] = words16(rows[i] + k, (c0 + c) * 128 + 128 <= a.K, rows[i] + a.K);
    }
  };
  unsigned char* const own = smem + wave * (NL * 1024);
  auto place = [](int r, int c) { return r * 128 + (c ^ ((r >> 1) & 7)) * 16; };
  v4i acc[RT][TT] = {};
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (u < n) load(u, u);
  compiler_fence();
  for (int c = 0; c < n; c += U) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c + u < n) {
        const int first = (c0 + c + u) * 128, left = a.K - first - part * 16;
        auto turn = [&](auto whole) {
#pragma unroll
          for (int i = 0; i < NL; ++i) {  // bytes behind K count as zero; it takes one operand to see to that
            constexpr bool kWhole = decltype(whole)::value;
            v4i v;
            if constexpr (ALIGNED) v = kWhole || i >= 2 * RT || left > 0 ? held[u][i] : v4i{0, 0, 0, 0};
            else if (kWhole || i >= 2 * RT) v = bytes16<true>(held[u][i], skip_of(rows[i]));
            else v = bytes16<false>(held[u][i], skip_of(rows[i]), left);
            *reinterpret_cast<v4i*>(own + place(i * 8 + (lane >> 3), part)) = v;
          }
        };
        if (first + 128 <= a.K) turn(std::true_type{});
        else turn(std::false_type{});
        if (c + u + U < n) load(u, c + u + U);
        wave_sync();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          v4i fw[RT], fa[TT];
#pragma unroll
          for (int i = 0; i < RT; ++i)
            fw[i] = *reinterpret_cast<const v4i*>(own + place(i * 16 + (lane & 15), h * 4 + (lane >> 4)));
#pragma unroll
          for (int j = 0; j < TT; ++j)
            fa[j] = *reinterpret_cast<const v4i*>(own + place((RT + j) * 16 + (lane & 15), h * 4 + (lane >> 4)));
#pragma unroll
          for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int j = 0; j < TT; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[i], fa[j], acc[i][j], 0, 0, 0);
        }
        wave_sync();
      }
  }
  // [wave][token][weight row], padded by four words a row
  constexpr int kRow = 16 * RT + 4, kTile = 16 * TT * kRow;
  int* const sums = reinterpret_cast<int*>(smem);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < TT; ++j)
      *reinterpret_cast<v4i*>(sums + wave * kTile + (j * 16 + (lane & 15)) * kRow + i * 16 + (lane >> 4) * 4) = acc[i][j];
  __syncthreads();
  using T = typename Elem<OUT>::T;
  for (int o = threadIdx.x; o < COLS * 16 * TT; o += 64 * WV) {
    const int64_t m = m0 + o / COLS;
    const int c = n0 + o % COLS;
    if (m >= a.M || c >= H) continue;
    const int* p = sums + o / COLS * kRow + o % COLS;
    int sum = 0, sum_up = 0;
#pragma unroll
    for (int v = 0; v < WV; ++v) {
      sum += p[v * kTile];
      if (SWIGLU) sum_up += p[v * kTile + 16];
    }
    const float sa = a.sa[m];
    float y = static_cast<float>(sum) * sa * a.sw[c] + (a.bias ? a.bias[c] : 0.0f);
    if (SWIGLU) y = silu(y) * (static_cast<float>(sum_up) * sa * a.sw[H + c] + (a.bias ? a.bias[H + c] : 0.0f));
    if (a.add) y += to_f32<OUT>(static_cast<const T*>(a.add)[m * a.ldadd + c]);
    static_cast<T*>(a.out)[m * a.ldo + c] = from_f32<OUT>(y);
  }
}

// ------------------------------------------------- linear: many tokens
// 16 bytes a lane from a buffer (base, extent in bytes) to LDS at lds + 16 * lane; lanes whose
// offset lies outside the extent write zeros and read nothing.  Written as asm so that the
// compiler does not drain the stream before every LDS read: its landing is awaited by count.
constexpr uint32_t kOutside = 0x80000000u;
__device__ __forceinline__ void dma16(v4i rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
               : "m0", "memory");
}
__device__ __forceinline__ void dma4(v4i rsrc, uint32_t voff, uint32_t lds) {  // 4 bytes a lane
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(rsrc)
               : "m0", "memory");
}
__device__ __forceinline__ v4i make_rsrc(const void* base, uint32_t bytes) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  v4i r;
  r[0] = __builtin_amdgcn_readfirstlane(static_cast<int>(b));
  r[1] = __builtin_amdgcn_readfirstlane(static_cast<int>((b >> 32) & 0xffffu));
  r[2] = __builtin_amdgcn_readfirstlane(static_cast<int>(bytes));
  r[3] = 0x00020000;
  return r;
}
template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

// Floats of LDS a wave needs to store its tile, and the storing: scales, bias, activation; 32
// tokens at a time go through LDS, so that whole rows' pieces are added to and stored.  acc is
// the wave's part of a tile (tokens m0 + wm.., tile rows wn..); sw, bias and sa are the whole
// tile's, in LDS.
template <int TM, int TN, bool SWIGLU>
constexpr int kEpilogue = 32 * ((SWIGLU ? TN * 16 : TN * 32) + 4);
template <int TM, int TN, int OUT, bool SWIGLU>
__device__ __forceinline__ void store_tile(const LinearArgs& a, const v16i (&acc)[TN][TM], float* buf, const float* sw,
                                           const float* bias, const float* sa, int64_t m0, int wm, int n0, int wn) {
  using T = typename Elem<OUT>::T;
  constexpr int kCols = SWIGLU ? TN * 16 : TN * 32, kRow = kCols + 4, PER = 16 / sizeof(T);
  const int lane = threadIdx.x & 63, H = SWIGLU ? a.N / 2 : a.N;
  const int nw = n0 + (SWIGLU ? wn / 2 : wn);
  const bool vec = (reinterpret_cast<uintptr_t>(a.out) | (a.ldo * sizeof(T))) % 16 == 0 &&
                   (!a.add || (reinterpret_cast<uintptr_t>(a.add) | (a.ldadd * sizeof(T))) % 16 == 0);
#pragma unroll
  for (int j = 0; j < TM; ++j) {
    const int64_t mt = m0 + wm + j * 32;
    const float scale = sa[wm + j * 32 + (lane & 31)];
#pragma unroll
    for (int i = 0; i < TN; i += SWIGLU ? 2 : 1)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int r = g * 8 + (lane >> 5) * 4, row = wn + i * 32 + r;
        const v4f ws = *reinterpret_cast<const v4f*>(sw + row), wb = *reinterpret_cast<const v4f*>(bias + row);
        v4f y;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = static_cast<float>(acc[i][j][g * 4 + e]) * scale * ws[e] + wb[e];
        if constexpr (SWIGLU) {
          const v4f us = *reinterpret_cast<const v4f*>(sw + row + 32), ub = *reinterpret_cast<const v4f*>(bias + row + 32);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            y[e] = silu(y[e]) * (static_cast<float>(acc[i + 1][j][g * 4 + e]) * scale * us[e] + ub[e]);
        }
        *reinterpret_cast<v4f*>(buf + (lane & 31) * kRow + (SWIGLU ? i * 16 : i * 32) + r) = y;
      }
    __builtin_amdgcn_wave_barrier();
    constexpr int kPieces = kCols / PER;  // 16-byte pieces of a row
    for (int p = lane; p < 32 * kPieces; p += 64) {
      const int row = p / kPieces, c = p % kPieces * PER, col = nw + c;
      const int64_t m = mt + row;
      if (m >= a.M || col >= H) continue;
      float y[PER];
#pragma unroll
      for (int e = 0; e < PER; ++e) y[e] = buf[row * kRow + c + e];
      T* out = static_cast<T*>(a.out) + m * a.ldo + col;
      const T* add = static_cast<const T*>(a.add) + m * a.ldadd + col;
      if (vec && col + PER <= H) {
        T v[PER];
        if (a.add) {
          __builtin_memcpy(v, __builtin_assume_aligned(add, 16), 16);
#pragma unroll
          for (int e = 0; e < PER; ++e) y[e] += to_f32<OUT>(v[e]);
        }
#pragma unroll
        for (int e = 0; e < PER; ++e) v[e] = from_f32<OUT>(y[e]);
        __builtin_memcpy(__builtin_assume_aligned(out, 16), v, 16);
      } else {
        for (int e = 0; e < PER && col + e < H; ++e)
          out[e] = from_f32<OUT>(a.add ? y[e] + to_f32<OUT>(add[e]) : y[e]);
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// Workgroup tile of BM tokens x BN weight rows, WM x WN waves, 32x32x32 MFMAs with the weight
// as the row operand (a lane then holds four neighbouring columns of out).  K goes through LDS
// in NS stages of KB bytes a row.  A row's 16-byte parts lie permuted by its index, so that the
// 16 lanes that LDS serves at once (0-3, 12-15, 20-27 and so on) meet all 64 banks once.
template <int BM, int BN, int WM, int WN, int KB, int NS, int OUT, bool SWIGLU>
__global__ __launch_bounds__(64 * WM * WN, (BM + BN) * KB * NS > 78 * 1024 ? 1 : 2) void linear_dma_kernel(
    LinearArgs a, uint32_t nm, uint32_t nn, uint32_t per_xcd) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  constexpr int NW = WM * WN, kStage = (BM + BN) * KB, PARTS = KB / 16, DR = 1024 / KB;  // rows of one DMA
  constexpr int RA = BM / DR / NW, RW = BN / DR / NW, US = KB / 32;
  constexpr int TM = BM / WM / 32, TN = BN / WN / 32;
  static_assert(!SWIGLU || TN % 2 == 0, "a wave holds whole gate and up pairs");
  static_assert(BM % (DR * NW) == 0 && BN % (DR * NW) == 0 && (KB == 64 || KB == 128), "whole DMAs");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // each XCD (workgroups go round the eight) takes a contiguous range of tiles, in groups of
  // eight token tiles: what runs at once on an XCD shares operands in its L2
  const uint32_t tile = blockIdx.x % 8 * per_xcd + blockIdx.x / 8;
  if (blockIdx.x / 8 >= per_xcd || tile >= nm * nn) return;
  const uint32_t band = tile / (8 * nn), left = nm - band * 8, height = left < 8 ? left : 8, in = tile - band * 8 * nn;
  const int64_t m0 = static_cast<int64_t>(band * 8 + in % height) * BM;
  const int H = SWIGLU ? a.N / 2 : a.N, n0 = static_cast<int>(in / height) * (SWIGLU ? BN / 2 : BN);
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) void*)smem));

  // place of part `c` of row r: parts go round by the row, by every second with 128-byte rows
  // (two rows span the banks) and every fourth with 64-byte rows
  auto place = [](int r, int c) { return c ^ ((KB == 128 ? r >> 1 : r >> 2) & (PARTS - 1)); };
  // what this lane moves: a part of row lane / PARTS of its wave's blocks of DR rows
  const int lr = lane / PARTS;
  const int mrows = a.M - m0 < BM ? static_cast<int>(a.M - m0) : BM;
  const v4i ra = make_rsrc(a.a + m0 * a.lda, static_cast<uint32_t>((mrows - 1) * a.lda + a.K));
  uint32_t va[RA], vw[RW];
  int ka[RA], kw[RW];  // the part's offset in the stage
  v4i rw[RW];
  {
    const int cols = SWIGLU ? BN / 2 : BN, nrows = H - n0 < cols ? H - n0 : cols;
    const uint32_t bytes = static_cast<uint32_t>((nrows - 1) * a.ldw + a.K);
#pragma unroll
    for (int i = 0; i < RA; ++i) {
      const int row = (wave * RA + i) * DR + lr;
      ka[i] = place(row, lane % PARTS) * 16;
      va[i] = row < mrows ? static_cast<uint32_t>(row * a.lda) + ka[i] : kOutside;
    }
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      // SwiGLU: 32 gate rows, then their 32 up rows, and so on
      const int first = (wave * RW + i) * DR, slot = first + lr, row = SWIGLU ? (slot >> 6) * 32 + (slot & 31) : slot;
      kw[i] = place(slot, lane % PARTS) * 16;
      rw[i] = make_rsrc(a.w + (n0 + (SWIGLU ? static_cast<int64_t>((first >> 5) & 1) * H : 0)) * a.ldw, bytes);
      vw[i] = row < nrows ? static_cast<uint32_t>(row * a.ldw) + kw[i] : kOutside;
    }
  }
  constexpr int kIssue = RA + RW;
  // DMA d of this wave for stage s into the LDS at buf; parts behind K, and whole stages behind
  // it, are zeros.  The bounds check holds a lane's offset against the extent less the scalar offset, so a
  // stage behind K has none: with few rows in the tile it could exceed the extent, and nothing says that
  // the difference does not wrap.
  auto issue = [&](int s, int buf, int d) {
    const int k0 = s * KB;
    const uint32_t soff = k0 < a.K ? k0 : 0;
    if (d < RA) {
      dma16(ra, k0 + ka[d] < a.K ? va[d] : kOutside, soff, lds0 + buf + (wave * RA + d) * 1024);
    } else {
      d -= RA;
      dma16(rw[d], k0 + kw[d] < a.K ? vw[d] : kOutside, soff, lds0 + buf + BM * KB + (wave * RW + d) * 1024);
    }
  };

  const int wm = wave % WM * (BM / WM), wn = wave / WM * (BN / WN);
  uint32_t la[US];  // this lane's operand inside a 32-row tile, for each 32 of K
#pragma unroll
  for (int u = 0; u < US; ++u) la[u] = (lane & 31) * KB + place(lane & 31, u * 2 + (lane >> 5)) * 16;
  v16i acc[TN][TM] = {};
  v4i fa[2][TM], fw[2][TN];
  // the TM + TN reads of a step, spread over the first half of the rows of MFMAs before it
  constexpr int kPart = TN > 1 ? (TM + TN + TN / 2 - 1) / (TN / 2) : TM + TN;
  auto read = [&](int buf, int u, int from) {
    const unsigned char* p = smem + buf + la[u];
#pragma unroll
    for (int f = from; f < from + kPart && f < TM + TN; ++f) {
      if (f < TM) fa[u & 1][f] = *reinterpret_cast<const v4i*>(p + (wm + f * 32) * KB);
      else fw[u & 1][f - TM] = *reinterpret_cast<const v4i*>(p + (BM + wn + (f - TM) * 32) * KB);
    }
  };
  auto mult = [&](int h, int i) {
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[h][i], fa[h][j], acc[i][j], 0, 0, 0);
  };
  // a stage's DMAs are issued over the US steps after its buffer is free, some behind each row
  auto slot = [](int p) { return p * kIssue / (US * TN); };
  const int n = (a.K + KB - 1) / KB;
  // scales and bias of the tile, behind the stages, in the order of its rows; they go the same
  // way, first: an ordinary load among the DMAs would have to wait for all of them
  const float* const sw = reinterpret_cast<const float*>(smem + NS * kStage);
  const float* const bias = sw + BN;
  const float* const sa = bias + BN;
  {
    const uint32_t dst = lds0 + NS * kStage;
    const int cols = H - n0;  // columns from here on
    for (int b = wave; b < BN / 64; b += NW) {
      // 64 tile rows: 64 columns, or 32 and then the same 32 of the other half
      const int c = SWIGLU ? b * 32 + (lane & 31) : b * 64 + lane;
      const uint32_t off = c < cols ? (c + (SWIGLU && lane >= 32 ? H : 0)) * 4u : kOutside;
      const uint32_t bytes = static_cast<uint32_t>(a.N - n0) * 4u;
      dma4(make_rsrc(a.sw + n0, bytes), off, dst + b * 256);
      dma4(make_rsrc(a.bias + n0, a.bias ? bytes : 0u), off, dst + (BN + b * 64) * 4);
    }
    for (int b = wave; b < BM / 64; b += NW)
      dma4(make_rsrc(a.sa + m0, static_cast<uint32_t>(mrows) * 4u), (b * 64 + lane) * 4u, dst + (2 * BN + b * 64) * 4);
  }
#pragma unroll
  for (int s = 0; s < NS; ++s) {
#pragma unroll
    for (int d = 0; d < (s < NS - 1 ? kIssue : slot(TN)); ++d) issue(s, s * kStage, d);
  }
  wait_vm<kIssue*(NS - 2) + slot(TN)>();
  __builtin_amdgcn_s_barrier();
  compiler_fence();
#pragma unroll
  for (int f = 0; f < TM + TN; f += kPart) read(0, 0, f);
  compiler_fence();
  // Each step multiplies what the step before read, a row of MFMAs at a time; the next step's
  // reads and the DMA issues (which hold a wave up for some 90 cycles each) go between the
  // rows, in the order written.
  int prev = (NS - 1) * kStage, cur = 0;  // LDS offsets of stages s - 1 and s
  for (int s = 0; s < n; ++s) {
    const int next = cur + kStage == NS * kStage ? 0 : cur + kStage;
#pragma unroll
    for (int u = 0; u < US; ++u) {
      if (u == US - 1) {
        // this stage is read out and the next has landed, for every wave
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        wait_vm<kIssue*(NS - 2)>();
        __builtin_amdgcn_s_barrier();
        compiler_fence();
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int i = 0; i < TN; ++i) {
        read(u == US - 1 ? next : cur, (u + 1) % US, i * kPart);
        mult(u & 1, i);
        const int p = (u + 1) % US * TN + i;
#pragma unroll
        for (int d = slot(p); d < slot(p + 1); ++d) {
          if (u == US - 1) issue(s + NS, cur, d);
          else issue(s + NS - 1, prev, d);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    prev = cur;
    cur = next;
    compiler_fence();
  }
  wait_vm<0>();
  __syncthreads();
  static_assert(NW * kEpilogue<TM, TN, SWIGLU> * 4 <= NS * kStage, "epilogue fits the stages");
  store_tile<TM, TN, OUT, SWIGLU>(a, acc, reinterpret_cast<float*>(smem) + wave * kEpilogue<TM, TN, SWIGLU>, sw, bias, sa, m0,
                                  wm, n0, wn);
}

// The same product for rows of any alignment: 128 tokens x 128 weight rows, four waves, stages of
// 128 bytes a row that pass through registers (LDS DMA wants 16-byte parts), the next stage's
// loads in flight while one is multiplied.
template <int OUT, bool SWIGLU>
__global__ __launch_bounds__(256, 2) void linear_any_kernel(LinearArgs a, uint32_t nx) {
  constexpr int BM = 128, BN = 128, KB = 128, kStage = (BM + BN) * KB, TM = 2, TN = 2;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t m0 = static_cast<int64_t>(blockIdx.x / nx) * BM;
  const int H = SWIGLU ? a.N / 2 : a.N, n0 = (blockIdx.x % nx) * (SWIGLU ? BN / 2 : BN);
  auto place = [](int r, int c) { return c ^ ((r >> 1) & 7); };
  auto wrow = [&](int r) -> int64_t {  // the weight row in row r of the tile, or -1
    const int c = n0 + (SWIGLU ? (r >> 6) * 32 + (r & 31) : r);
    return c < H ? c + (SWIGLU ? static_cast<int64_t>((r >> 5) & 1) * H : 0) : -1;
  };
  float* const sw = reinterpret_cast<float*>(smem + 2 * kStage);
  float* const bias = sw + BN;
  float* const sa = bias + BN;
  if (threadIdx.x < BN) {
    const int64_t r = wrow(threadIdx.x);
    sw[threadIdx.x] = r >= 0 ? a.sw[r] : 0.0f;
    bias[threadIdx.x] = r >= 0 && a.bias ? a.bias[r] : 0.0f;
  } else {
    const int r = threadIdx.x - BN;
    sa[r] = m0 + r < a.M ? a.sa[m0 + r] : 0.0f;
  }
  // this thread's parts: part threadIdx.x % 8 of rows threadIdx.x / 8 + 32 i
  const int part = threadIdx.x & 7, r0 = threadIdx.x >> 3;
  const int8_t *pa[4], *pw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + 32 * i;
    const int64_t n = wrow(r);  // rows outside: the last one, its products are not stored
    pa[i] = a.a + (m0 + r < a.M ? m0 + r : a.M - 1) * a.lda;
    pw[i] = a.w + (n >= 0 ? n : static_cast<int64_t>(a.N) - 1) * a.ldw;
  }
  Words ga[4], gw[4];
  auto load = [&](int s) {
    const int k = s * KB + part * 16;
    const bool whole = (s + 1) * KB <= a.K;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ga[i] = words16(pa[i] + k, whole, pa[i] + a.K);
      gw[i] = words16(pw[i] + k, whole, pw[i] + a.K);
    }
  };
  auto store = [&](int s, int buf) {
    auto turn = [&](auto whole) {
      const int left = a.K - s * KB - part * 16;  // bytes behind K count as zero
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = r0 + 32 * i;
        *reinterpret_cast<v4i*>(smem + buf + r * KB + place(r, part) * 16) = bytes16<true>(ga[i], skip_of(pa[i]));
        *reinterpret_cast<v4i*>(smem + buf + (BM + r) * KB + place(r, part) * 16) =
            bytes16<decltype(whole)::value>(gw[i], skip_of(pw[i]), left);
      }
    };
    if ((s + 1) * KB <= a.K) turn(std::true_type{});
    else turn(std::false_type{});
  };
  const int wm = (wave & 1) * 64, wn = (wave >> 1) * 64, n = (a.K + KB - 1) / KB;
  v16i acc[TN][TM] = {};
  load(0);
  store(0, 0);
  __syncthreads();
  for (int s = 0; s < n; ++s) {
    const int cur = (s & 1) * kStage;
    if (s + 1 < n) load(s + 1);
    compiler_fence();
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int off = (lane & 31) * KB + place(lane & 31, u * 2 + (lane >> 5)) * 16;
      v4i fa[TM], fw[TN];
#pragma unroll
      for (int j = 0; j < TM; ++j) fa[j] = *reinterpret_cast<const v4i*>(smem + cur + (wm + j * 32) * KB + off);
#pragma unroll
      for (int i = 0; i < TN; ++i) fw[i] = *reinterpret_cast<const v4i*>(smem + cur + (BM + wn + i * 32) * KB + off);
#pragma unroll
      for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[i], fa[j], acc[i][j], 0, 0, 0);
    }
    if (s + 1 < n) store(s + 1, kStage - cur);
    __syncthreads();
  }
  static_assert(4 * kEpilogue<TM, TN, SWIGLU> * 4 <= 2 * kStage, "epilogue fits the stages");
  store_tile<TM, TN, OUT, SWIGLU>(a, acc, reinterpret_cast<float*>(smem) + wave * kEpilogue<TM, TN, SWIGLU>, sw, bias, sa, m0,
                                  wm, n0, wn);
}

// ---------------------------------------------------------------------- host
hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }
int hip_failed() {
  (void)hipGetLastError();  // reported here, and not again by the thread's next caller
  return MOE_EHIP;
}
// Enqueue a kernel.  The status is this launch's own: the thread's last error may be an earlier call's, and would
// make a call that was enqueued look like one that was not.
template <typename T>
struct Same {
  using type = T;
};
template <typename... P>
int launch(void (*kernel)(P...), uint32_t grid, uint32_t block, size_t lds, hipStream_t st, typename Same<P>::type... p) {
  void* args[] = {const_cast<void*>(static_cast<const void*>(&p))...};
  const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(grid), dim3(block), args, lds, st);
  return e == hipSuccess ? MOE_OK : hip_failed();
}
constexpr int32_t kMaxRows = 1 << 22;  // tokens of one call: its grids stay within the launch limits
bool type_ok(int32_t t) { return t == MOE_BF16 || t == MOE_F16 || t == MOE_F32; }
bool gate_ok(int32_t E, int32_t D, int32_t wtype) {
  return E >= 1 && E <= 1024 && D >= 512 && D <= 16384 && D % 512 == 0 && (wtype == MOE_BF16 || wtype == MOE_F32);
}

template <int TYPE, int LPT, int NV>
int launch_route(const RouteArgs& a, hipStream_t st) {
  constexpr int per = 4 * (64 / LPT);
  return launch(route_kernel<TYPE, LPT, NV>, (a.B + per - 1) / per, 256, 0, st, a);
}

template <int TYPE>
int launch_route(const RouteArgs& a, hipStream_t st) {
  // 16 lanes a token do less work in all, 64 finish a token sooner (160 experts, top 16, bias: 4096
  // tokens 9.5 against 9.2 us, 6000 11.2 against 11.4, 16384 16.4 against 23).  A lane's list is sorted in a number of
  // steps that grows with the square of its room, hence three sizes of it (16384 tokens, top 8, bias: 64 experts
  // with room for 4 a lane 7.6 us; for 10 and for 16: 72 experts 11.4 and 18.3, 128 13.1 and 20.2, 160 14.3 and 21.7)
  if (a.B > 4096 && a.E <= 256 && a.groups <= 16) {
    if (a.E <= 64) return launch_route<TYPE, 16, 4>(a, st);
    if (a.E <= 160) return launch_route<TYPE, 16, 10>(a, st);
    return launch_route<TYPE, 16, 16>(a, st);
  }
  return a.E <= 256 ? launch_route<TYPE, 64, 4>(a, st) : launch_route<TYPE, 64, 16>(a, st);
}

template <int TYPE, int W, int NV>
int launch_quant(const void* x, int64_t ldx, int32_t M, int32_t K, int8_t* codes, int64_t ldc, float* scales,
                 hipStream_t st) {
  constexpr int per = 4 / W;
  return launch(quant_kernel<TYPE, W, NV>, (M + per - 1) / per, 256, 0, st, x, ldx, M, K, codes, ldc, scales);
}

template <int TYPE>
int launch_quant(const void* x, int64_t ldx, int32_t M, int32_t K, int8_t* codes, int64_t ldc, float* scales,
                 hipStream_t st) {
  constexpr int VE = 16 / static_cast<int>(elem_size(TYPE));
  const int pieces = (K + VE - 1) / VE;
  // many tokens: a wave each, no step waits for another wave; few: four waves each
  if (M >= 1024 && pieces <= 8 * 64) {
    if (pieces <= 64) return launch_quant<TYPE, 1, 1>(x, ldx, M, K, codes, ldc, scales, st);
    if (pieces <= 2 * 64) return launch_quant<TYPE, 1, 2>(x, ldx, M, K, codes, ldc, scales, st);
    if (pieces <= 4 * 64) return launch_quant<TYPE, 1, 4>(x, ldx, M, K, codes, ldc, scales, st);
    return launch_quant<TYPE, 1, 8>(x, ldx, M, K, codes, ldc, scales, st);
  }
  if (pieces <= 2 * 256) return launch_quant<TYPE, 4, 2>(x, ldx, M, K, codes, ldc, scales, st);
  if (pieces <= 8 * 256) return launch_quant<TYPE, 4, 8>(x, ldx, M, K, codes, ldc, scales, st);
  return launch_quant<TYPE, 4, 0>(x, ldx, M, K, codes, ldc, scales, st);
}

// Allow a kernel more than 64 KB of LDS, once per device.
template <typename F>
bool allow_lds(F fn, size_t bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (bytes <= 65536) return true;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return false;
  if (done.load(std::memory_order_relaxed) >> dev & 1) return true;
  if (hipFuncSetAttribute(reinterpret_cast<const void*>(fn), hipFuncAttributeMaxDynamicSharedMemorySize,
                          static_cast<int>(bytes)) != hipSuccess)
    return false;
  done.fetch_or(1ull << dev, std::memory_order_relaxed);
  return true;
}

template <int P, int TT, int ET, int WV>
int launch_gate_tile(const GateArgs& a, hipStream_t st) {
  static std::atomic<uint64_t> done{0};
  constexpr size_t lds = WV * std::max(64 * TT * (16 * ET + 4), 2048 * TT);
  static_assert(lds <= 160 * 1024, "gate tile");
  if (!allow_lds(gate_kernel<P, TT, ET, WV>, lds, done)) return hip_failed();
  const uint32_t cols = ((a.E + 15) / 16 + ET - 1) / ET, rows = static_cast<uint32_t>((a.B + 16 * TT - 1) / (16 * TT));
  return launch(gate_kernel<P, TT, ET, WV>, (rows + 7) / 8 * 8 * cols, 64 * WV, lds, st, a, cols, rows);
}

template <int P>
int launch_gate(const GateArgs& a, hipStream_t st) {
  // Rounds of tiles over 256 CUs, weighed with a tile's time (BF16 and FP32 weight): small tiles
  // fill the CUs, large ones read less.  The weights are fitted to 1 to 8192 tokens, 32 to 250
  // experts, 1024 to 5120 features, where the tile chosen is on average 4 % (BF16) and 2 % (FP32)
  // slower than the best of thirteen (at worst by a third: 2600 tokens with 250 experts).
  const int64_t tiles = (a.E + 15) / 16;
  auto cost = [&](int tt, int et, int bf16, int f32) {
    return ((a.B + 16 * tt - 1) / (16 * tt) * ((tiles + et - 1) / et) + 255) / 256 * (P == 3 ? f32 : bf16);
  };
  const int64_t c0 = cost(1, 1, 10, 10), c1 = cost(2, 1, 13, 13), c2 = cost(2, 2, 20, 18), c3 = cost(4, 2, 34, 33),
                c4 = cost(4, 3, 36, 43), c5 = cost(4, 5, 49, 44);
  const int64_t best = std::min(std::min(std::min(c0, c1), std::min(c2, c3)), std::min(c4, c5));
  if (best == c0) return launch_gate_tile<P, 1, 1, 16>(a, st);
  if (best == c1) return launch_gate_tile<P, 2, 1, 8>(a, st);
  if (best == c2) return launch_gate_tile<P, 2, 2, 16>(a, st);
  if (best == c3) return launch_gate_tile<P, 4, 2, 8>(a, st);
  if (best == c4) return launch_gate_tile<P, 4, 3, 8>(a, st);
  return launch_gate_tile<P, 4, 5, 4>(a, st);
}

template <int OUT, bool SWIGLU, bool ALIGNED, int RT, int TT, int WV>
int launch_stream(const LinearArgs& a, hipStream_t st) {
  static std::atomic<uint64_t> done{0};
  constexpr size_t lds = WV * std::max(2048 * (RT + TT), 64 * TT * (16 * RT + 4));
  static_assert(lds <= 160 * 1024, "LDS of a CU");
  if (!allow_lds(linear_stream_kernel<OUT, SWIGLU, ALIGNED, RT, TT, WV>, lds, done)) return hip_failed();
  const int cols = SWIGLU ? a.N / 2 : a.N, per = SWIGLU ? 16 : 16 * RT;
  const uint32_t nx = static_cast<uint32_t>((cols + per - 1) / per), ny = static_cast<uint32_t>((a.M + 16 * TT - 1) / (16 * TT));
  return launch(linear_stream_kernel<OUT, SWIGLU, ALIGNED, RT, TT, WV>, nx * ny, 64 * WV, lds, st, a, nx);
}

template <int BM, int BN, int WM, int WN, int KB, int NS, int OUT, bool SWIGLU>
int launch_dma(const LinearArgs& a, hipStream_t st) {
  static std::atomic<uint64_t> done{0};
  constexpr size_t lds = NS * (BM + BN) * KB + 4 * (BM + 2 * BN);
  static_assert(lds <= 160 * 1024, "LDS of a CU");
  if (!allow_lds(linear_dma_kernel<BM, BN, WM, WN, KB, NS, OUT, SWIGLU>, lds, done)) return hip_failed();
  const uint32_t nm = static_cast<uint32_t>((a.M + BM - 1) / BM), bn = SWIGLU ? BN / 2 : BN,
                 nn = static_cast<uint32_t>(((SWIGLU ? a.N / 2 : a.N) + bn - 1) / bn), per = (nm * nn + 7) / 8;
  return launch(linear_dma_kernel<BM, BN, WM, WN, KB, NS, OUT, SWIGLU>, per * 8, 64 * WM * WN, lds, st, a, nm, nn, per);
}

template <int OUT, bool SWIGLU, bool ALIGNED>
int launch_linear(const LinearArgs& a, hipStream_t st) {
  // The streaming kernel's workgroups of 16 columns, 64 tokens a block.  Beyond a round of 256, two
  // row tiles halve them and the reads of a.  With more than 64 tokens it is taken while it stays
  // in one round, when tiles would leave most CUs idle (us, it and tiles: 256 x 768 x 3584 7.1 and
  // 12.5, 512 x 768 x 3584 8.2 and 12.7, 128 x 4096 x 4096 9.3 and 13.9); where tiles cannot use LDS
  // DMA, two rounds (512 x 768 x 3583 14.9 and 37.7).
  constexpr int R1 = SWIGLU ? 2 : 1;
  const int64_t blocks = static_cast<int64_t>((a.M + 63) / 64) * (((SWIGLU ? a.N / 2 : a.N) + 15) / 16);
  const bool wide = !SWIGLU && blocks > 256;
  // (unaligned gate and up rows take more registers than sixteen waves leave)
  if (a.M <= 16) return launch_stream<OUT, SWIGLU, ALIGNED, R1, 1, SWIGLU && !ALIGNED ? 8 : 16>(a, st);
  if (a.M <= 32)
    return wide ? launch_stream<OUT, SWIGLU, ALIGNED, 2, 2, 8>(a, st) : launch_stream<OUT, SWIGLU, ALIGNED, R1, 2, 8>(a, st);
  if (a.M <= 64 || blocks <= (SWIGLU ? 256 : ALIGNED ? 512 : 1024))
    return wide ? launch_stream<OUT, SWIGLU, ALIGNED, 2, 4, 8>(a, st) : launch_stream<OUT, SWIGLU, ALIGNED, R1, 4, 8>(a, st);
  if constexpr (ALIGNED) {
    // Rounds of tiles over 256 CUs, weighed with a round's time at K = 4096 (us, less what every
    // call pays): large tiles move fewer bytes for each product, small ones fill the CUs.
    const int64_t cols = SWIGLU ? a.N / 2 : a.N;
    auto cost = [&](int bm, int bn, int us) {
      const int64_t b = SWIGLU ? bn / 2 : bn;
      return (((a.M + bm - 1) / bm) * ((cols + b - 1) / b) + 255) / 256 * us;
    };
    // (Timed over 32 to 6400 tokens, 256 to 8192 columns, K from 256 to 8192.)
    const int64_t c0 = cost(64, 128, 22), c1 = cost(128, 128, 37), c2 = cost(128, 256, 64), c3 = cost(256, 256, 124);
    const int64_t best = std::min(std::min(c0, c1), std::min(c2, c3));
    if constexpr (!SWIGLU) {  // (a wave's 32 rows hold no gate and up pair)
      if (cost(64, 64, 17) < best) return launch_dma<64, 64, 2, 2, 128, 4, OUT, SWIGLU>(a, st);
    }
    if (best == c3) return launch_dma<256, 256, 2, 4, 128, 2, OUT, SWIGLU>(a, st);
    if (best == c2) return launch_dma<128, 256, 2, 4, 128, 3, OUT, SWIGLU>(a, st);
    if (best == c1) return launch_dma<128, 128, 4, 2, 128, 4, OUT, SWIGLU>(a, st);
    return launch_dma<64, 128, 2, 2, 128, 3, OUT, SWIGLU>(a, st);
  }
  static std::atomic<uint64_t> done{0};
  constexpr size_t lds = 2 * 256 * 128 + 4 * (128 + 2 * 128);
  if (!allow_lds(linear_any_kernel<OUT, SWIGLU>, lds, done)) return hip_failed();
  const uint32_t ny = static_cast<uint32_t>((a.M + 127) / 128);
  const uint32_t nx = static_cast<uint32_t>(SWIGLU ? (a.N / 2 + 63) / 64 : (a.N + 127) / 128);
  return launch(linear_any_kernel<OUT, SWIGLU>, nx * ny, 256, lds, st, a, nx);
}

template <int OUT>
int launch_linear(const LinearArgs& a, bool swiglu, bool aligned, hipStream_t st) {
  if (aligned) return swiglu ? launch_linear<OUT, true, true>(a, st) : launch_linear<OUT, false, true>(a, st);
  return swiglu ? launch_linear<OUT, true, false>(a, st) : launch_linear<OUT, false, false>(a, st);
}

}  // namespace

extern "C" {

size_t moe_gate_packed_bytes(int32_t E, int32_t D, int32_t wtype) {
  if (!gate_ok(E, D, wtype)) return 0;
  return static_cast<size_t>((E + 15) / 16) * 16 * D * (wtype == MOE_F32 ? 6 : 2);
}

int moe_gate_pack(const void* w, int32_t wtype, int32_t E, int32_t D, void* packed, size_t packed_bytes,
                  void* stream) {
  if (!w || !packed || !gate_ok(E, D, wtype)) return MOE_EINVAL;
  if (packed_bytes < moe_gate_packed_bytes(E, D, wtype)) return MOE_ENOSPACE;
  const int64_t n = static_cast<int64_t>((E + 15) / 16) * (D / 32) * 64;
  const uint32_t grid = static_cast<uint32_t>((n + 255) / 256);
  if (wtype == MOE_F32)
    return launch(gate_pack_kernel<MOE_F32>, grid, 256, 0, as_stream(stream), static_cast<const float*>(w), E, D,
                  static_cast<uint16_t*>(packed));
  return launch(gate_pack_kernel<MOE_BF16>, grid, 256, 0, as_stream(stream), static_cast<const uint16_t*>(w), E, D,
                static_cast<uint16_t*>(packed));
}

int moe_gate(const moe_gate_t* g, const void* x, int64_t ldx, int32_t B, float* logits, int64_t ldl, void* stream) {
  if (!g || !g->packed || !x || !logits || !gate_ok(g->E, g->D, g->wtype) || B < 1 || B > kMaxRows || ldx < g->D || ldx % 8 ||
      ldl < g->E || reinterpret_cast<uintptr_t>(x) % 16 || reinterpret_cast<uintptr_t>(g->packed) % 16)
    return MOE_EINVAL;
  const GateArgs a = {static_cast<const uint16_t*>(x), ldx, g->packed, B, g->E, g->D, logits, ldl};
  return g->wtype == MOE_F32 ? launch_gate<3>(a, as_stream(stream)) : launch_gate<1>(a, as_stream(stream));
}

int moe_route(const void* logits, int32_t type, int64_t ldl, int32_t B, int32_t E, int32_t topk,
              const moe_route_opts_t* opts, int32_t* ids, float* weights, void* stream) {
  moe_route_opts_t o;
  std::memset(&o, 0, sizeof(o));
  if (opts) o = *opts;
  if (!logits || !ids || !weights || !type_ok(type) || B < 1 || B > kMaxRows || E < 1 || E > 1024 || ldl < E || topk < 1 ||
      topk > 64 || topk > E || o.score < 0 || o.score > 1 || o.renorm < 0 || o.renorm > 1 || !std::isfinite(o.scale) ||
      o.groups < 0 || o.groups > 64 || o.group_score < 0 || o.group_score > 1)
    return MOE_EINVAL;
  if (o.groups == 0 ? o.topk_groups != 0
                    : E % o.groups || o.topk_groups < 1 || o.topk_groups > o.groups ||
                          topk > o.topk_groups * (E / o.groups))
    return MOE_EINVAL;
  const RouteArgs a = {logits,        ldl,      B,     E, topk, o.score, o.groups, o.topk_groups, o.group_score, o.renorm,
                       o.scale == 0.0f ? 1.0f : o.scale, o.bias_dev, ids, weights};
  hipStream_t st = as_stream(stream);
  if (type == MOE_F32) return launch_route<MOE_F32>(a, st);
  return type == MOE_F16 ? launch_route<MOE_F16>(a, st) : launch_route<MOE_BF16>(a, st);
}

int moe_quant_i8(const void* x, int32_t type, int64_t ldx, int32_t M, int32_t K, int8_t* codes, int64_t ldc,
                 float* scales, void* stream) {
  if (!x || !codes || !scales || !type_ok(type) || M < 1 || M > kMaxRows || K < 1 || K > 131072 || ldx < K || ldc < K)
    return MOE_EINVAL;
  hipStream_t st = as_stream(stream);
  if (type == MOE_F32) return launch_quant<MOE_F32>(x, ldx, M, K, codes, ldc, scales, st);
  if (type == MOE_F16) return launch_quant<MOE_F16>(x, ldx, M, K, codes, ldc, scales, st);
  return launch_quant<MOE_BF16>(x, ldx, M, K, codes, ldc, scales, st);
}

int moe_linear_i8(const int8_t* a, int64_t lda, const float* sa, const int8_t* w, int64_t ldw, const float* sw,
                  int32_t M, int32_t N, int32_t K, const moe_linear_opts_t* opts, void* out, int32_t out_type,
                  int64_t ldo, void* stream) {
  moe_linear_opts_t o;
  std::memset(&o, 0, sizeof(o));
  if (opts) o = *opts;
  constexpr int64_t kMaxLd = 1 << 22;
  if (!a || !sa || !w || !sw || !out || !type_ok(out_type) || M < 1 || M > kMaxRows || N < 1 || N > 1 << 20 ||
      static_cast<int64_t>(M) * N > 1LL << 34 || K < 1 || K > 131071 || lda < K ||
      ldw < K || lda >= kMaxLd || ldw >= kMaxLd || o.act < 0 || o.act > 1 || (o.act == 1 && N % 2))
    return MOE_EINVAL;
  const int32_t cols = o.act == 1 ? N / 2 : N;
  if (ldo < cols || (o.add_dev && o.ldadd < cols)) return MOE_EINVAL;
  const LinearArgs r = {a, w, sa, sw, o.bias_dev, o.add_dev, out, lda, ldw, ldo, o.ldadd, M, N, K};
  const bool aligned =
      (reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(w) | lda | ldw | static_cast<uintptr_t>(K)) % 16 == 0;
  hipStream_t st = as_stream(stream);
  if (out_type == MOE_F32) return launch_linear<MOE_F32>(r, o.act == 1, aligned, st);
  if (out_type == MOE_F16) return launch_linear<MOE_F16>(r, o.act == 1, aligned, st);
  return launch_linear<MOE_BF16>(r, o.act == 1, aligned, st);
}

}  // extern "C"
