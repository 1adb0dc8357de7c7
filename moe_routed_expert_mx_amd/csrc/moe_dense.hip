// moe_dense.hip -- MI355X (gfx950) kernels of the dense side of a routed-experts layer: the
// router in front of the experts (product and top-k choice) and the int8 products of a
// shared expert beside them, behind the C ABI of include/moe_mx.h.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

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
  int32_t B, E, topk, groups, kept, group_score, renorm;
  float scale;
  const float* bias;
  int32_t* ids;
  float* weights;
};

// One wave per token; lane l holds experts l, l + 64, ...  The choice stays in FP64.
template <int TYPE, bool SIGMOID, int NV>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs a) {
  extern __shared__ double route_lds[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + wave;
  double* vals = route_lds + static_cast<size_t>(wave) * (a.E + 64);
  double* rank = vals + a.E;
  const bool live = t < a.B;
  const double kNone = -__builtin_huge_val();
  const typename Elem<TYPE>::T* row =
      static_cast<const typename Elem<TYPE>::T*>(a.logits) + (live ? t : 0) * a.ldl;
  float l[NV];
  float m = -__builtin_huge_valf();
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = lane + 64 * j;
    float v = -__builtin_huge_valf();
    if (e < a.E) {
      v = to_f32<TYPE>(row[e]);
      if (v != v) v = -__builtin_huge_valf();
    }
    l[j] = v;
    m = fmaxf(m, v);
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
  auto score_of = [&](float v) -> double {  // softmax: without the common denominator
    if (v == -__builtin_huge_valf()) return 0.0;
    if (SIGMOID) return 1.0 / (1.0 + exp(-static_cast<double>(v)));
    return v == m ? 1.0 : exp(static_cast<double>(v) - static_cast<double>(m));
  };
  double denom = 1.0;
  if (!SIGMOID && (!a.renorm || a.bias)) {
    denom = 0.0;
#pragma unroll
    for (int j = 0; j < NV; ++j) denom += score_of(l[j]);
#pragma unroll
    for (int d = 32; d; d >>= 1) denom += __shfl_xor(denom, d);
    if (denom < 1.0) denom = 1.0;  // every expert masked
  }
  double c[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = lane + 64 * j;
    double v = l[j];
    if (a.bias && e < a.E) v = score_of(l[j]) / denom + static_cast<double>(a.bias[e]);
    if (l[j] == -__builtin_huge_valf() || v != v) v = kNone;
    c[j] = v;
  }
  bool taken[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) taken[j] = lane + 64 * j >= a.E;
  if (a.groups) {
    const int size = a.E / a.groups;
    const bool sums = a.group_score == 1;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e = lane + 64 * j;
      if (e < a.E) vals[e] = sums && !a.bias && c[j] != kNone ? score_of(l[j]) / denom : c[j];
    }
    __syncthreads();
    double r = kNone;
    if (lane < a.groups) {
      double v1 = kNone, v2 = kNone;
      for (int i = 0; i < size; ++i) {
        const double v = vals[lane * size + i];
        if (v > v1) {
          v2 = v1;
          v1 = v;
        } else if (v > v2) {
          v2 = v;
        }
      }
      r = sums && v2 != kNone ? v1 + v2 : v1;
      rank[lane] = r;
    }
    __syncthreads();
    bool keep = false;
    if (lane < a.groups) {
      int before = 0;
      for (int g = 0; g < a.groups; ++g) before += rank[g] > r || (rank[g] == r && g < lane);
      keep = before < a.kept;
    }
    const uint64_t kept = __ballot(keep);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e = lane + 64 * j;
      if (e < a.E && !((kept >> (e / size)) & 1)) taken[j] = true;
    }
  }
  int my_id = 0;
  float my_logit = -__builtin_huge_valf();
  for (int k = 0; k < a.topk; ++k) {
    double bv = kNone;
    int bi = 0x7fffffff;
    float bl = -__builtin_huge_valf();
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (!taken[j] && (bi == 0x7fffffff || c[j] > bv)) {
        bv = c[j];
        bi = lane + 64 * j;
        bl = l[j];
      }
#pragma unroll
    for (int d = 32; d; d >>= 1) {
      const double ov = __shfl_xor(bv, d);
      const int oi = __shfl_xor(bi, d);
      const float ol = __shfl_xor(bl, d);
      if (ov > bv || (ov == bv && oi < bi)) {
        bv = ov;
        bi = oi;
        bl = ol;
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (lane + 64 * j == bi) taken[j] = true;
    if (lane == k) {
      my_id = bi;
      my_logit = bl;
    }
  }
  double w = lane < a.topk ? score_of(my_logit) : 0.0;
  if (a.renorm) {
    double total = w;
#pragma unroll
    for (int d = 32; d; d >>= 1) total += __shfl_xor(total, d);
    w = total > 0.0 ? w / total : 0.0;
  } else {
    w /= denom;
  }
  if (live && lane < a.topk) {
    a.ids[t * a.topk + lane] = my_id;
    a.weights[t * a.topk + lane] = static_cast<float>(w * static_cast<double>(a.scale));
  }
}

// --------------------------------------------------------------------- quant
// One workgroup per token: the row's largest magnitude, then the codes.
// code = x * 127 / amax, half to even, exactly: x * 127 - r * amax is exact in FP64, so the
// rounded guess r is corrected by comparing it with half a step.
__device__ __forceinline__ int quant_code(double x, double amax, double inv) {
  const double n = x * 127.0;
  double r = __builtin_rint(n * inv);
  const double d = 2.0 * (n - r * amax);
  const bool odd = (static_cast<int>(r) & 1) != 0;
  if (d > amax || (d == amax && odd)) r += 1.0;
  else if (d < -amax || (d == -amax && odd)) r -= 1.0;
  return static_cast<int>(r);
}

template <int TYPE>
__global__ __launch_bounds__(256) void quant_kernel(const void* x, int64_t ldx, int32_t M, int32_t K,
                                                    int8_t* codes, int64_t ldc, float* scales) {
  __shared__ uint32_t part[4];
  const int64_t row = blockIdx.x;
  const typename Elem<TYPE>::T* p = static_cast<const typename Elem<TYPE>::T*>(x) + row * ldx;
  uint32_t top = 0;  // magnitudes order as their bits, infinity and NaN above all
  for (int k = threadIdx.x; k < K; k += 256) {
    const uint32_t b = __float_as_uint(to_f32<TYPE>(p[k])) & 0x7fffffffu;
    top = b > top ? b : top;
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    const uint32_t o = static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), d));
    top = o > top ? o : top;
  }
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
  __syncthreads();
  for (int i = 0; i < 4; ++i) top = part[i] > top ? part[i] : top;
  const float amax = __uint_as_float(top);
  const bool finite = top < 0x7f800000u;
  int8_t* q = codes + row * ldc;
  if (top == 0 || !finite) {
    for (int k = threadIdx.x; k < K; k += 256) q[k] = 0;
    if (threadIdx.x == 0) scales[row] = finite ? 0.0f : __builtin_nanf("");
    return;
  }
  const double inv = 1.0 / static_cast<double>(amax);
  for (int k = threadIdx.x; k < K; k += 256)
    q[k] = static_cast<int8_t>(quant_code(static_cast<double>(to_f32<TYPE>(p[k])), static_cast<double>(amax), inv));
  if (threadIdx.x == 0) scales[row] = amax / 127.0f;
}

// ---------------------------------------------------------------------- gate
// Packed router weight: [E/16][D/32][plane][64 lanes][8 BF16], lane l of a run holding
// expert l % 16, features 8 * (l / 16) .. + 7 of the step: an operand of the 16x16x32 MFMA.
template <int WTYPE>
__global__ __launch_bounds__(256) void gate_pack_kernel(const void* w, int32_t E, int32_t D, uint16_t* packed) {
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
    uint16_t* out = packed + run * P * 512 + lane * 8 + j;
    if constexpr (WTYPE == MOE_F32) {
      // upper, middle and lower eight bits of the significand, each cut off towards zero
      // and exactly a BF16; the differences are exact
      float v = e < E ? static_cast<const float*>(w)[static_cast<int64_t>(e) * D + k + j] : 0.0f;
      for (int p = 0; p < 3; ++p) {
        const uint32_t b = __float_as_uint(v);
        const bool finite = (b & 0x7fffffffu) < 0x7f800000u;
        uint16_t h = static_cast<uint16_t>(b >> 16);
        if (!finite && (b & 0x7fffffu)) h |= 0x40;
        out[p * 512] = h;
        v = finite ? v - bf16_to_f32(h) : 0.0f;
      }
    } else {
      out[0] = e < E ? static_cast<const uint16_t*>(w)[static_cast<int64_t>(e) * D + k + j] : 0;
    }
  }
}

struct GateArgs {
  const uint16_t* x;
  int64_t ldx;
  const uint16_t* packed;
  int32_t B, E, D;
  float* logits;
  int64_t ldl;
};

// A workgroup's tile is 16 TT tokens x 16 ET experts; its WV waves take a share of the features
// each, read both operands straight into registers (no byte is read twice in a workgroup, so
// LDS would serve nothing) and add their FP32 tiles through LDS in wave order.
template <int P, int TT, int ET, int WV>
__global__ __launch_bounds__(64 * WV) void gate_kernel(GateArgs a, uint32_t cols, uint32_t rows) {
  extern __shared__ float gate_lds[];
  constexpr int kOut = 256 * TT * ET;           // outputs of the tile
  // steps in flight: of x, which comes from HBM, and of the weight, which L2 holds
  constexpr int UX = TT * ET >= 8 ? 8 : 4, UW = TT * ET >= 8 ? 2 : 4;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // the tiles of one token range run on one XCD (workgroups go round the eight), so that its L2
  // serves x to all of them
  const uint32_t span = 8 * cols, row = blockIdx.x / span * 8 + blockIdx.x % 8, col = blockIdx.x % span / 8;
  if (row >= rows) return;
  const int64_t t0 = static_cast<int64_t>(row) * (16 * TT);
  const int tiles = (a.E + 15) / 16, steps = a.D / 32, n = steps / WV, s0 = wave * n;
  const uint16_t* xp[TT];
  const uint16_t* wp[ET];
#pragma unroll
  for (int i = 0; i < TT; ++i) {
    const int64_t t = t0 + i * 16 + (lane & 15);
    xp[i] = a.x + (t < a.B ? t : a.B - 1) * a.ldx + s0 * 32 + (lane >> 4) * 8;
  }
#pragma unroll
  for (int i = 0; i < ET; ++i) {
    const int et = static_cast<int>(col) * ET + i;
    wp[i] = a.packed + (static_cast<int64_t>(et < tiles ? et : tiles - 1) * steps + s0) * (P * 512) + lane * 8;
  }
  v4f acc[TT][ET] = {};
  v8bf xb[UX][TT], wb[UW][ET][P];
  auto load_x = [&](int u, int s) {
    s = s < n ? s : n - 1;  // past the end: loaded again, not used
#pragma unroll
    for (int i = 0; i < TT; ++i) xb[u][i] = *reinterpret_cast<const v8bf*>(xp[i] + s * 32);
  };
  auto load_w = [&](int u, int s) {
    s = s < n ? s : n - 1;
#pragma unroll
    for (int i = 0; i < ET; ++i)
#pragma unroll
      for (int p = 0; p < P; ++p) wb[u][i][p] = *reinterpret_cast<const v8bf*>(wp[i] + (s * P + p) * 512);
  };
#pragma unroll
  for (int u = 0; u < UX; ++u) load_x(u, u);
#pragma unroll
  for (int u = 0; u < UW; ++u) load_w(u, u);
  compiler_fence();  // the loads stay where they are written, steps ahead of their use
  for (int s = 0; s < n; s += UX) {
#pragma unroll
    for (int u = 0; u < UX; ++u) {
      if (s + u < n) {
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int i = 0; i < ET; ++i)
#pragma unroll
            for (int j = 0; j < TT; ++j)
              acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[u % UW][i][p], xb[u][j], acc[j][i], 0, 0, 0);
        load_x(u, s + u + UX);
        load_w(u % UW, s + u + UW);
        compiler_fence();
      }
    }
  }
  // [wave][token][expert], padded by a word a row
  constexpr int kRow = 16 * ET + 4;
#pragma unroll
  for (int j = 0; j < TT; ++j)
#pragma unroll
    for (int i = 0; i < ET; ++i)
      *reinterpret_cast<v4f*>(gate_lds + (wave * 16 * TT + j * 16 + (lane & 15)) * kRow + i * 16 + (lane >> 4) * 4) =
          acc[j][i];
  __syncthreads();
  for (int o = threadIdx.x; o < kOut; o += 64 * WV) {
    const int tok = o / (16 * ET), e = o % (16 * ET);
    float v = gate_lds[tok * kRow + e];
#pragma unroll
    for (int w = 1; w < WV; ++w) v += gate_lds[(w * 16 * TT + tok) * kRow + e];
    const int64_t t = t0 + tok;
    const int ge = static_cast<int>(col) * 16 * ET + e;
    if (t < a.B && ge < a.E) a.logits[t * a.ldl + ge] = v;
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

// 16 bytes of a row from k on, zeros from K on; any alignment, nothing read past the row.
__device__ __forceinline__ uint4 row16(const int8_t* row, int k, int K, bool live) {
  uint4 v = {0, 0, 0, 0};
  if (!live || k >= K) return v;
  if (k + 16 <= K) {
    __builtin_memcpy(&v, row + k, 16);
    return v;
  }
  uint32_t u[4] = {0, 0, 0, 0};
  for (int i = 0; i < K - k; ++i)
    u[i >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(row[k + i])) << (8 * (i & 3));
  v = {u[0], u[1], u[2], u[3]};
  return v;
}

__device__ __forceinline__ v4i bits(uint4 v) {
  return v4i{static_cast<int>(v.x), static_cast<int>(v.y), static_cast<int>(v.z), static_cast<int>(v.w)};
}
__device__ __forceinline__ float silu(float g) { return g / (1.0f + __expf(-g)); }

// ------------------------------------------------- linear: up to 64 tokens
// The weight is read once, so its bytes bound the product.  A workgroup takes 16 weight rows
// (SwiGLU: 16 gate rows and their 16 up rows) and all tokens; its WV waves split K, read both
// operands straight into registers some chunks of 64 bytes ahead, and add their 32-bit sums
// through LDS.
template <int OUT, bool SWIGLU, bool ALIGNED, int TT, int WV>
__global__ __launch_bounds__(64 * WV) void linear_stream_kernel(LinearArgs a) {
  extern __shared__ int stream_lds[];
  constexpr int RT = SWIGLU ? 2 : 1, U = RT + TT >= 5 ? 4 : 8;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int H = SWIGLU ? a.N / 2 : a.N, n0 = blockIdx.x * 16;
  const int chunks = (a.K + 63) / 64, per = (chunks + WV - 1) / WV, c0 = wave * per;
  const int n = chunks - c0 < per ? (chunks > c0 ? chunks - c0 : 0) : per;
  const int r = lane & 15, q = lane >> 4;
  const int8_t *wp[RT], *ap[TT];
  const int row = n0 + r < H ? n0 + r : H - 1;
#pragma unroll
  for (int i = 0; i < RT; ++i) wp[i] = a.w + (static_cast<int64_t>(row) + i * H) * a.ldw;
#pragma unroll
  for (int i = 0; i < TT; ++i) ap[i] = a.a + static_cast<int64_t>(i * 16 + r < a.M ? i * 16 + r : a.M - 1) * a.lda;
  v4i acc[RT][TT] = {}, wb[U][RT], ab[U][TT];
  // aligned: an operand's 16 bytes lie wholly inside the row or wholly behind it; those behind
  // are read from the row's last 16 and set to zero when used
  auto load = [&](int u, int c) {
    const int k = (c0 + c) * 64 + q * 16;
    if constexpr (ALIGNED) {
      const int kc = k < a.K ? k : a.K - 16;
#pragma unroll
      for (int i = 0; i < RT; ++i) wb[u][i] = *reinterpret_cast<const v4i*>(wp[i] + kc);
#pragma unroll
      for (int i = 0; i < TT; ++i) ab[u][i] = *reinterpret_cast<const v4i*>(ap[i] + kc);
    } else {
#pragma unroll
      for (int i = 0; i < RT; ++i) wb[u][i] = bits(row16(wp[i], k, a.K, true));
#pragma unroll
      for (int i = 0; i < TT; ++i) ab[u][i] = bits(row16(ap[i], k, a.K, true));
    }
  };
  if (n > 0) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (u < n) load(u, u);
    compiler_fence();
    for (int c = 0; c < n; c += U) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c + u < n) {
          if (ALIGNED && (c0 + c + u) * 64 + 64 > a.K) {
            const bool in = (c0 + c + u) * 64 + q * 16 < a.K;
#pragma unroll
            for (int i = 0; i < RT; ++i) wb[u][i] = in ? wb[u][i] : v4i{0, 0, 0, 0};
          }
#pragma unroll
          for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int j = 0; j < TT; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wb[u][i], ab[u][j], acc[i][j], 0, 0, 0);
          if (c + u + U < n) load(u, c + u + U);
          compiler_fence();
        }
    }
  }
  // [wave][token][weight row], padded by four words a row
  constexpr int kRow = 16 * RT + 4, kTile = 16 * TT * kRow;
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < TT; ++j)
      *reinterpret_cast<v4i*>(stream_lds + wave * kTile + (j * 16 + r) * kRow + i * 16 + q * 4) = acc[i][j];
  __syncthreads();
  using T = typename Elem<OUT>::T;
  for (int o = threadIdx.x; o < 256 * TT; o += 64 * WV) {
    const int m = o >> 4, c = n0 + (o & 15);
    if (m >= a.M || c >= H) continue;
    const int* p = stream_lds + m * kRow + (o & 15);
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
               : "memory");
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

// Workgroup tile of BM tokens x BN weight rows, four waves of half by half each, 32x32x32
// MFMAs with the weight as the row operand (a lane then holds four neighbouring columns of out).
// K goes through LDS in stages of 64 bytes a row, four in flight; a row's four 16-byte parts lie
// permuted by its index, so that eight neighbouring rows' reads meet all banks once.
template <int BM, int BN, int OUT, bool SWIGLU>
__global__ __launch_bounds__(256, BM * BN >= 65536 ? 1 : 2) void linear_dma_kernel(LinearArgs a, uint32_t nm,
                                                                                   uint32_t nn, uint32_t per_xcd) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  constexpr int NS = 4, kStage = (BM + BN) * 64, RA = BM / 64, RW = BN / 64;
  static_assert(!SWIGLU || BN >= 128, "a wave holds whole gate and up pairs");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // each XCD (workgroups go round the eight) takes a contiguous range of tiles, in groups of
  // eight token tiles: what runs at once on an XCD shares operands in its L2
  const uint32_t tile = blockIdx.x % 8 * per_xcd + blockIdx.x / 8;
  if (blockIdx.x / 8 >= per_xcd || tile >= nm * nn) return;
  const uint32_t band = tile / (8 * nn), left = nm - band * 8, height = left < 8 ? left : 8, in = tile - band * 8 * nn;
  const int64_t m0 = static_cast<int64_t>(band * 8 + in % height) * BM;
  const int H = SWIGLU ? a.N / 2 : a.N, n0 = static_cast<int>(in / height) * (SWIGLU ? BN / 2 : BN);
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) void*)smem));

  // what this lane moves: 16-byte part `ch` of rows lane / 4 of its wave's 16-row blocks
  const int ch = (lane & 3) ^ ((lane >> 3) & 3), lr = lane >> 2;
  const int mrows = a.M - m0 < BM ? static_cast<int>(a.M - m0) : BM;
  const v4i ra = make_rsrc(a.a + m0 * a.lda, static_cast<uint32_t>((mrows - 1) * a.lda + a.K));
  uint32_t va[RA], vw[RW];
  v4i rw[RW];
  {
    const int cols = SWIGLU ? BN / 2 : BN, nrows = H - n0 < cols ? H - n0 : cols;
    const uint32_t bytes = static_cast<uint32_t>((nrows - 1) * a.ldw + a.K);
#pragma unroll
    for (int i = 0; i < RA; ++i) {
      const int row = (wave * RA + i) * 16 + lr;
      va[i] = row < mrows ? static_cast<uint32_t>(row * a.lda) + ch * 16 : kOutside;
    }
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      // SwiGLU: 32 gate rows, then their 32 up rows, and so on
      const int b = wave * RW + i, row = SWIGLU ? (b >> 2) * 32 + (b & 1) * 16 + lr : b * 16 + lr;
      rw[i] = make_rsrc(a.w + (n0 + (SWIGLU ? static_cast<int64_t>((b >> 1) & 1) * H : 0)) * a.ldw, bytes);
      vw[i] = row < nrows ? static_cast<uint32_t>(row * a.ldw) + ch * 16 : kOutside;
    }
  }
  auto issue = [&](int s) {
    const int k0 = s * 64;
    const uint32_t dst = lds0 + (s % NS) * kStage;
    const bool in_k = k0 + ch * 16 < a.K;  // parts behind K, and whole stages behind it: zeros
#pragma unroll
    for (int i = 0; i < RA; ++i) dma16(ra, in_k ? va[i] : kOutside, k0, dst + (wave * RA + i) * 1024);
#pragma unroll
    for (int i = 0; i < RW; ++i) dma16(rw[i], in_k ? vw[i] : kOutside, k0, dst + BM * 64 + (wave * RW + i) * 1024);
  };

  const int wm = (wave & 1) * (BM / 2), wn = (wave >> 1) * (BN / 2);
  constexpr int TM = BM / 64, TN = BN / 64;
  uint32_t la[2];  // this lane's operand inside a 32-row tile, for the stage's two halves
#pragma unroll
  for (int h = 0; h < 2; ++h) la[h] = (lane & 31) * 64 + (((h * 2 + (lane >> 5)) ^ ((lane >> 1) & 3)) << 4);
  v16i acc[TN][TM] = {};
  v4i fa[2][TM], fw[2][TN];
  auto read = [&](int buf, int h) {
    const unsigned char* p = smem + buf * kStage + la[h];
#pragma unroll
    for (int j = 0; j < TM; ++j) fa[h][j] = *reinterpret_cast<const v4i*>(p + (wm + j * 32) * 64);
#pragma unroll
    for (int i = 0; i < TN; ++i) fw[h][i] = *reinterpret_cast<const v4i*>(p + (BM + wn + i * 32) * 64);
  };
  auto mult = [&](int h) {
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[h][i], fa[h][j], acc[i][j], 0, 0, 0);
  };
  const int n = (a.K + 63) / 64;
  constexpr int kIssue = RA + RW;
#pragma unroll
  for (int s = 0; s < NS; ++s) issue(s);
  wait_vm<kIssue * (NS - 1)>();
  __builtin_amdgcn_s_barrier();
  compiler_fence();
  read(0, 0);
  for (int s = 0; s < n; ++s) {
    read(s % NS, 1);
    mult(0);
    // this stage is read out and the next has landed, for every wave
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    wait_vm<kIssue * (NS - 2)>();
    __builtin_amdgcn_s_barrier();
    compiler_fence();
    issue(s + NS);
    read((s + 1) % NS, 0);
    mult(1);
  }
  wait_vm<0>();
  __syncthreads();

  // 32 tokens at a time through LDS, so that whole rows' pieces are stored
  using T = typename Elem<OUT>::T;
  constexpr int kCols = SWIGLU ? BN / 4 : BN / 2, kRow = kCols + 4, PER = 16 / sizeof(T);
  static_assert(4 * 32 * kRow * 4 <= NS * kStage, "epilogue fits the stages");
  float* buf = reinterpret_cast<float*>(smem) + wave * 32 * kRow;
  const int nw = n0 + (SWIGLU ? wn / 2 : wn);
  const bool vec = (reinterpret_cast<uintptr_t>(a.out) | (a.ldo * sizeof(T))) % 16 == 0 &&
                   (!a.add || (reinterpret_cast<uintptr_t>(a.add) | (a.ldadd * sizeof(T))) % 16 == 0);
#pragma unroll
  for (int j = 0; j < TM; ++j) {
    const int64_t mt = m0 + wm + j * 32, mrow = mt + (lane & 31);
    const float sa = a.sa[mrow < a.M ? mrow : a.M - 1];
#pragma unroll
    for (int i = 0; i < TN; i += SWIGLU ? 2 : 1)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int c = (SWIGLU ? i * 16 : i * 32) + g * 8 + (lane >> 5) * 4;
        v4f y;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int col = nw + c + e < H ? nw + c + e : H - 1;
          y[e] = static_cast<float>(acc[i][j][g * 4 + e]) * sa * a.sw[col] + (a.bias ? a.bias[col] : 0.0f);
          if (SWIGLU)
            y[e] = silu(y[e]) * (static_cast<float>(acc[i + (SWIGLU ? 1 : 0)][j][g * 4 + e]) * sa * a.sw[H + col] +
                                 (a.bias ? a.bias[H + col] : 0.0f));
        }
        *reinterpret_cast<v4f*>(buf + (lane & 31) * kRow + c) = y;
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

// Workgroup tile of 64 tokens x 64 weight rows, 128 bytes of K a step, through LDS.
template <int OUT, bool SWIGLU>
__global__ __launch_bounds__(256) void linear_tile_kernel(LinearArgs a, uint32_t nx) {
  __shared__ uint4 lds_a[64 * 8], lds_w[64 * 8];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x / nx) * 64;
  const int H = SWIGLU ? a.N / 2 : a.N;
  const int n0 = (blockIdx.x % nx) * (SWIGLU ? 32 : 64);
  // weight row of the tile's row r: with SwiGLU 16 gate rows, then their 16 up rows, twice
  auto wrow = [&](int r) {
    if (!SWIGLU) return n0 + r < a.N ? n0 + r : -1;
    const int j = n0 + (r >> 5) * 16 + (r & 15);
    return j < H ? j + ((r >> 4) & 1) * H : -1;
  };
  const int wm = (wave & 1) * 32, wn = (wave >> 1) * 32;
  v4i acc[2][2] = {};
  for (int k0 = 0; k0 < a.K; k0 += 128) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = threadIdx.x + 256 * i, r = c >> 3, ch = c & 7;
      lds_a[r * 8 + (ch ^ (r & 7))] = row16(a.a + (m0 + r) * a.lda, k0 + ch * 16, a.K, m0 + r < a.M);
      const int n = wrow(r);
      lds_w[r * 8 + (ch ^ (r & 7))] = row16(a.w + static_cast<int64_t>(n) * a.ldw, k0 + ch * 16, a.K, n >= 0);
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      v4i fw[2], fa[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int rw = wn + i * 16 + (lane & 15), ra = wm + i * 16 + (lane & 15), ch = s * 4 + (lane >> 4);
        fw[i] = *reinterpret_cast<const v4i*>(&lds_w[rw * 8 + (ch ^ (rw & 7))]);
        fa[i] = *reinterpret_cast<const v4i*>(&lds_a[ra * 8 + (ch ^ (ra & 7))]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[i], fa[j], acc[i][j], 0, 0, 0);
    }
  }
  using T = typename Elem<OUT>::T;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t m = m0 + wm + j * 16 + (lane & 15);
    if (m >= a.M) continue;
    const float sa = a.sa[m];
#pragma unroll
    for (int i = 0; i < (SWIGLU ? 1 : 2); ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = SWIGLU ? n0 + (wn >> 1) + (lane >> 4) * 4 + q : n0 + wn + i * 16 + (lane >> 4) * 4 + q;
        if (n >= H) continue;
        float y = static_cast<float>(acc[i][j][q]) * sa * a.sw[n] + (a.bias ? a.bias[n] : 0.0f);
        if (SWIGLU) {
          const float up = static_cast<float>(acc[1][j][q]) * sa * a.sw[H + n] + (a.bias ? a.bias[H + n] : 0.0f);
          y = silu(y) * up;
        }
        if (a.add) y += to_f32<OUT>(static_cast<const T*>(a.add)[m * a.ldadd + n]);
        static_cast<T*>(a.out)[m * a.ldo + n] = from_f32<OUT>(y);
      }
  }
}

// ---------------------------------------------------------------------- host
hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }
int launch_status() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_EHIP; }
constexpr int32_t kMaxRows = 1 << 22;  // tokens of one call: its grids stay within the launch limits
bool type_ok(int32_t t) { return t == MOE_BF16 || t == MOE_F16 || t == MOE_F32; }
bool gate_ok(int32_t E, int32_t D, int32_t wtype) {
  return E >= 1 && E <= 1024 && D >= 512 && D <= 16384 && D % 512 == 0 && (wtype == MOE_BF16 || wtype == MOE_F32);
}

template <int TYPE, bool SIG>
void launch_route(const RouteArgs& a, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>((a.B + 3LL) / 4));
  const size_t lds = a.groups ? 4 * sizeof(double) * (a.E + 64) : 0;
  if (a.E <= 256) hipLaunchKernelGGL((route_kernel<TYPE, SIG, 4>), grid, dim3(256), lds, st, a);
  else hipLaunchKernelGGL((route_kernel<TYPE, SIG, 16>), grid, dim3(256), lds, st, a);
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
  constexpr size_t lds = sizeof(float) * WV * 16 * TT * (16 * ET + 4);
  static_assert(lds <= 160 * 1024, "gate tile");
  if (!allow_lds(gate_kernel<P, TT, ET, WV>, lds, done)) return MOE_EHIP;
  const uint32_t cols = ((a.E + 15) / 16 + ET - 1) / ET, rows = static_cast<uint32_t>((a.B + 16 * TT - 1) / (16 * TT));
  hipLaunchKernelGGL((gate_kernel<P, TT, ET, WV>), dim3((rows + 7) / 8 * 8 * cols), dim3(64 * WV), lds, st, a, cols,
                     rows);
  return launch_status();
}

template <int P>
int launch_gate(const GateArgs& a, hipStream_t st) {
  if (a.B <= 1024) return launch_gate_tile<P, 1, 1, 16>(a, st);
  return launch_gate_tile<P, 4, 5, 4>(a, st);
}

template <int OUT, bool SWIGLU, bool ALIGNED, int TT, int WV>
int launch_stream(const LinearArgs& a, hipStream_t st) {
  static std::atomic<uint64_t> done{0};
  constexpr size_t lds = sizeof(int) * WV * 16 * TT * ((SWIGLU ? 32 : 16) + 4);
  if (!allow_lds(linear_stream_kernel<OUT, SWIGLU, ALIGNED, TT, WV>, lds, done)) return MOE_EHIP;
  const int cols = SWIGLU ? a.N / 2 : a.N;
  hipLaunchKernelGGL((linear_stream_kernel<OUT, SWIGLU, ALIGNED, TT, WV>), dim3((cols + 15) / 16), dim3(64 * WV), lds, st,
                     a);
  return launch_status();
}

template <int BM, int BN, int OUT, bool SWIGLU>
int launch_dma(const LinearArgs& a, hipStream_t st) {
  static std::atomic<uint64_t> done{0};
  constexpr size_t lds = 4 * (BM + BN) * 64;
  if (!allow_lds(linear_dma_kernel<BM, BN, OUT, SWIGLU>, lds, done)) return MOE_EHIP;
  const uint32_t nm = static_cast<uint32_t>((a.M + BM - 1) / BM), bn = SWIGLU ? BN / 2 : BN,
                 nn = static_cast<uint32_t>(((SWIGLU ? a.N / 2 : a.N) + bn - 1) / bn), per = (nm * nn + 7) / 8;
  hipLaunchKernelGGL((linear_dma_kernel<BM, BN, OUT, SWIGLU>), dim3(per * 8), dim3(256), lds, st, a, nm, nn, per);
  return launch_status();
}

template <int OUT, bool SWIGLU, bool ALIGNED>
int launch_linear(const LinearArgs& a, hipStream_t st) {
  if (a.M <= 16) return launch_stream<OUT, SWIGLU, ALIGNED, 1, 16>(a, st);
  if (a.M <= 32) return launch_stream<OUT, SWIGLU, ALIGNED, 2, 8>(a, st);
  if (a.M <= 64) return launch_stream<OUT, SWIGLU, ALIGNED, 4, 8>(a, st);
  if constexpr (ALIGNED) {
    // rounds of tiles over the CUs, weighed with the time of a tile
    const int64_t cols = SWIGLU ? a.N / 2 : a.N;
    auto rounds = [&](int bm, int bn) {
      const int64_t b = SWIGLU ? bn / 2 : bn;
      return (((a.M + bm - 1) / bm) * ((cols + b - 1) / b) + 255) / 256;
    };
    const int64_t big = rounds(256, 256) * 40, mid = rounds(128, 128) * 16;
    if (big <= mid) return launch_dma<256, 256, OUT, SWIGLU>(a, st);
    return launch_dma<128, 128, OUT, SWIGLU>(a, st);
  }
  const unsigned my = static_cast<unsigned>((a.M + 63) / 64);
  const unsigned nx = static_cast<unsigned>(SWIGLU ? (a.N / 2 + 31) / 32 : (a.N + 63) / 64);
  hipLaunchKernelGGL((linear_tile_kernel<OUT, SWIGLU>), dim3(nx * my), dim3(256), 0, st, a, nx);
  return launch_status();
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
  return static_cast<size_t>((E + 15) / 16) * 16 * D * 2 * (wtype == MOE_F32 ? 3 : 1);
}

int moe_gate_pack(const void* w, int32_t wtype, int32_t E, int32_t D, void* packed, size_t packed_bytes,
                  void* stream) {
  if (!w || !packed || !gate_ok(E, D, wtype)) return MOE_EINVAL;
  if (packed_bytes < moe_gate_packed_bytes(E, D, wtype)) return MOE_ENOSPACE;
  const int64_t n = static_cast<int64_t>((E + 15) / 16) * (D / 32) * 64;
  const dim3 grid(static_cast<unsigned>((n + 255) / 256));
  if (wtype == MOE_F32)
    hipLaunchKernelGGL(gate_pack_kernel<MOE_F32>, grid, dim3(256), 0, as_stream(stream), w, E, D,
                       static_cast<uint16_t*>(packed));
  else
    hipLaunchKernelGGL(gate_pack_kernel<MOE_BF16>, grid, dim3(256), 0, as_stream(stream), w, E, D,
                       static_cast<uint16_t*>(packed));
  return launch_status();
}

int moe_gate(const moe_gate_t* g, const void* x, int64_t ldx, int32_t B, float* logits, int64_t ldl, void* stream) {
  if (!g || !g->packed || !x || !logits || !gate_ok(g->E, g->D, g->wtype) || B < 1 || B > kMaxRows || ldx < g->D || ldx % 8 ||
      ldl < g->E || reinterpret_cast<uintptr_t>(x) % 16 || reinterpret_cast<uintptr_t>(g->packed) % 16)
    return MOE_EINVAL;
  const GateArgs a = {static_cast<const uint16_t*>(x), ldx,    static_cast<const uint16_t*>(g->packed), B, g->E, g->D,
                      logits,                          ldl};
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
  const RouteArgs a = {logits,        ldl,      B,      E,   topk,   o.groups, o.topk_groups,
                       o.group_score, o.renorm, o.scale == 0.0f ? 1.0f : o.scale, o.bias_dev, ids, weights};
  hipStream_t st = as_stream(stream);
  const int v = type * 2 + o.score;
  switch (v) {
    case MOE_BF16 * 2: launch_route<MOE_BF16, false>(a, st); break;
    case MOE_BF16 * 2 + 1: launch_route<MOE_BF16, true>(a, st); break;
    case MOE_F16 * 2: launch_route<MOE_F16, false>(a, st); break;
    case MOE_F16 * 2 + 1: launch_route<MOE_F16, true>(a, st); break;
    case MOE_F32 * 2: launch_route<MOE_F32, false>(a, st); break;
    default: launch_route<MOE_F32, true>(a, st); break;
  }
  return launch_status();
}

int moe_quant_i8(const void* x, int32_t type, int64_t ldx, int32_t M, int32_t K, int8_t* codes, int64_t ldc,
                 float* scales, void* stream) {
  if (!x || !codes || !scales || !type_ok(type) || M < 1 || M > kMaxRows || K < 1 || K > 131072 || ldx < K || ldc < K)
    return MOE_EINVAL;
  const dim3 grid(static_cast<unsigned>(M));
  hipStream_t st = as_stream(stream);
  if (type == MOE_F32) hipLaunchKernelGGL(quant_kernel<MOE_F32>, grid, dim3(256), 0, st, x, ldx, M, K, codes, ldc, scales);
  else if (type == MOE_F16)
    hipLaunchKernelGGL(quant_kernel<MOE_F16>, grid, dim3(256), 0, st, x, ldx, M, K, codes, ldc, scales);
  else hipLaunchKernelGGL(quant_kernel<MOE_BF16>, grid, dim3(256), 0, st, x, ldx, M, K, codes, ldc, scales);
  return launch_status();
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
