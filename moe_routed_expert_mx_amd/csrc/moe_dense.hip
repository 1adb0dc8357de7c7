// moe_dense.hip -- MI355X (gfx950) kernels of the dense side of a routed-experts layer: the
// router in front of the experts (product and top-k choice) and the int8 products of a
// shared expert beside them, behind the C ABI of include/moe_mx.h.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "moe_mx.h"

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

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

template <int P>
__global__ __launch_bounds__(256) void gate_kernel(GateArgs a) {
  constexpr int ET = 5;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 64 + wave * 16 + (lane & 15);
  const int et0 = blockIdx.y * ET, tiles = (a.E + 15) / 16, steps = a.D / 32;
  const uint16_t* xr = a.x + (t < a.B ? t : a.B - 1) * a.ldx + (lane >> 4) * 8;
  v4f acc[ET] = {};
  for (int s = 0; s < steps; ++s) {
    const v8bf b = *reinterpret_cast<const v8bf*>(xr + s * 32);
#pragma unroll
    for (int i = 0; i < ET; ++i) {
      const int et = et0 + i < tiles ? et0 + i : tiles - 1;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const v8bf w = *reinterpret_cast<const v8bf*>(
            a.packed + ((static_cast<int64_t>(et) * steps + s) * P + p) * 512 + lane * 8);
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, b, acc[i], 0, 0, 0);
      }
    }
  }
  if (t >= a.B) return;
#pragma unroll
  for (int i = 0; i < ET; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = (et0 + i) * 16 + (lane >> 4) * 4 + j;
      if (e < a.E) a.logits[t * a.ldl + e] = acc[i][j];
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

__device__ __forceinline__ float silu(float g) { return g / (1.0f + __expf(-g)); }

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

template <int OUT>
void launch_linear(const LinearArgs& a, bool swiglu, hipStream_t st) {
  const unsigned my = static_cast<unsigned>((a.M + 63) / 64);
  const unsigned nx = static_cast<unsigned>(swiglu ? (a.N / 2 + 31) / 32 : (a.N + 63) / 64);
  if (swiglu) hipLaunchKernelGGL((linear_tile_kernel<OUT, true>), dim3(nx * my), dim3(256), 0, st, a, nx);
  else hipLaunchKernelGGL((linear_tile_kernel<OUT, false>), dim3(nx * my), dim3(256), 0, st, a, nx);
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
  const dim3 grid(static_cast<unsigned>((B + 63LL) / 64), ((g->E + 15) / 16 + 4) / 5);
  if (g->wtype == MOE_F32) hipLaunchKernelGGL(gate_kernel<3>, grid, dim3(256), 0, as_stream(stream), a);
  else hipLaunchKernelGGL(gate_kernel<1>, grid, dim3(256), 0, as_stream(stream), a);
  return launch_status();
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
  hipStream_t st = as_stream(stream);
  if (out_type == MOE_F32) launch_linear<MOE_F32>(r, o.act == 1, st);
  else if (out_type == MOE_F16) launch_linear<MOE_F16>(r, o.act == 1, st);
  else launch_linear<MOE_BF16>(r, o.act == 1, st);
  return launch_status();
}

}  // extern "C"
