// moe_norm.hip -- MI355X (gfx950) kernels in front of a layer's products: the root-mean-square norm
// with the residual's addition and codes in 8 bits, and the quantization into blocks of e4m3, behind
// the C ABI of include/moe_mx.h.
#include <cmath>
#include <cstring>
#include <type_traits>

#include "dense_common.h"

namespace {

constexpr int VE = 8;  // elements of a lane's piece: 16 lanes hold a block of 128

template <int TYPE>
__device__ __forceinline__ void load8(float (&v)[VE], const typename Elem<TYPE>::T* p, int i, int K) {
  typename Elem<TYPE>::T t[VE];
  if ((i + 1) * VE <= K) {  // any alignment
    __builtin_memcpy(t, p + i * VE, sizeof(t));
  } else {
#pragma unroll
    for (int e = 0; e < VE; ++e) t[e] = i * VE + e < K ? p[i * VE + e] : typename Elem<TYPE>::T(0);
  }
#pragma unroll
  for (int e = 0; e < VE; ++e) v[e] = to_f32<TYPE>(t[e]);
}
__device__ __forceinline__ void store_codes(uint8_t* p, int i, int K, const uint32_t (&c)[2]) {
  if ((i + 1) * VE <= K) {
    __builtin_memcpy(p + i * VE, c, VE);
  } else {
#pragma unroll
    for (int e = 0; e < VE; ++e)
      if (i * VE + e < K) p[i * VE + e] = static_cast<uint8_t>(c[e / 4] >> (8 * (e & 3)));
  }
}
// Largest magnitude of the piece, as FP32 bits (which order as magnitudes, infinity and NaN above all).
__device__ __forceinline__ uint32_t top_of(const float (&v)[VE]) {
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < VE; ++e) {
    const uint32_t b = __float_as_uint(v[e]) & 0x7fffffffu;
    top = b > top ? b : top;
  }
  return top;
}

// The piece's e4m3 codes, 16 lanes sharing a block; returns the block's scale.  amax = m 2^k with
// 1 <= m < 2 and 448 = 1.75 * 2^8, so e = k - 8, or one more where m > 1.75.
__device__ __forceinline__ float codes_e4m3(const float (&v)[VE], uint32_t (&c)[2]) {
  const uint32_t top = lanes_max<16>(top_of(v));
  int e = static_cast<int>(top >> 23) - 135 + ((top & 0x7fffffu) > 0x600000u);
  e = e < -126 ? -126 : e;
  const bool finite = top < 0x7f800000u;
  const float inverse = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * g] * inverse, v[4 * g + 1] * inverse, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * g + 2] * inverse, v[4 * g + 3] * inverse, w, true);
    c[g] = finite ? static_cast<uint32_t>(w) : 0u;
  }
  if (!finite) return __builtin_nanf("");
  return top ? __uint_as_float(static_cast<uint32_t>(e + 127) << 23) : 0.0f;
}

// ------------------------------------------------------------- blocks of e4m3
// 16 lanes a block, four blocks a wave at once; a wave takes P runs of four blocks, all loaded before
// the first is used.  Bytes bound it: 16384 x 4096 BF16, 203 MB, 41.6 us, 4.9 TB/s (a copy 5.15).  Rows of less than 512
// leave lanes idle: 65536 x 128 13.1 us, 1.9 TB/s, 65536 x 384 18.8, 4.1.
template <int TYPE, int P>
__global__ __launch_bounds__(256) void quant_f8_kernel(const void* x, int64_t ldx, int32_t M, int32_t K, uint8_t* codes,
                                                       int64_t ldc, float* scales, int64_t lds, uint32_t runs) {
  using T = typename Elem<TYPE>::T;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint64_t u0 = (static_cast<uint64_t>(blockIdx.x) * 4 + wave) * P;
  float v[P][VE];
  int64_t row[P];
  int piece[P];
  row[0] = static_cast<int64_t>(u0 / runs);
  uint32_t run = static_cast<uint32_t>(u0 - static_cast<uint64_t>(row[0]) * runs);
#pragma unroll
  for (int p = 0; p < P; ++p) {
    if (p) {
      row[p] = row[p - 1];
      if (++run == runs) {
        run = 0;
        ++row[p];
      }
    }
    piece[p] = static_cast<int>(run) * 64 + lane;
#pragma unroll
    for (int e = 0; e < VE; ++e) v[p][e] = 0.0f;
    if (row[p] < M && piece[p] * VE < K) load8<TYPE>(v[p], static_cast<const T*>(x) + row[p] * ldx, piece[p], K);
  }
#pragma unroll
  for (int p = 0; p < P; ++p) {
    uint32_t c[2];
    const float scale = codes_e4m3(v[p], c);
    if (row[p] < M && piece[p] * VE < K) {
      store_codes(codes + row[p] * ldc, piece[p], K, c);
      if (lane % 16 == 0) scales[row[p] * lds + piece[p] / 16] = scale;
    }
  }
}

// ----------------------------------------------------------------------- norm
struct NormArgs {
  const void *x, *residual, *weight;
  void *total, *out;
  uint8_t* codes;
  float* scales;
  int64_t ldx, ldr, ldt, ldo, ldc, lds;
  double eps;
  int32_t M, K, format;
};

// Two values as 16-bit ones in a word.
template <int TYPE>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  typedef std::conditional_t<TYPE == MOE_BF16, __bf16, _Float16> E;
  typedef E v2 __attribute__((ext_vector_type(2)));
  const v2 v = {static_cast<E>(a), static_cast<E>(b)};
  uint32_t w;
  __builtin_memcpy(&w, &v, 4);
  return w;
}
// 8 elements as they lie in memory.
template <int TYPE>
struct Piece {
  static constexpr int N = TYPE == MOE_F32 ? 8 : 4;
  uint32_t w[N];
  __device__ __forceinline__ float at(int e) const {
    if constexpr (TYPE == MOE_F32) return __uint_as_float(w[e]);
    else return to_f32<TYPE>(static_cast<uint16_t>(e & 1 ? w[e >> 1] >> 16 : w[e >> 1]));
  }
  __device__ __forceinline__ void set2(int e, float a, float b) {
    if constexpr (TYPE == MOE_F32) {
      w[e] = __float_as_uint(a);
      w[e + 1] = __float_as_uint(b);
    } else {
      w[e >> 1] = pack2<TYPE>(a, b);
    }
  }
  __device__ __forceinline__ void load(const typename Elem<TYPE>::T* p, int i, int K) {  // any alignment; zeros behind K
    if ((i + 1) * VE <= K) {
      __builtin_memcpy(w, p + i * VE, sizeof(w));
    } else {
      typename Elem<TYPE>::T t[VE];
#pragma unroll
      for (int e = 0; e < VE; ++e) t[e] = i * VE + e < K ? p[i * VE + e] : typename Elem<TYPE>::T(0);
      __builtin_memcpy(w, t, sizeof(w));
    }
  }
  __device__ __forceinline__ void store(typename Elem<TYPE>::T* p, int i, int K) const {
    if ((i + 1) * VE <= K) {
      __builtin_memcpy(p + i * VE, w, sizeof(w));
    } else {
      typename Elem<TYPE>::T t[VE];
      __builtin_memcpy(t, w, sizeof(w));
#pragma unroll
      for (int e = 0; e < VE; ++e)
        if (i * VE + e < K) p[i * VE + e] = t[e];
    }
  }
};

// W waves a row, which they hold in registers, in its own type: NV pieces of 8 elements a lane.  One pass over
// the data; bytes bound it: 16384 x 3584 BF16 with residual, total, out and e4m3 codes, 530 MB, 98 us, 5.4 TB/s (a copy
// 5.15; half of the input came from the memory-side cache; held as FP32 instead it took 177 us).  The sum of squares is FP64 (two instructions an element, hidden behind the
// loads), so that r, and with it every code, is the same however the sum is cut.
template <int TYPE, int WTYPE, int W, int NV>
__global__ __launch_bounds__(256) void norm_kernel(NormArgs a) {
  using T = typename Elem<TYPE>::T;
  using TW = typename Elem<WTYPE>::T;
  __shared__ double part_sum[4];
  __shared__ uint32_t part_top[4];
  const int lane = threadIdx.x % (64 * W), wave = threadIdx.x >> 6;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (4 / W) + threadIdx.x / (64 * W);
  if (W == 1 && row >= a.M) return;
  const int K = a.K;
  const T* const x = static_cast<const T*>(a.x) + row * a.ldx;
  const T* const residual = static_cast<const T*>(a.residual) + row * a.ldr;
  Piece<TYPE> h[NV] = {};
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = lane + 64 * W * j;
    if (i * VE < K) h[j].load(x, i, K);
  }
  if (a.residual) {
    Piece<TYPE> r[NV] = {};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = lane + 64 * W * j;
      if (i * VE < K) r[j].load(residual, i, K);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < VE; e += 2) h[j].set2(e, h[j].at(e) + r[j].at(e), h[j].at(e + 1) + r[j].at(e + 1));
  }
  double sum = 0.0;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const double v = static_cast<double>(h[j].at(e));
      sum = __builtin_fma(v, v, sum);
    }
  if (a.total) {
    T* const total = static_cast<T*>(a.total) + row * a.ldt;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = lane + 64 * W * j;
      if (i * VE < K) h[j].store(total, i, K);
    }
  }
  sum = lanes_sum<64>(sum);
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) part_sum[wave] = sum;
    __syncthreads();
    sum = 0.0;
#pragma unroll
    for (int i = 0; i < W; ++i) sum += part_sum[i];
  }
  const float r = static_cast<float>(1.0 / __builtin_sqrt(sum / K + a.eps));
  const TW* const weight = static_cast<const TW*>(a.weight);
  T* const out = static_cast<T*>(a.out) + row * a.ldo;
  uint8_t* const codes = a.codes + row * a.ldc;
  uint32_t top = 0;
  float v[NV][VE];  // y, zeros behind K
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = lane + 64 * W * j;
    Piece<WTYPE> w = {};
    if (i * VE < K) w.load(weight, i, K);
#pragma unroll
    for (int e = 0; e < VE; ++e) v[j][e] = i * VE + e < K ? (h[j].at(e) * r) * w.at(e) : 0.0f;
    if (a.out) {
#pragma unroll
      for (int e = 0; e < VE; e += 2) h[j].set2(e, v[j][e], v[j][e + 1]);
      if (i * VE < K) h[j].store(out, i, K);
    }
    if (a.format == MOE_CODES_E4M3) {
      uint32_t c[2];
      const float scale = codes_e4m3(v[j], c);
      if (i * VE < K) {
        store_codes(codes, i, K, c);
        if (lane % 16 == 0) a.scales[row * a.lds + i / 16] = scale;
      }
    }
  }
  if (a.format == MOE_CODES_I8) {
    constexpr float kMagic = 12582912.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const uint32_t t = top_of(v[j]);
      top = t > top ? t : top;
    }
    top = lanes_max<64>(top);
    if constexpr (W > 1) {
      if ((threadIdx.x & 63) == 0) part_top[wave] = top;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < W; ++i) top = part_top[i] > top ? part_top[i] : top;
    }
    const float amax = __uint_as_float(top);
    const bool finite = top < 0x7f800000u, some = top != 0 && finite, quick = some && amax >= 0x1p-100f;
    QuantScale s = {0, 1.0f, 0.0f};
    if (some) {
      s.exp = __builtin_amdgcn_frexp_expf(amax) - 1;
      s.amax = __builtin_ldexpf(amax, -s.exp);
      s.inv = 127.0f / s.amax;
    }
    const float inv = quick ? __uint_as_float(__float_as_uint(127.0f / amax) + 1) : 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int i = lane + 64 * W * j;
      uint32_t c[2] = {0, 0};
      bool redo = some && !quick;
      if (quick) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          uint32_t b[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float t = v[j][4 * g + e], y = __builtin_fmaf(t, inv, kMagic);
            b[e] = __float_as_uint(y);
            redo |= __builtin_fabsf(__builtin_fmaf(t, inv, kMagic - y)) >= 0.5f - 0x1p-14f;
          }
          const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400), hi = __builtin_amdgcn_perm(b[3], b[2], 0x0c0c0400);
          c[g] = lo | hi << 16;
        }
      }
      if (redo) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          c[g] = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) c[g] |= static_cast<uint32_t>(quant_exact(v[j][4 * g + e], s) & 255) << (8 * e);
        }
      }
      if (i * VE < K) store_codes(codes, i, K, c);
    }
    if (lane == 0) a.scales[row] = finite ? amax / 127.0f : __builtin_nanf("");
  }
}

// ----------------------------------------------------------------------- host
template <int TYPE>
int launch_quant_f8(const void* x, int64_t ldx, int32_t M, int32_t K, uint8_t* codes, int64_t ldc, float* scales,
                    int64_t lds, hipStream_t st) {
  const uint32_t runs = static_cast<uint32_t>((K + 511) / 512);
  const uint64_t units = static_cast<uint64_t>(M) * runs;
  // two runs a wave where that leaves more waves than the GPU holds at once
  if (units >= 65536)
    return launch(quant_f8_kernel<TYPE, 2>, static_cast<uint32_t>((units + 7) / 8), 256, 0, st, x, ldx, M, K, codes, ldc,
                  scales, lds, runs);
  return launch(quant_f8_kernel<TYPE, 1>, static_cast<uint32_t>((units + 3) / 4), 256, 0, st, x, ldx, M, K, codes, ldc,
                scales, lds, runs);
}

template <int TYPE, int WTYPE, int W, int NV>
int launch_norm(const NormArgs& a, hipStream_t st) {
  constexpr int per = 4 / W;
  return launch(norm_kernel<TYPE, WTYPE, W, NV>, static_cast<uint32_t>((a.M + per - 1) / per), 256, 0, st, a);
}
template <int TYPE, int WTYPE>
int launch_norm(const NormArgs& a, hipStream_t st) {
  const int pieces = (a.K + VE - 1) / VE;
  // many short rows: a wave each, no step waits for another wave (us, against four waves: 16384 x 512 14.9 and 36.9,
  // 16384 x 1024 33 and 42); few or long ones: four waves each (16384 x 3584 101, against 110)
  if (a.M >= 1024 && pieces <= 4 * 64) {
    if (pieces <= 64) return launch_norm<TYPE, WTYPE, 1, 1>(a, st);
    if (pieces <= 2 * 64) return launch_norm<TYPE, WTYPE, 1, 2>(a, st);
    return launch_norm<TYPE, WTYPE, 1, 4>(a, st);
  }
  if (pieces <= 2 * 256) return launch_norm<TYPE, WTYPE, 4, 2>(a, st);
  return launch_norm<TYPE, WTYPE, 4, 8>(a, st);
}
template <int TYPE>
int launch_norm(const NormArgs& a, int32_t wtype, hipStream_t st) {
  if (wtype == MOE_F32) return launch_norm<TYPE, MOE_F32>(a, st);
  return launch_norm<TYPE, TYPE>(a, st);
}

}  // namespace

extern "C" {

int moe_quant_f8(const void* x, int32_t type, int64_t ldx, int32_t M, int32_t K, uint8_t* codes, int64_t ldc,
                 float* scales, int64_t lds, void* stream) {
  if (!x || !codes || !scales || !type_ok(type) || M < 1 || M > kMaxRows || K < 1 || K > 131072 || ldx < K || ldc < K ||
      lds < (K + 127) / 128 || static_cast<int64_t>(M) * ((K + 511) / 512) >= 1 << 27)  // (2^32 threads)
    return MOE_EINVAL;
  hipStream_t st = as_stream(stream);
  if (type == MOE_F32) return launch_quant_f8<MOE_F32>(x, ldx, M, K, codes, ldc, scales, lds, st);
  if (type == MOE_F16) return launch_quant_f8<MOE_F16>(x, ldx, M, K, codes, ldc, scales, lds, st);
  return launch_quant_f8<MOE_BF16>(x, ldx, M, K, codes, ldc, scales, lds, st);
}

int moe_rms_norm(const void* x, int32_t type, int64_t ldx, int32_t M, int32_t K, const void* weight, int32_t wtype,
                 const moe_norm_opts_t* opts, void* stream) {
  moe_norm_opts_t o;
  std::memset(&o, 0, sizeof(o));
  if (opts) o = *opts;
  if (!x || !weight || !type_ok(type) || (wtype != MOE_F32 && wtype != type) || M < 1 || M > kMaxRows || K < 1 || K > 16384 ||
      ldx < K || !(o.eps >= 0.0) || !std::isfinite(o.eps) || o.codes < MOE_CODES_NONE || o.codes > MOE_CODES_E4M3)
    return MOE_EINVAL;
  if ((!o.out_dev && o.codes == MOE_CODES_NONE) || (o.residual_dev && o.ldr < K) || (o.total_dev && o.ldt < K) ||
      (o.out_dev && o.ldo < K))
    return MOE_EINVAL;
  if (o.codes != MOE_CODES_NONE &&
      (!o.codes_dev || !o.scales_dev || o.ldc < K || (o.codes == MOE_CODES_E4M3 && o.lds < (K + 127) / 128)))
    return MOE_EINVAL;
  const NormArgs a = {x,     o.residual_dev, weight, o.total_dev, o.out_dev, static_cast<uint8_t*>(o.codes_dev), o.scales_dev,
                      ldx,   o.ldr,          o.ldt,  o.ldo,       o.ldc,     o.lds,
                      o.eps, M,              K,      o.codes};
  hipStream_t st = as_stream(stream);
  if (type == MOE_F32) return launch_norm<MOE_F32, MOE_F32>(a, st);
  if (type == MOE_F16) return launch_norm<MOE_F16>(a, wtype, st);
  return launch_norm<MOE_BF16>(a, wtype, st);
}

}  // extern "C"
