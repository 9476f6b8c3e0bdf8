// Rotary positions with several axes, forward and gradient (include/jca.h states the layout).
//
// Each token has one position per axis and each axis turns its own pairs (j, j + d/2) of every head:
//   (a, b) -> (a cos x - b sin x, a sin x + b cos x),  x = position[token, axis(j)] * theta_j.
// The gradient of a rotation is the rotation by -x.
//
// What bounds it: memory. q and k are read and written once, so a token of H + Hkv heads moves
// 2 (H + Hkv) d elements; the cosines and sines depend on the token and the pair alone. A block
// takes a tile of tokens, forms the tile's (cos, sin) once into shared memory (512 entries, two per
// thread) and then turns every head of q and k of those tokens with 16-byte accesses, so the
// trigonometry is paid once per token and not once per head, and one launch serves q and k.
//
// Angles: the turn count position * theta / 2 pi is formed in fp64, with theta / 2 pi as a sum of two
// numbers and the product's rounding recovered by an FMA, and its whole part removed there: with one
// fp64 factor a position of 2^31 (seconds since an epoch) would already cost 2^-22 of a radian, as
// much as fp32 elements can show. The nearest quarter turn is
// split off there too, and only the remainder in [-1/8, 1/8] turns goes to the fp32 sine and cosine:
// its rounding is then at most pi 2^-27, where that of a whole half turn would be pi 2^-25, more
// than the sine's own error. theta / 2 pi comes from the host as a kernel argument. The
// rotation is fp32, rounded once to the element type; pairs past the sections keep their bits.
#include <climits>
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "jca_internal.h"

namespace jca {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeEntries = 512;   // (cos, sin) pairs of a tile
constexpr int kMaxHalf = 64;
constexpr int kMaxAxes = 4;

struct RopeAxesArgs {
  const void* q;
  const void* k;
  void* q_out;
  void* k_out;
  const void* pos;
  int64_t T, q_stride, k_stride, qo_stride, ko_stride;
  int H, Hkv, n_axes;
  int n_turned;                     // pairs [0, n_turned) turn, the rest stay as they are
  float sign;                       // -1 turns backwards (the gradient)
  double turns[kMaxHalf];           // theta_j / 2 pi, and what its rounding to fp64 left out
  double turns_lo[kMaxHalf];
  uint8_t axis[kMaxHalf];
};

// 16 bytes of elements as floats and back.
template <typename E>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void load(uint4 w, float* f) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 store(const float* f) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      u[i] = *reinterpret_cast<uint32_t*>(&h);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <>
struct Vec<__half> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void load(uint4 w, float* f) {
    uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = __half22float2(*reinterpret_cast<__half2*>(&u[i]));
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  }
  static __device__ __forceinline__ uint4 store(const float* f) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      u[i] = *reinterpret_cast<uint32_t*>(&h);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void load(uint4 w, float* f) {
    f[0] = __uint_as_float(w.x);
    f[1] = __uint_as_float(w.y);
    f[2] = __uint_as_float(w.z);
    f[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 store(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};

// The first n elements of `a`, the others of `b`.
template <typename E>
__device__ __forceinline__ uint4 keep_tail(uint4 a, uint4 b, int n) {
  uint32_t x[4] = {a.x, a.y, a.z, a.w};
  const uint32_t y[4] = {b.x, b.y, b.z, b.w};
  constexpr int PER = 4 / (int)sizeof(E);   // elements of a word
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (n <= i * PER) x[i] = y[i];
    else if (PER == 2 && n == i * PER + 1) x[i] = (x[i] & 0xffffu) | (y[i] & 0xffff0000u);
  }
  return make_uint4(x[0], x[1], x[2], x[3]);
}

template <typename E, typename IdxT, int D>
__global__ void __launch_bounds__(kRopeThreads)
    rope_axes_kernel(const __grid_constant__ RopeAxesArgs a) {
  constexpr int HALF = D / 2;
  constexpr int ROWS = kRopeEntries / HALF;      // tokens of a tile
  constexpr int N = Vec<E>::N;
  constexpr int CH = HALF / N;                   // 16-byte chunks of half a head
  __shared__ __align__(16) float2 cs[kRopeEntries];
  const int64_t t0 = (int64_t)blockIdx.x * ROWS;
  const int rows = (int)min((int64_t)ROWS, a.T - t0);
  const IdxT* pos = static_cast<const IdxT*>(a.pos);
#pragma unroll
  for (int e = threadIdx.x; e < kRopeEntries; e += kRopeThreads) {
    const int r = e / HALF, j = e % HALF;
    if (r < rows) {
      const double p = (double)pos[(t0 + r) * a.n_axes + a.axis[j]];
      double n = p * a.turns[j];
      const double left = fma(p, a.turns[j], -n) + p * a.turns_lo[j];
      n = 4.0 * ((n - rint(n)) + left);
      const double k = rint(n);
      float s, c;
      sincospif((float)(0.5 * (n - k)), &s, &c);
      const int quarter = (int)k;   // -2..2: a quarter turn swaps the two and flips one
      const float s1 = (quarter & 1) ? c : s, c1 = (quarter & 1) ? -s : c;
      cs[e] = make_float2((quarter & 2) ? -c1 : c1, a.sign * ((quarter & 2) ? -s1 : s1));
    }
  }
  __syncthreads();
  // Units of the tile: (token, head, chunk of half a head), the chunk fastest.
  const uint32_t per_row = (uint32_t)(a.H + a.Hkv) * CH;
  const uint32_t units = per_row * (uint32_t)rows;
  for (uint32_t u = threadIdx.x; u < units; u += kRopeThreads) {
    const uint32_t r = u / per_row, x = u - r * per_row;
    const int head = (int)(x / CH), j0 = (int)(x % CH) * N;
    const bool is_q = head < a.H;
    const E* src = is_q ? static_cast<const E*>(a.q) + (t0 + r) * a.q_stride + (int64_t)head * D
                        : static_cast<const E*>(a.k) + (t0 + r) * a.k_stride +
                              (int64_t)(head - a.H) * D;
    E* dst = is_q ? static_cast<E*>(a.q_out) + (t0 + r) * a.qo_stride + (int64_t)head * D
                  : static_cast<E*>(a.k_out) + (t0 + r) * a.ko_stride +
                        (int64_t)(head - a.H) * D;
    float lo[N], hi[N];
    const uint4 wlo = *reinterpret_cast<const uint4*>(src + j0);
    const uint4 whi = *reinterpret_cast<const uint4*>(src + HALF + j0);
    Vec<E>::load(wlo, lo);
    Vec<E>::load(whi, hi);
    const float4* t4 = reinterpret_cast<const float4*>(cs + r * HALF + j0);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float4 t = t4[i / 2];
      const float a0 = lo[i], b0 = hi[i], a1 = lo[i + 1], b1 = hi[i + 1];
      lo[i] = fmaf(a0, t.x, -(b0 * t.y));
      hi[i] = fmaf(a0, t.y, b0 * t.x);
      lo[i + 1] = fmaf(a1, t.z, -(b1 * t.w));
      hi[i + 1] = fmaf(a1, t.w, b1 * t.z);
    }
    uint4 olo = Vec<E>::store(lo), ohi = Vec<E>::store(hi);
    if (j0 + N > a.n_turned) {
      olo = keep_tail<E>(olo, wlo, a.n_turned - j0);
      ohi = keep_tail<E>(ohi, whi, a.n_turned - j0);
    }
    *reinterpret_cast<uint4*>(dst + j0) = olo;
    *reinterpret_cast<uint4*>(dst + HALF + j0) = ohi;
  }
}

template <typename E, typename IdxT>
void launch_rope_axes(const RopeAxesArgs& a, int d, cudaStream_t st) {
  const int rows = kRopeEntries / (d / 2);
  const unsigned grid = (unsigned)((a.T + rows - 1) / rows);
  switch (d) {
    case 16: rope_axes_kernel<E, IdxT, 16><<<grid, kRopeThreads, 0, st>>>(a); break;
    case 32: rope_axes_kernel<E, IdxT, 32><<<grid, kRopeThreads, 0, st>>>(a); break;
    case 64: rope_axes_kernel<E, IdxT, 64><<<grid, kRopeThreads, 0, st>>>(a); break;
    default: rope_axes_kernel<E, IdxT, 128><<<grid, kRopeThreads, 0, st>>>(a); break;
  }
}

int rope_axes(const void* q, const void* k, void* q_out, void* k_out, const void* positions,
              const int32_t* sections, int n_axes, int per_axis, int64_t T, int H, int Hkv, int d,
              int64_t qs, int64_t ks, int64_t qos, int64_t kos, float base, int dtype,
              int idx_bits, float sign, jca_stream_t stream) {
  if (idx_bits != 32 && idx_bits != 64) return JCA_ERR_IDX_BITS;
  if (!head_dim_ok(d)) return JCA_ERR_HEAD_DIM;
  if (dtype != JCA_BF16 && dtype != JCA_FP16 && dtype != JCA_FP32) return JCA_ERR_DTYPE;
  if (!k) Hkv = 0;
  if (T < 0 || T >= (int64_t)INT_MAX || H < 1 || H >= 65536 || (k && (Hkv < 1 || Hkv >= 65536)) ||
      n_axes < 1 || n_axes > kMaxAxes || !(base > 1.f) || !(base < INFINITY))
    return JCA_ERR_SHAPE;
  if (!sections) return JCA_ERR_NULL;
  const int half = d / 2;
  int64_t sum = 0;
  for (int a = 0; a < n_axes; ++a) {
    if (sections[a] < 0) return JCA_ERR_SHAPE;
    sum += sections[a];
  }
  if (sum > half) return JCA_ERR_SHAPE;
  if (qs < (int64_t)H * d || qos < (int64_t)H * d ||
      (k && (ks < (int64_t)Hkv * d || kos < (int64_t)Hkv * d)))
    return JCA_ERR_SHAPE;
  if (T == 0) return JCA_OK;
  if (!q || !q_out || !positions || (k && !k_out)) return JCA_ERR_NULL;
  const int64_t per16 = dtype == JCA_FP32 ? 4 : 8;
  if (!aligned(q, 16) || !aligned(q_out, 16) || qs % per16 || qos % per16 ||
      (k && (!aligned(k, 16) || !aligned(k_out, 16) || ks % per16 || kos % per16)))
    return JCA_ERR_ALIGN;
  int dev = 0, sms = 0;
  const int rc = current_device(&dev, &sms);
  if (rc) return rc;
  RopeAxesArgs a = {};
  a.q = q;
  a.k = k;
  a.q_out = q_out;
  a.k_out = k_out;
  a.pos = positions;
  a.T = T;
  a.q_stride = qs;
  a.k_stride = ks;
  a.qo_stride = qos;
  a.ko_stride = kos;
  a.H = H;
  a.Hkv = Hkv;
  a.n_axes = n_axes;
  a.sign = sign;
  const long double log2_base = log2l((long double)base);
  const long double inv_2pi = 0.159154943091895335768883763372514362L;
  int j = 0;
  for (int ax = 0; ax < n_axes; ++ax)
    for (int i = 0; i < sections[ax]; ++i, ++j) {
      const long double e = per_axis ? (long double)i / sections[ax] : (long double)j / half;
      const long double t = exp2l(-e * log2_base) * inv_2pi;
      a.turns[j] = (double)t;
      a.turns_lo[j] = (double)(t - (long double)a.turns[j]);
      a.axis[j] = (uint8_t)ax;
    }
  a.n_turned = j;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (idx_bits == 32) {
    if (dtype == JCA_BF16) launch_rope_axes<__nv_bfloat16, int32_t>(a, d, st);
    else if (dtype == JCA_FP16) launch_rope_axes<__half, int32_t>(a, d, st);
    else launch_rope_axes<float, int32_t>(a, d, st);
  } else {
    if (dtype == JCA_BF16) launch_rope_axes<__nv_bfloat16, int64_t>(a, d, st);
    else if (dtype == JCA_FP16) launch_rope_axes<__half, int64_t>(a, d, st);
    else launch_rope_axes<float, int64_t>(a, d, st);
  }
  return cudaGetLastError() == cudaSuccess ? JCA_OK : JCA_ERR_CUDA;
}

}  // namespace
}  // namespace jca

extern "C" int jca_rope_axes_fwd(const void* q, const void* k, void* q_out, void* k_out,
                                 const void* positions, const int32_t* sections, int n_axes,
                                 int per_axis, int64_t T, int H, int Hkv, int d_head,
                                 int64_t q_stride, int64_t k_stride, int64_t q_out_stride,
                                 int64_t k_out_stride, float base, int dtype, int idx_bits,
                                 jca_stream_t stream) {
  return jca::rope_axes(q, k, q_out, k_out, positions, sections, n_axes, per_axis, T, H, Hkv,
                        d_head, q_stride, k_stride, q_out_stride, k_out_stride, base, dtype,
                        idx_bits, 1.f, stream);
}

extern "C" int jca_rope_axes_bwd(const void* dq_out, const void* dk_out, void* dq, void* dk,
                                 const void* positions, const int32_t* sections, int n_axes,
                                 int per_axis, int64_t T, int H, int Hkv, int d_head,
                                 int64_t dq_out_stride, int64_t dk_out_stride, int64_t dq_stride,
                                 int64_t dk_stride, float base, int dtype, int idx_bits,
                                 jca_stream_t stream) {
  return jca::rope_axes(dq_out, dk_out, dq, dk, positions, sections, n_axes, per_axis, T, H, Hkv,
                        d_head, dq_out_stride, dk_out_stride, dq_stride, dk_stride, base, dtype,
                        idx_bits, -1.f, stream);
}
