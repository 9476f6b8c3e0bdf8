// Rotary positions with several axes, forward and gradient (include/jca.h states the layout).
//
// Each token has one position per axis and each axis turns its own pairs (j, j + d/2) of every head:
//   (a, b) -> (a cos x - b sin x, a sin x + b cos x),  x = position[token, axis(j)] * theta_j.
// The gradient of a rotation is the rotation by -x.
//
// What bounds it: memory (256 users, 16 heads of 128: 202 us, 0.85 of the copy bandwidth; fp32 gradient
// of 64 users 47 us, 0.90). q and k are read and written once; the cosines and sines depend on the
// token and the pair alone. A warp takes a few tokens at a time, starts its first loads, forms the
// tokens' (cos, sin) once into its part of shared memory while they are under way (frequencies in
// registers, positions fetched a step ahead) and turns every head of q and k of them with 16-byte
// accesses: the trigonometry is paid once per token, one launch serves q and k, and no warp waits
// for another. With one barrier per block and tile instead it took 254 us, with half the entries
// per step 249 us, with more warps that each spill 208 to 260 us.
//
// Angles are counted in turns, in 64-bit fixed point: theta / 2 pi is an integer multiple of 2^-64 (the
// host rounds it from extended precision), and the position times that integer, wrapped to 64 bits,
// is the fraction of the turn, whatever the position: one integer product in place of a chain of fp64
// operations and their reduction (a third of the time on the 256-user batch), off by at most 2^-61
// of a turn per unit of position, 2^-30 at a position of 2^31 (seconds since an epoch), where an
// fp64 product would be off by 2^-22 of a radian. The nearest quarter turn is split off and the
// remainder in [-1/8, 1/8] turns goes to fp32 series for sine and cosine: its rounding there is at
// most 2^-24, where that of a whole half turn would be four times as much. The rotation is fp32,
// rounded once to the element type; pairs past the sections keep their bits.
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
constexpr int kRopeEntries = 128;   // (cos, sin) pairs of a warp's tile
constexpr int kRopeBlocks = 2;      // blocks per SM
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
  uint64_t turns[kMaxHalf];         // theta_j / 2 pi in units of 2^-64
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

// Sine and cosine of |x| <= pi / 4 by their Taylor series, to x^9 and x^10: the next terms are below
// 2^-29. A dozen multiply-adds where the library's function also reduces any argument.
__device__ __forceinline__ void sin_cos_eighth(float x, float& s, float& c) {
  const float y = x * x;
  s = fmaf(y, fmaf(y, fmaf(y, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f);
  s = fmaf(s * y, x, x);
  c = fmaf(y, fmaf(y, fmaf(y, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f);
  c = fmaf(y, fmaf(y, c, -0.5f), 1.f);
}

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
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks)
    rope_axes_kernel(const __grid_constant__ RopeAxesArgs a) {
  constexpr int HALF = D / 2;
  constexpr int ROWS = kRopeEntries / HALF;      // tokens of a tile
  constexpr int N = Vec<E>::N;
  constexpr int CH = HALF / N;                   // 16-byte chunks of half a head
  constexpr int U = 4;                           // units a lane has in flight
  constexpr int EPL = kRopeEntries / 32;         // entries a lane forms
  __shared__ __align__(16) float2 table[kRopeThreads / 32][kRopeEntries];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float2* cs = table[warp];
  const IdxT* pos = static_cast<const IdxT*>(a.pos);
  // The lane's pairs: their frequencies, and where their entries lie. Entries of a token: the first
  // two pairs of every chunk, then the next two of every chunk, ..., so that the lanes that read a
  // chunk each read consecutive 16 bytes.
  uint64_t turns[EPL];
  int axis[EPL], at[EPL], row[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 32 * i, j = e % HALF;
    turns[i] = a.turns[j];
    axis[i] = a.axis[j];
    row[i] = e / HALF;
    at[i] = row[i] * HALF + (j % N / 2 * CH + j / N) * 2 + (j & 1);
  }
  // Units of a tile: (token, head, chunk of half a head), the chunk fastest.
  const uint32_t per_row = (uint32_t)(a.H + a.Hkv) * CH;
  const int64_t tiles = (a.T + ROWS - 1) / ROWS;
  const int64_t first = blockIdx.x * (int64_t)(kRopeThreads / 32) + warp;
  const int64_t stride = gridDim.x * (int64_t)(kRopeThreads / 32);
  // Positions are loaded a tile ahead: behind the tile's own loads they would hold up its angles.
  IdxT next[EPL] = {};
  auto fetch = [&](int64_t tile) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int64_t r = tile * ROWS + row[i];
      if (r < a.T) next[i] = pos[r * a.n_axes + axis[i]];
    }
  };
  fetch(first);
  for (int64_t tile = first; tile < tiles; tile += stride) {
    const int64_t t0 = tile * ROWS;
    const int rows = (int)min((int64_t)ROWS, a.T - t0);
    const uint32_t units = per_row * (uint32_t)rows;
    for (uint32_t u0 = 0; u0 < units; u0 += 32 * U) {
      uint4 lo[U], hi[U];
      uint32_t r[U], x[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const uint32_t u = u0 + 32 * i + lane;
        r[i] = ROWS == 1 ? 0u : u / per_row;
        x[i] = u - r[i] * per_row;
        if (u < units) {
          const int head = (int)(x[i] / CH);
          const bool is_q = head < a.H;
          const E* s = static_cast<const E*>(is_q ? a.q : a.k) +
                       (t0 + r[i]) * (is_q ? a.q_stride : a.k_stride) +
                       (is_q ? head : head - a.H) * (int64_t)D + x[i] % CH * N;
          lo[i] = *reinterpret_cast<const uint4*>(s);
          hi[i] = *reinterpret_cast<const uint4*>(s + HALF);
        }
      }
      if (u0 == 0) {
        // The tile's cosines and sines, formed while the first loads are under way.
        __syncwarp();
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          const uint64_t f = (uint64_t)(int64_t)next[i] * turns[i];   // of a turn, in 2^-64
          const uint32_t quarter = (uint32_t)((f + (1ull << 61)) >> 62);
          const int32_t rest = (int32_t)((f - ((uint64_t)quarter << 62)) >> 32);
          float s, c;
          sin_cos_eighth((float)rest * 1.4629180792671596e-9f, s, c);   // 2 pi 2^-32
          // A quarter turn swaps the two and flips one.
          const float s1 = (quarter & 1) ? c : s, c1 = (quarter & 1) ? -s : c;
          cs[at[i]] = make_float2((quarter & 2) ? -c1 : c1, a.sign * ((quarter & 2) ? -s1 : s1));
        }
        fetch(tile + stride);
        __syncwarp();
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (u0 + 32 * i + lane >= units) continue;
        const int c = (int)(x[i] % CH), head = (int)(x[i] / CH);
        float u[N], v[N];
        Vec<E>::load(lo[i], u);
        Vec<E>::load(hi[i], v);
        const float4* t4 = reinterpret_cast<const float4*>(cs + r[i] * HALF) + c;
#pragma unroll
        for (int k = 0; k < N; k += 2) {
          const float4 t = t4[k / 2 * CH];
          const float a0 = u[k], b0 = v[k], a1 = u[k + 1], b1 = v[k + 1];
          u[k] = fmaf(a0, t.x, -(b0 * t.y));
          v[k] = fmaf(a0, t.y, b0 * t.x);
          u[k + 1] = fmaf(a1, t.z, -(b1 * t.w));
          v[k + 1] = fmaf(a1, t.w, b1 * t.z);
        }
        uint4 olo = Vec<E>::store(u), ohi = Vec<E>::store(v);
        const int turned = a.n_turned - c * N;   // of the chunk's pairs
        if (turned < N) {
          olo = keep_tail<E>(olo, lo[i], turned);
          ohi = keep_tail<E>(ohi, hi[i], turned);
        }
        const bool is_q = head < a.H;
        E* d = static_cast<E*>(is_q ? a.q_out : a.k_out) +
               (t0 + r[i]) * (is_q ? a.qo_stride : a.ko_stride) +
               (is_q ? head : head - a.H) * (int64_t)D + c * N;
        *reinterpret_cast<uint4*>(d) = olo;
        *reinterpret_cast<uint4*>(d + HALF) = ohi;
      }
    }
  }
}

template <typename E, typename IdxT>
void launch_rope_axes(const RopeAxesArgs& a, int d, int sms, cudaStream_t st) {
  const int rows = kRopeEntries / (d / 2) * (kRopeThreads / 32);   // tokens of a block's warps
  const int64_t want = (a.T + rows - 1) / rows;
  const unsigned grid = (unsigned)(want < (int64_t)sms * kRopeBlocks ? want : sms * kRopeBlocks);
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
  // In place row by row only: with another stride a row's result would land in one not yet read.
  if (T > 1 && ((q == q_out && qs != qos) || (k && k == k_out && ks != kos))) return JCA_ERR_SHAPE;
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
  // Frequency i of n is base^(-i / n): the product of those of i's bits, so that a call pays for a few
  // exponentials instead of one per pair (they were half of its time on the host). Six factors
  // and products, each off by at most 2^-63 of its value, and a first frequency of 1 / 2 pi turns.
  long double freq[64], power[6];
  auto frequencies = [&](int n, int count) {
    for (int b = 0; b < 6 && (1 << b) < count; ++b)
      power[b] = exp2l(-log2_base * (1 << b) / n);
    freq[0] = ldexpl(inv_2pi, 64);
    for (int i = 1; i < count; ++i) freq[i] = freq[i & (i - 1)] * power[__builtin_ctz(i)];
  };
  if (!per_axis) frequencies(half, (int)sum);
  int j = 0;
  for (int ax = 0; ax < n_axes; ++ax) {
    if (per_axis) frequencies(sections[ax], sections[ax]);
    for (int i = 0; i < sections[ax]; ++i, ++j) {
      a.turns[j] = (uint64_t)(freq[per_axis ? i : j] + 0.5L);
      a.axis[j] = (uint8_t)ax;
    }
  }
  a.n_turned = j;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (idx_bits == 32) {
    if (dtype == JCA_BF16) launch_rope_axes<__nv_bfloat16, int32_t>(a, d, sms, st);
    else if (dtype == JCA_FP16) launch_rope_axes<__half, int32_t>(a, d, sms, st);
    else launch_rope_axes<float, int32_t>(a, d, sms, st);
  } else {
    if (dtype == JCA_BF16) launch_rope_axes<__nv_bfloat16, int64_t>(a, d, sms, st);
    else if (dtype == JCA_FP16) launch_rope_axes<__half, int64_t>(a, d, sms, st);
    else launch_rope_axes<float, int64_t>(a, d, sms, st);
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
