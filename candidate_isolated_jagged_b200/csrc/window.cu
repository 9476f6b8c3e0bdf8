// Causal attention over packed rows with a sliding window and first tokens that stay visible:
// forward and backward (include/jca.h states the mask and the layout).
#include <climits>
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "jca_device.cuh"
#include "jca_internal.h"

namespace jca {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kMaxSinks = 128;

struct WindowArgs {
  const bf16* q;
  const bf16* k;
  const bf16* v;
  const bf16* out;
  const bf16* dout;
  const float* lse;
  bf16* o;
  float* lse_out;
  bf16* dq;
  bf16* dk;
  bf16* dv;
  const uint8_t* valid;
  const int32_t* row_start;   // [T] first row of the row's user
  const int32_t* row_end;     // [T] one past its last
  const int32_t* status;
  int64_t T, q_stride, k_stride, v_stride;
  int H, Hkv, window, n_sinks;
  float scale;
};

// Checks the offsets and writes each row's user bounds; one block per user.
template <typename IdxT>
__global__ void __launch_bounds__(128)
    window_plan_kernel(const IdxT* __restrict__ off, int64_t B, int64_t T,
                       int32_t* __restrict__ row_start, int32_t* __restrict__ row_end,
                       int32_t* status) {
  if (*status != 0) return;
  for (int64_t b = blockIdx.x; b < B; b += gridDim.x) {
    const long long s = (long long)off[b], e = (long long)off[b + 1];
    if (s < 0 || s > e || e > T || (b == 0 && s != 0) || (b == B - 1 && e != T)) {
      if (threadIdx.x == 0) atomicCAS(status, 0, (int32_t)JCA_STATUS_BAD_OFFSETS);
      continue;
    }
    for (long long i = s + threadIdx.x; i < e; i += blockDim.x) {
      row_start[i] = (int32_t)s;
      if (row_end) row_end[i] = (int32_t)e;
    }
  }
}

// One warp per (row, head); lane l holds elements l * EPL ... of the head.
template <int D>
struct Row {
  static constexpr int EPL = D >= 32 ? D / 32 : 1;
  float x[EPL];
  __device__ __forceinline__ void load(const bf16* p, int lane) {
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      x[i] = lane * EPL < D ? __bfloat162float(p[lane * EPL + i]) : 0.f;
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < EPL; ++i) x[i] = 0.f;
  }
  __device__ __forceinline__ float dot(const Row& o) const {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) s = fmaf(x[i], o.x[i], s);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    return s;
  }
  __device__ __forceinline__ void axpy(float a, const Row& o) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) x[i] = fmaf(a, o.x[i], x[i]);
  }
  __device__ __forceinline__ void store(bf16* p, float a, int lane) const {
    if (lane * EPL < D)
#pragma unroll
      for (int i = 0; i < EPL; ++i) p[lane * EPL + i] = __float2bfloat16(x[i] * a);
  }
};

template <int D>
__global__ void __launch_bounds__(128) window_fwd_kernel(const WindowArgs a) {
  if (*a.status != 0) return;
  const int lane = threadIdx.x & 31;
  const int64_t w = blockIdx.x * (int64_t)4 + (threadIdx.x >> 5);
  if (w >= a.T * a.H) return;
  const int64_t i = w / a.H;
  const int h = (int)(w % a.H), hk = h / (a.H / a.Hkv);
  Row<D> q, acc, x;
  q.load(a.q + i * a.q_stride + (int64_t)h * D, lane);
  acc.zero();
  float m = -INFINITY, l = 0.f;
  const bool real = !a.valid || a.valid[i];
  if (real) {
    const int64_t s = a.row_start[i];
    const int64_t lo = max(s, i - a.window + 1);
    const int64_t first = min(s + a.n_sinks, lo);   // sinks [s, first), then [lo, i]
    for (int64_t j = s; j <= i; ++j) {
      if (j == first && first < lo) {
        j = lo;
      }
      if (a.valid && !a.valid[j]) continue;
      x.load(a.k + j * a.k_stride + (int64_t)hk * D, lane);
      const float sc = q.dot(x) * a.scale;
      const float mn = fmaxf(m, sc);
      const float al = m == -INFINITY ? 0.f : __expf(m - mn), p = __expf(sc - mn);
#pragma unroll
      for (int t = 0; t < Row<D>::EPL; ++t) acc.x[t] *= al;
      x.load(a.v + j * a.v_stride + (int64_t)hk * D, lane);
      acc.axpy(p, x);
      l = l * al + p;
      m = mn;
    }
  }
  acc.store(a.o + (i * a.H + h) * D, l > 0.f ? 1.f / l : 0.f, lane);
  if (a.lse_out && lane == 0) a.lse_out[i * a.H + h] = l > 0.f ? m + logf(l) : -INFINITY;
}

template <int D>
__global__ void __launch_bounds__(128) window_dq_kernel(const WindowArgs a) {
  if (*a.status != 0) return;
  const int lane = threadIdx.x & 31;
  const int64_t w = blockIdx.x * (int64_t)4 + (threadIdx.x >> 5);
  if (w >= a.T * a.H) return;
  const int64_t i = w / a.H;
  const int h = (int)(w % a.H), hk = h / (a.H / a.Hkv);
  Row<D> q, dov, acc, x;
  acc.zero();
  if (!a.valid || a.valid[i]) {
    q.load(a.q + i * a.q_stride + (int64_t)h * D, lane);
    dov.load(a.dout + (i * a.H + h) * D, lane);
    x.load(a.out + (i * a.H + h) * D, lane);
    const float dl = dov.dot(x), lse = a.lse[i * a.H + h];
    const int64_t s = a.row_start[i];
    const int64_t lo = max(s, i - a.window + 1);
    const int64_t first = min(s + a.n_sinks, lo);
    for (int64_t j = s; j <= i; ++j) {
      if (j == first && first < lo) j = lo;
      if (a.valid && !a.valid[j]) continue;
      x.load(a.v + j * a.v_stride + (int64_t)hk * D, lane);
      const float dp = dov.dot(x);
      x.load(a.k + j * a.k_stride + (int64_t)hk * D, lane);
      const float p = __expf(q.dot(x) * a.scale - lse);
      acc.axpy(p * (dp - dl), x);
    }
  }
  acc.store(a.dq + (i * a.H + h) * D, a.scale, lane);
}

template <int D>
__global__ void __launch_bounds__(128) window_dkv_kernel(const WindowArgs a) {
  if (*a.status != 0) return;
  const int lane = threadIdx.x & 31;
  const int64_t w = blockIdx.x * (int64_t)4 + (threadIdx.x >> 5);
  if (w >= a.T * a.Hkv) return;
  const int64_t j = w / a.Hkv;
  const int hk = (int)(w % a.Hkv), G = a.H / a.Hkv;
  Row<D> k, v, dk, dv, x, y;
  dk.zero();
  dv.zero();
  if (!a.valid || a.valid[j]) {
    k.load(a.k + j * a.k_stride + (int64_t)hk * D, lane);
    v.load(a.v + j * a.v_stride + (int64_t)hk * D, lane);
    const int64_t s = a.row_start[j], e = a.row_end[j];
    const int64_t end = j - s < a.n_sinks ? e : min(e, j + a.window);
    for (int64_t i = j; i < end; ++i) {
      if (a.valid && !a.valid[i]) continue;
      for (int h = hk * G; h < hk * G + G; ++h) {
        x.load(a.dout + (i * a.H + h) * D, lane);
        y.load(a.out + (i * a.H + h) * D, lane);
        const float dl = x.dot(y), dp = x.dot(v);
        y.load(a.q + i * a.q_stride + (int64_t)h * D, lane);
        const float p = __expf(y.dot(k) * a.scale - a.lse[i * a.H + h]);
        dv.axpy(p, x);
        dk.axpy(p * (dp - dl), y);
      }
    }
  }
  dk.store(a.dk + (j * a.Hkv + hk) * D, a.scale, lane);
  dv.store(a.dv + (j * a.Hkv + hk) * D, 1.f, lane);
}

struct WindowLayout {
  size_t row_start = 0, row_end = 0, total = 0;
};

WindowLayout window_layout(int64_t T, bool bwd) {
  WindowLayout L;
  L.row_end = align_up(4 * (size_t)T, 256);
  L.total = align_up(L.row_end + (bwd ? 4 * (size_t)T : 0), 256);
  if (L.total == 0) L.total = 256;
  return L;
}

bool window_sizes_ok(int64_t B, int64_t T, int H, int Hkv, int n_sinks) {
  return B >= 0 && T >= 0 && T < (int64_t)INT_MAX - kItemRows && B < (int64_t)INT_MAX && H >= 1 &&
         H < 65536 && Hkv >= 1 && H % Hkv == 0 && n_sinks >= 0 && n_sinks <= kMaxSinks &&
         (B > 0 || T == 0);
}

int window_check(int64_t B, int64_t T, int H, int Hkv, int d, int64_t window, int n_sinks,
                 int64_t qs, int64_t ks, int64_t vs, int idx_bits) {
  if (idx_bits != 32 && idx_bits != 64) return JCA_ERR_IDX_BITS;
  if (!head_dim_ok(d)) return JCA_ERR_HEAD_DIM;
  if (!window_sizes_ok(B, T, H, Hkv, n_sinks) || window < 1) return JCA_ERR_SHAPE;
  if (qs < (int64_t)H * d || ks < (int64_t)Hkv * d || vs < (int64_t)Hkv * d) return JCA_ERR_SHAPE;
  if (qs % 8 || ks % 8 || vs % 8) return JCA_ERR_ALIGN;
  return JCA_OK;
}

int window_plan(const void* offsets, int64_t B, int64_t T, int idx_bits, int32_t* row_start,
                int32_t* row_end, int32_t* status, cudaStream_t st) {
  const unsigned grid = (unsigned)(B < (1 << 20) ? B : (1 << 20));
  if (idx_bits == 32)
    window_plan_kernel<int32_t><<<grid, 128, 0, st>>>(static_cast<const int32_t*>(offsets), B, T,
                                                      row_start, row_end, status);
  else
    window_plan_kernel<int64_t><<<grid, 128, 0, st>>>(static_cast<const int64_t*>(offsets), B, T,
                                                      row_start, row_end, status);
  return cudaGetLastError() == cudaSuccess ? JCA_OK : JCA_ERR_CUDA;
}

}  // namespace
}  // namespace jca

using namespace jca;

extern "C" size_t jca_window_workspace_bytes(int64_t B, int64_t T, int H, int Hkv, int d_head,
                                             int n_sinks) {
  if (!window_sizes_ok(B, T, H, Hkv, n_sinks) || !head_dim_ok(d_head)) return 0;
  return window_layout(T, false).total;
}

extern "C" size_t jca_window_bwd_workspace_bytes(int64_t B, int64_t T, int H, int Hkv, int d_head,
                                                 int n_sinks) {
  if (!window_sizes_ok(B, T, H, Hkv, n_sinks) || !head_dim_ok(d_head)) return 0;
  return window_layout(T, true).total;
}

extern "C" int jagged_window_attn_fwd(const void* q, const void* k, const void* v, void* out,
                                      float* lse, const void* offsets, const uint8_t* valid,
                                      int64_t B, int64_t T, int H, int Hkv, int d_head,
                                      int64_t window, int n_sinks, int64_t q_stride,
                                      int64_t k_stride, int64_t v_stride, float scale,
                                      int idx_bits, void* workspace, size_t workspace_bytes,
                                      int32_t* status, jca_stream_t stream) {
  int rc = window_check(B, T, H, Hkv, d_head, window, n_sinks, q_stride, k_stride, v_stride,
                        idx_bits);
  if (rc) return rc;
  if (!status || !offsets || !workspace) return JCA_ERR_NULL;
  if (T > 0 && (!q || !k || !v || !out)) return JCA_ERR_NULL;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) ||
      !aligned(lse, 4) || !aligned(workspace, 256))
    return JCA_ERR_ALIGN;
  const WindowLayout L = window_layout(T, false);
  if (workspace_bytes < L.total) return JCA_ERR_WORKSPACE;
  if (B == 0) return JCA_OK;
  int dev = 0, sms = 0;
  rc = current_device(&dev, &sms);
  if (rc) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  WindowArgs a = {};
  a.q = static_cast<const bf16*>(q);
  a.k = static_cast<const bf16*>(k);
  a.v = static_cast<const bf16*>(v);
  a.o = static_cast<bf16*>(out);
  a.lse_out = lse;
  a.valid = valid;
  a.row_start = reinterpret_cast<int32_t*>(ws + L.row_start);
  a.status = status;
  a.T = T;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.H = H;
  a.Hkv = Hkv;
  a.window = (int)(window < T ? window : (T > 0 ? T : 1));
  a.n_sinks = n_sinks;
  a.scale = scale > 0.f ? scale : 1.0f / sqrtf((float)d_head);
  rc = window_plan(offsets, B, T, idx_bits, reinterpret_cast<int32_t*>(ws + L.row_start), nullptr,
                   status, st);
  if (rc || T == 0) return rc;
  const int64_t blocks = (T * H + 3) / 4;
  if (blocks >= (int64_t)INT_MAX) return JCA_ERR_SHAPE;
  switch (d_head) {
    case 16: window_fwd_kernel<16><<<(unsigned)blocks, 128, 0, st>>>(a); break;
    case 32: window_fwd_kernel<32><<<(unsigned)blocks, 128, 0, st>>>(a); break;
    case 64: window_fwd_kernel<64><<<(unsigned)blocks, 128, 0, st>>>(a); break;
    default: window_fwd_kernel<128><<<(unsigned)blocks, 128, 0, st>>>(a); break;
  }
  return cudaGetLastError() == cudaSuccess ? JCA_OK : JCA_ERR_CUDA;
}

namespace jca {
namespace {
template <int D>
void launch_window_bwd(const WindowArgs& a, cudaStream_t st) {
  window_dq_kernel<D><<<(unsigned)((a.T * a.H + 3) / 4), 128, 0, st>>>(a);
  window_dkv_kernel<D><<<(unsigned)((a.T * a.Hkv + 3) / 4), 128, 0, st>>>(a);
}
}  // namespace
}  // namespace jca

extern "C" int jagged_window_attn_bwd(const void* q, const void* k, const void* v, const void* out,
                                      const void* dout, const float* lse, void* dq, void* dk,
                                      void* dv, const void* offsets, const uint8_t* valid,
                                      int64_t B, int64_t T, int H, int Hkv, int d_head,
                                      int64_t window, int n_sinks, int64_t q_stride,
                                      int64_t k_stride, int64_t v_stride, float scale,
                                      int idx_bits, void* workspace, size_t workspace_bytes,
                                      int32_t* status, jca_stream_t stream) {
  int rc = window_check(B, T, H, Hkv, d_head, window, n_sinks, q_stride, k_stride, v_stride,
                        idx_bits);
  if (rc) return rc;
  if (!status || !offsets || !workspace) return JCA_ERR_NULL;
  if (T > 0 && (!q || !k || !v || !out || !dout || !lse || !dq || !dk || !dv)) return JCA_ERR_NULL;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) ||
      !aligned(dout, 16) || !aligned(lse, 4) || !aligned(dq, 16) || !aligned(dk, 16) ||
      !aligned(dv, 16) || !aligned(workspace, 256))
    return JCA_ERR_ALIGN;
  const WindowLayout L = window_layout(T, true);
  if (workspace_bytes < L.total) return JCA_ERR_WORKSPACE;
  if (B == 0) return JCA_OK;
  int dev = 0, sms = 0;
  rc = current_device(&dev, &sms);
  if (rc) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  WindowArgs a = {};
  a.q = static_cast<const bf16*>(q);
  a.k = static_cast<const bf16*>(k);
  a.v = static_cast<const bf16*>(v);
  a.out = static_cast<const bf16*>(out);
  a.dout = static_cast<const bf16*>(dout);
  a.lse = lse;
  a.dq = static_cast<bf16*>(dq);
  a.dk = static_cast<bf16*>(dk);
  a.dv = static_cast<bf16*>(dv);
  a.valid = valid;
  a.row_start = reinterpret_cast<int32_t*>(ws + L.row_start);
  a.row_end = reinterpret_cast<int32_t*>(ws + L.row_end);
  a.status = status;
  a.T = T;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.H = H;
  a.Hkv = Hkv;
  a.window = (int)(window < T ? window : (T > 0 ? T : 1));
  a.n_sinks = n_sinks;
  a.scale = scale > 0.f ? scale : 1.0f / sqrtf((float)d_head);
  rc = window_plan(offsets, B, T, idx_bits, reinterpret_cast<int32_t*>(ws + L.row_start),
                   reinterpret_cast<int32_t*>(ws + L.row_end), status, st);
  if (rc || T == 0) return rc;
  switch (d_head) {
    case 16: launch_window_bwd<16>(a, st); break;
    case 32: launch_window_bwd<32>(a, st); break;
    case 64: launch_window_bwd<64>(a, st); break;
    default: launch_window_bwd<128>(a, st); break;
  }
  return cudaGetLastError() == cudaSuccess ? JCA_OK : JCA_ERR_CUDA;
}
