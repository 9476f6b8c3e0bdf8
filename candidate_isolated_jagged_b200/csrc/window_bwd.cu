// Causal attention over packed rows with a sliding window and first tokens that stay visible:
// forward and backward (include/jca.h states the mask and the layout).
#include <climits>
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "jca_device.cuh"
#include "jca_internal.h"
#include "window.h"

namespace jca {
namespace {

using bf16 = __nv_bfloat16;

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

struct BwdLayout {
  size_t row_start = 0, row_end = 0, counters = 0, total = 0;
};

BwdLayout bwd_layout(int64_t T) {
  BwdLayout L;
  L.row_end = align_up(4 * (size_t)T, 256);
  L.counters = align_up(L.row_end + 4 * (size_t)T, 256);
  L.total = L.counters + 256;
  return L;
}

}  // namespace
}  // namespace jca

using namespace jca;

extern "C" size_t jca_window_bwd_workspace_bytes(int64_t B, int64_t T, int H, int Hkv, int d_head,
                                                 int n_sinks) {
  if (!window_sizes_ok(B, T, H, Hkv, n_sinks) || !head_dim_ok(d_head)) return 0;
  return bwd_layout(T).total;
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
  const BwdLayout L = bwd_layout(T);
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
                   reinterpret_cast<int32_t*>(ws + L.row_end),
                   reinterpret_cast<int32_t*>(ws + L.counters), 1, status, st);
  if (rc || T == 0) return rc;
  switch (d_head) {
    case 16: launch_window_bwd<16>(a, st); break;
    case 32: launch_window_bwd<32>(a, st); break;
    case 64: launch_window_bwd<64>(a, st); break;
    default: launch_window_bwd<128>(a, st); break;
  }
  return cudaGetLastError() == cudaSuccess ? JCA_OK : JCA_ERR_CUDA;
}
