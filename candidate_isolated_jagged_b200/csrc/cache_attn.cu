// Attention of a few new tokens per user over the user's cached history: one new token with a sliding
// window and visible first tokens (jagged_window_decode_fwd), and a tree of drafted tokens
// (cand_tree_attn_fwd); include/jca.h states both.
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

constexpr int kMaxTree = 1024;

struct CacheArgs {
  const bf16* q;
  const bf16* k;            // decode: the new tokens; tree: the drafted tokens
  const bf16* v;
  bf16* kc;
  bf16* vc;
  bf16* out;
  const void* off;          // decode: cache regions; tree: drafted runs
  const void* hist_off;     // tree: cache regions
  const void* len;          // tokens in each region (tree: may be null)
  const int32_t* parent;
  int32_t* status;
  int64_t B, N, R, window, n_sinks, q_stride, k_stride, v_stride;
  int H, Hkv, max_cand;
  float scale;
};

template <int D>
struct Vecs {
  static constexpr int EPL = D >= 32 ? D / 32 : 1;
  float q[EPL], acc[EPL], m, l;
  __device__ __forceinline__ void see(const bf16* k, const bf16* v, float scale, int lane) {
    float s = 0.f;
    if (lane * EPL < D)
#pragma unroll
      for (int i = 0; i < EPL; ++i) s = fmaf(q[i], __bfloat162float(k[lane * EPL + i]), s);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= scale;
    const float mn = fmaxf(m, s), al = m == -INFINITY ? 0.f : __expf(m - mn), p = __expf(s - mn);
    if (lane * EPL < D)
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        acc[i] = fmaf(p, __bfloat162float(v[lane * EPL + i]), acc[i] * al);
    l = l * al + p;
    m = mn;
  }
  __device__ __forceinline__ void start(const bf16* p, int lane) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      q[i] = lane * EPL < D ? __bfloat162float(p[lane * EPL + i]) : 0.f;
      acc[i] = 0.f;
    }
    m = -INFINITY;
    l = 0.f;
  }
  __device__ __forceinline__ void store(bf16* p, int lane) const {
    if (lane * EPL < D)
#pragma unroll
      for (int i = 0; i < EPL; ++i) p[lane * EPL + i] = __float2bfloat16(l > 0.f ? acc[i] / l : 0.f);
  }
};

__device__ __forceinline__ void set_status(int32_t* status, int code) {
  atomicCAS(status, 0, (int32_t)code);
}

// One warp per (user, head).
template <int D, typename IdxT>
__global__ void __launch_bounds__(128) decode_kernel(const CacheArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t w = blockIdx.x * (int64_t)4 + (threadIdx.x >> 5);
  if (w >= a.B * a.H || *a.status != 0) return;
  const int64_t b = w / a.H;
  const int h = (int)(w % a.H), G = a.H / a.Hkv, hk = h / G;
  const IdxT* off = static_cast<const IdxT*>(a.off);
  const int64_t s = off[b], e = off[b + 1], p = static_cast<const IdxT*>(a.len)[b];
  if (s < 0 || s > e || e > a.R) {
    if (lane == 0) set_status(a.status, JCA_STATUS_BAD_OFFSETS);
    return;
  }
  if (p < -1 || (p >= 0 && p >= e - s)) {
    if (lane == 0) set_status(a.status, JCA_STATUS_BAD_LENGTH);
    return;
  }
  Vecs<D> x;
  x.start(a.q + b * a.q_stride + (int64_t)h * D, lane);
  if (p >= 0) {
    const bf16* kn = a.k + b * a.k_stride + (int64_t)hk * D;
    const bf16* vn = a.v + b * a.v_stride + (int64_t)hk * D;
    const int64_t lo = max((int64_t)0, p - a.window + 1), first = min(a.n_sinks, lo);
    for (int64_t j = 0; j < p; ++j) {
      if (j == first && first < lo) j = lo;
      if (j >= p) break;
      const int64_t at = ((s + j) * a.Hkv + hk) * D;
      x.see(a.kc + at, a.vc + at, a.scale, lane);
    }
    x.see(kn, vn, a.scale, lane);
    if (h == hk * G && lane * Vecs<D>::EPL < D) {
      const int64_t at = ((s + p) * a.Hkv + hk) * D;
#pragma unroll
      for (int i = 0; i < Vecs<D>::EPL; ++i) {
        a.kc[at + lane * Vecs<D>::EPL + i] = kn[lane * Vecs<D>::EPL + i];
        a.vc[at + lane * Vecs<D>::EPL + i] = vn[lane * Vecs<D>::EPL + i];
      }
    }
  }
  x.store(a.out + (b * a.H + h) * D, lane);
}

// One block per (user, token): the block checks the user, then each warp takes heads.
template <int D, typename IdxT>
__global__ void __launch_bounds__(128) tree_kernel(const CacheArgs a) {
  if (*a.status != 0) return;
  const int lane = threadIdx.x & 31;
  const int64_t b = blockIdx.y;
  const IdxT *off = static_cast<const IdxT*>(a.off), *ho = static_cast<const IdxT*>(a.hist_off);
  const int64_t s = off[b], e = off[b + 1], hs = ho[b], he = ho[b + 1];
  int bad = 0;
  int64_t hl = he - hs;
  if (s < 0 || s > e || e > a.N || (b == 0 && s != 0) || (b == a.B - 1 && e != a.N) || hs < 0 ||
      hs > he || he > a.R) {
    bad = JCA_STATUS_BAD_OFFSETS;
  } else if (e - s > a.max_cand) {
    bad = JCA_STATUS_BAD_TREE;
  } else if (a.len) {
    hl = static_cast<const IdxT*>(a.len)[b];
    if (hl < 0 || hl > he - hs) bad = JCA_STATUS_BAD_LENGTH;
  }
  if (!bad) {
    int wrong = 0;
    for (int i = threadIdx.x; i < e - s; i += blockDim.x) {
      const int p = a.parent[s + i];
      wrong |= p < -1 || p >= i;
    }
    if (__syncthreads_or(wrong)) bad = JCA_STATUS_BAD_TREE;
  }
  if (bad) {
    if (threadIdx.x == 0) set_status(a.status, bad);
    return;
  }
  const int64_t t = blockIdx.x;
  if (t >= e - s) return;
  const int G = a.H / a.Hkv;
  for (int h = threadIdx.x >> 5; h < a.H; h += 4) {
    const int hk = h / G;
    Vecs<D> x;
    x.start(a.q + (s + t) * a.q_stride + (int64_t)h * D, lane);
    for (int64_t j = 0; j < hl; ++j) {
      const int64_t at = ((hs + j) * a.Hkv + hk) * D;
      x.see(a.kc + at, a.vc + at, a.scale, lane);
    }
    for (int j = (int)t; j >= 0; j = a.parent[s + j])
      x.see(a.k + (s + j) * a.k_stride + (int64_t)hk * D,
            a.v + (s + j) * a.v_stride + (int64_t)hk * D, a.scale, lane);
    x.store(a.out + ((s + t) * a.H + h) * D, lane);
  }
}

int cache_check(int64_t B, int64_t rows, int64_t R, int H, int Hkv, int d, int64_t qs, int64_t ks,
                int64_t vs, int idx_bits) {
  if (idx_bits != 32 && idx_bits != 64) return JCA_ERR_IDX_BITS;
  if (!head_dim_ok(d)) return JCA_ERR_HEAD_DIM;
  if (B < 0 || rows < 0 || rows >= (int64_t)INT_MAX || R < 0 || R >= (int64_t)INT_MAX ||
      B >= (int64_t)INT_MAX || H < 1 || H >= 65536 || Hkv < 1 || H % Hkv)
    return JCA_ERR_SHAPE;
  if (qs < (int64_t)H * d || ks < (int64_t)Hkv * d || vs < (int64_t)Hkv * d) return JCA_ERR_SHAPE;
  if (qs % 8 || ks % 8 || vs % 8) return JCA_ERR_ALIGN;
  return JCA_OK;
}

template <int D>
void launch_decode(const CacheArgs& a, int idx_bits, cudaStream_t st) {
  const unsigned grid = (unsigned)((a.B * a.H + 3) / 4);
  if (idx_bits == 32) decode_kernel<D, int32_t><<<grid, 128, 0, st>>>(a);
  else decode_kernel<D, int64_t><<<grid, 128, 0, st>>>(a);
}

template <int D>
void launch_tree(const CacheArgs& a, int idx_bits, cudaStream_t st) {
  const dim3 grid((unsigned)a.max_cand, (unsigned)a.B);
  if (idx_bits == 32) tree_kernel<D, int32_t><<<grid, 128, 0, st>>>(a);
  else tree_kernel<D, int64_t><<<grid, 128, 0, st>>>(a);
}

}  // namespace
}  // namespace jca

using namespace jca;

extern "C" int jagged_window_decode_fwd(const void* q, const void* k_new, const void* v_new,
                                        void* k_cache, void* v_cache, void* out,
                                        const void* cache_offsets, const void* cache_len,
                                        int64_t B, int64_t R, int H, int Hkv, int d_head,
                                        int64_t window, int64_t n_sinks, int64_t q_stride,
                                        int64_t k_stride, int64_t v_stride, float scale,
                                        int idx_bits, int32_t* status, jca_stream_t stream) {
  int rc = cache_check(B, B, R, H, Hkv, d_head, q_stride, k_stride, v_stride, idx_bits);
  if (rc) return rc;
  if (window < 1 || n_sinks < 0) return JCA_ERR_SHAPE;
  if (B == 0) return JCA_OK;
  if (!status || !q || !k_new || !v_new || !out || !cache_offsets || !cache_len ||
      (R > 0 && (!k_cache || !v_cache)))
    return JCA_ERR_NULL;
  if (!aligned(q, 16) || !aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16) || !aligned(out, 16))
    return JCA_ERR_ALIGN;
  int dev = 0, sms = 0;
  rc = current_device(&dev, &sms);
  if (rc) return rc;
  CacheArgs a = {};
  a.q = static_cast<const bf16*>(q);
  a.k = static_cast<const bf16*>(k_new);
  a.v = static_cast<const bf16*>(v_new);
  a.kc = static_cast<bf16*>(k_cache);
  a.vc = static_cast<bf16*>(v_cache);
  a.out = static_cast<bf16*>(out);
  a.off = cache_offsets;
  a.len = cache_len;
  a.status = status;
  a.B = B;
  a.N = B;
  a.R = R;
  a.window = window;
  a.n_sinks = n_sinks;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.H = H;
  a.Hkv = Hkv;
  a.scale = scale > 0.f ? scale : 1.0f / sqrtf((float)d_head);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  switch (d_head) {
    case 16: launch_decode<16>(a, idx_bits, st); break;
    case 32: launch_decode<32>(a, idx_bits, st); break;
    case 64: launch_decode<64>(a, idx_bits, st); break;
    default: launch_decode<128>(a, idx_bits, st); break;
  }
  return cudaGetLastError() == cudaSuccess ? JCA_OK : JCA_ERR_CUDA;
}

extern "C" int cand_tree_attn_fwd(const void* cand_q, const void* own_k, const void* own_v,
                                  const void* cand_offsets, const int32_t* parent,
                                  const void* hist_k, const void* hist_v,
                                  const void* hist_offsets, const void* hist_len, void* out,
                                  int64_t B, int64_t Nc, int64_t R, int H, int Hkv, int d_head,
                                  int max_cand, int64_t q_stride, int64_t k_stride,
                                  int64_t v_stride, float scale, int idx_bits, int32_t* status,
                                  jca_stream_t stream) {
  int rc = cache_check(B, Nc, R, H, Hkv, d_head, q_stride, k_stride, v_stride, idx_bits);
  if (rc) return rc;
  if (max_cand < 1 || max_cand > kMaxTree || (B == 0 && Nc > 0) || B > 65535) return JCA_ERR_SHAPE;
  if (B == 0) return JCA_OK;
  if (!status || !cand_offsets || !hist_offsets ||
      (Nc > 0 && (!cand_q || !own_k || !own_v || !parent || !out)) ||
      (R > 0 && (!hist_k || !hist_v)))
    return JCA_ERR_NULL;
  if (!aligned(cand_q, 16) || !aligned(own_k, 16) || !aligned(own_v, 16) || !aligned(hist_k, 16) ||
      !aligned(hist_v, 16) || !aligned(out, 16))
    return JCA_ERR_ALIGN;
  int dev = 0, sms = 0;
  rc = current_device(&dev, &sms);
  if (rc) return rc;
  CacheArgs a = {};
  a.q = static_cast<const bf16*>(cand_q);
  a.k = static_cast<const bf16*>(own_k);
  a.v = static_cast<const bf16*>(own_v);
  a.kc = static_cast<bf16*>(const_cast<void*>(hist_k));
  a.vc = static_cast<bf16*>(const_cast<void*>(hist_v));
  a.out = static_cast<bf16*>(out);
  a.off = cand_offsets;
  a.hist_off = hist_offsets;
  a.len = hist_len;
  a.parent = parent;
  a.status = status;
  a.B = B;
  a.N = Nc;
  a.R = R;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.H = H;
  a.Hkv = Hkv;
  a.max_cand = max_cand;
  a.scale = scale > 0.f ? scale : 1.0f / sqrtf((float)d_head);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  switch (d_head) {
    case 16: launch_tree<16>(a, idx_bits, st); break;
    case 32: launch_tree<32>(a, idx_bits, st); break;
    case 64: launch_tree<64>(a, idx_bits, st); break;
    default: launch_tree<128>(a, idx_bits, st); break;
  }
  return cudaGetLastError() == cudaSuccess ? JCA_OK : JCA_ERR_CUDA;
}
