// Attention of a few new tokens per user over the user's cached history: one new token with a sliding
// window and visible first tokens (jagged_window_decode_fwd), and a tree of drafted tokens
// (cand_tree_attn_fwd); include/jca.h states both.
//
// Mathematics: softmax(scale q K^T) V over the list of keys a user's tokens see, with a running
// maximum m and sum l in fp32 (p = 2^(s - m) in log2 units), so the keys are read once.
//
// What bounds it: reading the cache. A user's n tokens times the G = H / Hkv query heads of a key
// head are the rows of one product against that head's keys, so a key's 4 d bytes (K and V) serve
// n G rows. With few rows (256 users, one token each, 4 heads to a key head: 68 us, 0.90 of the copy
// bandwidth) nothing else counts. With 64 rows (256 users with trees of 64 tokens: 151 us, 0.60) a
// key of d = 128 takes an SM 22 cycles to read at the copy bandwidth, 16 of the warp-level tensor
// instruction (m16n8k16, 8 cycles each) and 20 of shared-memory reads, which three warps per
// scheduler overlap (two: 165 us), and the longest history, 65 tiles in one block, ends last. A
// 128-row tcgen05 tile would leave half or more of its rows empty here and would have to clear the
// ends of the cache in shared memory; here the copies zero-fill what lies behind the last key.
// One user alone (4,096 keys: 10.9 us) pays for its launch, three dependent reads and the joining.
//
// Shape: a block of 4 warps takes up to 64 rows of one (user, key head) and walks 64-key tiles
// through a ring of stages filled by 16-byte asynchronous copies. With 64 rows each warp owns 16 of
// them and sees all 64 keys; with at most 16 rows (one token, shared heads) the four warps take 16
// keys each and their partial results are joined at the end. When there are few (user, head) pairs,
// the key list is split further over a cluster of up to 8 blocks, which join through distributed
// shared memory in rank order: one launch, no workspace, equal bits for equal calls.
// The keys of a tile that a copy does not reach (behind the list) are zeros, so whatever the cache
// holds there never meets a weight.
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "jca_device.cuh"
#include "jca_internal.h"

namespace jca {
namespace {

namespace cg = cooperative_groups;
using bf16 = __nv_bfloat16;

constexpr int kMaxTree = 1024;
constexpr int kThr = 128;          // threads of a block
constexpr int kBK = 64;            // keys of a tile
// Blocks of a cluster. (Sixteen: one user's token 10.8 us too, 4 users with trees 10.9 us, not 9.7.)
constexpr int kMaxSplit = 8;
constexpr int kTreeWords = kMaxTree / 32;
constexpr int kGroup = 256;        // users that are put in order together

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
  int H, Hkv, max_cand, row_blocks, split;
  int longest_first;        // tree: users in the order of longest_first()
  float scale_log2;
};

__device__ __forceinline__ void set_status(int32_t* status, int code) {
  atomicCAS(status, 0, (int32_t)code);
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool real) {
  const int n = real ? 16 : 0;   // 0: the 16 bytes are zero-filled, nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// RW warps of 16 rows, times KW warps that share the rows and split the keys of a tile. (Eight warps
// for 64 rows, two to a row group, measured slower: 272 us against 222 on the 256 users with trees,
// with the users in the order of the batch.)
template <int D, int RW, bool TREE>
struct CCfg {
  static constexpr int CH = D / 8;                        // 16-byte chunks of a row
  static constexpr int RB = 16 * RW;                      // rows of a block
  static constexpr int KW = 4 / RW;
  static constexpr int KPW = kBK / KW;                    // keys of a tile per warp
  static constexpr int TILE = kBK * D * 2;                // bytes of a K or V tile
  static constexpr int STAGE = 2 * TILE;
  static constexpr int STAGES = D == 128 ? (RW == 4 ? 2 : 3) : 4;
  static constexpr int BPS = RW == 4 ? 3 : 2;             // blocks per SM
  static constexpr int OFF_ML = STAGES * STAGE;           // [KW][RB] m and l, then [RB] joined
  static constexpr int OFF_BITS = OFF_ML + (2 * KW + 2) * RB * 4;
  static constexpr int OFF_PAR = 0;                       // in the ring, before its first tile
  static constexpr int OFF_TILES = OFF_BITS + (TREE ? RB * kTreeWords * 4 : 0);
  static constexpr int SMEM = OFF_TILES + (TREE ? 128 : 16);
  // Partial results [KW][RB][D] fp32 reuse the ring.
  static_assert(KW * RB * D * 4 <= STAGES * STAGE, "partials fit the ring");
  static_assert(RB * D * 2 <= STAGE, "Q fits one stage");
  static_assert(BPS * (SMEM + 1024) <= 228 * 1024, "blocks per SM");
};

// Shared-memory byte offset of chunk c of row r: chunks are XORed with the row so that eight rows'
// chunks of one column fall into different banks.
template <int D>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  constexpr int CH = D / 8;
  constexpr int RPL = CH >= 8 ? 1 : 8 / CH;               // rows of a 128-byte line
  constexpr int MASK = (CH >= 8 ? 8 : CH) - 1;
  return (uint32_t)(r * CH + (c ^ ((r / RPL) & MASK))) * 16u;
}

// The keys a block walks: rows of the cache and the new tokens' own rows.
struct Keys {
  int64_t base;       // first cache row of the list
  int64_t base2;      // decode: first cache row behind the visible first tokens
  int n1, n2;         // decode: first tokens, window tokens before the new one; tree: history, 0
  int64_t own;        // first own row
  int n_own;          // own rows
  int own_tile;       // tree: first tile of own rows
};

// The user that takes place b when the users of each group of 256 go by the length of their history,
// longest first. Blocks start in the order of their index, so a long history that starts late runs
// on alone after the others (256 users with trees of 64 tokens, two blocks to an SM: 222 us in the
// order of the batch, 165 us so).
// A sort by quarter octaves is close enough and cheap: counts, a scan, the bucket that holds the
// place, the place's bit among its members. It depends on the lengths only, so all blocks agree
// whatever the lengths hold. `w`: 128 + 10 words of shared memory.
template <typename IdxT>
__device__ int64_t longest_first(const CacheArgs& a, int64_t b, uint32_t* w) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t g0 = b - b % kGroup;
  const IdxT* ho = static_cast<const IdxT*>(a.hist_off);
  const IdxT* len = static_cast<const IdxT*>(a.len);
  int bucket[kGroup / kThr];
  w[tid] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kGroup / kThr; ++i) {
    const int64_t u = g0 + i * kThr + tid;
    bucket[i] = -1;
    if (u < a.B) {
      const int64_t n = len ? (int64_t)len[u] : (int64_t)ho[u + 1] - (int64_t)ho[u];
      const uint32_t x = (uint32_t)max((int64_t)4, min(n, (int64_t)INT_MAX));
      const int e = 31 - __clz(x);
      bucket[i] = 127 - (4 * e + (int)((x >> (e - 2)) & 3));
      atomicAdd(&w[bucket[i]], 1u);
    }
  }
  __syncthreads();
  if (warp == 0) {
    uint32_t c[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) sum += c[i] = w[4 * lane + i];
    uint32_t at = sum;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, at, d);
      if (lane >= d) at += y;
    }
    at -= sum;
    const uint32_t place = (uint32_t)(b - g0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (place >= at && place < at + c[i]) {
        w[128] = 4 * lane + i;
        w[129] = place - at;
      }
      at += c[i];
    }
  }
  __syncthreads();
  const int want = (int)w[128], k = (int)w[129];
  uint32_t mine[kGroup / kThr];   // members of the bucket in this warp's 32 users
#pragma unroll
  for (int i = 0; i < kGroup / kThr; ++i) {
    mine[i] = __ballot_sync(0xffffffffu, bucket[i] == want);
    if (lane == 0) w[130 + i * (kThr / 32) + warp] = __popc(mine[i]);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kGroup / kThr; ++i) {
    int before = __popc(mine[i] & ((1u << lane) - 1u));
    for (int x = 0; x < i * (kThr / 32) + warp; ++x) before += (int)w[130 + x];
    if (bucket[i] == want && before == k) w[0] = i * kThr + tid;
  }
  __syncthreads();
  const int64_t user = g0 + w[0];
  __syncthreads();
  return user;
}

template <int D, int RW, bool TREE, typename IdxT>
__global__ void __launch_bounds__(kThr, CCfg<D, RW, TREE>::BPS) cache_attn_kernel(const CacheArgs a) {
  using C = CCfg<D, RW, TREE>;
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)(blockIdx.x % (unsigned)a.split);
  int64_t unit = blockIdx.x / (unsigned)a.split;
  const int rb = (int)(unit % a.row_blocks);
  unit /= a.row_blocks;
  const int hk = (int)(unit % a.Hkv);
  int64_t b = unit / a.Hkv;
  if constexpr (TREE)
    if (a.longest_first) b = longest_first<IdxT>(a, b, reinterpret_cast<uint32_t*>(smem));
  const int G = a.H / a.Hkv;
  const IdxT* off = static_cast<const IdxT*>(a.off);

  // The user's numbers, all loads under way before the first is used.
  const int64_t off0 = off[b], off1 = off[b + 1];
  int64_t h0 = 0, h1 = 0, len = 0;
  if constexpr (TREE) {
    h0 = static_cast<const IdxT*>(a.hist_off)[b];
    h1 = static_cast<const IdxT*>(a.hist_off)[b + 1];
  }
  if (a.len) len = static_cast<const IdxT*>(a.len)[b];
  const int before = *a.status;
  // An error recorded earlier makes the call a no-op. Threads and blocks of a cluster could see a
  // status that another user's block sets meanwhile at different times, so all threads of a block
  // go by one vote, and a block that sees an error keeps in step with its cluster and only tells
  // the others, at the joining, that it has nothing to add.
  const bool skip = __syncthreads_or(tid == 0 && before != 0);
  if (skip && a.split == 1) return;

  // The user's keys and rows; every block of a user takes the same decisions.
  Keys k;
  int rows = 0;                       // rows of this block
  int nt = 0;                         // key tiles
  int64_t row0 = 0;                   // token of row 0 of the user in q
  if constexpr (TREE) {
    const int64_t s = off0, e = off1, hs = h0, he = h1;
    int bad = 0;
    int64_t hl = he - hs;
    if (s < 0 || s > e || e > a.N || (b == 0 && s != 0) || (b == a.B - 1 && e != a.N) || hs < 0 ||
        hs > he || he > a.R) {
      bad = JCA_STATUS_BAD_OFFSETS;
    } else if (e - s > a.max_cand) {
      bad = JCA_STATUS_BAD_TREE;
    } else if (a.len) {
      hl = len;
      if (hl < 0 || hl > he - hs) bad = JCA_STATUS_BAD_LENGTH;
    }
    const int n = bad ? 0 : (int)(e - s);
    // Every block looks at all parents of its user, so that all of them see a bad one.
    int16_t* par = reinterpret_cast<int16_t*>(smem + C::OFF_PAR);
    int wrong = 0;
    for (int i = tid; i < n; i += kThr) {
      const int p = a.parent[s + i];
      wrong |= p < -1 || p >= i;
      par[i] = (int16_t)p;
    }
    if (__syncthreads_or(wrong)) bad = JCA_STATUS_BAD_TREE;
    if (bad) {
      if (tid == 0 && !skip) set_status(a.status, bad);
      return;
    }
    rows = min(C::RB, n * G - rb * C::RB);
    if (rows <= 0) return;
    row0 = s;
    k.base = hs;
    k.n1 = (int)hl;
    k.own = s;
    k.n_own = n;
    k.own_tile = (int)((hl + kBK - 1) / kBK);
    // Ancestors of the block's tokens, a bit per drafted token, and the own tiles that hold any.
    uint32_t* bits = reinterpret_cast<uint32_t*>(smem + C::OFF_BITS);
    int* tiles = reinterpret_cast<int*>(smem + C::OFF_TILES);   // [16] tiles, [16] count, [17] flags
    const int tok0 = rb * C::RB / G, ntok = (rb * C::RB + rows - 1) / G - tok0 + 1;
    const int words = 2 * ((n + kBK - 1) / kBK);   // whole tiles
    for (int i = tid; i < ntok * words; i += kThr) bits[i / words * kTreeWords + i % words] = 0;
    if (tid == 0) tiles[17] = 0;
    __syncthreads();
    if (tid < ntok) {
      int flags = 0;
      for (int j = tok0 + tid; j >= 0; j = par[j]) {
        bits[tid * kTreeWords + (j >> 5)] |= 1u << (j & 31);
        flags |= 1 << (j / kBK);
      }
      atomicOr(&tiles[17], flags);
    }
    __syncthreads();
    if (tid == 0) {
      int c = 0;
      for (int f = tiles[17]; f; f &= f - 1) tiles[c++] = __ffs(f) - 1;
      tiles[16] = c;
    }
    __syncthreads();
    nt = k.own_tile + tiles[16];
  } else {
    const int64_t s = off0, e = off1, p = len;
    int bad = 0;
    if (s < 0 || s > e || e > a.R) bad = JCA_STATUS_BAD_OFFSETS;
    else if (p < -1 || (p >= 0 && p >= e - s)) bad = JCA_STATUS_BAD_LENGTH;
    if (bad) {
      if (tid == 0 && !skip) set_status(a.status, bad);
      return;
    }
    rows = min(C::RB, G - rb * C::RB);
    row0 = b;
    if (p < 0) {   // an empty slot of the batch
      if (rank == 0 && !skip)
        for (int i = tid; i < rows * C::CH; i += kThr)
          reinterpret_cast<uint4*>(a.out + (b * a.H + (int64_t)hk * G + rb * C::RB) * D)[i] =
              make_uint4(0u, 0u, 0u, 0u);
      return;
    }
    const int64_t lo = max((int64_t)0, p - a.window + 1);
    k.n1 = (int)min(a.n_sinks, lo);
    k.n2 = (int)(p - lo);
    k.base = s;
    k.base2 = s + lo;
    k.own = b;
    k.n_own = 1;
    nt = (k.n1 + k.n2) / kBK + 1;   // of n1 + n2 + 1 keys; rounding up would pass 2^31 on the longest
    // The new token's key and value go behind the cached ones; no block reads them from there.
    if (rank == 0 && rb == 0 && !skip && tid < 2 * C::CH) {
      const int c = tid % C::CH;
      const bool is_k = tid < C::CH;
      const bf16* src = is_k ? a.k + b * a.k_stride : a.v + b * a.v_stride;
      bf16* dst = (is_k ? a.kc : a.vc) + ((s + p) * a.Hkv + hk) * D;
      reinterpret_cast<uint4*>(dst)[c] = reinterpret_cast<const uint4*>(src + (int64_t)hk * D)[c];
    }
  }
  const int per = (nt + a.split - 1) / a.split;
  const int t0 = min(nt, rank * per), t1 = skip ? t0 : min(nt, t0 + per);

  // This thread's share of a tile: chunk tid % CH of rows r0, r0 + kStep, ...
  constexpr int kStep = kThr / C::CH, kRows = kBK / kStep;
  const int64_t cstride = (int64_t)a.Hkv * D, hoff = (int64_t)hk * D;
  const int ch = tid % C::CH, r0 = tid / C::CH;
  auto copy = [&](uint32_t st, int i, const bf16* pk, const bf16* pv, bool real) {
    const uint32_t at = st + swz<D>(r0 + i * kStep, ch);
    cp16(at, pk, real);
    cp16(at + C::TILE, pv, real);
  };
  // Rows [row, row + 64) of the cache, of which the first n are real; 0 < n.
  auto load_run = [&](uint32_t st, int64_t row, int n) {
    const int64_t at = (row + r0) * cstride + hoff + ch * 8;
    const bf16 *pk = a.kc + at, *pv = a.vc + at;
    const int64_t step = kStep * cstride;
    if (n >= kBK) {
#pragma unroll
      for (int i = 0; i < kRows; ++i, pk += step, pv += step) copy(st, i, pk, pv, true);
    } else {
#pragma unroll 2
      for (int i = 0; i < kRows; ++i, pk += step, pv += step) {
        const bool real = r0 + i * kStep < n;
        copy(st, i, real ? pk : a.k, real ? pv : a.v, real);
      }
    }
  };
  auto load_tile = [&](int t) {
    const uint32_t st = sb + (uint32_t)(t - t0) % C::STAGES * C::STAGE;
    if constexpr (TREE) {
      if (t < k.own_tile) {
        load_run(st, k.base + (int64_t)t * kBK, k.n1 - t * kBK);
        return;
      }
      const int x0 = reinterpret_cast<const int*>(smem + C::OFF_TILES)[t - k.own_tile] * kBK;
#pragma unroll 2
      for (int i = 0; i < kRows; ++i) {
        const int x = x0 + r0 + i * kStep;
        const bool real = x < k.n_own;
        copy(st, i, real ? a.k + (k.own + x) * a.k_stride + hoff + ch * 8 : a.k,
             real ? a.v + (k.own + x) * a.v_stride + hoff + ch * 8 : a.v, real);
      }
    } else {
      const int x0 = t * kBK, cached = k.n1 + k.n2;
      if (x0 >= k.n1 && cached - x0 >= kBK) {
        load_run(st, k.base2 + (x0 - k.n1), kBK);
        return;
      }
      // A tile with first tokens, or with the new token at its end.
#pragma unroll 2
      for (int i = 0; i < kRows; ++i) {
        const int x = x0 + r0 + i * kStep;
        const bf16 *pk = a.k, *pv = a.v;
        if (x < cached) {
          const int64_t row = x < k.n1 ? k.base + x : k.base2 + (x - k.n1);
          pk = a.kc + row * cstride + hoff + ch * 8;
          pv = a.vc + row * cstride + hoff + ch * 8;
        } else if (x == cached) {
          pk = a.k + k.own * a.k_stride + hoff + ch * 8;
          pv = a.v + k.own * a.v_stride + hoff + ch * 8;
        }
        copy(st, i, pk, pv, x <= cached);
      }
    }
  };

  // Q through the last stage's memory into registers, behind it the first tiles.
  const uint32_t q_at = sb + (C::STAGES - 1) * C::STAGE;
  for (int i = tid; i < C::RB * C::CH; i += kThr) {
    const int r = i / C::CH, c = i % C::CH, g = rb * C::RB + r;
    const bool real = r < rows;
    const bf16* src = real ? a.q + (row0 + g / G) * a.q_stride + (int64_t)(hk * G + g % G) * D + c * 8
                           : a.q;
    cp16(q_at + swz<D>(r, c), src, real);
  }
  cp_commit();
#pragma unroll
  for (int i = 0; i < C::STAGES - 1; ++i) {
    if (t0 + i < t1) load_tile(t0 + i);
    cp_commit();
  }
  cp_wait<C::STAGES - 1>();
  __syncthreads();
  const int wr = warp / C::KW, wk = warp % C::KW;   // row group and key group of the warp
  uint32_t qf[D / 16][4];
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk)
    ldsm4(q_at + swz<D>(wr * 16 + (lane & 15), 2 * kk + (lane >> 4)), qf[kk]);

  float o[D / 8][4];
#pragma unroll
  for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  const int ra = wr * 16 + (lane >> 2);             // this thread's rows: ra and ra + 8

  for (int t = t0; t < t1; ++t) {
    cp_wait<C::STAGES - 2>();
    __syncthreads();
    if (t + C::STAGES - 1 < t1) load_tile(t + C::STAGES - 1);
    cp_commit();
    const uint32_t st = sb + (uint32_t)(t - t0) % C::STAGES * C::STAGE;
    // S = Q K^T of the warp's keys, 16 at a time.
    float s[C::KPW / 8][4];
#pragma unroll
    for (int n = 0; n < C::KPW / 8; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
    // Step by step along the head, so that consecutive products go to different sums.
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      uint32_t f[C::KPW / 16][4];
#pragma unroll
      for (int n = 0; n < C::KPW / 16; ++n) {
        const int key = wk * C::KPW + n * 16 + (lane & 7) + ((lane >> 4) << 3);
        ldsm4(st + swz<D>(key, 2 * kk + ((lane >> 3) & 1)), f[n]);
      }
#pragma unroll
      for (int n = 0; n < C::KPW / 16; ++n) {
        mma16816(s[2 * n], qf[kk], f[n][0], f[n][1]);
        mma16816(s[2 * n + 1], qf[kk], f[n][2], f[n][3]);
      }
    }
    // Keys behind the list, and drafted tokens off the path, drop out.
    int limit = kBK;                                // visible columns of a tile of cached keys
    bool own = false;
    if constexpr (TREE) {
      own = t >= k.own_tile;
      if (!own) limit = min(kBK, k.n1 - t * kBK);
    } else {
      limit = min(kBK, k.n1 + k.n2 + 1 - t * kBK);
    }
    if (own || limit < kBK) {
      const int col0 = wk * C::KPW + 2 * (lane & 3);   // columns col0 + 8 n + {0, 1}
      uint64_t seen[2];
      seen[0] = seen[1] = limit >= 64 ? ~0ull : (1ull << limit) - 1;
      if constexpr (TREE) {
        if (own) {
          const uint32_t* bits = reinterpret_cast<const uint32_t*>(smem + C::OFF_BITS);
          const int w = 2 * reinterpret_cast<const int*>(smem + C::OFF_TILES)[t - k.own_tile];
          const int tok0 = rb * C::RB / G;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = min(ra + 8 * h, rows - 1);
            const uint32_t* x = bits + ((rb * C::RB + r) / G - tok0) * kTreeWords + w;
            seen[h] = (uint64_t)x[0] | ((uint64_t)x[1] << 32);
          }
        }
      }
      seen[0] >>= col0;
      seen[1] >>= col0;
#pragma unroll
      for (int n = 0; n < C::KPW / 8; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (!((seen[j >> 1] >> (8 * n + (j & 1))) & 1)) s[n][j] = -INFINITY;
    }
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int n = 0; n < C::KPW / 8; ++n) {
      mx[0] = fmax3(mx[0], s[n][0], s[n][1]);
      mx[1] = fmax3(mx[1], s[n][2], s[n][3]);
    }
    float al[2], ref[2];
    bool grew = false;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
      // Log2 units (the scale is positive). The reference moves only when the maximum grows by
      // more than 2^8: the weights stay below 2^8, and O and l keep the same reference.
      const float top = fmaxf(m[h], mx[h] * a.scale_log2);
      const bool moves = top > m[h] + 8.0f;
      al[h] = moves ? (m[h] == -INFINITY ? 0.f : fast_exp2(m[h] - top)) : 1.f;
      m[h] = moves ? top : m[h];
      ref[h] = m[h] == -INFINITY ? 0.f : m[h];
      l[h] *= al[h];
      grew |= moves;
    }
    if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        o[n][0] *= al[0];
        o[n][1] *= al[0];
        o[n][2] *= al[1];
        o[n][3] *= al[1];
      }
    }
    // O += P V, P rounded to bf16 as the tensor instruction's operand; l sums it in fp32.
#pragma unroll
    for (int n = 0; n < C::KPW / 16; ++n) {
      uint32_t p[4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float* x = s[2 * n + j];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = fast_exp2(fmaf(x[i], a.scale_log2, -ref[i >> 1]));
        l[0] += x[0] + x[1];
        l[1] += x[2] + x[3];
        p[2 * j] = pack_bf16x2(x[0], x[1]);
        p[2 * j + 1] = pack_bf16x2(x[2], x[3]);
      }
      const int key = wk * C::KPW + n * 16 + (lane & 15);
#pragma unroll
      for (int d2 = 0; d2 < D / 16; ++d2) {
        uint32_t f[4];
        ldsm4t(st + C::TILE + swz<D>(key, 2 * d2 + (lane >> 4)), f);
        mma16816(o[2 * d2], p, f[0], f[1]);
        mma16816(o[2 * d2 + 1], p, f[2], f[3]);
      }
    }
  }
  cp_wait<0>();
  __syncthreads();

#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
  }
  // Row r of the block in the output.
  auto out_row = [&](int r) -> bf16* {
    const int g = rb * C::RB + r;
    return a.out + ((row0 + g / G) * a.H + (int64_t)hk * G + g % G) * D;
  };
  if (C::KW == 1 && a.split == 1) {
    // Nothing to join: each warp puts its 16 rows into shared memory as bf16 and writes them out.
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float inv = 1.f / l[h];
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
        *reinterpret_cast<uint32_t*>(smem + swz<D>(ra + 8 * h, n) + 4 * (lane & 3)) =
            pack_bf16x2(o[n][2 * h] * inv, o[n][2 * h + 1] * inv);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 16 * C::CH / 32; ++i) {
      const int r = wr * 16 + (lane + 32 * i) / C::CH, c = (lane + 32 * i) % C::CH;
      if (r < rows)
        *reinterpret_cast<uint4*>(out_row(r) + c * 8) =
            *reinterpret_cast<const uint4*>(smem + swz<D>(r, c));
    }
    return;
  }

  // Joining: every warp's (m, l, O) to shared memory, then the block's key groups, then the cluster.
  float* part = reinterpret_cast<float*>(smem);                       // [KW][RB][D]
  float* pm = reinterpret_cast<float*>(smem + C::OFF_ML);             // [KW][RB]
  float* pl = pm + C::KW * C::RB;
  float* jm = pl + C::KW * C::RB;                                     // [RB] of the block
  float* jl = jm + C::RB;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = ra + 8 * h;
    if ((lane & 3) == 0) {
      pm[wk * C::RB + r] = m[h];
      pl[wk * C::RB + r] = l[h];
    }
    float* x = part + (wk * C::RB + r) * D + 2 * (lane & 3);
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
      *reinterpret_cast<float2*>(x + 8 * n) = make_float2(o[n][2 * h], o[n][2 * h + 1]);
  }
  __syncthreads();
  if (tid < C::RB) {
    float mm = -INFINITY, ll = 0.f;
#pragma unroll
    for (int w = 0; w < C::KW; ++w) mm = fmaxf(mm, pm[w * C::RB + tid]);
#pragma unroll
    for (int w = 0; w < C::KW; ++w) {
      const float x = pm[w * C::RB + tid], f = x == -INFINITY ? 0.f : fast_exp2(x - mm);
      ll += pl[w * C::RB + tid] * f;
      pm[w * C::RB + tid] = f;
    }
    jm[tid] = mm;
    jl[tid] = skip ? -1.f : ll;   // a block that saw an error: nothing of the cluster is written
  }
  __syncthreads();
  if (C::KW > 1 && a.split > 1) {
    for (int i = tid; i < C::RB * D / 4; i += kThr) {
      const int r = i / (D / 4);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < C::KW; ++w) {
        const float f = pm[w * C::RB + r];
        const float4 y = reinterpret_cast<const float4*>(part)[w * C::RB * D / 4 + i];
        x.x = fmaf(f, y.x, x.x);
        x.y = fmaf(f, y.y, x.y);
        x.z = fmaf(f, y.z, x.z);
        x.w = fmaf(f, y.w, x.w);
      }
      reinterpret_cast<float4*>(part)[i] = x;
    }
  }
  const int n4 = rows * D / 4;
  auto store = [&](int i, float4 x) {
    *reinterpret_cast<uint2*>(out_row(i / (D / 4)) + i % (D / 4) * 4) =
        make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
  };
  if (a.split == 1) {
    for (int i = tid; i < n4; i += kThr) {
      const int r = i / (D / 4);
      const float inv = 1.f / jl[r];
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < C::KW; ++w) {
        const float f = pm[w * C::RB + r] * inv;
        const float4 y = reinterpret_cast<const float4*>(part)[w * C::RB * D / 4 + i];
        x.x = fmaf(f, y.x, x.x);
        x.y = fmaf(f, y.y, x.y);
        x.z = fmaf(f, y.z, x.z);
        x.w = fmaf(f, y.w, x.w);
      }
      store(i, x);
    }
    return;
  }
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  for (int i = rank * kThr + tid; i < n4; i += a.split * kThr) {
    const int r = i / (D / 4);
    float mm = -INFINITY, total = 0.f;
    bool whole = true;
    float w[kMaxSplit];
#pragma unroll
    for (int x = 0; x < kMaxSplit; ++x) {
      w[x] = x < a.split ? *cluster.map_shared_rank(jm + r, x) : -INFINITY;
      mm = fmaxf(mm, w[x]);
    }
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int x = 0; x < kMaxSplit; ++x) {
      if (x >= a.split) break;
      const float f = w[x] == -INFINITY ? 0.f : fast_exp2(w[x] - mm);
      const float lx = *cluster.map_shared_rank(jl + r, x);
      whole &= lx >= 0.f;
      total = fmaf(f, lx, total);
      const float4 y = reinterpret_cast<const float4*>(cluster.map_shared_rank(part, x))[i];
      acc.x = fmaf(f, y.x, acc.x);
      acc.y = fmaf(f, y.y, acc.y);
      acc.z = fmaf(f, y.z, acc.z);
      acc.w = fmaf(f, y.w, acc.w);
    }
    const float inv = 1.f / total;
    if (whole) store(i, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
  }
  cluster.sync();   // no block leaves while another still reads its shared memory
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

constexpr int kMaxDevices = 64;

// `keys`: no unit walks more. The key list is split while the blocks fit the device at two per SM and
// the longest list leaves each part a tile: with few units the longest list sets the time (4 users
// with trees: 14.3 us whole, 11.2 in two parts, 9.7 in eight; one token over 4,096 keys: 24.6 us in
// two parts, 10.9 in eight), with many the parts only cost (256 users with trees, longest first: 156
// to 158 us whole, every list in two parts 242, in four 377). Parts for the few longest lists alone have
// not been measured in this order; before users went by length, parts for lists of more than 16
// tiles took 290 us against 222.
template <int D, int RW, bool TREE, typename IdxT>
int launch_cache(CacheArgs a, int64_t max_rows, int64_t keys, int dev, int sms, cudaStream_t st) {
  using C = CCfg<D, RW, TREE>;
  a.row_blocks = (int)((max_rows + C::RB - 1) / C::RB);
  const int64_t units = a.B * a.Hkv * a.row_blocks;
  const int64_t tiles = (keys + kBK - 1) / kBK;
  a.split = 1;
  while (a.split < kMaxSplit && units * a.split <= sms && tiles >= 2 * a.split) a.split *= 2;
  if (units * a.split >= (int64_t)INT_MAX) return JCA_ERR_SHAPE;
  // Blocks that all fit the device at once start together, in whatever order.
  a.longest_first = TREE && a.B > 1 && units > C::BPS * (int64_t)sms;
  auto kernel = cache_attn_kernel<D, RW, TREE, IdxT>;
  static std::atomic<bool> set[kMaxDevices];
  if (!set[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) !=
        cudaSuccess)
      return JCA_ERR_CUDA;
    set[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * a.split));
  cfg.blockDim = dim3(kThr);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)a.split;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = a.split > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? JCA_OK : JCA_ERR_CUDA;
}

template <int D, bool TREE, typename IdxT>
int launch_rows(const CacheArgs& a, int64_t max_rows, int64_t keys, int dev, int sms,
                cudaStream_t st) {
  if (max_rows <= 16) return launch_cache<D, 1, TREE, IdxT>(a, max_rows, keys, dev, sms, st);
  if (max_rows <= 32) return launch_cache<D, 2, TREE, IdxT>(a, max_rows, keys, dev, sms, st);
  return launch_cache<D, 4, TREE, IdxT>(a, max_rows, keys, dev, sms, st);
}

template <bool TREE, typename IdxT>
int launch_heads(const CacheArgs& a, int d, int64_t max_rows, int64_t keys, int dev, int sms,
                 cudaStream_t st) {
  switch (d) {
    case 16: return launch_rows<16, TREE, IdxT>(a, max_rows, keys, dev, sms, st);
    case 32: return launch_rows<32, TREE, IdxT>(a, max_rows, keys, dev, sms, st);
    case 64: return launch_rows<64, TREE, IdxT>(a, max_rows, keys, dev, sms, st);
    default: return launch_rows<128, TREE, IdxT>(a, max_rows, keys, dev, sms, st);
  }
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
  a.scale_log2 = (scale > 0.f ? scale : 1.0f / sqrtf((float)d_head)) * 1.4426950408889634f;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int64_t span = window < R ? window : R, first = n_sinks < R ? n_sinks : R;
  const int64_t keys = span + first < R ? span + first : R;
  return idx_bits == 32
             ? launch_heads<false, int32_t>(a, d_head, H / Hkv, keys, dev, sms, st)
             : launch_heads<false, int64_t>(a, d_head, H / Hkv, keys, dev, sms, st);
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
  if (max_cand < 1 || max_cand > kMaxTree || (B == 0 && Nc > 0)) return JCA_ERR_SHAPE;
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
  a.scale_log2 = (scale > 0.f ? scale : 1.0f / sqrtf((float)d_head)) * 1.4426950408889634f;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int64_t max_rows = (int64_t)max_cand * (H / Hkv), keys = R + max_cand;
  return idx_bits == 32 ? launch_heads<true, int32_t>(a, d_head, max_rows, keys, dev, sms, st)
                        : launch_heads<true, int64_t>(a, d_head, max_rows, keys, dev, sms, st);
}
