// Backward pass of the causal attention with a sliding window and visible first tokens (window.cu;
// include/jca.h states the mask and the layout).
//
// Mathematics, with P rebuilt tile by tile from the forward's log-sum-exp:
//   dV = P^T dO,   dS = P * (dO V^T - D),  D = rowsum(dO * O),   dQ = scale dS K,   dK = scale dS^T Q,
// dK and dV of a key head summed over its query heads. Three disjoint parts, no atomics:
//   * dQ: a 128-row query tile of one head walks the key tiles that the forward walks;
//   * dKV: a 128-row key tile of one key head walks the query tiles that see it through the window
//     (rows j <= i < min(j + window, end)) for each of its query heads;
//   * first tokens are also seen from behind their window, by every later row of the user: a unit
//     takes a user's first tokens as its key tile and walks up to kChunk of those rows, leaving an
//     fp32 partial sum. The dKV unit leaves the window's sum of such a key in fp32 too, and a last
//     kernel adds them in order and rounds. Without this split one key tile would walk a whole
//     long history for its few first tokens.
// Row tiles are cut from the packed rows whatever users they hold, as in the forward.
//
// Kernel (one persistent block per SM, 16 warps; tcgen05 with TMEM accumulators, TMA loads). O1/O2 are
// the unit's outer tiles, I1/I2 the inner tiles streamed through a ring:
//   S = O1 I1^T,  dP = O2 I2^T  (SS MMAs)   ->   dS (and P) as bf16 in TMEM   ->   TS MMAs
//   dQ  (O1 = Q, O2 = dO, I1 = K, I2 = V):   acc0 += dS I1
//   dKV (O1 = K, O2 = V, I1 = Q, I2 = dO):   acc0 (dV) += P^T I2,  acc1 (dK) += dS^T I1
// The blocks of the three parts share one launch.
// A step takes 64 inner rows, so that S and dP fit two or three times beside the accumulators in TMEM
// and the tensor core works ahead of the compute warps. Columns a warp's rows do not see are
// decided per 32 columns: none (zeros are written), all (no masking) or some.
//   warp 0      lane 0: TMA loads, lane 1: claims units and posts them to a ring;
//   warps 1, 2  one thread each issues the SS and the TS MMAs;
//   warp 3      with padding: zeroes the padding rows of the inner tiles;
//   warps 4..11 compute, a row a thread, two warps per 32 rows (32 of the 64 columns each);
//   warps 12..15 write a unit's accumulators out while the others are at the next unit.
//
// What bounds it (256 users, window 256, d = 128, in a short run: dKV 437 us, dQ 373, first tokens 118,
// 1.02 ms with the statistics before and the joining behind, 0.34 of the copy bandwidth; 1.10 to 1.22 ms
// under the power limit of a long run, 0.31 to 0.28): the tensor core's part of the chain
// S, dP -> dS -> products. Seven products are formed per pair instead of five (S and dP in both
// passes), and those of 64 columns take nearly as long as those of 128 (about 60 cycles for 16 of
// the head) but leave room for three score buffers, which overlap the exponentials and conversions
// (256 users 1.10 ms in steps of 128 columns, 1.04 ms in steps of 64, short runs). For first tokens a 128-row
// tile holds n_sinks keys.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "jca_device.cuh"
#include "jca_internal.h"
#include "window.h"

namespace jca {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kDQ = 0, kDKV = 1, kSink = 2;   // kSink: dKV of first tokens from behind the window
constexpr int kThreads = 512;
constexpr int kCompute = 256;
constexpr int kEpilogue = 128;
// Registers a thread: 512 x 128 at launch, shared out anew (72 + 2 x 168 + 104 = 4 x 128).
constexpr int kRegsRoles = 72, kRegsCompute = 168, kRegsEpilogue = 104;
constexpr int kStep = 64;        // inner rows of a step
// Query rows of a kSink unit: 256 rows keep the longest unit short (16 users: 14 us alone, with 1024
// rows 36 us; on 256 users 1024 rows took 7 % more).
constexpr int kChunk = 256;
// A unit's accumulators are taken over into fp32 sums in memory after so many steps. The tensor core
// cuts each addition off, which costs a sum about 2^-25 of itself for every 16 products (a key seen by
// 4,096 rows of 8,192 heads lost 3 % of dV); within 4,096 steps of four additions that is 2^-11.
constexpr int kSpill = 4096;
constexpr int kRing = 4;
constexpr int kEntry = 6;        // ints of a ring entry

struct BwdArgs {
  bf16* dq;
  bf16* dk;
  bf16* dv;
  const uint8_t* valid;       // [T] or null
  const int32_t* row_start;   // [T]
  const int32_t* row_end;     // [T]
  const int32_t* row_number;  // [T], for first tokens of users longer than the window: the user's
                              // place in sink_users
  const float* lse2;          // [H][T] log2 units; +inf: the row sees no key
  const float* dsum;          // [H][T] D
  float* part;                // partials of first tokens [slot][Hkv][n_sinks][2][D]: dV, dK / scale
  int window_slot;            // slot of the window's own sums: this + the user's place in sink_users
  const int4* sinks;          // kSink units {first row, end, chunk, slot}
  const int4* sink_users;     // their users {first row, end, slot of the first unit, 0}
  float* spill;               // [block][128][2][D], where a unit has more than kSpill steps
  const int32_t* n_sink_units;
  const int32_t* n_sink_users;
  int32_t* counter;           // [3] next unit of each part
  int32_t* status;
  // Limit of the wait for room in the ring, which is one for a whole unit: the other waits are for
  // kSpill steps at most, and an abort there ends this one too. 10 us a step of the longest unit; a
  // step takes 0.8 to 1.
  uint64_t unit_ns;
  int T, H, Hkv, group, window, n_sinks;
  int units_dq, units_dkv;
  int blocks_sink, blocks_dkv;   // the launch's blocks in this order, those of kDQ last
  int v8;                     // gradients can be written with 32-byte stores
  float scale, scale_log2;
};

template <int D, int MODE>
struct Cfg {
  static constexpr int BM = kTileM;
  static constexpr int ROW_BYTES = D * 2;
  static constexpr int SW = ROW_BYTES >= 128 ? 128 : ROW_BYTES;
  static constexpr int NBLK = ROW_BYTES / SW;
  static constexpr int BOX_X = SW / 2;
  static constexpr int TILE_BYTES = BM * ROW_BYTES;
  static constexpr int BLK_BYTES = BM * SW;
  static constexpr uint32_t LAYOUT = SW == 128 ? 2u : (SW == 64 ? 4u : 6u);
  static constexpr int KSTEPS_QK = D / 16;
  static constexpr int KSTEPS_PER_BLK = SW / 32;
  static constexpr int IN_BLK = kStep * SW;                           // column block of an inner tile
  static constexpr int IN_TILE = kStep * ROW_BYTES;
  static constexpr int IN_STAGE = 2 * IN_TILE;                        // I1, I2
  static constexpr int STAGES = D == 128 ? 3 : 6;
  // S and dP buffers, 128 columns each: what the accumulators leave of the 512 columns.
  static constexpr int BUFS = (MODE == kDQ || D <= 64) ? 3 : 2;
  static constexpr int OFF_OUT = 0;                                   // [2] O1, O2
  static constexpr int OFF_IN = 4 * TILE_BYTES;
  static constexpr int OFF_BAR = OFF_IN + STAGES * IN_STAGE;
  static constexpr int B_OUTFULL = 0;                                 // [2]
  static constexpr int B_OUTEMPTY = 2;                                // [2]
  static constexpr int B_INFULL = 4;                                  // [STAGES]
  static constexpr int B_INREADY = B_INFULL + STAGES;                 // padding rows zeroed
  static constexpr int B_INEMPTY = B_INREADY + STAGES;
  static constexpr int B_SPFULL = B_INEMPTY + STAGES;                 // [BUFS] S and dP written
  static constexpr int B_DSFULL = B_SPFULL + BUFS;                    // [BUFS] dS (and P) written
  static constexpr int B_BUFFREE = B_DSFULL + BUFS;                   // [BUFS] read by TS
  static constexpr int B_ACCFULL = B_BUFFREE + BUFS;
  static constexpr int B_ACCFREE = B_ACCFULL + 1;
  static constexpr int B_COLS = B_ACCFREE + 1;                        // [2] column statistics
  static constexpr int B_DRAIN = B_COLS + 2;                          // [2] MMA threads
  static constexpr int B_RINGFULL = B_DRAIN + 2;
  static constexpr int B_RINGEMPTY = B_RINGFULL + kRing;
  static constexpr int NUM_BARS = B_RINGEMPTY + kRing;
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
  static constexpr int OFF_RING = OFF_MISC + 16;
  static constexpr int OFF_COLS = (OFF_RING + kRing * kEntry * 4 + 15) / 16 * 16;   // [2][2][64]
  static constexpr int SMEM_USED = OFF_COLS + 2 * 2 * kStep * 4;
  static constexpr int SMEM_RAW = SMEM_USED + 1024;
  // At least 120 KB so that a second block never shares the SM (and its TMEM).
  static constexpr int SMEM_ALLOC = SMEM_RAW > 120 * 1024 ? SMEM_RAW : 120 * 1024;
  static constexpr uint32_t TMEM_S = 0, TMEM_P = 64, TMEM_BUF = 128, TMEM_A0 = BUFS * 128,
                            TMEM_A1 = TMEM_A0 + (D < 64 ? 64 : D), TMEM_COLS = 512;
  static_assert(TMEM_A0 + (MODE == kDQ ? 1 : 2) * D <= TMEM_COLS, "TMEM budget");
  static_assert(SMEM_ALLOC <= 227 * 1024, "shared memory budget");
};

// A unit as every role derives it from a ring entry: its outer tile, and the rows that its inner steps
// walk, up to 64 at a time.
struct Unit {
  int orow0, oh;                // outer rows and head (dQ: query head, else key head)
  int n_in;                     // steps
  int base, end, n_run;         // rows [base, end) in n_run steps (dKV, kSink: once per query head)
  int sink0, n_sink, n_first;   // dQ: rows of the first tokens, which come first, in n_first steps
  int slot, uend;               // kSink: partial sum's slot, end of the user
};

template <int MODE>
__device__ __forceinline__ Unit make_unit(const volatile int* e, const BwdArgs& a) {
  Unit u;
  u.orow0 = e[0];
  u.oh = e[1];
  u.sink0 = u.n_sink = u.n_first = u.slot = u.uend = 0;
  if (MODE == kDQ) {
    const int lo = e[2], start = e[3];
    u.base = lo & ~(kStep - 1);
    u.end = min(u.orow0 + kTileM, a.T);
    u.sink0 = start;
    u.n_sink = max(0, min(a.n_sinks, u.base - start));
    u.n_first = (u.n_sink + kStep - 1) / kStep;
    u.n_run = (u.end - u.base + kStep - 1) / kStep;
    u.n_in = u.n_first + u.n_run;
  } else {
    u.base = e[2];
    u.end = e[3];
    u.n_run = (u.end - u.base + kStep - 1) / kStep;
    u.n_in = u.n_run * a.group;
    u.slot = e[4];
    u.uend = e[5];
  }
  return u;
}

// A unit's steps in order: rows [row, row + valid) of head `head`.
template <int MODE>
struct Walk {
  int i, t, row, valid, head;
  __device__ __forceinline__ void place(const Unit& u) {
    if (MODE == kDQ && i < u.n_first) {
      row = u.sink0 + i * kStep;
      valid = min(kStep, u.n_sink - i * kStep);
    } else {
      row = u.base + t * kStep;
      valid = min(kStep, u.end - row);
    }
  }
  __device__ __forceinline__ void begin(const Unit& u, const BwdArgs& a) {
    i = t = 0;
    head = MODE == kDQ ? u.oh / a.group : u.oh * a.group;
    place(u);
  }
  // The next step; false behind the last.
  __device__ __forceinline__ bool next(const Unit& u) {
    if (MODE != kDQ || i >= u.n_first) ++t;
    ++i;
    if (MODE != kDQ && t == u.n_run) {
      t = 0;
      ++head;
    }
    place(u);
    return i < u.n_in;
  }
};

template <int MODE>
__device__ __forceinline__ bool ring_take(Ring& r, const BwdArgs& a, Unit& u,
                                          volatile int* abort_flag, bool& ok) {
  const int s = (int)(r.k % kRing);
  ok = mbar_wait(r.full + 8 * s, (r.k / kRing) & 1, abort_flag, a.status);
  if (!ok) return false;
  const volatile int* e = r.slot + kEntry * s;
  const bool more = e[0] >= 0;
  if (more) u = make_unit<MODE>(e, a);
  mbar_arrive(r.empty + 8 * s);
  ++r.k;
  return more;
}

template <int MODE>
__device__ void claim_role(const BwdArgs& a, Ring r, volatile int* abort_flag) {
  const int heads = MODE == kDQ ? a.H : a.Hkv;
  const int n = MODE == kSink  ? *a.n_sink_units * heads
                : MODE == kDQ ? a.units_dq
                              : a.units_dkv;
  for (;;) {
    const int v = atomicAdd(a.counter + MODE, 1);
    int e[kEntry] = {-1, 0, 0, 0, 0, 0};
    if (v < n) {
      e[1] = v % heads;
      if (MODE == kSink) {
        const int4 x = a.sinks[v / heads];   // {first row, end, chunk, slot}
        e[0] = x.x;
        e[2] = max(x.x + a.window, x.z * kChunk) & ~(kStep - 1);
        e[3] = (int)min((long long)x.y, (long long)(x.z + 1) * kChunk);
        e[4] = x.w;
        e[5] = x.y;
      } else {
        // Under a long window the later query tiles and the earlier key tiles are the longer units.
        const int t = MODE == kDQ ? (n - 1 - v) / heads : v / heads;
        e[0] = t * kTileM;
        if (MODE == kDQ) {
          e[3] = a.row_start[e[0]];
          e[2] = max(e[3], e[0] - a.window + 1);
        } else {
          const int last = min(e[0] + kTileM, a.T) - 1;
          e[2] = e[0];
          e[3] = (int)min((long long)a.row_end[last], (long long)last + a.window);
        }
      }
    }
    const int s = (int)(r.k % kRing);
    if (!mbar_wait(r.empty + 8 * s, ((r.k / kRing) & 1) ^ 1, abort_flag, a.status, a.unit_ns)) return;
#pragma unroll
    for (int i = 0; i < kEntry; ++i) r.slot[kEntry * s + i] = e[i];
    mbar_arrive(r.full + 8 * s);
    ++r.k;
    if (e[0] < 0) return;
  }
}

template <int D, int MODE>
__device__ void producer_role(const CUtensorMap* tmO1, const CUtensorMap* tmO2,
                              const CUtensorMap* tmI1, const CUtensorMap* tmI2, const BwdArgs& a,
                              uint32_t sbase, uint32_t bars, volatile int* abort_flag, Ring ring) {
  using C = Cfg<D, MODE>;
  uint32_t units = 0, g = 0;
  bool ok = true;
  Unit u;
  Walk<MODE> w;
  while (ok && ring_take<MODE>(ring, a, u, abort_flag, ok)) {
    // The outer tiles have two slots, so a unit's arrive while the one before is worked on.
    const int slot = (int)(units & 1);
    ok = mbar_wait(bars + 8 * (C::B_OUTEMPTY + slot), ((units >> 1) & 1) ^ 1, abort_flag, a.status);
    if (!ok) break;
    const uint32_t obar = bars + 8 * (C::B_OUTFULL + slot);
    mbar_arrive_expect_tx(obar, 2 * C::TILE_BYTES);
    ++units;
    const uint32_t out = sbase + C::OFF_OUT + slot * 2 * C::TILE_BYTES;
#pragma unroll
    for (int c = 0; c < C::NBLK; ++c)
#pragma unroll
      for (int x = 0; x < kTileM / kStep; ++x) {
        const uint32_t at = out + c * C::BLK_BYTES + x * C::IN_BLK;
        tma_load_3d(at, tmO1, obar, c * C::BOX_X, u.oh, u.orow0 + x * kStep);
        tma_load_3d(at + C::TILE_BYTES, tmO2, obar, c * C::BOX_X, u.oh, u.orow0 + x * kStep);
      }
    w.begin(u, a);
    for (bool more = true; more; more = w.next(u)) {
      const int s = (int)(g % C::STAGES);
      ok = mbar_wait(bars + 8 * (C::B_INEMPTY + s), ((g / C::STAGES) & 1) ^ 1, abort_flag, a.status);
      if (!ok) break;
      const uint32_t ibar = bars + 8 * (C::B_INFULL + s);
      mbar_arrive_expect_tx(ibar, C::IN_STAGE);
      const uint32_t dst = sbase + C::OFF_IN + s * C::IN_STAGE;
#pragma unroll
      for (int c = 0; c < C::NBLK; ++c) {
        tma_load_3d(dst + c * C::IN_BLK, tmI1, ibar, c * C::BOX_X, w.head, w.row);
        tma_load_3d(dst + C::IN_TILE + c * C::IN_BLK, tmI2, ibar, c * C::BOX_X, w.head, w.row);
      }
      ++g;
    }
  }
  if (!ok) {
    // Aborting: let the copies this thread started land before the block exits.
    for (uint32_t n = units > 2 ? units - 2 : 0; n < units; ++n)
      mbar_wait_drain(bars + 8 * (C::B_OUTFULL + (int)(n & 1)), (n >> 1) & 1);
    for (uint32_t n = g > (uint32_t)C::STAGES ? g - C::STAGES : 0; n < g; ++n)
      mbar_wait_drain(bars + 8 * (C::B_INFULL + (int)(n % C::STAGES)), (n / C::STAGES) & 1);
  }
}

// Zeroes the rows of padding in both inner tiles; one warp.
template <int D, int MODE>
__device__ void padding_role(const BwdArgs& a, uint32_t sbase, uint32_t bars,
                             volatile int* abort_flag, int lane, Ring ring) {
  using C = Cfg<D, MODE>;
  uint32_t g = 0;
  bool ok = true;
  Unit u;
  Walk<MODE> w;
  for (;;) {
    const bool taken = ring_take<MODE>(ring, a, u, abort_flag, ok);
    if (!__all_sync(0xffffffffu, taken)) return;
    w.begin(u, a);
    for (bool more = true; more; more = w.next(u), ++g) {
      const int s = (int)(g % C::STAGES);
      uint32_t pad[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int k = w.row + 32 * c + lane;
        pad[c] = __ballot_sync(0xffffffffu, k < a.T && !a.valid[k]);
      }
      ok = mbar_wait_long(bars + 8 * (C::B_INFULL + s), (g / C::STAGES) & 1, abort_flag, a.status);
      if (!__all_sync(0xffffffffu, ok)) return;
      const uint32_t tile = sbase + C::OFF_IN + s * C::IN_STAGE;
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (pad[c]) zero_rows<C::ROW_BYTES, C::SW, C::IN_BLK, C::IN_TILE>(tile, 32 * c, pad[c], lane);
      fence_proxy_async_smem();
      mbar_arrive(bars + 8 * (C::B_INREADY + s));
    }
  }
}

// The S and dP products of every step, one thread. A buffer is formed anew once the TS products that
// read it last are done.
template <int D, int MODE>
__device__ void ss_role(const BwdArgs& a, uint32_t sbase, uint32_t bars, uint32_t tmem,
                        volatile int* abort_flag, Ring ring) {
  using C = Cfg<D, MODE>;
  constexpr uint32_t kIdescSS = idesc_bf16_f32(C::BM, kStep, false, false);
  constexpr uint32_t kIdesc0 = kIdescSS & ~(0x3Fu << 17);
  const int infull = a.valid ? C::B_INREADY : C::B_INFULL;
  const uint64_t out = smem_desc(sbase + C::OFF_OUT, 16, 8 * C::SW, C::LAYOUT);
  const uint64_t in = smem_desc(sbase + C::OFF_IN, 16, 8 * C::SW, C::LAYOUT);
  uint32_t units = 0, g = 0;
  bool ok = true;
  Unit u;
  Walk<MODE> w;
  while (ok && ring_take<MODE>(ring, a, u, abort_flag, ok)) {
    const int slot = (int)(units & 1);
    ok = mbar_wait_long(bars + 8 * (C::B_OUTFULL + slot), (units >> 1) & 1, abort_flag, a.status);
    if (!ok) break;
    ++units;
    const uint64_t o1 = out + (uint64_t)((slot * 2 * C::TILE_BYTES) >> 4);
    w.begin(u, a);
    for (bool more = true; more; ++g) {
      const int s = (int)(g % C::STAGES), b = (int)(g % C::BUFS);
      ok = mbar_wait_long(bars + 8 * (infull + s), (g / C::STAGES) & 1, abort_flag, a.status);
      if (ok && g >= (uint32_t)C::BUFS)
        ok = mbar_wait_long(bars + 8 * (C::B_BUFFREE + b), (g / C::BUFS - 1) & 1, abort_flag,
                            a.status);
      if (!ok) break;
      tc_fence_after();
      const uint32_t idesc = kIdesc0 | ((uint32_t)(((w.valid + 15) & ~15) >> 3) << 17);
      const uint64_t i1 = in + (uint64_t)((s * C::IN_STAGE) >> 4);
      const uint32_t buf = tmem + b * C::TMEM_BUF;
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int kk = 0; kk < C::KSTEPS_QK; ++kk) {
          constexpr int PB = C::KSTEPS_PER_BLK;
          const uint32_t k32 = (kk % PB) * 32;
          tc_mma(buf + (x ? C::TMEM_P : C::TMEM_S),
                 o1 + (uint32_t)((x * C::TILE_BYTES + kk / PB * C::BLK_BYTES + k32) >> 4),
                 i1 + (uint32_t)((x * C::IN_TILE + kk / PB * C::IN_BLK + k32) >> 4), idesc,
                 kk > 0 ? 1u : 0u);
        }
      tc_commit(bars + 8 * (C::B_SPFULL + b));
      more = w.next(u);
      if (!more) tc_commit(bars + 8 * (C::B_OUTEMPTY + slot));
    }
  }
  if (!ok) {
    // Aborting: wait until every MMA this thread issued has completed.
    tc_commit(bars + 8 * C::B_DRAIN);
    mbar_wait_drain(bars + 8 * C::B_DRAIN, 0);
  }
}

// The TS products, which add to the unit's accumulators; another thread, so that neither its waits
// for the compute warps nor its issue hold up the next S and dP (one thread for both: 2,400 cycles
// a step at d = 128, of which the tensor core needs about 1,250).
template <int D, int MODE>
__device__ void ts_role(const BwdArgs& a, uint32_t sbase, uint32_t bars, uint32_t tmem,
                        volatile int* abort_flag, Ring ring) {
  using C = Cfg<D, MODE>;
  constexpr uint32_t kIdescTS = idesc_bf16_f32(C::BM, D, false, true);
  constexpr uint32_t kRows16 = (16 * C::SW) >> 4;
  const int infull = a.valid ? C::B_INREADY : C::B_INFULL;
  const uint64_t in = smem_desc(sbase + C::OFF_IN, C::IN_BLK, 8 * C::SW, C::LAYOUT);
  uint32_t g = 0, sums = 0;
  bool ok = true;
  Unit u;
  Walk<MODE> w;
  // The pairs of a step sit in two 16-column runs, one per compute warp of a lane quarter.
  auto ts = [&](uint32_t acc, uint32_t p, uint64_t y, int ksteps, bool overwrite) {
#pragma unroll
    for (int kk = 0; kk < kStep / 16; ++kk)
      if (kk < ksteps)
        tc_mma_ts(acc, p + (uint32_t)(kk >> 1) * 32u + (uint32_t)(kk & 1) * 8u,
                  y + (uint64_t)(kk * kRows16), kIdescTS, (overwrite && kk == 0) ? 0u : 1u);
  };
  while (ok && ring_take<MODE>(ring, a, u, abort_flag, ok)) {
    w.begin(u, a);
    for (bool more = true; more; ++g, more = w.next(u)) {
      const int s = (int)(g % C::STAGES), b = (int)(g % C::BUFS);
      const bool first = w.i % kSpill == 0;   // of the accumulators' sums
      if (first && w.i > 0) {
        tc_commit(bars + 8 * C::B_ACCFULL);
        ++sums;
      }
      // The tile has landed (S was formed from it); this thread sees that for itself.
      ok = mbar_wait_long(bars + 8 * (infull + s), (g / C::STAGES) & 1, abort_flag, a.status);
      if (ok && first && sums > 0)
        ok = mbar_wait_long(bars + 8 * C::B_ACCFREE, (sums - 1) & 1, abort_flag, a.status);
      if (ok)
        ok = mbar_wait_long(bars + 8 * (C::B_DSFULL + b), (g / C::BUFS) & 1, abort_flag, a.status);
      if (!ok) break;
      tc_fence_after();
      const int ksteps = (w.valid + 15) >> 4;
      const uint32_t buf = tmem + b * C::TMEM_BUF;
      const uint64_t i1 = in + (uint64_t)((s * C::IN_STAGE) >> 4);
      if (MODE == kDQ) {
        ts(tmem + C::TMEM_A0, buf + C::TMEM_P, i1, ksteps, first);
      } else {
        ts(tmem + C::TMEM_A0, buf + C::TMEM_S, i1 + (uint64_t)(C::IN_TILE >> 4), ksteps, first);
        ts(tmem + C::TMEM_A1, buf + C::TMEM_P, i1, ksteps, first);
      }
      tc_commit(bars + 8 * (C::B_BUFFREE + b));
      tc_commit(bars + 8 * (C::B_INEMPTY + s));
    }
    if (!ok) break;
    tc_commit(bars + 8 * C::B_ACCFULL);
    ++sums;
  }
  if (!ok) {
    tc_commit(bars + 8 * (C::B_DRAIN + 1));
    mbar_wait_drain(bars + 8 * (C::B_DRAIN + 1), 0);
  }
}

template <int D, int MODE>
__device__ void compute_role(const BwdArgs& a, uint32_t bars, uint32_t tmem, float* cols,
                             volatile int* abort_flag, int warp, int lane, Ring ring) {
  using C = Cfg<D, MODE>;
  const int quarter = warp & 3;
  const int ch = (warp - 4) >> 2;               // 32-column half of every step
  const int tid = (warp - 4) * 32 + lane;
  const int r = quarter * 32 + lane;            // outer row of this thread inside its tile
  const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
  const uint32_t t_s = t_lane + C::TMEM_S + 32 * ch, t_p = t_lane + C::TMEM_P + 32 * ch;
  const float2 sl2v = make_float2(a.scale_log2, a.scale_log2);
  const size_t T = (size_t)a.T;
  uint32_t g = 0;                               // steps so far
  bool ok = true;
  Unit u;
  Walk<MODE> w;
  for (;;) {
    const bool more = ring_take<MODE>(ring, a, u, abort_flag, ok);
    if (!__all_sync(0xffffffffu, more)) break;
    const int row = u.orow0 + r;                // this thread's row
    const bool row_ok = row < a.T;
    const bool real = row_ok && (!a.valid || a.valid[row]);
    const int start = row_ok ? a.row_start[row] : 0;
    // Inner rows the outer row pairs with: [lo, hi), and for dQ the first tokens [start, first).
    int lo = 0, hi = 0, first = start;
    if (real) {
      if (MODE == kDQ) {
        lo = max(start, row - a.window + 1);
        hi = row + 1;
        first = min(start + a.n_sinks, lo);
      } else if (MODE == kDKV) {
        lo = row;
        hi = (int)min((long long)a.row_end[row], (long long)row + a.window);
      } else if (row < min(u.orow0 + a.n_sinks, u.uend)) {
        hi = u.uend;
        lo = (int)min((long long)hi, (long long)row + a.window);
      }
    }
    // dQ: this row's statistics.
    const size_t own = (size_t)u.oh * T + (size_t)row;
    const float lse2 = (MODE == kDQ && row_ok) ? a.lse2[own] : INFINITY;
    const float dsum = (MODE == kDQ && row_ok) ? a.dsum[own] : 0.f;
    const float2 nlv = make_float2(-lse2, -lse2), ndv = make_float2(-dsum, -dsum);
    // dKV: column statistics of a step's query rows, negated in shared memory (-lse2 of the 64 rows,
    // then -D), one value from each of 128 threads; the next step's are fetched while this one is
    // computed.
    auto col_stat = [&](const Walk<MODE>& x) -> float {
      const int q = x.row + (tid & 63);
      if (tid >= 2 * kStep || q >= a.T) return tid < kStep ? -INFINITY : 0.f;
      const size_t at = (size_t)x.head * T + (size_t)q;
      return tid < kStep ? -a.lse2[at] : -a.dsum[at];
    };
    w.begin(u, a);
    float stat = MODE != kDQ ? col_stat(w) : 0.f;
    for (bool more = true; more; ++g) {
      const int b = (int)(g % C::BUFS), c0 = w.row + 32 * ch;
      const int cvalid = w.valid - 32 * ch;     // of this warp's columns
      const float* cl = cols + (g & 1) * 2 * kStep;
      more = w.next(u);
      if (MODE != kDQ) {
        if (tid < 2 * kStep) cols[(g & 1) * 2 * kStep + tid] = stat;
        mbar_arrive(bars + 8 * (C::B_COLS + (int)(g & 1)));
        if (more) stat = col_stat(w);
        ok = __all_sync(0xffffffffu, mbar_wait_long(bars + 8 * (C::B_COLS + (int)(g & 1)),
                                                    (g >> 1) & 1, abort_flag, a.status));
        if (!ok) break;
      }
      {
        // Which of the warp's 32 columns each row pairs with.
        uint32_t bits = range_bits(lo - c0, hi - c0);
        if (MODE == kDQ) bits |= range_bits(start - c0, first - c0);
        if (cvalid < 32) bits &= range_bits(0, cvalid);
        if (a.valid) {
          const int k = c0 + lane;
          bits &= __ballot_sync(0xffffffffu, k < a.T && a.valid[k]);
        }
        const bool any = __any_sync(0xffffffffu, bits != 0u);
        const bool all = __all_sync(0xffffffffu, bits == 0xffffffffu);
        ok = __all_sync(0xffffffffu, mbar_wait_long(bars + 8 * (C::B_SPFULL + b), (g / C::BUFS) & 1,
                                                    abort_flag, a.status));
        if (!ok) break;
        tc_fence_after();
        const uint32_t buf = b * C::TMEM_BUF;
        // The bf16 pairs go to the first 16 columns of the warp's own chunk of S (P) and dP (dS).
        uint32_t pk_ds[16], pk_p[16];
        if (any) {
          uint32_t sv[32], dp[32];
          tmem_ld_x32(t_s + buf, sv);
          tmem_ld_x32(t_p + buf, dp);
          tmem_wait_ld();
          reg_fence16(sv);
          reg_fence16(sv + 16);
          reg_fence16(dp);
          reg_fence16(dp + 16);
          if (!all) {
            // Off the mask P = 0, and dP (from padding it may not be finite) counts as 0.
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              sv[j] = ((bits >> j) & 1u) ? sv[j] : 0xff800000u;
              dp[j] = ((bits >> j) & 1u) ? dp[j] : 0u;
            }
          }
          const float* cln = cl + 32 * ch;
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            float2 nl = nlv, nd = ndv;
            if (MODE != kDQ) {
              nl = *reinterpret_cast<const float2*>(cln + j);
              nd = *reinterpret_cast<const float2*>(cln + kStep + j);
            }
            const float2 x = __ffma2_rn(make_float2(__uint_as_float(sv[j]),
                                                    __uint_as_float(sv[j + 1])), sl2v, nl);
            const float2 pp = make_float2(fast_exp2(x.x), fast_exp2(x.y));
            const float2 dd = __fadd2_rn(make_float2(__uint_as_float(dp[j]),
                                                     __uint_as_float(dp[j + 1])), nd);
            const float2 ds = __fmul2_rn(pp, dd);
            // bf16: the operand type of the gradient products.
            pk_ds[j / 2] = pack_bf16x2(ds.x, ds.y);
            if (MODE != kDQ) pk_p[j / 2] = pack_bf16x2(pp.x, pp.y);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) pk_ds[j] = pk_p[j] = 0u;
        }
        tmem_st_x16(t_p + buf, pk_ds);
        if (MODE != kDQ) tmem_st_x16(t_s + buf, pk_p);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bars + 8 * (C::B_DSFULL + b));
      }
    }
    if (!ok) break;
  }
}

// 16 fp32 values in memory: written, and added to.
__device__ __forceinline__ void put16(float* to, const uint32_t* x) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
    reinterpret_cast<uint4*>(to)[k] = make_uint4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
}
__device__ __forceinline__ void add16(uint32_t* x, const float* from) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float4 y = reinterpret_cast<const float4*>(from)[k];
    x[4 * k] = __float_as_uint(__uint_as_float(x[4 * k]) + y.x);
    x[4 * k + 1] = __float_as_uint(__uint_as_float(x[4 * k + 1]) + y.y);
    x[4 * k + 2] = __float_as_uint(__uint_as_float(x[4 * k + 2]) + y.z);
    x[4 * k + 3] = __float_as_uint(__uint_as_float(x[4 * k + 3]) + y.w);
  }
}

// Writes a unit's accumulators out, a row a thread, while the compute warps are at the next unit. Of a
// unit of more than kSpill steps they come several times; a thread adds its row up in its own place.
template <int D, int MODE>
__device__ void epilogue_role(const BwdArgs& a, uint32_t bars, uint32_t tmem,
                              volatile int* abort_flag, int warp, int lane, Ring ring) {
  using C = Cfg<D, MODE>;
  constexpr int CW = 16;
  const int r = (warp & 3) * 32 + lane;
  const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
  const uint32_t t_a0 = t_lane + C::TMEM_A0, t_a1 = t_lane + C::TMEM_A1;
  float* spill = a.spill + ((size_t)blockIdx.x * kTileM + r) * 2 * D;
  uint32_t seen = 0;
  bool ok = true;
  Unit u;
  auto put = [&](bf16* dst, const uint32_t* x, float f) {
    uint32_t p[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      p[k] = pack_bf16x2(__uint_as_float(x[2 * k]) * f, __uint_as_float(x[2 * k + 1]) * f);
    if (a.v8) {
      st_global_v8(dst, p);
    } else {
      reinterpret_cast<uint4*>(dst)[0] = make_uint4(p[0], p[1], p[2], p[3]);
      reinterpret_cast<uint4*>(dst)[1] = make_uint4(p[4], p[5], p[6], p[7]);
    }
  };
  for (;;) {
    const bool more = ring_take<MODE>(ring, a, u, abort_flag, ok);
    if (!__all_sync(0xffffffffu, more)) break;
    const int row = u.orow0 + r;
    const bool row_ok = row < a.T;
    // Sums of first tokens that rows behind the window see too stay in fp32 partials.
    float* mine = nullptr;
    bool writes = row_ok;
    if (MODE == kSink) {
      writes = r < a.n_sinks;
      mine = a.part + (((size_t)u.slot * a.Hkv + u.oh) * a.n_sinks + r) * 2 * D;
    } else if (MODE == kDKV && a.part && row_ok) {
      const int start = a.row_start[row];
      if (row - start < a.n_sinks && a.row_end[row] - start > a.window) {
        const size_t slot = (size_t)a.window_slot + a.row_number[row];
        mine = a.part + ((slot * a.Hkv + u.oh) * a.n_sinks + (row - start)) * 2 * D;
      }
    }
    const size_t base = ((size_t)row * (MODE == kDQ ? a.H : a.Hkv) + u.oh) * D;
    for (int done = 0; done < u.n_in; done += kSpill) {
      const bool last = u.n_in - done <= kSpill;
      ok = __all_sync(0xffffffffu,
                      mbar_wait_long(bars + 8 * C::B_ACCFULL, seen & 1, abort_flag, a.status));
      if (!ok) break;
      ++seen;
      tc_fence_after();
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += CW) {
        uint32_t x[CW], y[CW];
        tmem_ld_x16(t_a0 + c0, x);
        if (MODE != kDQ) tmem_ld_x16(t_a1 + c0, y);
        tmem_wait_ld();
        reg_fence16(x);
        if (MODE != kDQ) reg_fence16(y);
        if (c0 + CW >= D) {
          tc_fence_before();
          mbar_arrive(bars + 8 * C::B_ACCFREE);
        }
        if (!writes) continue;
        if (done > 0) {
          add16(x, spill + c0);
          if (MODE != kDQ) add16(y, spill + D + c0);
        }
        if (!last) {
          put16(spill + c0, x);
          if (MODE != kDQ) put16(spill + D + c0, y);
        } else if (MODE == kDQ) {
          put(a.dq + base + c0, x, a.scale);
        } else if (mine) {
          put16(mine + c0, x);
          put16(mine + D + c0, y);
        } else if (MODE == kDKV) {
          put(a.dv + base + c0, x, 1.f);
          put(a.dk + base + c0, y, a.scale);
        }
      }
    }
    if (!ok) break;
  }
}

template <int D, int MODE>
__device__ __forceinline__ void bwd_block(const CUtensorMap& tmO1, const CUtensorMap& tmO2,
                                          const CUtensorMap& tmI1, const CUtensorMap& tmI2,
                                          const BwdArgs& a) {
  using C = Cfg<D, MODE>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw);
  const uint32_t bars = sbase + C::OFF_BAR;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  volatile int* skip = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 8);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NUM_BARS; ++i) {
      uint32_t n = 1;
      if (i >= C::B_DSFULL && i < C::B_DSFULL + C::BUFS) n = kCompute;
      if (i >= C::B_COLS && i < C::B_COLS + 2) n = kCompute;
      if (i == C::B_ACCFREE) n = kEpilogue;
      if (i >= C::B_INREADY && i < C::B_INREADY + C::STAGES) n = 32;
      // Readers of the ring: producer and MMA threads, compute, epilogue and padding warps.
      if (i >= C::B_RINGEMPTY) n = 3 + kCompute + kEpilogue + (a.valid ? 32 : 0);
      mbar_init(bars + 8 * i, n);
    }
    *abort_flag = 0;
    mbar_fence_init();
    fence_proxy_async_smem();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&tmO1);
    tma_prefetch_map(&tmO2);
    tma_prefetch_map(&tmI1);
    tma_prefetch_map(&tmI2);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
    tc_fence_before();
  }
  grid_dep_wait();
  if (threadIdx.x == 0) *skip = *a.status != 0;   // an error recorded earlier makes the launch a no-op
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Ring ring{reinterpret_cast<volatile int*>(smem + C::OFF_RING), bars + 8 * C::B_RINGFULL,
            bars + 8 * C::B_RINGEMPTY, 0u};
  if (warp < 4) {
    set_max_regs_dec<kRegsRoles>();
    if (*skip) {
    } else if (warp == 0) {
      if (lane == 0)
        producer_role<D, MODE>(&tmO1, &tmO2, &tmI1, &tmI2, a, sbase, bars, abort_flag, ring);
      else if (lane == 1)
        claim_role<MODE>(a, ring, abort_flag);
    } else if (warp == 1) {
      if (lane == 0) ss_role<D, MODE>(a, sbase, bars, tmem, abort_flag, ring);
    } else if (warp == 2) {
      if (lane == 0) ts_role<D, MODE>(a, sbase, bars, tmem, abort_flag, ring);
    } else if (a.valid) {
      padding_role<D, MODE>(a, sbase, bars, abort_flag, lane, ring);
    }
  } else if (warp < 12) {
    set_max_regs_inc<kRegsCompute>();
    if (!*skip)
      compute_role<D, MODE>(a, bars, tmem, reinterpret_cast<float*>(smem + C::OFF_COLS),
                            abort_flag, warp, lane, ring);
  } else {
    set_max_regs_dec<kRegsEpilogue>();
    if (!*skip) epilogue_role<D, MODE>(a, bars, tmem, abort_flag, warp, lane, ring);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// The three parts are independent, so one launch holds the blocks of all: a small batch's parts run side
// by side (16 users 16 us; three launches 38 us), and a large one's blocks of the next part start
// where blocks of the one before end (256 users 919 us, one after the other 928 us). First tokens
// come first: behind the others a few blocks would take all their units in a row (16 users 43 us).
// Blocks of dKV and dQ in turn, to share tiles in L2, took 25 and 958 us.
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    window_bwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmDO,
                      const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const BwdArgs a) {
  const int b = (int)blockIdx.x;
  if (b < a.blocks_sink) bwd_block<D, kSink>(tmK, tmV, tmQ, tmDO, a);
  else if (b < a.blocks_sink + a.blocks_dkv) bwd_block<D, kDKV>(tmK, tmV, tmQ, tmDO, a);
  else bwd_block<D, kDQ>(tmQ, tmDO, tmK, tmV, a);
}

// Statistics of every row and head, [H][T]: the log-sum-exp in log2 units (+inf for a row that sees no
// key) and D = rowsum(dO * O); D / 8 lanes per row and head. Also the lists of kSink units and their
// users, one thread per user; their order does not touch any result.
template <int D, typename IdxT>
__global__ void __launch_bounds__(256)
    window_prep_kernel(const bf16* __restrict__ out, const bf16* __restrict__ dout,
                       const float* __restrict__ lse, const uint8_t* __restrict__ valid, int T,
                       int H, float* __restrict__ lse2, float* __restrict__ dsum,
                       const IdxT* __restrict__ off, int64_t B, int window, int n_sinks,
                       int4* sinks, int4* sink_users, int32_t* row_number, int32_t* n_sink_units,
                       int32_t* n_sink_users, const int32_t* status) {
  grid_dep_launch();
  grid_dep_wait();
  if (*status != 0) return;
  constexpr int L = D / 8;
  const int64_t n = (int64_t)T * H;
  const int64_t step = (int64_t)gridDim.x * (256 / L);
  const int sub = threadIdx.x % L;
  // Every lane of a warp takes the same number of turns: the reduction needs them all.
  for (int64_t x0 = (int64_t)blockIdx.x * (256 / L); x0 < n; x0 += step) {
    const int64_t x = x0 + threadIdx.x / L;
    const bool in = x < n;
    const int64_t row = in ? x / H : 0;
    const int h = in ? (int)(x - row * H) : 0;
    const bool real = in && (!valid || valid[row]);
    float acc = 0.f;
    if (real) {
      const uint4 o = ld_global_nc_v4(out + x * D + sub * 8), g = ld_global_nc_v4(dout + x * D + sub * 8);
      const uint32_t ow[4] = {o.x, o.y, o.z, o.w}, gw[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc = fmaf(bf16_lo(ow[i]), bf16_lo(gw[i]), fmaf(bf16_hi(ow[i]), bf16_hi(gw[i]), acc));
    }
#pragma unroll
    for (int m = L / 2; m > 0; m >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, m);
    if (in && sub == 0) {
      const float l = real ? lse[x] : -INFINITY;
      lse2[(size_t)h * T + row] = l == -INFINITY ? INFINITY : l * 1.4426950408889634f;
      dsum[(size_t)h * T + row] = real ? acc : 0.f;
    }
  }
  if (!sinks) return;
  for (int64_t b = blockIdx.x * (int64_t)256 + threadIdx.x; b < B;
       b += (int64_t)gridDim.x * 256) {
    const int s = (int)off[b], e = (int)off[b + 1];
    if (e - s <= window) continue;
    const int first = (s + window) / kChunk, chunks = (e - 1) / kChunk - first + 1;
    const int number = atomicAdd(n_sink_users, 1), slot = atomicAdd(n_sink_units, chunks);
    sink_users[number] = make_int4(s, e, slot, 0);
    for (int c = 0; c < chunks; ++c) sinks[slot + c] = make_int4(s, e, first + c, slot + c);
    for (int i = 0; i < min(n_sinks, e - s); ++i) row_number[s + i] = number;
  }
}

// dK and dV of the first tokens of users longer than the window: the window's sum, then the chunks' in
// order. One block per user and key head, four elements a thread.
template <int D>
__global__ void __launch_bounds__(256) window_join_kernel(const BwdArgs a) {
  grid_dep_wait();
  if (*a.status != 0) return;
  const int64_t n = *a.n_sink_users;
  for (int64_t x = blockIdx.x; x < n * a.Hkv; x += gridDim.x) {
    const int64_t number = x / a.Hkv;
    const int4 user = a.sink_users[number];      // {first row, end, slot of the first unit, -}
    const int hk = (int)(x % a.Hkv), s = user.x, e = user.y;
    const int c0 = (s + a.window) / kChunk, chunks = (e - 1) / kChunk - c0 + 1;
    const size_t step = (size_t)a.Hkv * a.n_sinks * 2 * D / 4;
    const size_t head = (size_t)hk * a.n_sinks * 2 * D / 4;
    const float4* part = reinterpret_cast<const float4*>(a.part);
    const float4* own = part + (size_t)(a.window_slot + number) * step + head;
    part += (size_t)user.z * step + head;
    const int keys = min(a.n_sinks, e - s);      // a user may be shorter than the first tokens
    for (int i = threadIdx.x; i < keys * 2 * D / 4; i += 256) {
      float4 v = own[i];
#pragma unroll 8
      for (int c = 0; c < chunks; ++c) {
        const float4 y = part[c * step + i];
        v.x += y.x;
        v.y += y.y;
        v.z += y.z;
        v.w += y.w;
      }
      const int key = i / (D / 2), is_k = i / (D / 4) % 2, d = i % (D / 4) * 4;
      const float f = is_k ? a.scale : 1.f;
      bf16* dst = (is_k ? a.dk : a.dv) + ((size_t)(s + key) * a.Hkv + hk) * D + d;
      *reinterpret_cast<uint2*>(dst) =
          make_uint2(pack_bf16x2(v.x * f, v.y * f), pack_bf16x2(v.z * f, v.w * f));
    }
  }
}

struct BwdLayout {
  size_t row_start = 0, row_end = 0, row_number = 0, lse2 = 0, dsum = 0, sinks = 0, users = 0,
         part = 0, spill = 0, counters = 0, total = 0;
  int64_t slots = 0, sink_users = 0;   // chunk partials, users that can have any
  bool spills = false;                 // some unit may have more than kSpill steps
};

// Only users longer than the window leave partial sums: at most T / (window + 1) of them. Their rows
// behind the window are disjoint runs, so that of their (user, chunk) pairs no more than one a user
// share a chunk with a pair before.
BwdLayout bwd_layout(int64_t B, int64_t T, int H, int Hkv, int d, int64_t window, int n_sinks) {
  BwdLayout L;
  const size_t t4 = align_up(4 * (size_t)T, 256);
  if (n_sinks > 0 && window < T) {
    L.sink_users = std::min(B, T / (window + 1));
    L.slots = T / kChunk + 1 + L.sink_users;
  }
  L.row_end = t4;
  L.row_number = 2 * t4;
  L.lse2 = 3 * t4;
  L.dsum = L.lse2 + align_up(4 * (size_t)T * H, 256);
  L.sinks = L.dsum + align_up(4 * (size_t)T * H, 256);
  L.users = L.sinks + align_up(16 * (size_t)L.slots, 256);
  L.part = L.users + align_up(16 * (size_t)L.sink_users, 256);
  L.spill = L.part + align_up(8 * (size_t)(L.slots + L.sink_users) * Hkv * n_sinks * d, 256);
  L.spills = std::max(T / kStep + 3, (T / kStep + 1) * (H / Hkv)) > kSpill;
  L.counters = L.spill + (L.spills ? (size_t)3 * kMaxSms * kTileM * 2 * d * 4 : 0);
  L.total = L.counters + 256;
  return L;
}

struct Maps {
  CUtensorMap q, k, v, dout;
};

// Every part gets a block per unit, or per SM where it has more units than the device SMs.
template <int D>
int launch_parts(BwdArgs a, const Maps& m, int64_t sink_units, int dev, int sms, cudaStream_t st) {
  constexpr int kBytes = std::max({Cfg<D, kDQ>::SMEM_ALLOC, Cfg<D, kDKV>::SMEM_ALLOC,
                                   Cfg<D, kSink>::SMEM_ALLOC});
  static std::atomic<bool> set[64];
  if (!set[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(window_bwd_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kBytes) != cudaSuccess)
      return JCA_ERR_CUDA;
    set[dev].store(true, std::memory_order_release);
  }
  sms = std::min(sms, kMaxSms);
  a.blocks_sink = (int)std::min<int64_t>(sink_units, sms);
  a.blocks_dkv = std::min(a.units_dkv, sms);
  const int grid = a.blocks_sink + a.blocks_dkv + std::min(a.units_dq, sms);
  return launch_dependent(window_bwd_kernel<D>, grid, kThreads, kBytes, st, m.q, m.dout, m.k, m.v, a);
}

template <int D>
int launch_bwd(BwdArgs a, const void* q, const void* k, const void* v, const void* out,
               const void* dout, const float* lse, const void* offsets, int64_t B, int64_t qs,
               int64_t ks, int64_t vs, int idx_bits, float* lse2, float* dsum, int4* sinks,
               int4* sink_users, int32_t* row_number, int32_t* n_listed, const BwdLayout& L, int dev,
               int sms, cudaStream_t st) {
  Maps m;
  if (!make_strided_map_bf16(&m.q, q, a.T, a.H, D, qs, kStep) ||
      !make_strided_map_bf16(&m.k, k, a.T, a.Hkv, D, ks, kStep) ||
      !make_strided_map_bf16(&m.v, v, a.T, a.Hkv, D, vs, kStep) ||
      !make_rows_map_bf16(&m.dout, dout, a.T, a.H, D, kStep))
    return JCA_ERR_CUDA;
  const int64_t want = ((int64_t)a.T * a.H * (D / 8) + 255) / 256;
  const int grid = (int)(want < (int64_t)sms * 16 ? want : (int64_t)sms * 16);
  const bf16 *o = static_cast<const bf16*>(out), *g = static_cast<const bf16*>(dout);
  int rc;
  if (idx_bits == 32)
    rc = launch_dependent(window_prep_kernel<D, int32_t>, grid, 256, 0, st, o, g, lse, a.valid, a.T,
                          a.H, lse2, dsum, static_cast<const int32_t*>(offsets), B, a.window,
                          a.n_sinks, sinks, sink_users, row_number, n_listed, n_listed + 1, a.status);
  else
    rc = launch_dependent(window_prep_kernel<D, int64_t>, grid, 256, 0, st, o, g, lse, a.valid, a.T,
                          a.H, lse2, dsum, static_cast<const int64_t*>(offsets), B, a.window,
                          a.n_sinks, sinks, sink_users, row_number, n_listed, n_listed + 1, a.status);
  if (rc) return rc;
  const int tiles = (a.T + kTileM - 1) / kTileM;
  a.units_dq = tiles * a.H;
  a.units_dkv = tiles * a.Hkv;
  // The list of kSink units is counted on the device; no more than this.
  rc = launch_parts<D>(a, m, sinks ? L.slots * a.Hkv : 0, dev, sms, st);
  if (rc || !sinks) return rc;
  const int64_t most = L.sink_users * a.Hkv;
  return launch_dependent(window_join_kernel<D>, (int)(most < (int64_t)sms * 64 ? most : sms * 64), 256,
                          0, st, a);
}

}  // namespace
}  // namespace jca

using namespace jca;

extern "C" size_t jca_window_bwd_workspace_bytes(int64_t B, int64_t T, int H, int Hkv, int d_head,
                                                 int n_sinks) {
  return jca_window_bwd_workspace_bytes_for(B, T, H, Hkv, d_head, n_sinks, 1);
}

extern "C" size_t jca_window_bwd_workspace_bytes_for(int64_t B, int64_t T, int H, int Hkv,
                                                     int d_head, int n_sinks, int64_t window) {
  if (!window_sizes_ok(B, T, H, Hkv, n_sinks) || !head_dim_ok(d_head) || window < 1) return 0;
  return bwd_layout(B, T, H, Hkv, d_head, window, n_sinks).total;
}

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
  const BwdLayout L = bwd_layout(B, T, H, Hkv, d_head, window, n_sinks);
  if (workspace_bytes < L.total) return JCA_ERR_WORKSPACE;
  if (B == 0) return JCA_OK;
  int dev = 0, sms = 0;
  rc = current_device(&dev, &sms);
  if (rc) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  // A window as long as the batch leaves no row behind it.
  const bool sinks = L.sink_users > 0;
  BwdArgs a = {};
  a.dq = static_cast<bf16*>(dq);
  a.dk = static_cast<bf16*>(dk);
  a.dv = static_cast<bf16*>(dv);
  a.valid = valid;
  a.row_start = reinterpret_cast<int32_t*>(ws + L.row_start);
  a.row_end = reinterpret_cast<int32_t*>(ws + L.row_end);
  int32_t* row_number = reinterpret_cast<int32_t*>(ws + L.row_number);
  a.row_number = row_number;
  a.lse2 = reinterpret_cast<float*>(ws + L.lse2);
  a.dsum = reinterpret_cast<float*>(ws + L.dsum);
  a.part = sinks ? reinterpret_cast<float*>(ws + L.part) : nullptr;
  a.spill = L.spills ? reinterpret_cast<float*>(ws + L.spill) : nullptr;
  a.window_slot = (int)L.slots;
  a.sinks = reinterpret_cast<int4*>(ws + L.sinks);
  a.sink_users = reinterpret_cast<int4*>(ws + L.users);
  a.counter = reinterpret_cast<int32_t*>(ws + L.counters);   // [3] claims, kSink units, users
  a.n_sink_units = a.counter + 3;
  a.n_sink_users = a.counter + 4;
  a.status = status;
  a.T = (int)T;
  a.H = H;
  a.Hkv = Hkv;
  a.group = H / Hkv;
  a.window = (int)(window < T ? window : (T > 0 ? T : 1));
  a.n_sinks = n_sinks;
  a.unit_ns = kWaitTimeoutNs + 10000ull * (uint64_t)(T / kStep + 3) * (uint64_t)a.group;
  a.v8 = aligned(dq, 32) && aligned(dk, 32) && aligned(dv, 32);
  a.scale = scale > 0.f ? scale : 1.0f / sqrtf((float)d_head);
  a.scale_log2 = a.scale * 1.4426950408889634f;
  rc = window_plan(offsets, B, T, idx_bits, reinterpret_cast<int32_t*>(ws + L.row_start),
                   reinterpret_cast<int32_t*>(ws + L.row_end), a.counter, 5, status, st);
  if (rc || T == 0) return rc;
  float* lse2 = reinterpret_cast<float*>(ws + L.lse2);
  float* dsum = reinterpret_cast<float*>(ws + L.dsum);
  int4* list = sinks ? reinterpret_cast<int4*>(ws + L.sinks) : nullptr;
  auto run = [&](auto fn) {
    return fn(a, q, k, v, out, dout, lse, offsets, B, q_stride, k_stride, v_stride, idx_bits, lse2,
              dsum, list, reinterpret_cast<int4*>(ws + L.users), row_number, a.counter + 3, L, dev,
              sms, st);
  };
  switch (d_head) {
    case 16: return run(launch_bwd<16>);
    case 32: return run(launch_bwd<32>);
    case 64: return run(launch_bwd<64>);
    default: return run(launch_bwd<128>);
  }
}
