// Causal attention over packed rows with a sliding window and first tokens that stay visible, forward
// (include/jca.h states the mask and the layout). The backward pass is in window_bwd.cu.
//
// Mathematics: row i of a user that starts at row s sees the keys of the two intervals
//   [max(s, i - window + 1), i]   and   [s, min(s + n_sinks, that lower end)),
// padding left out; softmax with a running maximum (p = 2^(scale log2e s - m), moved only when it
// grows by 2^8) and sum in fp32, so each key is visited once.
//
// Tiling. The packed rows are cut into blocks of 256 whatever users they hold: both lower ends never
// fall from row to row, so the keys that a 128-row tile needs are one run of packed rows ending
// at the tile itself, plus the first tokens of the tile's first user (every later user of the
// tile starts inside it). Short users therefore share tiles, every block costs about
// (window + 256) / 128 key tiles, and no list of work is needed beyond each row's user start, which a
// small kernel writes while it checks the offsets. Key tiles start at multiples of 128 rows, so
// most tiles are visible whole or not at all to a warp's 32 rows; the visible columns of a tile
// are decided for 32 columns at a time and per warp: chunks that no row sees are not read, chunks that
// every row sees are not masked.
//
// Kernel (one persistent block per SM, 16 warps; tcgen05 with TMEM accumulators, TMA loads):
//   warp 0       lane 0 loads Q and K tiles, lane 1 loads V tiles (rings of stages);
//   warps 1, 2   one thread each issues the MMAs of query tile A (rows 0..127 of the block) and B: the
//                two tiles share every K and V tile they both need, but neither waits for the
//                other's softmax (warp 1 also allocates TMEM);
//   warp 3       with padding: zeroes the padding rows of each landed V tile (a weight of 0 does not
//                undo an Inf or NaN there), otherwise idle;
//   warps 4..11  two softmax groups, one per query tile, one row a thread (TMEM lane = row); P goes
//                back to TMEM as bf16 and is read from there by the PV MMA; the group finishes its
//                own rows. They take over registers of the other warps, so that a row's 128 scores
//                stay in registers;
//   warp 12      claims the next block from a counter, reads where its rows' users start and passes
//                both to every role through a ring, several blocks ahead of the loads.
// The roles' code is kept small: instruction fetch of a larger kernel cost more than the steps
// themselves (256 users: 663 us with the softmax specialised by the number of visible chunks, against
// 350 in the same short run).
//
// What bounds it (256 users, window 256, d = 128: 350 us in a short run, 360 to 400 in a long one, 0.49
// to 0.43 of the copy bandwidth; 12 long users, window 1024, d = 64: 515 to 520 us): the chain
// QK -> softmax -> PV of each query tile. Cycles of a softmax group per tile, with timestamps:
//   d = 64    4,340: exponentials and weights 1,610 (1,024 at the unit's full rate), maximum 700, which
//             columns are visible 690, scores awaited and read 460, PV awaited 270, weights stored 180;
//             a block's output 2,520 of waiting and 1,410 of writing, over 9 tiles;
//   d = 128   6,570: scores awaited 1,630 (the weights lie over them, so QK follows PV), exponentials
//             1,215, visible columns 1,140, maximum 740; a block's output 2,570 and 2,940 over 3.3 tiles.
// TMEM holds the scores of two tiles only. Exponential unit busy 0.42 (d = 64), tensor core 0.23. What
// did not help, times of short runs:
// eight warps on one tile at a time (64 columns a thread; 350 and 657 us), sixteen with two threads to a
// row that exchange their maxima (460 and 745 us), one thread issuing both tiles' MMAs (350 and
// 562 us), the two groups taking turns at their exponentials (363 and 540 us), the products of a
// tile's first 64 weights started while the others are formed (379 us at d = 128).
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

// Checks the offsets and writes each row's user bounds; a block per user and share of its rows.
// Zeroes the counters from which the attention kernels claim their blocks.
template <typename IdxT>
__global__ void __launch_bounds__(128)
    window_plan_kernel(const IdxT* __restrict__ off, int64_t B, int64_t T,
                       int32_t* __restrict__ row_start, int32_t* __restrict__ row_end,
                       int32_t* counters, int n_counters, int32_t* status) {
  grid_dep_launch();
  if (blockIdx.x == 0 && blockIdx.y == 0 && (int)threadIdx.x < n_counters) counters[threadIdx.x] = 0;
  if (*status != 0) return;
  for (int64_t b = blockIdx.x; b < B; b += gridDim.x) {
    const long long s = (long long)off[b], e = (long long)off[b + 1];
    if (s < 0 || s > e || e > T || (b == 0 && s != 0) || (b == B - 1 && e != T)) {
      if (threadIdx.x == 0) atomicCAS(status, 0, (int32_t)JCA_STATUS_BAD_OFFSETS);
      continue;
    }
    for (long long i = s + blockIdx.y * 128 + threadIdx.x; i < e; i += gridDim.y * 128) {
      row_start[i] = (int32_t)s;
      if (row_end) row_end[i] = (int32_t)e;
    }
  }
}

struct FwdArgs {
  bf16* out;
  float* lse;                 // [T, H] or null
  const uint8_t* valid;       // [T] or null
  const int32_t* row_start;   // [T]
  int32_t* counter;           // next block to claim
  float* spill;               // [block][256][D], LONG: where a row may see more than kSpill key tiles
  int32_t* status;
  uint64_t item_ns;           // limit of the wait for room in the ring, which a block's work frees
  int T, H, group, window, n_sinks, n_items;
  int out_v8;                 // rows can be written with 32-byte stores
  float scale_log2;
};

// O is taken over into fp32 sums in memory after so many key tiles. The tensor core cuts each addition
// to its accumulators off, which costs sums of one sign about 2^-23 of themselves for every 16 keys
// (a row of 500,000 visible keys came out 0.3 % small, one of 2 million 1.2 %); within 1,024 tiles of
// eight additions that is 2^-10.
constexpr int kSpill = 1024;
constexpr int kRing = 4;
constexpr int kEntry = 8 + kItemRows;   // first row, head, then each row's user start from 8 on
constexpr int kThreads = 512;
constexpr int kGroup = 128;   // softmax threads of a query tile
// Registers a thread: 512 x 128 at launch, of which the softmax warps take what the others give up
// (72 + 40 + 2 x 200 = 4 x 128).
constexpr int kRegsRoles = 72, kRegsClaim = 40, kRegsSoftmax = 200;

template <int D>
struct Cfg {
  static constexpr int BM = kTileM, BN = kTileN;
  static constexpr int ROW_BYTES = D * 2;
  static constexpr int SW = ROW_BYTES >= 128 ? 128 : ROW_BYTES;    // swizzle span (bytes)
  static constexpr int NBLK = ROW_BYTES / SW;                      // column blocks of a tile
  static constexpr int BOX_X = SW / 2;
  static constexpr int TILE_BYTES = BM * ROW_BYTES;
  static constexpr int BLK_BYTES = BM * SW;
  static constexpr uint32_t LAYOUT = SW == 128 ? 2u : (SW == 64 ? 4u : 6u);
  static constexpr int KSTEPS_QK = D / 16;
  static constexpr int KSTEPS_PER_BLK = SW / 32;
  // Ring depths; d = 128 fills shared memory (192 KB) with one Q buffer per tile and two stages.
  static constexpr int QS = D >= 128 ? 1 : 2;
  static constexpr int KVS = D >= 128 ? 2 : 4;
  static constexpr int OFF_Q = 0;                                  // [group][QS]
  static constexpr int OFF_K = OFF_Q + 2 * QS * TILE_BYTES;
  static constexpr int OFF_V = OFF_K + KVS * TILE_BYTES;
  static constexpr int OFF_BAR = OFF_V + KVS * TILE_BYTES;
  static constexpr int B_QFULL = 0;                                // [group][QS]
  static constexpr int B_QEMPTY = B_QFULL + 2 * QS;
  static constexpr int B_KFULL = B_QEMPTY + 2 * QS;                // [KVS]
  static constexpr int B_KEMPTY = B_KFULL + KVS;
  static constexpr int B_VFULL = B_KEMPTY + KVS;
  static constexpr int B_VREADY = B_VFULL + KVS;                   // padding rows zeroed
  static constexpr int B_VEMPTY = B_VREADY + KVS;
  static constexpr int B_SFULL = B_VEMPTY + KVS;                   // [group]
  static constexpr int B_PFULL = B_SFULL + 2;
  static constexpr int B_OREADY = B_PFULL + 2;
  static constexpr int B_OFREE = B_OREADY + 2;
  static constexpr int B_SREAD = B_OFREE + 2;                      // SEP_P: S_w is in registers
  static constexpr int B_PVDONE = B_SREAD + 2;                     // SEP_P: P_w was read
  static constexpr int B_DRAIN = B_PVDONE + 2;                     // [group]
  static constexpr int B_RINGFULL = B_DRAIN + 2;                   // [kRing]
  static constexpr int B_RINGEMPTY = B_RINGFULL + kRing;
  static constexpr int NUM_BARS = B_RINGEMPTY + kRing;
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
  static constexpr int OFF_RING = OFF_MISC + 16;                   // [kRing][kEntry] ints
  static constexpr int SMEM_USED = OFF_RING + kRing * kEntry * 4;
  static constexpr int SMEM_RAW = SMEM_USED + 1024;                // slack for 1 KB alignment
  // At least 120 KB so that a second block never shares the SM (and its TMEM).
  static constexpr int SMEM_ALLOC = SMEM_RAW > 120 * 1024 ? SMEM_RAW : 120 * 1024;
  // TMEM columns: S_A | S_B (128 each), then O_A | O_B. Heads of up to 64 leave room for the weights
  // beside the scores: the next QK of a query tile is then issued as soon as its scores are in
  // registers, and the softmax never waits for a PV and a QK in a row. At d = 128 the weights lie
  // over the scores.
  static constexpr bool SEP_P = D <= 64;
  static constexpr uint32_t TMEM_COLS = 512;
  static __device__ __forceinline__ uint32_t s_col(int grp) { return 128u * grp; }
  static __device__ __forceinline__ uint32_t o_col(int grp) { return 256u + (SEP_P ? 64u : 128u) * grp; }
  static __device__ __forceinline__ uint32_t p_col(int grp) { return SEP_P ? 384u + 64u * grp : 128u * grp; }
  static_assert(SMEM_ALLOC <= 227 * 1024, "shared memory budget");
};

// A block of up to 256 rows of one head, as every role derives it from the ring entry. Its key tiles
// are, in order, the first tokens of A's first user (when they lie below the others; trimmed to
// n_sink keys) and the 128-row tiles from kstart to the block's own rows.
struct Item {
  int q0, h, kstart, n_sink, sink0, n_tiles;
  int last_a;                 // A reads tiles [0, last_a]; the last holds its own rows
  int b0, sb0, sb1;           // B reads tiles [b0, n_tiles) and, for first tokens, [sb0, sb1)
  bool has_b;

  __device__ __forceinline__ bool is_sink(int j) const { return n_sink && j == 0; }
  __device__ __forceinline__ int key_row(int j) const {
    return is_sink(j) ? sink0 : kstart + (j - (n_sink ? 1 : 0)) * kTileN;
  }
  __device__ __forceinline__ bool a_reads(int j) const { return j <= last_a; }
  __device__ __forceinline__ bool b_reads(int j) const { return j >= b0 || (j >= sb0 && j < sb1); }
};

__device__ __forceinline__ Item make_item(const volatile int* e, const FwdArgs& a) {
  Item w;
  w.q0 = e[0];
  w.h = e[1];
  w.has_b = w.q0 + kTileM < a.T;
  const int start_a = e[8], start_b = e[8 + kTileM];
  const int lo_a = max(start_a, w.q0 - a.window + 1);
  const int lo_b = max(start_b, w.q0 + kTileM - a.window + 1);
  w.sink0 = start_a;
  w.kstart = lo_a & ~(kTileN - 1);
  w.n_sink = max(0, min(a.n_sinks, w.kstart - start_a));
  const int x = w.n_sink ? 1 : 0;
  w.last_a = x + (w.q0 - w.kstart) / kTileN;
  w.n_tiles = w.last_a + (w.has_b ? 2 : 1);
  w.b0 = w.has_b ? x + max(0, lo_b - w.kstart) / kTileN : w.n_tiles;
  // First tokens of B's first user: in A's tile of them, in the tiles from kstart on, or both.
  const int first_b = min(start_b + a.n_sinks, lo_b);
  w.sb0 = start_b < w.kstart ? 0 : x + (start_b - w.kstart) / kTileN;
  w.sb1 = !w.has_b || first_b <= start_b ? 0
          : first_b <= w.kstart          ? 1
                                         : x + (first_b - 1 - w.kstart) / kTileN + 1;
  return w;
}

// Takes the next entry, and the user start of row `r` of the block; false when aborting or at the end.
__device__ __forceinline__ bool ring_take(Ring& r, const FwdArgs& a, Item& w,
                                          volatile int* abort_flag, bool& ok, int row = 0,
                                          int* start = nullptr) {
  const int s = (int)(r.k % kRing);
  ok = mbar_wait(r.full + 8 * s, (r.k / kRing) & 1, abort_flag, a.status);
  if (!ok) return false;
  const volatile int* e = r.slot + kEntry * s;
  const bool more = e[0] >= 0;
  if (more) w = make_item(e, a);
  if (start) *start = e[8 + row];
  mbar_arrive(r.empty + 8 * s);
  ++r.k;
  return more;
}

// Claims blocks until none is left and posts them, then the end marker; one warp.
__device__ void claim_role(const FwdArgs& a, Ring r, volatile int* abort_flag, int lane) {
  for (;;) {
    int v = lane == 0 ? atomicAdd(a.counter, 1) : 0;
    v = __shfl_sync(0xffffffffu, v, 0);
    // Heads fastest: concurrent blocks share rows, and with shared heads K and V. Rows from the
    // end: under a long window the later blocks of a user are the longer ones.
    const int left = a.n_items - 1 - v;
    const int q0 = left < 0 ? -1 : left / a.H * kItemRows;
    int start[kItemRows / 32];
    if (left >= 0) {
#pragma unroll
      for (int i = 0; i < kItemRows / 32; ++i)
        start[i] = a.row_start[min(q0 + 32 * i + lane, a.T - 1)];
    }
    const int s = (int)(r.k % kRing);
    const bool ok = mbar_wait_long(r.empty + 8 * s, ((r.k / kRing) & 1) ^ 1, abort_flag, a.status,
                                   a.item_ns);
    if (!__all_sync(0xffffffffu, ok)) return;
    volatile int* e = r.slot + kEntry * s;
    if (lane == 0) e[0] = q0;
    if (left >= 0) {
      if (lane == 0) e[1] = left % a.H;
#pragma unroll
      for (int i = 0; i < kItemRows / 32; ++i) e[8 + 32 * i + lane] = start[i];
    }
    mbar_arrive(r.full + 8 * s);
    ++r.k;
    if (left < 0) return;
  }
}

template <int D>
__device__ void producer_role(const CUtensorMap* tmQ, const CUtensorMap* tmKV, const FwdArgs& a,
                              uint32_t sbase, uint32_t bars, volatile int* abort_flag,
                              bool loads_v, Ring ring) {
  using C = Cfg<D>;
  uint32_t nq[2] = {0, 0}, g = 0;
  const int empty = loads_v ? C::B_VEMPTY : C::B_KEMPTY, full = loads_v ? C::B_VFULL : C::B_KFULL;
  const int off = loads_v ? C::OFF_V : C::OFF_K;
  bool ok = true;
  Item w;
  while (ring_take(ring, a, w, abort_flag, ok)) {
    const int hk = w.h / a.group;
    for (int j = 0; ok && j < w.n_tiles; ++j) {
      const int s = (int)(g % C::KVS);
      ok = mbar_wait(bars + 8 * (empty + s), ((g / C::KVS) & 1) ^ 1, abort_flag, a.status);
      if (!ok) break;
      mbar_arrive_expect_tx(bars + 8 * (full + s), C::TILE_BYTES);
#pragma unroll
      for (int c = 0; c < C::NBLK; ++c)
        tma_load_3d(sbase + off + s * C::TILE_BYTES + c * C::BLK_BYTES, tmKV,
                    bars + 8 * (full + s), c * C::BOX_X, hk, w.key_row(j));
      ++g;
      if (loads_v || j > 0) continue;
      // The item's Q tiles go out behind its first K tile, whose stage was freed earlier.
      for (int t = 0; t < (w.has_b ? 2 : 1); ++t) {
        const int slot = t * C::QS + (int)(nq[t] % C::QS);
        ok = mbar_wait(bars + 8 * (C::B_QEMPTY + slot), ((nq[t] / C::QS) & 1) ^ 1, abort_flag,
                       a.status);
        if (!ok) break;
        mbar_arrive_expect_tx(bars + 8 * (C::B_QFULL + slot), C::TILE_BYTES);
        ++nq[t];
#pragma unroll
        for (int c = 0; c < C::NBLK; ++c)
          tma_load_3d(sbase + C::OFF_Q + slot * C::TILE_BYTES + c * C::BLK_BYTES, tmQ,
                      bars + 8 * (C::B_QFULL + slot), c * C::BOX_X, w.h, w.q0 + t * C::BM);
      }
    }
    if (!ok) break;
  }
  if (!ok) {
    // Aborting: let every copy this thread started land before the block exits.
    for (int t = 0; t < 2; ++t)
      for (uint32_t n = nq[t] > (uint32_t)C::QS ? nq[t] - C::QS : 0; n < nq[t]; ++n)
        mbar_wait_drain(bars + 8 * (C::B_QFULL + t * C::QS + (int)(n % C::QS)), (n / C::QS) & 1);
    for (uint32_t n = g > (uint32_t)C::KVS ? g - C::KVS : 0; n < g; ++n)
      mbar_wait_drain(bars + 8 * (full + (int)(n % C::KVS)), (n / C::KVS) & 1);
  }
}

// Zeroes the rows of padding in every V tile; one warp.
template <int D>
__device__ void padding_role(const FwdArgs& a, uint32_t sbase, uint32_t bars,
                             volatile int* abort_flag, int lane, Ring ring) {
  using C = Cfg<D>;
  uint32_t g = 0;
  bool ok = true;
  Item w;
  for (;;) {
    const bool more = ring_take(ring, a, w, abort_flag, ok);
    if (!__all_sync(0xffffffffu, more)) return;
    for (int j = 0; j < w.n_tiles; ++j, ++g) {
      const int s = (int)(g % C::KVS), row = w.key_row(j);
      uint32_t pad[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int k = row + 32 * c + lane;
        pad[c] = __ballot_sync(0xffffffffu, k < a.T && !a.valid[k]);
      }
      ok = mbar_wait_long(bars + 8 * (C::B_VFULL + s), (g / C::KVS) & 1, abort_flag, a.status);
      if (!__all_sync(0xffffffffu, ok)) return;
      const uint32_t tile = sbase + C::OFF_V + s * C::TILE_BYTES;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (pad[c]) zero_rows<C::ROW_BYTES, C::SW, C::BLK_BYTES>(tile, 32 * c, pad[c], lane);
      fence_proxy_async_smem();
      mbar_arrive(bars + 8 * (C::B_VREADY + s));
    }
  }
}

// One query tile's products; a thread for A and one for B, so that neither waits for the other's
// softmax. QK(t) is followed by PV(t), or with SEP_P by PV(t - 1).
template <int D, bool LONG>
__device__ void mma_role(const FwdArgs& a, uint32_t sbase, uint32_t bars, uint32_t tmem,
                         volatile int* abort_flag, int grp, Ring ring) {
  using C = Cfg<D>;
  constexpr uint32_t kIdescFull = idesc_bf16_f32(C::BM, C::BN, false, false);
  constexpr uint32_t kIdesc0 = kIdescFull & ~(0x3Fu << 17);
  constexpr uint32_t kIdescPV = idesc_bf16_f32(C::BM, D, false, true);
  constexpr uint32_t kVStep = (16 * C::SW) >> 4;   // 16 key rows of V
  const int vfull = a.valid ? C::B_VREADY : C::B_VFULL;
  const uint32_t ts = tmem + C::s_col(grp), to = tmem + C::o_col(grp), tp = tmem + C::p_col(grp);
  const uint64_t dq = smem_desc(sbase + C::OFF_Q + grp * C::QS * C::TILE_BYTES, 16, 8 * C::SW,
                                C::LAYOUT);
  const uint64_t dk = smem_desc(sbase + C::OFF_K, 16, 8 * C::SW, C::LAYOUT);
  const uint64_t dv = smem_desc(sbase + C::OFF_V, C::BLK_BYTES, 8 * C::SW, C::LAYOUT);
  uint32_t g = 0, steps = 0, pvs = 0, sums = 0, qn = 0;
  bool ok = true;
  // A PV whose weights are not known to be there yet (key tile, 16-key steps, first and last of O's
  // sums).
  uint32_t pv_g = 0;
  int pv_k = 0;
  bool pv_first = false, pv_last = false;
  auto issue_pv = [&]() -> bool {
    const int s = (int)(pv_g % C::KVS);
    if (!mbar_wait_long(bars + 8 * (vfull + s), (pv_g / C::KVS) & 1, abort_flag, a.status)) return false;
    if (pv_k == 0) {   // not read by this query tile
      mbar_arrive(bars + 8 * (C::B_VEMPTY + s));
      return true;
    }
    if (pv_first && sums > 0 &&
        !mbar_wait_long(bars + 8 * (C::B_OFREE + grp), (sums - 1) & 1, abort_flag, a.status))
      return false;
    if (!mbar_wait_long(bars + 8 * (C::B_PFULL + grp), pvs & 1, abort_flag, a.status)) return false;
    ++pvs;
    tc_fence_after();
    // O (+)= P V; P sits in TMEM as bf16 pairs, 8 columns per 16 keys.
    const uint64_t v = dv + (uint64_t)((s * C::TILE_BYTES) >> 4);
#pragma unroll 4
    for (int kk = 0; kk < pv_k; ++kk)
      tc_mma_ts(to, tp + (uint32_t)kk * 8u, v + (uint64_t)(kk * kVStep), kIdescPV,
                (pv_first && kk == 0) ? 0u : 1u);
    tc_commit(bars + 8 * (C::B_VEMPTY + s));
    if (C::SEP_P) tc_commit(bars + 8 * (C::B_PVDONE + grp));
    if (pv_last) {
      tc_commit(bars + 8 * (C::B_OREADY + grp));
      ++sums;
    }
    return true;
  };
  bool pending = false;
  Item w;
  while (ok && ring_take(ring, a, w, abort_flag, ok)) {
    bool seen = false;
    int in_sums = 0;                               // LONG: tiles in O's present sums
    const int last = grp ? (w.has_b ? w.n_tiles - 1 : -1) : w.last_a;
    const int slot = grp * C::QS + (int)(qn % C::QS);
    const uint64_t q = dq + (uint64_t)(((int)(qn % C::QS) * C::TILE_BYTES) >> 4);
#pragma unroll 1
    for (int j = 0; j < w.n_tiles; ++j, ++g) {
      const int s = (int)(g % C::KVS);
      const bool reads = grp ? w.b_reads(j) : w.a_reads(j);
      const int keys = w.is_sink(j) ? (w.n_sink + 15) & ~15 : C::BN;
      ok = mbar_wait_long(bars + 8 * (C::B_KFULL + s), (g / C::KVS) & 1, abort_flag, a.status);
      if (!ok) break;
      if (reads) {
        if (!seen)
          ok = mbar_wait_long(bars + 8 * (C::B_QFULL + slot), (qn / C::QS) & 1, abort_flag, a.status);
        if (C::SEP_P && ok && steps > 0)
          ok = mbar_wait_long(bars + 8 * (C::B_SREAD + grp), (steps - 1) & 1, abort_flag, a.status);
        if (!ok) break;
        tc_fence_after();
        const uint64_t k = dk + (uint64_t)((s * C::TILE_BYTES) >> 4);
        const uint32_t idesc = kIdesc0 | ((uint32_t)(keys >> 3) << 17);
#pragma unroll
        for (int kk = 0; kk < C::KSTEPS_QK; ++kk) {
          const uint32_t off = ((kk / C::KSTEPS_PER_BLK) * C::BLK_BYTES +
                                (kk % C::KSTEPS_PER_BLK) * 32) >> 4;
          tc_mma(ts, q + off, k + off, idesc, kk > 0 ? 1u : 0u);
        }
        ++steps;
        tc_commit(bars + 8 * (C::B_SFULL + grp));
        tc_commit(bars + 8 * (C::B_KEMPTY + s));
        if (j == last) tc_commit(bars + 8 * (C::B_QEMPTY + slot));
      } else {
        mbar_arrive(bars + 8 * (C::B_KEMPTY + s));
      }
      if (C::SEP_P && pending) {
        ok = issue_pv();
        if (!ok) break;
      }
      pv_g = g;
      pv_k = reads ? keys >> 4 : 0;
      pv_first = reads && !seen;
      pv_last = j == last;
      seen |= reads;
      if constexpr (LONG) {
        pv_first = reads && in_sums == 0;
        in_sums += reads ? 1 : 0;
        pv_last |= in_sums == kSpill;
        if (pv_last) in_sums = 0;
      }
      pending = C::SEP_P;
      if (!C::SEP_P) {
        ok = issue_pv();
        if (!ok) break;
      }
    }
    if (last >= 0) ++qn;
  }
  if (ok && pending) ok = issue_pv();
  if (!ok) {
    // Aborting: wait until every MMA this thread issued has completed.
    tc_commit(bars + 8 * (C::B_DRAIN + grp));
    mbar_wait_drain(bars + 8 * (C::B_DRAIN + grp), 0);
  }
}

// Weights p = 2^(scale_log2 s - m) of 32 scores, their sum added to (acc0, acc1), and the weights
// rounded to bf16 pairs, the operand type of the PV product.
__device__ __forceinline__ void weights32(const uint32_t* x, float2 sl2v, float2 negv, float2& acc0,
                                          float2& acc1, uint32_t* pk) {
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const float2 xs = __ffma2_rn(
        make_float2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])), sl2v, negv);
    float2 p;
    p.x = fast_exp2(xs.x);
    p.y = fast_exp2(xs.y);
    if (k & 1) acc1 = __fadd2_rn(acc1, p);
    else acc0 = __fadd2_rn(acc0, p);
    pk[k] = pack_bf16x2(p.x, p.y);
  }
}

__device__ __forceinline__ float max32(const uint32_t* x) {
  float m0 = -INFINITY, m1 = -INFINITY, m2 = -INFINITY, m3 = -INFINITY;
#pragma unroll
  for (int k = 0; k < 32; k += 8) {
    m0 = fmax3(m0, __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
    m1 = fmax3(m1, __uint_as_float(x[k + 2]), __uint_as_float(x[k + 3]));
    m2 = fmax3(m2, __uint_as_float(x[k + 4]), __uint_as_float(x[k + 5]));
    m3 = fmax3(m3, __uint_as_float(x[k + 6]), __uint_as_float(x[k + 7]));
  }
  return fmaxf(fmaxf(m0, m1), fmaxf(m2, m3));
}

template <int D, bool LONG>
__device__ void softmax_role(const FwdArgs& a, uint32_t bars, uint32_t tmem,
                             volatile int* abort_flag, int warp, int lane, Ring ring) {
  using C = Cfg<D>;
  const int grp = (warp - 4) >> 2;
  const int quarter = warp & 3;
  const int r = quarter * 32 + lane;
  const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
  const uint32_t t_s = t_lane + C::s_col(grp), t_o = t_lane + C::o_col(grp);
  const uint32_t t_p = t_lane + C::p_col(grp);
  const float sl2 = a.scale_log2;
  float* spill = LONG ? a.spill + ((size_t)blockIdx.x * kItemRows + grp * C::BM + r) * D : nullptr;
  uint32_t lt = 0, oi = 0;
  bool ok = true;
  Item w;
  for (;;) {
    int start = 0;
    const bool more = ring_take(ring, a, w, abort_flag, ok, grp * C::BM + r, &start);
    if (!__all_sync(0xffffffffu, more)) break;
    if (grp == 1 && !w.has_b) continue;
    const int i = w.q0 + grp * C::BM + r;           // this thread's row
    const bool row_ok = i < a.T;
    const bool sees = row_ok && (!a.valid || a.valid[i]);
    // Visible keys: [lo, hi) and [start, first).
    const int lo = sees ? max(start, i - a.window + 1) : 0, hi = sees ? i + 1 : 0;
    const int first = sees ? min(start + a.n_sinks, lo) : start;
    float m = -INFINITY, l = 0.f;
    float m_spill = -INFINITY;                      // reference of the sums in `spill`
    int j = 0;
    do {
      bool fresh = true;
      int in_sums = 0;
      const bool spilled = LONG && j > 0;
      for (; j < w.n_tiles && !(LONG && in_sums == kSpill); ++j) {
        if (!(grp ? w.b_reads(j) : w.a_reads(j))) continue;
        const int kr = w.key_row(j), cols = w.is_sink(j) ? w.n_sink : C::BN;
        // Chunks of 32 columns that some row, and that every row of the warp sees.
        uint32_t bits[4], any = 0xfu, all = 0xfu;
        if (!__all_sync(0xffffffffu,
                        cols == C::BN && !a.valid && lo <= kr && hi >= kr + C::BN)) {
          any = all = 0;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int k0 = kr + 32 * c;
            uint32_t b = range_bits(lo - k0, hi - k0) | range_bits(start - k0, first - k0);
            b &= range_bits(0, cols - 32 * c);
            if (a.valid) {
              const int k = k0 + lane;
              b &= __ballot_sync(0xffffffffu, k < a.T && a.valid[k]);
            }
            bits[c] = b;
            any |= __any_sync(0xffffffffu, b != 0u) ? 1u << c : 0u;
            all |= __all_sync(0xffffffffu, b == 0xffffffffu) ? 1u << c : 0u;
          }
        }
        ok = __all_sync(0xffffffffu,
                        mbar_wait_long(bars + 8 * (C::B_SFULL + grp), lt & 1, abort_flag, a.status));
        if (!ok) break;
        ++lt;
        tc_fence_after();
        uint32_t x[128];
        tmem_ld_x32(t_s + 0, x);
        tmem_ld_x32(t_s + 32, x + 32);
        tmem_ld_x32(t_s + 64, x + 64);
        tmem_ld_x32(t_s + 96, x + 96);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 128; c += 16) reg_fence16(x + c);
        if (C::SEP_P) {
          tc_fence_before();
          mbar_arrive(bars + 8 * (C::B_SREAD + grp));
        }
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (!((any >> c) & 1)) continue;
          if (!((all >> c) & 1)) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
              x[32 * c + k] = ((bits[c] >> k) & 1u) ? x[32 * c + k] : 0xff800000u;   // -inf
          }
          mx = fmaxf(mx, max32(x + 32 * c));
        }
        // The reference maximum moves only when it grows by more than 2^8: the weights stay below 2^8,
        // and O and l keep the same reference.
        const float m_new = fmaxf(m, mx * sl2);
        const bool rescale = m_new > m + 8.0f;
        const float m_use = rescale ? m_new : m;
        const float neg_m = (m_use == -INFINITY) ? 0.f : -m_use;
        const float alpha = (rescale && m != -INFINITY) ? fast_exp2(m - m_use) : 1.f;
        const float2 sl2v = make_float2(sl2, sl2), negv = make_float2(neg_m, neg_m);
        float2 acc0 = make_float2(0.f, 0.f), acc1 = acc0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t* pk = x + 32 * c;   // in place: each pair goes where a pair before it was read
          if ((any >> c) & 1) {
            weights32(x + 32 * c, sl2v, negv, acc0, acc1, pk);
          } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) pk[k] = 0u;
          }
          if (!C::SEP_P) tmem_st_x16(t_p + 16 * c, pk);
        }
        if (C::SEP_P) {
          if (lt > 1) {
            // The PV before has read the weights that these replace, and O is stable.
            ok = __all_sync(0xffffffffu, mbar_wait_long(bars + 8 * (C::B_PVDONE + grp), lt & 1, abort_flag,
                                                   a.status));
            if (!ok) break;
            tc_fence_after();
          }
#pragma unroll
          for (int c = 0; c < 4; ++c)
            tmem_st_x16(t_p + 16 * c, x + 32 * c);
        }
        // O is stable here: without SEP_P its last PV was issued before the QK that filled S, and a
        // commit fires only after every earlier MMA of its thread.
        if (__any_sync(0xffffffffu, rescale && !fresh)) scale_row<D, 1>(t_o, alpha);
        l = l * alpha + ((acc0.x + acc0.y) + (acc1.x + acc1.y));
        m = m_use;
        fresh = false;
        ++in_sums;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bars + 8 * (C::B_PFULL + grp));
      }
      if (!ok) break;
      ok = __all_sync(0xffffffffu,
                      mbar_wait_long(bars + 8 * (C::B_OREADY + grp), oi & 1, abort_flag, a.status));
      if (!ok) break;
      ++oi;
      tc_fence_after();
      // O is complete, or (LONG) handed over: the sums that the row's thread keeps in memory come in
      // under the present reference.
      const bool end = !LONG || j > (grp ? w.n_tiles - 1 : w.last_a);
      float old = 0.f;
      if constexpr (LONG) {
        if (m_spill != -INFINITY) old = fast_exp2(m_spill - m);
        m_spill = m;
      }
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const size_t row = (size_t)i * a.H + w.h;
      constexpr int CW = D < 32 ? D : 32;
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += CW) {
        uint32_t u[CW];
        tmem_ld_cols<CW>(t_o + c0, u);
        tmem_wait_ld();
        reg_fence_cols<CW>(u);
        if (c0 + CW >= D) {
          tc_fence_before();
          mbar_arrive(bars + 8 * (C::B_OFREE + grp));
        }
        if (!row_ok) continue;
        if (spilled) {
#pragma unroll
          for (int c = 0; c < CW; ++c)
            u[c] = __float_as_uint(fmaf(old, spill[c0 + c], __uint_as_float(u[c])));
        }
        if (!end) {
#pragma unroll
          for (int c = 0; c < CW; ++c) spill[c0 + c] = __uint_as_float(u[c]);
          continue;
        }
#pragma unroll
        for (int c = 0; c < CW; c += 16) {
          uint32_t p[8];
#pragma unroll
          for (int k = 0; k < 8; ++k)
            p[k] = pack_bf16x2(__uint_as_float(u[c + 2 * k]) * inv,
                               __uint_as_float(u[c + 2 * k + 1]) * inv);
          bf16* dst = a.out + row * D + c0 + c;
          if (a.out_v8) {
            st_global_v8(dst, p);
          } else {
            reinterpret_cast<uint4*>(dst)[0] = make_uint4(p[0], p[1], p[2], p[3]);
            reinterpret_cast<uint4*>(dst)[1] = make_uint4(p[4], p[5], p[6], p[7]);
          }
        }
      }
      if (end && a.lse && row_ok)
        a.lse[row] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
      if (end) break;
    } while (LONG);
    if (!ok) break;
  }
}

template <int D, bool LONG>
__global__ void __launch_bounds__(kThreads, 1)
    window_fwd_kernel(const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const FwdArgs a) {
  using C = Cfg<D>;
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
      if (i >= C::B_KEMPTY && i < C::B_KEMPTY + C::KVS) n = 2;   // both MMA threads
      if (i >= C::B_VEMPTY && i < C::B_VEMPTY + C::KVS) n = 2;
      if (i >= C::B_PFULL && i < C::B_PFULL + 2) n = kGroup;
      if (i >= C::B_OFREE && i < C::B_OFREE + 2) n = kGroup;
      if (i >= C::B_SREAD && i < C::B_SREAD + 2) n = kGroup;
      if (i >= C::B_VREADY && i < C::B_VREADY + C::KVS) n = 32;
      if (i >= C::B_RINGFULL) n = 32;
      // Readers of the ring: the two producer and MMA threads, both groups, the padding warp.
      if (i >= C::B_RINGEMPTY) n = 4 + 2 * kGroup + (a.valid ? 32 : 0);
      mbar_init(bars + 8 * i, n);
    }
    *abort_flag = 0;
    mbar_fence_init();
    fence_proxy_async_smem();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&tmQ);
    tma_prefetch_map(&tmK);
    tma_prefetch_map(&tmV);
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
      if (lane < 2)
        producer_role<D>(&tmQ, lane == 1 ? &tmV : &tmK, a, sbase, bars, abort_flag, lane == 1,
                         ring);
    } else if (warp < 3) {
      if (lane == 0) mma_role<D, LONG>(a, sbase, bars, tmem, abort_flag, warp - 1, ring);
    } else if (a.valid) {
      padding_role<D>(a, sbase, bars, abort_flag, lane, ring);
    }
  } else if (warp < 12) {
    set_max_regs_inc<kRegsSoftmax>();
    if (!*skip) softmax_role<D, LONG>(a, bars, tmem, abort_flag, warp, lane, ring);
  } else {
    set_max_regs_dec<kRegsClaim>();
    if (!*skip && warp == 12) claim_role(a, ring, abort_flag, lane);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int D, bool LONG>
int launch_fwd(FwdArgs a, const void* q, const void* k, const void* v, int Hkv, int64_t qs,
               int64_t ks, int64_t vs, int dev, int sms, cudaStream_t st) {
  using C = Cfg<D>;
  static std::atomic<bool> set[64];
  if (!set[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(window_fwd_kernel<D, LONG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::SMEM_ALLOC) != cudaSuccess)
      return JCA_ERR_CUDA;
    set[dev].store(true, std::memory_order_release);
  }
  CUtensorMap tmQ, tmK, tmV;
  if (!make_strided_map_bf16(&tmQ, q, a.T, a.H, D, qs, C::BM) ||
      !make_strided_map_bf16(&tmK, k, a.T, Hkv, D, ks, C::BN) ||
      !make_strided_map_bf16(&tmV, v, a.T, Hkv, D, vs, C::BN))
    return JCA_ERR_CUDA;
  sms = sms < kMaxSms ? sms : kMaxSms;
  const int grid = a.n_items < sms ? a.n_items : sms;
  return launch_dependent(window_fwd_kernel<D, LONG>, grid, kThreads, C::SMEM_ALLOC, st, tmQ, tmK, tmV,
                          a);
}

struct FwdLayout {
  size_t row_start = 0, spill = 0, counter = 0, total = 0;
  bool spills = false;   // some row may see more than kSpill key tiles
};

FwdLayout fwd_layout(int64_t T, int d) {
  FwdLayout L;
  L.spill = align_up(4 * (size_t)T, 256);
  L.spills = T / kTileN + 2 > kSpill;
  L.counter = L.spill + (L.spills ? (size_t)kMaxSms * kItemRows * d * 4 : 0);
  L.total = L.counter + 256;
  return L;
}

}  // namespace

bool window_sizes_ok(int64_t B, int64_t T, int H, int Hkv, int n_sinks) {
  return B >= 0 && T >= 0 && T < (int64_t)INT_MAX - kItemRows && B < (int64_t)INT_MAX && H >= 1 &&
         H < 65536 && Hkv >= 1 && H % Hkv == 0 && n_sinks >= 0 && n_sinks <= kWindowMaxSinks &&
         (B > 0 || T == 0) && (T / kTileM + 1) * H < (int64_t)INT_MAX;
}

int window_check(int64_t B, int64_t T, int H, int Hkv, int d, int64_t window, int n_sinks,
                 int64_t qs, int64_t ks, int64_t vs, int idx_bits) {
  if (idx_bits != 32 && idx_bits != 64) return JCA_ERR_IDX_BITS;
  if (!head_dim_ok(d)) return JCA_ERR_HEAD_DIM;
  if (!window_sizes_ok(B, T, H, Hkv, n_sinks) || window < 1) return JCA_ERR_SHAPE;
  const int64_t far = (int64_t)1 << 38;   // row strides of a tensor map stay below 2^40 bytes
  if (qs < (int64_t)H * d || ks < (int64_t)Hkv * d || vs < (int64_t)Hkv * d || qs >= far ||
      ks >= far || vs >= far)
    return JCA_ERR_SHAPE;
  if (qs % 8 || ks % 8 || vs % 8) return JCA_ERR_ALIGN;
  return JCA_OK;
}

int window_plan(const void* offsets, int64_t B, int64_t T, int idx_bits, int32_t* row_start,
                int32_t* row_end, int32_t* counters, int n_counters, int32_t* status,
                cudaStream_t st) {
  // About four rows a thread on average, so that a few long users do not wait for one block each.
  const int64_t x = B < (1 << 20) ? B : (1 << 20), share = T / (B * 512);
  const dim3 grid((unsigned)x, (unsigned)(share < 1 ? 1 : share < 256 ? share : 256));
  if (idx_bits == 32)
    window_plan_kernel<int32_t><<<grid, 128, 0, st>>>(static_cast<const int32_t*>(offsets), B, T,
                                                      row_start, row_end, counters, n_counters,
                                                      status);
  else
    window_plan_kernel<int64_t><<<grid, 128, 0, st>>>(static_cast<const int64_t*>(offsets), B, T,
                                                      row_start, row_end, counters, n_counters,
                                                      status);
  return cudaGetLastError() == cudaSuccess ? JCA_OK : JCA_ERR_CUDA;
}

}  // namespace jca

using namespace jca;

extern "C" size_t jca_window_workspace_bytes(int64_t B, int64_t T, int H, int Hkv, int d_head,
                                             int n_sinks) {
  if (!window_sizes_ok(B, T, H, Hkv, n_sinks) || !head_dim_ok(d_head)) return 0;
  return fwd_layout(T, d_head).total;
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
  const FwdLayout L = fwd_layout(T, d_head);
  if (workspace_bytes < L.total) return JCA_ERR_WORKSPACE;
  if (B == 0) return JCA_OK;
  int dev = 0, sms = 0;
  rc = current_device(&dev, &sms);
  if (rc) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  FwdArgs a = {};
  a.out = static_cast<bf16*>(out);
  a.lse = lse;
  a.valid = valid;
  a.row_start = reinterpret_cast<int32_t*>(ws + L.row_start);
  a.counter = reinterpret_cast<int32_t*>(ws + L.counter);
  a.spill = L.spills ? reinterpret_cast<float*>(ws + L.spill) : nullptr;
  a.status = status;
  a.T = (int)T;
  a.H = H;
  a.group = H / Hkv;
  a.window = (int)(window < T ? window : (T > 0 ? T : 1));
  a.n_sinks = n_sinks;
  a.item_ns = kWaitTimeoutNs + 20000ull * (uint64_t)(T / kTileN + 3);   // a key tile takes 2 us
  a.n_items = (int)((T + kItemRows - 1) / kItemRows) * H;
  a.out_v8 = aligned(out, 32) ? 1 : 0;
  a.scale_log2 = (scale > 0.f ? scale : 1.0f / sqrtf((float)d_head)) * 1.4426950408889634f;
  rc = window_plan(offsets, B, T, idx_bits, reinterpret_cast<int32_t*>(ws + L.row_start), nullptr,
                   a.counter, 1, status, st);
  if (rc || T == 0) return rc;
  // Only where a row can see more than kSpill key tiles: with the taking over in every instantiation
  // the others were 3 to 6 % slower (256 users 366 -> 389 us).
  const bool spills = (a.window + kItemRows) / kTileN + 3 > kSpill && L.spills;
  auto run = [&](auto fn) {
    return fn(a, q, k, v, Hkv, q_stride, k_stride, v_stride, dev, sms, st);
  };
  switch (d_head) {
    case 16: return spills ? run(launch_fwd<16, true>) : run(launch_fwd<16, false>);
    case 32: return spills ? run(launch_fwd<32, true>) : run(launch_fwd<32, false>);
    case 64: return spills ? run(launch_fwd<64, true>) : run(launch_fwd<64, false>);
    default: return spills ? run(launch_fwd<128, true>) : run(launch_fwd<128, false>);
  }
}
