// Shared by the forward and the backward of the windowed causal attention (not part of the ABI).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "jca.h"
#include "jca_device.cuh"

namespace jca {

constexpr int kWindowMaxSinks = 128;   // the visible first tokens of a user fit one key tile
constexpr int kMaxSms = 160;           // no persistent launch, or part of one, has more blocks

bool window_sizes_ok(int64_t B, int64_t T, int H, int Hkv, int n_sinks);

// Host argument checks of both entry points; JCA_OK or a negative code.
int window_check(int64_t B, int64_t T, int H, int Hkv, int d, int64_t window, int n_sinks,
                 int64_t q_stride, int64_t k_stride, int64_t v_stride, int idx_bits);

// Checks the offsets (JCA_STATUS_BAD_OFFSETS), writes the first row of each row's user and, unless
// null, one past its last, and zeroes the counters. No other check: callers validate first.
int window_plan(const void* offsets, int64_t B, int64_t T, int idx_bits, int32_t* row_start,
                int32_t* row_end, int32_t* counters, int n_counters, int32_t* status,
                cudaStream_t st);

// The kernels of a call follow one another by programmatic dependent launch: a kernel's blocks may be
// placed, and its barriers and TMEM set up, while the kernel before still runs. Every thread of a
// dependent kernel waits (grid_dep_wait) before its first access to global memory, until the kernel
// before is complete and its writes are visible; since that kernel waited for its own predecessor,
// the whole chain is then complete. A call's first kernel is launched in the ordinary way, behind
// everything that the stream held.
__device__ __forceinline__ void grid_dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the dependent kernel's blocks be placed once every block here has got this far.
__device__ __forceinline__ void grid_dep_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// A ring of entries in shared memory from which every role of a block takes its next piece of work.
struct Ring {
  volatile int* slot;
  uint32_t full, empty, k;
};

// Bits [a, b) of a word, for any a and b.
__device__ __forceinline__ uint32_t range_bits(int a, int b) {
  a = min(max(a, 0), 32);
  b = min(max(b, 0), 32);
  const uint32_t below_b = b >= 32 ? 0xffffffffu : (1u << b) - 1u;
  return a >= 32 ? 0u : below_b & (0xffffffffu << a);
}

// Zeroes the rows r0 + i of a tile for which bit i is set; one warp. A row's bytes of a column block (SW
// of them, blocks BLK bytes apart) are contiguous; the swizzle only reorders them. TWIN: also those of
// a tile so many bytes behind (in a second turn the padded gradient of 256 users took 4 % more).
template <int ROW_BYTES, int SW, int BLK, int TWIN = 0>
__device__ __forceinline__ void zero_rows(uint32_t tile, int r0, uint32_t rows, int lane) {
  constexpr int CH = ROW_BYTES / 16, CB = SW / 16;
#pragma unroll 1
  for (int i = lane; i < 32 * CH; i += 32) {
    const int r = i / CH, x = i % CH;
    if (!((rows >> r) & 1)) continue;
    const uint32_t at = tile + (x / CB) * BLK + (r0 + r) * SW + (x % CB) * 16;
    st_shared_v4(at, 0u, 0u, 0u, 0u);
    if (TWIN) st_shared_v4(at + TWIN, 0u, 0u, 0u, 0u);
  }
}

template <typename... Params, typename... Args>
int launch_dependent(void (*kernel)(Params...), int grid, int threads, size_t smem, cudaStream_t st,
                     const Args&... args) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, Params(args)...) == cudaSuccess) return JCA_OK;
  cudaGetLastError();
  return JCA_ERR_CUDA;
}

}  // namespace jca
