// Shared by the forward and the backward of the windowed causal attention (not part of the ABI).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace jca {

constexpr int kWindowMaxSinks = 128;   // the visible first tokens of a user fit one key tile

bool window_sizes_ok(int64_t B, int64_t T, int H, int Hkv, int n_sinks);

// Host argument checks of both entry points; JCA_OK or a negative code.
int window_check(int64_t B, int64_t T, int H, int Hkv, int d, int64_t window, int n_sinks,
                 int64_t q_stride, int64_t k_stride, int64_t v_stride, int idx_bits);

// Checks the offsets (JCA_STATUS_BAD_OFFSETS), writes the first row of each row's user and, unless
// null, one past its last and the user's index, and zeroes the counters. No other check: callers validate first.
int window_plan(const void* offsets, int64_t B, int64_t T, int idx_bits, int32_t* row_start,
                int32_t* row_end, int32_t* row_user, int32_t* counters, int n_counters,
                int32_t* status, cudaStream_t st);

}  // namespace jca
