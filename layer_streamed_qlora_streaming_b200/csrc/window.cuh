// Causal GQA attention with a sliding window and sinks (host interface). See window.cu.
#pragma once

#include "attention.cuh"

namespace lst {

// Key j of a sequence is visible to its query i when j <= i and (i - j < window or j < sinks).
struct WinArgs : AttnArgs {
  int window;  // >= 1
  int sinks;   // >= 0
};
struct WinBwdArgs : AttnBwdArgs {  // D: scratch of window_scratch() floats, D itself in front
  int window;
  int sinks;
};

bool window_shape_ok(int64_t T, int S, int hq, int hkv, int hd, int window, int sinks);
// fp32 values of scratch that window_bwd needs: D [T, hq], then what its dK / dV sums are split into.
int64_t window_scratch(int64_t T, int S, int hq, int hkv, int hd, int window, int sinks);

cudaError_t window_fwd(const WinArgs& a, cudaStream_t s);
cudaError_t window_bwd(const WinBwdArgs& a, cudaStream_t s);

}  // namespace lst
