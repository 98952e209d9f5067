// Causal GQA attention with a sliding window and sinks (host interface). See window.cu.
#pragma once

#include "attention.cuh"

namespace lst {

// Key j of a sequence is visible to its query i when j <= i and (i - j < window or j < sinks).
struct WinArgs : AttnArgs {
  int window;     // >= 1
  int sinks;      // >= 0
  int parts = 1;  // bf16 values that hold a probability in P V: 1 (8 bits) or 2 (16 bits)
  int heads;   // T / S * hq, set by window_fwd (window_bwd)
};
struct WinBwdArgs : AttnBwdArgs {  // D: window_scratch() floats, 16-byte aligned
  int window;
  int sinks;
  int heads;
};

bool window_shape_ok(int64_t T, int S, int hq, int hkv, int hd, int window, int sinks);
// fp32 values of scratch that window_bwd needs: (lse, D) of every query, then what its dK / dV sums are
// split into.
int64_t window_scratch(int64_t T, int S, int hq, int hkv, int hd, int window, int sinks);

cudaError_t window_fwd(WinArgs a, cudaStream_t s);
cudaError_t window_bwd(WinBwdArgs a, cudaStream_t s);

}  // namespace lst
