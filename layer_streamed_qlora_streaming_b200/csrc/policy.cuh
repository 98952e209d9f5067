// Clipped policy loss with a KL term (host interface). See policy.cu.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace lst {

// Per token t with mask_t != 0 (all when mask is null), logits row x_t, target y_t:
//   logp = x[y] - lse(x);  r = exp(logp - old);  u = min(r A, clip(r, 1 - lo, 1 + hi) A);
//   kl = exp(ref - logp) - (ref - logp) - 1;     l = -u + beta kl,
// (u = 0 where A = 0, no KL term where beta = 0, whatever overflows beside them), weighted by w_t of `norm` (0: m / sum m; 1: m / (nseq sum_seq m); 2: m / T).
struct PolicyArgs {
  const float* logits;  // rows [row0, row0 + rows) of [T, V]
  int64_t T;
  int V, S;             // S tokens a sequence, T a multiple of S
  const int32_t* y;     // [T], like the pointers below
  const float* old_logp;  // null: old = logp (r = 1)
  const float* ref_logp;  // null: no KL term
  const float* adv;       // [T], or [T / S] with adv_per_seq
  const int32_t* mask;    // null: every token counts
  float lo, hi, beta;
  int norm, adv_per_seq;
  float* logp;          // [T], 0 where masked
  float* out;           // [4]: sum of w times l, kl, [clipped], r
  __nv_bfloat16* dlog;  // rows [row0, row0 + rows) of [T, V], null: loss only
  float* scratch;       // policy_scratch() floats, 16-byte aligned
};

int64_t policy_scratch(int64_t T, int S);
constexpr int kPolicyMaxV = 1 << 20;
bool policy_cfg_ok(float lo, float hi, float beta, int norm);
bool policy_args_ok(const PolicyArgs& a);
// The call is policy_begin, then policy_rows over ranges of rows that cover [0, T) once; the last row
// to finish adds the terms of all rows up in a fixed order and writes out. The ranges may share one logits
// buffer. The results have the same bytes whatever the ranges, as long as V is a multiple of 4 and every range's
// logits lie alike in 16 bytes: a row's sum is added by its 16-byte slots.
// early: policy_begin is the launch right in front on the stream, so that the rows' loads need not wait for it.
cudaError_t policy_begin(const PolicyArgs& a, cudaStream_t s);
cudaError_t policy_rows(const PolicyArgs& a, int64_t row0, int64_t rows, bool early, cudaStream_t s);

}  // namespace lst
