// Clipped policy loss with a KL term, from logits to loss, log-probabilities and dlogits (the surrogate
// of Schulman et al., "Proximal Policy Optimization Algorithms", 2017, with the per-token KL estimate
// k3 of Shao et al., "DeepSeekMath", 2024; formulas in policy.cuh). Its gradient:
//   dl/dlogp = -r A [u is r A] + beta (1 - exp(ref - logp)),  dlogits = w dl/dlogp (onehot(y) - softmax(x)).
// Each logit crosses HBM once: a warp (k_policy_warp) or a cluster of CTAs (k_policy_cluster) holds a row in
// registers from its load to the store of dlogits; only rows too long for that are read twice (k_policy_rows).
#include "common.cuh"
#include "sync.cuh"
#include "pdl.cuh"
#include "ex2.cuh"
#include "policy.cuh"

#include <algorithm>

namespace lst {
namespace {

using bf16 = __nv_bfloat16;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ void bulk_store(uintptr_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"((uint64_t)dst), "r"(smem_u32(src)),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_store_wait() {  // this thread's bulk stores have been made
  asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group 0;" ::: "memory");
}
// 8 bytes into a cluster CTA's shared memory, counted by the mbarrier there
__device__ __forceinline__ void st_async_f2(uint32_t dst, float x, float y, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(dst), "f"(x),
               "f"(y), "r"(bar)
               : "memory");
}

// scratch: [0] rows done so far (as unsigned), then 4 floats a row, then the weight of each sequence's tokens
__host__ __device__ inline float* row_terms(float* scratch) { return scratch + 4; }
__host__ __device__ inline float* seq_weight(float* scratch, int64_t T) { return scratch + 4 + 4 * T; }

// A value from L2, loaded here and not next to its use.
__device__ __forceinline__ float load_cg(const float* p) {
  float v;
  asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}

// exp(d) - d - 1 without its cancellation near zero: the power series there
__device__ __forceinline__ float k3_term(float d) {
  if (fabsf(d) < 0.125f) {
    float t = 1.f / 720.f;
    t = fmaf(t, d, 1.f / 120.f);
    t = fmaf(t, d, 1.f / 24.f);
    t = fmaf(t, d, 1.f / 6.f);
    t = fmaf(t, d, 0.5f);
    return t * d * d;
  }
  return d < INFINITY ? expm1f(d) - d : d;
}

// One token's terms (l, kl, clipped, r) and dl/dlogp. Factors of zero take out what overflowed beside them: an
// advantage of 0 the ratio, a weight of 0 the KL term.
struct Token {
  float4 terms;
  float slope;
};
__device__ __forceinline__ Token policy_token(const PolicyArgs& a, float A, float old, float ref, float logp) {
  const float r = a.old_logp ? expf(logp - old) : 1.f;
  const float ra = A != 0.f ? r : 1.f, in = ra * A, cl = fminf(fmaxf(ra, 1.f - a.lo), 1.f + a.hi) * A;
  const bool cut = in > cl;  // the clip lowers the surrogate: no gradient
  float kl = 0.f, dkl = 0.f;
  if (a.ref_logp) {
    const float d = ref - logp;
    kl = k3_term(d);
    dkl = -expm1f(d);
  }
  const bool on = a.beta != 0.f;
  return {make_float4(fmaf(a.beta, on ? kl : 0.f, -(cut ? cl : in)), kl, cut ? 1.f : 0.f, r),
          fmaf(a.beta, on ? dkl : 0.f, cut ? 0.f : -in)};
}

// One CTA: counts the mask and leaves the weight of a counted token of each sequence. What is counted:
// the whole mask (mean over tokens), each sequence's (mean over sequences), nothing (fixed). A warp takes up
// to 256 tokens at a time, its loads independent; the counts are whole numbers, added in shared memory in
// any order. More sequences than fit there are counted by a warp each, or by a thread each where they are
// short (65536 sequences of one token: 2048 rounds of a load's latency by warps, 64 by threads).
constexpr int kSeqs = 1024;
__global__ void __launch_bounds__(1024) k_policy_weights(const int32_t* __restrict__ mask, int64_t T, int S, int norm,
                                                         float* __restrict__ scratch) {
  pdl_wait();
  pdl_trigger();
  __shared__ int count[kSeqs];
  float* w = seq_weight(scratch, T);
  const int nseq = (int)(T / S), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) reinterpret_cast<unsigned*>(scratch)[0] = 0;
  if (norm == 1 && nseq > kSeqs) {
    const bool wide = S >= 32;
    for (int64_t u = wide ? warp : (int)threadIdx.x; u < nseq; u += wide ? 32 : 1024) {
      int n = S;
      if (mask) {
        n = 0;
        for (int i = wide ? lane : 0; i < S; i += wide ? 32 : 1) n += mask[u * S + i] != 0;
        if (wide) n = __reduce_add_sync(0xffffffffu, n);
      }
      if (!wide || lane == 0) w[u] = n > 0 ? 1.f / ((float)nseq * (float)n) : 0.f;
    }
    return;
  }
  const int groups = norm == 0 ? 1 : norm == 1 ? nseq : 0, len = (int)(norm == 0 ? T : S);
  for (int b = threadIdx.x; b < groups; b += 1024) count[b] = 0;
  __syncthreads();
  const int parts = (int)(((int64_t)len + 255) / 256);
  for (int64_t u = warp; u < (int64_t)groups * parts; u += 32) {
    const int b = (int)(u / parts);
    const int64_t i0 = u % parts * 256, i1 = min((int64_t)len, i0 + 256);
    int n = 0;
    if (mask) {
      const int32_t* m = mask + (int64_t)b * len + i0;
      const int left = (int)(i1 - i0) - lane;
#pragma unroll
      for (int e = 0; e < 8; ++e) n += 32 * e < left && m[lane + 32 * e] != 0;
      n = __reduce_add_sync(0xffffffffu, n);
    } else {
      n = (int)(i1 - i0);
    }
    if (lane == 0) atomicAdd(&count[b], n);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < nseq; b += 1024) {
    const float n = norm == 2 ? (float)T : norm == 0 ? (float)count[0] : (float)nseq * (float)count[b];
    w[b] = n > 0.f ? 1.f / n : 0.f;
  }
}

// The maximum of a warp's values, none of them NaN, by their order as whole numbers: one instruction and not
// five shuffles, on the way that every row takes.
__device__ __forceinline__ float warp_max_of(float x) {
  const int i = __float_as_int(x), k = __reduce_max_sync(0xffffffffu, i ^ (i >> 31 & 0x7fffffff));
  return __int_as_float(k ^ (k >> 31 & 0x7fffffff));
}
// The sum of lanes 0 .. N - 1 (N a power of two), in them.
template <int N>
__device__ __forceinline__ float lane_sum(float x) {
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Once thread 0 has stored the terms of its `done` rows: the last CTA of the call to get here adds the
// terms of all rows in a fixed order (fp64) and writes out. For the first nt threads of a CTA (whole
// warps), all of them; part: 128 values of shared memory.
__device__ __forceinline__ void finish_rows(const PolicyArgs& a, int done, int nt, double* part) {
  __shared__ bool last;
  if (threadIdx.x == 0) {
    __threadfence();
    last = done > 0 && atomicAdd(reinterpret_cast<unsigned*>(a.scratch), (unsigned)done) + (unsigned)done == (unsigned)a.T;
  }
  named_sync(1, nt);
  if (!last) return;
  __threadfence();
  const float4* rows = reinterpret_cast<const float4*>(row_terms(a.scratch));
  double s[4] = {0, 0, 0, 0};
  constexpr int kAhead = 8;  // loads under way at once: one after another they take most of a call on many short rows
  for (int64_t i = threadIdx.x; i < a.T; i += kAhead * nt) {
    float4 v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) v[u] = i + u * nt < a.T ? __ldcg(rows + i + u * nt) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      s[0] += v[u].x;
      s[1] += v[u].y;
      s[2] += v[u].z;
      s[3] += v[u].w;
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    for (int o = 16; o > 0; o >>= 1) s[e] += __shfl_xor_sync(0xffffffffu, s[e], o);
    if ((threadIdx.x & 31) == 0) part[e * 32 + (threadIdx.x >> 5)] = s[e];
  }
  named_sync(1, nt);
  if (threadIdx.x < 4) {
    double v = 0;
    for (int i = 0; i < (nt >> 5); ++i) v += part[threadIdx.x * 32 + i];
    a.out[threadIdx.x] = (float)v;
  }
}

// One counted row's scalars, brought in ahead of it; lrow < 0 ends the rows.
struct RowInfo {
  int64_t lrow;
  int y;
  float xy, adv, old, ref;
};
constexpr int kZeroBytes = 1024;

// Persistent clusters of cs CTAs, cluster g taking rows g, g + clusters, ... CTA z owns slots
// [z * slice, (z + 1) * slice) of a row's 16-byte slots (slot i: logits 4 i - off .. 4 i - off + 3, off =
// how far the row starts behind a 16-byte boundary).
//  - The last warp is the producer: it reads the scalars of 32 rows at once, a lane each. A row that
//    does not count it finishes by itself, by bulk stores from a kilobyte of zeros. A counted row's slice it
//    brings into shared memory by bulk copies, in two halves of a ring of three. The consumers take a
//    half to registers at once, so up to one and a half rows are in flight under a row's arithmetic,
//    exchange and stores.
//  - A consumer warp holds 32 NV / 2 neighbouring slots of each half, lane by lane, 4 NV logits a thread: NV large
//    and the threads few, so that two slices fit an SM's registers without spills. With m its own
//    maximum it forms e = 2^((x - m) log2 e) once; maxima and sums are merged by warp, CTA and cluster
//    (st.async of each CTA's pair into its peers, onto their mbarrier), in a fixed order; the row's
//    factor coef 2^((m - lse) log2 e) then turns e into dlogits with one product.
// Each logit crosses HBM once and takes one exponential. Bound by HBM: 4 + 2 bytes a logit, 2 bytes on rows that
// do not count: 4096 rows of 151936 logits, most of them counted, take 442 to 458 us from card to card, 0.92 to 0.95 of the
// rate of a plain copy; 2048 rows of 128256 250 us (0.97), with half of them counted 179 us (0.90); 999 rows of 32003, of which
// less than half count, 25 us (0.57): a few rows a cluster, each a chain of load, exchange and stores.
// (A CTA a row, read twice: 3896 us for the first, 1461 for the half counted, 75 for the last. The slots of a thread
// as many apart as there are threads, each looked at: 2048 counted rows took 337 us instead of 265. dlogits by bulk
// stores through shared memory, which leaves two halves to load into: 358. Rows in an order that mixes counted
// ones with others: the half counted 196 instead of 190. Slices of half the size, on twice the CTAs: 8192 rows of
// 32000 take 322 us instead of 301.)
// ALIGNED: every row starts and ends with a slot (V a multiple of 4, the logits 16-byte aligned). Told apart for the
// code around the stores: with the ends' code in it, 2048 rows of 128256 take 278 us instead of 250; without it,
// each slot looked at, 4096 rows of 50257 take 257 us instead of 236.
template <int NV, int THREADS, int PER_SM, bool ALIGNED>
__global__ void __launch_bounds__(THREADS, PER_SM)
k_policy_cluster(const PolicyArgs a, int64_t row0, int64_t rows, int slice, int early) {
  static_assert(NV % 2 == 0 && kZeroBytes >= 128 * 8, "two halves; the zeros' space is reused");
  constexpr int kRun = 32 * (NV / 2);  // slots of a warp in each half
  extern __shared__ __align__(16) float ring[];  // three halves of a slice
  __shared__ __align__(16) uint8_t zeros[kZeroBytes];
  __shared__ uint64_t full[3], empty[3], pair_bar[2];
  // by counted row: rewritten for the fourth row after it, which waits for a buffer that the consumers
  // free behind this row
  __shared__ RowInfo info[4];
  __shared__ float2 pair[2][8];  // (max, sum) of each CTA of the cluster, by row parity
  __shared__ float2 wpair[32];   // of each warp of this CTA
  __shared__ float2 factor;      // lse and the row's coefficient
  const int cs = (int)cluster_size_x(), z = (int)cluster_rank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nc = (int)blockDim.x - 32, ncw = nc >> 5;  // consumers
  const int half = (slice + 1) / 2;
  const int64_t clusters = gridDim.x / cs, first = blockIdx.x / cs;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 3; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], (uint32_t)ncw);
    }
    mbar_init(&pair_bar[0], 1);
    mbar_init(&pair_bar[1], 1);
    fence_mbar_init();
  }
  for (int i = threadIdx.x; i < kZeroBytes / 4; i += blockDim.x) reinterpret_cast<uint32_t*>(zeros)[i] = 0;
  fence_proxy_async();  // the zeros are read by bulk stores
  __syncthreads();
  cluster_sync_all();  // every CTA's barriers are set up before a peer's pair can arrive
  // early: the kernel in front is k_policy_weights, which lets this one start once its own predecessors
  // have completed. All that it leaves is read by thread 0, which waits for it there.
  if (!early) pdl_wait();
  pdl_trigger();

  if (warp == ncw) {  // producer
    int it = 0, g = 0;  // counted rows, halves
    bool ok = true;
    const auto claim = [&] {  // the next buffer of the ring, once it is free
      if (g >= 3 && !__all_sync(0xffffffffu, mbar_wait(&empty[g % 3], (g / 3 - 1) & 1))) ok = false;
      return ok;
    };
    for (int64_t base = first; base < rows && ok; base += 32 * clusters) {
      const int64_t mine = base + lane * clusters;
      RowInfo r{mine, 0, 0.f, 0.f, 0.f, 0.f};
      bool live = false;
      if (mine < rows) {
        const int64_t t = row0 + mine;
        r.y = a.y[t];
        live = !a.mask || a.mask[t] != 0;
        if (live && (r.y < 0 || r.y >= a.V)) {
          if (z == 0) dev_fail(DEV_ERR_BAD_INDEX);
          live = false;
        }
        if (live) {
          r.xy = a.logits[mine * a.V + r.y];
          r.adv = a.adv[a.adv_per_seq ? t / a.S : t];
          r.old = a.old_logp ? a.old_logp[t] : 0.f;
          r.ref = a.ref_logp ? a.ref_logp[t] : 0.f;
        } else if (z == 0) {
          a.logp[t] = 0.f;
          reinterpret_cast<float4*>(row_terms(a.scratch))[t] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
      const uint32_t lives = __ballot_sync(0xffffffffu, live);
      for (int i = 0; i < 32 && ok; ++i) {
        const int64_t lrow = base + i * clusters;
        if (lrow >= rows) break;
        if (!(lives >> i & 1)) {  // zeros to this CTA's part of the row, whole 16 bytes of it by bulk stores
          if (a.dlog) {
            const int64_t per = (a.V + cs - 1) / cs;
            const bf16* d0 = a.dlog + lrow * a.V + min((int64_t)a.V, z * per);
            const bf16* d1 = a.dlog + lrow * a.V + min((int64_t)a.V, (z + 1) * per);
            const uintptr_t p0 = reinterpret_cast<uintptr_t>(d0), p1 = reinterpret_cast<uintptr_t>(d1);
            uintptr_t q0 = (p0 + 15) & ~uintptr_t(15), q1 = p1 & ~uintptr_t(15);
            if (q0 > q1) q0 = q1 = p1;
            if (p0 + 2 * lane < min(q0, p1)) *reinterpret_cast<bf16*>(p0 + 2 * lane) = __float2bfloat16_rn(0.f);
            if (max(q1, p0) + 2 * lane < p1) *reinterpret_cast<bf16*>(max(q1, p0) + 2 * lane) = __float2bfloat16_rn(0.f);
            for (uintptr_t q = q0 + lane * kZeroBytes; q < q1; q += 32 * kZeroBytes)
              bulk_store(q, zeros, (uint32_t)min((uintptr_t)kZeroBytes, q1 - q));
          }
          continue;
        }
        const float* x = a.logits + lrow * a.V;
        const int off = ALIGNED ? 0 : (int)(reinterpret_cast<uintptr_t>(x) >> 2) & 3, end = (a.V + off + 3) / 4;
        for (int h = 0; h < 2 && claim(); ++h, ++g) {
          const int k = g % 3;
          if (h == 0 && lane == i) info[it & 3] = r;
          float* buf = ring + 4 * k * half;
          const int b = z * slice + h * half, e = min(min(b + half, (z + 1) * slice), end);
          // [lo, hi): slots without a logit of a neighbouring row; the row's first and last slot may have
          // one and are filled in by hand then
          const int lo = max(b, off ? 1 : 0), hi = min(e, (a.V + off) / 4);
          for (int c = b; c < e; c = c < lo ? lo : max(c + 1, hi)) {
            if (c >= lo && c < hi) continue;
            const int at = 4 * c - off + lane;
            if (lane < 4) buf[4 * (c - b) + lane] = at >= 0 && at < a.V ? x[at] : -INFINITY;
            if (!ALIGNED) fence_proxy_async();  // a later row's bulk copy writes where these stores have written
          }
          __syncwarp();
          if (lane == 0) {
            if (hi > lo) {
              mbar_arrive_expect_tx(&full[k], (uint32_t)(hi - lo) * 16);
              const int q = (hi - lo + 1) / 2;
              for (int c = lo; c < hi; c += q)
                bulk_load(buf + 4 * (c - b), x + (4 * c - off), (uint32_t)min(q, hi - c) * 16, &full[k]);
            } else {
              mbar_arrive(&full[k]);
            }
          }
        }
        ++it;
      }
    }
    bulk_store_wait();
    __syncwarp();  // with the row terms of the other lanes, too, in front of the arrival
    if (ok && claim()) {  // (the zeros are the consumers' from here on)
      if (lane == 0) {
        info[it & 3].lrow = -1;
        mbar_arrive(&full[g % 3]);
      }
    }
    __syncwarp();
    cluster_sync_all();
    return;
  }

  if (threadIdx.x == 0) pdl_wait();
  int it = 0, g = 0;  // counted rows, halves
  bool ok = true;
  for (; ok; ++it) {
    if (!mbar_wait(&full[g % 3], (g / 3) & 1)) {  // for every consumer alike: the phase does not end
      ok = false;
      break;
    }
    const int64_t lrow = info[it & 3].lrow, t = row0 + lrow;
    if (lrow < 0) break;
    const int y = info[it & 3].y;
    const float* x = a.logits + lrow * a.V;
    bf16* d = a.dlog ? a.dlog + lrow * a.V : nullptr;
    const int off = ALIGNED ? 0 : (int)(reinterpret_cast<uintptr_t>(x) >> 2) & 3;
    const int b = z * slice, s1 = min((a.V + off + 3) / 4, b + slice);
    const bool dvec = (reinterpret_cast<uintptr_t>(d - off) & 7) == 0;
    float w = 0.f;  // thread 0: the row's weight, under the arithmetic
    if (threadIdx.x == 0) w = load_cg(seq_weight(a.scratch, a.T) + (uint32_t)t / (uint32_t)a.S);
    float v[4 * NV];
    // this thread's first slot of each half, and the half's slots from there on
    const int at[2] = {warp * kRun + lane, half + warp * kRun + lane};
    const int left[2] = {min(half, s1 - b) - at[0], s1 - b - at[1]};
#pragma unroll
    for (int h = 0; h < 2; ++h, ++g) {
      if (h == 1 && !mbar_wait(&full[g % 3], (g / 3) & 1)) ok = false;
      const float4* src = reinterpret_cast<const float4*>(ring + 4 * (g % 3) * half) + at[0];
#pragma unroll
      for (int n = 0; n < NV / 2; ++n) {
        float4 q = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (32 * n < left[h]) q = src[32 * n];
        float* o = v + 4 * (h * (NV / 2) + n);
        o[0] = q.x;
        o[1] = q.y;
        o[2] = q.z;
        o[3] = q.w;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[g % 3]);
    }
    // everything in units of log2: e = 2^(x log2 e - m), m the thread's rounded maximum; what matters is
    // that one m is used throughout (a thread without a finite logit takes 0 and adds zeros)
    float m4[4] = {v[0], v[1], v[2], v[3]}, s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int n = 4; n < 4 * NV; ++n) m4[n & 3] = fmaxf(m4[n & 3], v[n]);
    float m = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
    m = m > -INFINITY ? m * kLog2e : 0.f;
#pragma unroll
    for (int n = 0; n < 4 * NV; ++n) {
      v[n] = ex2_approx(fmaf(v[n], kLog2e, -m));
      s4[n & 3] += v[n];
    }
    const float s = (s4[0] + s4[1]) + (s4[2] + s4[3]);
    if (s == 0.f) m = -INFINITY;
    const float wm = warp_max_of(m);
    const float ws = warp_sum(m > -INFINITY ? s * ex2_approx(m - wm) : s);
    if (lane == 0) wpair[warp] = make_float2(wm, ws);
    named_sync(1, nc);
    if (warp == 0) {
      float2 p = lane < ncw ? wpair[lane] : make_float2(-INFINITY, 0.f);
      float rm = warp_max_of(p.x);
      float rs = lane_sum<16>(p.x > -INFINITY ? p.y * ex2_approx(p.x - rm) : p.y);
      if (cs > 1) {
        const int k = it & 1;
        if (lane == 0) mbar_arrive_expect_tx(&pair_bar[k], (uint32_t)cs * 8);
        if (lane < cs)
          st_async_f2(cluster_map(smem_u32(&pair[k][z]), (uint32_t)lane), rm, rs,
                      cluster_map(smem_u32(&pair_bar[k]), (uint32_t)lane));
        if (!mbar_wait(&pair_bar[k], (it >> 1) & 1)) ok = false;
        p = lane < cs ? pair[k][lane] : make_float2(-INFINITY, 0.f);
        rm = warp_max_of(p.x);
        rs = lane_sum<8>(p.x > -INFINITY ? p.y * ex2_approx(p.x - rm) : p.y);
      }
      if (lane == 0) {
        const RowInfo& r = info[it & 3];
        const float l2 = log2f(rs), logp = (fmaf(r.xy, kLog2e, -rm) - l2) * kLn2;
        const Token k = policy_token(a, r.adv, r.old, r.ref, logp);
        factor = make_float2(rm + l2, -w * k.slope);
        if (z == 0) {
          a.logp[t] = logp;
          reinterpret_cast<float4*>(row_terms(a.scratch))[t] =
              make_float4(w * k.terms.x, w * k.terms.y, w * k.terms.z, w * k.terms.w);
        }
      }
    }
    ok = sync_all(1, nc, ok);  // a lost pair ends the loop for every consumer
    if (!d) continue;
    const float lse2 = factor.x, coef = factor.y, f = coef * ex2_approx(m - lse2);
    const auto packed = [&](int n) {
      const __nv_bfloat162 lo = __floats2bfloat162_rn(v[4 * n] * f, v[4 * n + 1] * f);
      const __nv_bfloat162 hi = __floats2bfloat162_rn(v[4 * n + 2] * f, v[4 * n + 3] * f);
      return make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    };
    const int ys = (y + off) / 4 - b;
    // slots [f0, f1) of the slice are all this row's
    const int f0 = !ALIGNED && b == 0 && off ? 1 : 0, f1 = ALIGNED ? s1 - b : min(s1, (a.V + off) / 4) - b;
    if (dvec) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint2* dst = reinterpret_cast<uint2*>(d + 4 * (b + at[h]) - off);
        const int full = ALIGNED ? left[h] : (h ? f1 : min(half, f1)) - at[h];
#pragma unroll
        for (int n = 0; n < NV / 2; ++n) {
          const uint2 g4 = packed(h * (NV / 2) + n);
          if (32 * n < full && (n > 0 || at[h] >= f0)) dst[32 * n] = g4;
        }
      }
      if (!ALIGNED && warp == 0 && lane < 8) {  // the row's ends one by one
        const int c = lane < 4 ? lane : 4 * (b + f1) - off + lane - 4;
        if (lane < 4 ? f0 == 1 && lane < 4 - off && lane < a.V : f1 < s1 - b && c >= 0 && c < a.V)
          d[c] = __float2bfloat16_rn(coef * (ex2_approx(fmaf(x[c], kLog2e, -lse2)) - (c == y ? 1.f : 0.f)));
      }
    } else {  // dlogits that lie otherwise than the logits modulo 16 bytes
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const int h = n / (NV / 2), k = 32 * (n - h * (NV / 2));
        const uint2 g4 = packed(n);
        if (k >= left[h]) continue;
        const int c = 4 * (b + at[h] + k) - off;
        const bf16* q = reinterpret_cast<const bf16*>(&g4);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + e >= 0 && c + e < a.V) d[c + e] = q[e];
      }
    }
    // the target's own element, by the thread that has just stored its slot
    const int yh = ys < half ? ys : ys - half;  // its place in its half
    if (ys >= (dvec ? f0 : 0) && ys < (dvec ? f1 : slice) && yh / kRun == warp && yh % 32 == lane)
      d[y] = __float2bfloat16_rn(coef * (ex2_approx(fmaf(info[it & 3].xy, kLog2e, -lse2)) - 1.f));
  }
  if (z == 0 && ok)
    finish_rows(a, (int)((rows - first + clusters - 1) / clusters), nc, reinterpret_cast<double*>(zeros));
  __syncwarp();
  cluster_sync_all();  // no CTA leaves before its peers have their pairs
}

// Short rows, a warp each (slots as above, slot lane + 32 k in the lane's registers): no exchange, and as many
// rows in flight as the warps of all SMs. Bound by latency (a row's loads and merge, then the sum of the rows'
// terms): 128 rows of 512 logits 6.1 us, where clusters take 8.4; 3344 rows of 1427 14.5 against 25, of 4000
// (the longest: 32 slots a lane leave three CTAs an SM) 21 against 27.
template <int NV>
__global__ void __launch_bounds__(128, NV <= 4 ? 10 : NV <= 16 ? 5 : 3) k_policy_warp(const PolicyArgs a, int64_t row0, int64_t rows, int early) {
  if (!early) pdl_wait();
  pdl_trigger();
  __shared__ double part[128];
  const int lane = threadIdx.x & 31;
  const int64_t lrow = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5), t = row0 + lrow;
  if (lrow < rows) {
    const float* x = a.logits + lrow * a.V;
    bf16* d = a.dlog ? a.dlog + lrow * a.V : nullptr;
    const int off = (int)(reinterpret_cast<uintptr_t>(x) >> 2) & 3, n = (a.V + off + 3) / 4;
    const bool dvec = (reinterpret_cast<uintptr_t>(d - off) & 7) == 0;
    const int y = a.y[t];
    bool live = !a.mask || a.mask[t] != 0;
    if (live && (y < 0 || y >= a.V)) {
      if (lane == 0) dev_fail(DEV_ERR_BAD_INDEX);
      live = false;
    }
    float v[4 * NV], m = 0.f, lse2 = 0.f, coef = 0.f, xy = 0.f;
    if (live) {
      const int seq = (int)((uint32_t)t / (uint32_t)a.S);
      const float adv = a.adv[a.adv_per_seq ? seq : t], old = a.old_logp ? a.old_logp[t] : 0.f;
      const float ref = a.ref_logp ? a.ref_logp[t] : 0.f;
      xy = x[y];
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int i = lane + 32 * k, c = 4 * i - off;
        float4 q = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (i < n) {
          if (c >= 0 && c + 4 <= a.V) {
            q = *reinterpret_cast<const float4*>(x + c);
          } else {
            if (c >= 0) q.x = x[c];
            if (c + 1 >= 0 && c + 1 < a.V) q.y = x[c + 1];
            if (c + 2 >= 0 && c + 2 < a.V) q.z = x[c + 2];
            if (c + 3 < a.V) q.w = x[c + 3];
          }
        }
        v[4 * k] = q.x, v[4 * k + 1] = q.y, v[4 * k + 2] = q.z, v[4 * k + 3] = q.w;
      }
      float m4[4] = {v[0], v[1], v[2], v[3]}, s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 4; k < 4 * NV; ++k) m4[k & 3] = fmaxf(m4[k & 3], v[k]);
      m = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
      m = m > -INFINITY ? m * kLog2e : 0.f;
#pragma unroll
      for (int k = 0; k < 4 * NV; ++k) {
        v[k] = ex2_approx(fmaf(v[k], kLog2e, -m));
        s4[k & 3] += v[k];
      }
      const float s = (s4[0] + s4[1]) + (s4[2] + s4[3]);
      if (s == 0.f) m = -INFINITY;
      const float rm = warp_max_of(m), l2 = log2f(lane_sum<32>(m > -INFINITY ? s * ex2_approx(m - rm) : s));
      lse2 = rm + l2;
      const float logp = (fmaf(xy, kLog2e, -rm) - l2) * kLn2;
      const Token k = policy_token(a, adv, old, ref, logp);
      pdl_wait();
      const float w = load_cg(seq_weight(a.scratch, a.T) + seq);
      coef = -w * k.slope;
      if (lane == 0) {
        a.logp[t] = logp;
        reinterpret_cast<float4*>(row_terms(a.scratch))[t] =
            make_float4(w * k.terms.x, w * k.terms.y, w * k.terms.z, w * k.terms.w);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4 * NV; ++k) v[k] = 0.f;
      if (lane == 0) {
        a.logp[t] = 0.f;
        reinterpret_cast<float4*>(row_terms(a.scratch))[t] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
    if (d) {
      const float f = live ? coef * ex2_approx(m - lse2) : 0.f;
      const bf16 gy = __float2bfloat16_rn(coef * (ex2_approx(fmaf(xy, kLog2e, -lse2)) - 1.f));
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int i = lane + 32 * k, c = 4 * i - off;
        if (i >= n) continue;
        bf16 g[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) g[e] = live && c + e == y ? gy : __float2bfloat16_rn(v[4 * k + e] * f);
        if (dvec && c >= 0 && c + 4 <= a.V) {
          const __nv_bfloat162 lo(g[0], g[1]), hi(g[2], g[3]);
          *reinterpret_cast<uint2*>(d + c) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (c + e >= 0 && c + e < a.V) d[c + e] = g[e];
        }
      }
    }
  }
  pdl_wait();  // the count of rows done is set to zero in front
  __syncthreads();
  finish_rows(a, (int)min((int64_t)4, rows - (int64_t)blockIdx.x * 4), 128, part);
}

// Rows longer than a cluster's registers (V above 300,000): one CTA a row, read twice.
__global__ void __launch_bounds__(512) k_policy_rows(const PolicyArgs a, int64_t row0) {
  pdl_wait();
  pdl_trigger();
  __shared__ float red[16];
  __shared__ float coef_s;
  __shared__ double part[128];
  const int64_t lrow = blockIdx.x, t = row0 + lrow;
  const float* x = a.logits + lrow * a.V;
  bf16* d = a.dlog ? a.dlog + lrow * a.V : nullptr;
  const int y = a.y[t];
  const bool counted = !a.mask || a.mask[t] != 0;
  const bool bad = counted && (y < 0 || y >= a.V);
  if (bad && threadIdx.x == 0) dev_fail(DEV_ERR_BAD_INDEX);
  if (!counted || bad) {
    if (d)
      for (int c = threadIdx.x; c < a.V; c += blockDim.x) d[c] = __float2bfloat16_rn(0.f);
    if (threadIdx.x == 0) {
      a.logp[t] = 0.f;
      reinterpret_cast<float4*>(row_terms(a.scratch))[t] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    finish_rows(a, 1, blockDim.x, part);
    return;
  }
  float m = -INFINITY, s = 0.f;
  for (int c = threadIdx.x; c < a.V; c += blockDim.x) m = fmaxf(m, x[c]);
  m = warp_max(m);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
  for (int i = 0; i < (int)(blockDim.x >> 5); ++i) m = fmaxf(m, red[i]);
  for (int c = threadIdx.x; c < a.V; c += blockDim.x) s += expf(x[c] - m);
  s = warp_sum(s);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  s = 0.f;
  for (int i = 0; i < (int)(blockDim.x >> 5); ++i) s += red[i];
  const float ls = logf(s);
  if (threadIdx.x == 0) {
    const float logp = (x[y] - m) - ls;
    const Token k = policy_token(a, a.adv[a.adv_per_seq ? t / a.S : t], a.old_logp ? a.old_logp[t] : 0.f,
                                 a.ref_logp ? a.ref_logp[t] : 0.f, logp);
    const float w = seq_weight(a.scratch, a.T)[t / a.S];
    a.logp[t] = logp;
    coef_s = -w * k.slope;
    reinterpret_cast<float4*>(row_terms(a.scratch))[t] =
        make_float4(w * k.terms.x, w * k.terms.y, w * k.terms.z, w * k.terms.w);
  }
  __syncthreads();
  if (d) {
    const float coef = coef_s;
    for (int c = threadIdx.x; c < a.V; c += blockDim.x) {
      const float p = expf(x[c] - m - ls);
      d[c] = __float2bfloat16_rn(coef * (c == y ? p - 1.f : p));
    }
  }
  finish_rows(a, 1, blockDim.x, part);
}

// As many clusters as are resident at once (they take the rows in turn), at most one a row.
template <int NV, int THREADS, int PER_SM, bool ALIGNED>
cudaError_t launch_cluster_as(const PolicyArgs& a, int64_t row0, int64_t rows, int cs, int slice, bool early,
                              cudaStream_t s) {
  const auto kernel = k_policy_cluster<NV, THREADS, PER_SM, ALIGNED>;
  const int half = (slice + 1) / 2;
  const int run = 32 * (NV / 2), threads = std::max(1, (half + run - 1) / run) * 32 + 32, smem = 3 * half * 16;
  static std::atomic<unsigned long long> attr_done{0};
  if (!done_on_device(attr_done)) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               std::min((THREADS - 32) * NV / 2 * 3 * 16, 224 * 1024));
    if (e != cudaSuccess) return e;
    mark_done_on_device(attr_done);
  }
  struct Fit {
    int device, cs, slice, clusters;
  };
  static thread_local Fit fit{-1, 0, 0, 0};  // of this thread's last call
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (fit.device != dev || fit.cs != cs || fit.slice != slice) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)cs);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)cs;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    if ((e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg)) != cudaSuccess) return e;
    fit = Fit{dev, cs, slice, std::max(1, n)};
  }
  const int64_t clusters = std::min<int64_t>(rows, fit.clusters);
  return launch_k(kernel, dim3((unsigned)(clusters * cs)), dim3((unsigned)threads), (size_t)smem, s, (unsigned)cs, a, row0,
                  rows, slice, early ? 1 : 0);
}

// Every row starts and ends with a 16-byte slot.
bool rows_aligned(const PolicyArgs& a) { return a.V % 4 == 0 && (reinterpret_cast<uintptr_t>(a.logits) & 15) == 0; }

// PER_SM, PER_SM_U: CTAs an SM where rows are aligned and where they are not.
template <int NV, int THREADS, int PER_SM, int PER_SM_U = PER_SM>
cudaError_t launch_cluster(const PolicyArgs& a, int64_t row0, int64_t rows, int cs, int slice, bool early,
                           cudaStream_t s) {
  return rows_aligned(a)
             ? launch_cluster_as<NV, THREADS, PER_SM, true>(a, row0, rows, cs, slice, early, s)
             : launch_cluster_as<NV, THREADS, PER_SM_U, false>(a, row0, rows, cs, slice, early, s);
}

}  // namespace

int64_t policy_scratch(int64_t T, int S) { return 4 + 4 * T + T / S; }

bool policy_cfg_ok(float lo, float hi, float beta, int norm) {
  return lo >= 0.f && lo <= 1.f && hi >= 0.f && beta >= 0.f && beta < INFINITY && norm >= 0 && norm <= 2;
}

bool policy_args_ok(const PolicyArgs& a) {
  return a.T > 0 && a.T <= INT32_MAX && a.V > 0 && a.V <= kPolicyMaxV && a.S > 0 && a.T % a.S == 0 &&
         policy_cfg_ok(a.lo, a.hi, a.beta, a.norm) && (a.beta == 0.f || a.ref_logp);
}

cudaError_t policy_begin(const PolicyArgs& a, cudaStream_t s) {
  if (!policy_args_ok(a)) return cudaErrorInvalidValue;
  const cudaError_t e = launch_k(k_policy_weights, dim3(1), dim3(1024), 0, s, 0, a.mask, a.T, a.S, a.norm, a.scratch);
  note_launch(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t policy_rows(const PolicyArgs& a, int64_t row0, int64_t rows, bool early, cudaStream_t s) {
  if (!policy_args_ok(a) || row0 < 0 || rows <= 0 || row0 + rows > a.T) return cudaErrorInvalidValue;
  // A warp takes up to 1024 slots, in registers for 4, 16 or 32 a lane (3344 rows of 500 logits 10 us, of 4000 21 us;
  // by clusters 29 and 27). A CTA of a cluster takes up to 4750 slots (224 consumers of 22, three half slices of
  // shared memory), two CTAs an SM. A few rows are spread further, so that every SM has some of them, and a
  // shorter slice is a shorter chain for a row. All of it goes by the call's rows, not by this range's: the order in
  // which a row's sum and the rows' terms are added follows from it, and is the same however the rows are cut.
  const int slots = (a.V + 6) / 4;
  int cs = 1;
  while (cs < 8 && ((slots + cs - 1) / cs > 4750 || (a.T * cs < 2 * device_sm_count() && slots / cs > 1024))) cs *= 2;
  const int slice = (slots + cs - 1) / cs;
  // Short slices are held by threads of 6 slots, four CTAs an SM, up to what those hold, 1536 (3000 rows of 4100 logits
  // 20.7 us, of 6136 25.3, 48 rows of 9000 7.8; by threads of 22 slots 21.7, 25.5 and 8.5). Where rows are not aligned,
  // whose code needs more registers, three an SM and only to 1152 (3000 rows of 4099 logits 22.1 us against 23.5, 48
  // rows of 9001 7.9 against 8.8; with longer slices 3000 rows of 5003 took 26.1 against 24.1, of 6131 29.2 against 28.4;
  // at four an SM, with spills, 25.2 and 29.0).
  const int small = rows_aligned(a) ? 1536 : 1152;
  cudaError_t e;
  const auto warps = [&](auto kernel) {
    return launch_k(kernel, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, s, 0, a, row0, rows, early ? 1 : 0);
  };
  if (slots <= 32 * 4) e = warps(k_policy_warp<4>);
  else if (slots <= 32 * 16) e = warps(k_policy_warp<16>);
  else if (slots <= 32 * 32) e = warps(k_policy_warp<32>);
  else if (slice <= small) e = launch_cluster<6, 288, 4, 3>(a, row0, rows, cs, slice, early, s);
  else if (slice <= 4750) e = launch_cluster<22, 256, 2>(a, row0, rows, cs, slice, early, s);
  else if (slice <= 9400) e = launch_cluster<22, 512, 1>(a, row0, rows, cs, slice, early, s);
  else e = launch_k(k_policy_rows, dim3((unsigned)rows), dim3(512), 0, s, 0, a, row0);
  note_launch(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace lst
