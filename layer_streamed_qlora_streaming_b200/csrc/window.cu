// Causal GQA attention with a sliding window and sinks: key j of a sequence is visible to its query
// i when j <= i and (i - j < window or j < sinks).
//   s_ij = q_i . k_j / sqrt(hd),  P = softmax of s over the visible keys,  o_i = sum_j P_ij v_j,
//   lse_i = log sum_j exp s_ij;
//   D_i = do_i . o_i,  dS_ij = P_ij (do_i . v_j - D_i),
//   dq_i = sum_j dS_ij k_j / sqrt(hd),  dk_j = sum_{h, i} dS_ij q_i / sqrt(hd),  dv_j = sum_{h, i} P_ij do_i,
// the last two over the query heads h that share the kv head.
//
// Three kernels on tcgen05 (bf16 operands, fp32 in TMEM), each walking only the tiles that hold a
// visible pair: the forward, dQ (which forms D first), and dK / dV, whose sums over heads and queries
// are split over CTAs where there would be too few, or, for the keys that are sinks, too long ones.
// Tiles come by 3D TMA maps (column, row of the sequence, sequence): rows behind a sequence read as
// zeros, never as the next sequence. P and dS are rounded to bf16 as operands (half a step of 2^-8
// relative, independent of the output's own rounding); everything else is fp32.
#include "common.cuh"
#include "pdl.cuh"
#include "ex2.cuh"
#include "gemm.cuh"
#include "window.cuh"

#include <algorithm>
#include <cudaTypedefs.h>
#include <type_traits>

namespace lst {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn();  // gemm.cu

namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kQB = 128;  // rows of a query tile (the TMEM lanes), and of a key tile

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// D += A B with A [128, 16] bf16 in TMEM (two values a column, row = lane) and B by descriptor
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t db, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(db), "r"(idesc), "r"(accumulate)
      : "memory");
}
// The descriptor of a tile `bytes` further. Descriptors are made once a block: building two for every MMA
// cost the issuing thread about 110 cycles each, of the 64 that an MMA of 128 x 128 x 16 takes.
__device__ __forceinline__ uint64_t at(uint64_t desc, uint32_t bytes) { return desc + (bytes >> 4); }
// True for one lane of a converged warp, always the same one. The TMA and MMA warps run their loops with all
// lanes and issue under this, so that no lane runs ahead while the instructions' uniform operands live.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// Wait of a whole warp; false (for all of it) once it ran out.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

__host__ __device__ __forceinline__ int up(int a, int b) { return (a + b - 1) / b * b; }

// The key blocks that the queries [q0, q0 + 128) of a sequence see, in order: sinks in front of the
// window's first block, then the window's blocks. A block starts at a multiple of 128; its width is a
// multiple of 16 that covers its last visible key.
struct Blocks {
  int nsink, n, jb0, front, end;
  __device__ __forceinline__ Blocks(int q0, int S, int window, int sinks) {
    const int w0 = max(0, q0 - window + 1);
    jb0 = w0 / kQB;
    front = min(sinks, jb0 * kQB);  // sinks that the window's blocks do not hold
    nsink = (front + kQB - 1) / kQB;
    end = min(S, q0 + kQB);
    n = nsink + (end + kQB - 1) / kQB - jb0;
  }
  __device__ __forceinline__ int k0(int j) const { return (j < nsink ? j : jb0 + j - nsink) * kQB; }
  __device__ __forceinline__ int width(int j) const {
    const int left = (j < nsink ? front : end) - k0(j);
    return left >= kQB ? kQB : up(left, 16);
  }
};
// every pair of queries [q0, q0 + nq) and keys [k0, k0 + nk) is visible
__device__ __forceinline__ bool all_visible(int q0, int nq, int k0, int nk, int window, int sinks) {
  return k0 + nk - 1 <= q0 && (q0 + nq - 1 - k0 < window || k0 + nk <= sinks);
}

// rows [row, row + rows) of a [S, 64 CHUNKS] tile column block as CHUNKS swizzled tiles of `chunk` bytes; the
// map's box is `rows` rows
template <int HD>
__device__ __forceinline__ void load_tile(uint8_t* dst, uint32_t chunk, const CUtensorMap* m, uint64_t* bar, int col,
                                          int row, int b) {
#pragma unroll
  for (int c = 0; c < HD / 64; ++c) tma_load_3d(dst + c * chunk, m, bar, col + c * 64, row, b);
}

// w rows of a key tile (w a multiple of 16), in one box where they are more than 32
template <int HD>
__device__ __forceinline__ void load_keys(uint8_t* dst, uint32_t chunk, const CUtensorMap* m, const CUtensorMap* m16,
                                          uint64_t* bar, int col, int row, int w, int b) {
  mbar_arrive_expect_tx(bar, (uint32_t)(w <= 32 ? w : kQB) * 2 * HD);
  if (w <= 32) {
    for (int r = 0; r < w; r += 16) load_tile<HD>(dst + r * 128, chunk, m16, bar, col, row + r, b);
  } else {
    load_tile<HD>(dst, chunk, m, bar, col, row, b);
  }
}
// D = A B^T over HD columns, both K-major in chunks of 64 columns
template <int HD>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint32_t achunk, uint64_t bb, uint32_t bchunk, uint32_t id) {
#pragma unroll
  for (int kk = 0; kk < HD / 16; ++kk)
    umma_bf16(d, at(a, (kk >> 2) * achunk + (kk & 3) * 32), at(bb, (kk >> 2) * bchunk + (kk & 3) * 32), id, kk != 0);
}
// D (+)= A B over w <= N rows of B (MN-major, 128-byte rows): A bf16 in TMEM, 16 rows of B every 8 columns; with HALF,
// rows [HALF, ...) of it HALF columns behind the first
template <int N, int HALF>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t bb, uint32_t id, int w, bool add) {
  const auto step = [&](int kk, uint32_t acc) {
    umma_ts(d, a + (HALF ? kk * 16 / HALF * HALF + kk * 16 % HALF / 2 : kk * 8), at(bb, kk * 16 * 128), id, acc);
  };
  if (w == N) {
#pragma unroll
    for (int kk = 0; kk < N / 16; ++kk) step(kk, kk > 0 || add);
  } else {
#pragma unroll 1
    for (int kk = 0; kk * 16 < w; ++kk) step(kk, kk > 0 || add);
  }
}

// ---------------------------------------------------------------------------------- forward
// One CTA per query tile of one head, two CTAs an SM: a tile's chain S -> softmax -> P V is serial, so
// the tensor cores work on one CTA's products while the other's softmax runs, and a CTA's start and
// end hide behind the other's blocks. 192 threads: warp 0 TMA (one K and one V tile: K j+1 arrives
// under softmax j, V j+1 under softmax j+1), warp 1 issues the MMAs, warps 2-5 one thread a query row.
//   S = Q K^T into TMEM; P = 2^(S' - m) as bf16 over S itself, the A operand of O += P V.
// The reference m of a row moves only when a block's maximum exceeds it by 2^8, with O rescaled in
// TMEM then: S of block j has completed, so have the products issued before it, P V of j - 1 among
// them. Blocks of up to 32 keys (the usual few sinks) run a short form.
template <int HD>
struct FwdCfg {
  static constexpr uint32_t CH = kQB * 128;  // [128 rows x 64] bf16
  static constexpr uint32_t TILE = (HD / 64) * CH;
  static constexpr uint32_t SMEM = 3 * TILE + 1024 + 128;
};

template <int HD>
__global__ void __launch_bounds__(192, 2)
k_window_fwd(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
             const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmK16,
             const __grid_constant__ CUtensorMap tmV16, const WinArgs p) {
  using C = FwdCfg<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *sQ = smem, *sK = smem + C::TILE, *sV = smem + 2 * C::TILE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + 3 * C::TILE);
  uint64_t *q_full = bars, *k_full = bars + 1, *v_full = bars + 2, *k_empty = bars + 3, *v_empty = bars + 4,
           *s_full = bars + 5, *p_full = bars + 6, *o_full = bars + 7;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 8);

  const int nq = (p.S + kQB - 1) / kQB;
  const int h = blockIdx.x % p.hq, u = blockIdx.x / p.hq;
  const int b = u / nq, q0 = (nq - 1 - u % nq) * kQB;
  const int kvh = h / (p.hq / p.hkv);
  const Blocks kb(q0, p.S, p.window, p.sinks);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 8; ++i) mbar_init(bars + i, bars + i == p_full ? 128 : 1);
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tS = *tmem_slot, tO = tS + 128;
  pdl_wait();
  pdl_trigger();

  if (warp == 0) {
    if (elect_one()) {
      mbar_arrive_expect_tx(q_full, C::TILE);
      load_tile<HD>(sQ, C::CH, &tmQ, q_full, h * HD, q0, b);
    }
    __syncwarp();
    bool ok = true;
    for (int j = 0; j < kb.n && ok; ++j) {
      const int k0 = kb.k0(j), w = kb.width(j);
      for (int kv = 0; kv < 2; ++kv) {
        if (j > 0 && !(ok = warp_wait(kv ? v_empty : k_empty, (j - 1) & 1))) break;
        if (elect_one())
          load_keys<HD>(kv ? sV : sK, C::CH, kv ? &tmV : &tmK, kv ? &tmV16 : &tmK16, kv ? v_full : k_full, kvh * HD, k0, w, b);
        __syncwarp();
      }
    }
  } else if (warp == 1) {
    constexpr uint32_t idO = umma_idesc_bf16(128, HD, 0, 1);
    bool ok = warp_wait(q_full, 0);
    for (int j = 0; j <= kb.n && ok; ++j) {
      if (j > 0) {  // O += P_{j-1} V_{j-1}
        if (!(ok = warp_wait(p_full, (j - 1) & 1) && warp_wait(v_full, (j - 1) & 1))) break;
        tc_fence_after();
        if (elect_one()) {
          mma_ts<kQB, 0>(tO, tS, umma_desc(smem_u32(sV), C::CH, 1024), idO, kb.width(j - 1), j > 1);
          umma_commit(j < kb.n ? v_empty : o_full);
        }
        __syncwarp();
      }
      if (j < kb.n) {  // S = Q K_j^T
        if (!(ok = warp_wait(k_full, j & 1))) break;
        tc_fence_after();
        if (elect_one()) {
          mma_ss<HD>(tS, umma_desc(smem_u32(sQ), 16, 1024), C::CH, umma_desc(smem_u32(sK), 16, 1024), C::CH,
                     umma_idesc_bf16(128, kb.width(j), 0, 0));
          umma_commit(s_full);
          umma_commit(k_empty);
        }
        __syncwarp();
      }
    }
  } else {
    const int r = (warp & 3) * 32 + lane, i = q0 + r;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const float sl2 = p.scale * kLog2e;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    // one block of NC columns (those from `cols` on are not visible to any row)
    const auto block = [&](auto nc, bool masked, int k0, int j) {
      constexpr int NC = decltype(nc)::value;
      float x[NC];
#pragma unroll
      for (int c = 0; c < NC; c += 32) tmem_ld32(tS + lanes + c, *reinterpret_cast<uint32_t(*)[32]>(x + c));
      tmem_ld_wait();
      if (masked) {  // visible: [i - window + 1, i] and [0, sinks), both up to i, as columns
        const int hi = i - k0, lo = hi - p.window, sc = p.sinks - k0;
#pragma unroll
        for (int c = 0; c < NC; ++c)
          if (c > hi || (c <= lo && c >= sc)) x[c] = -INFINITY;
      }
      float pm[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
      for (int c = 4; c < NC; ++c) pm[c & 3] = fmaxf(pm[c & 3], x[c]);
      const float bm = fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3])) * sl2;
      float corr = 1.f;
      if (bm > m + 8.f) {
        corr = ex2_approx(m - bm);  // 0 where nothing was visible before
        m = bm;
        l *= corr;
      }
      if (j > 0 && __any_sync(0xffffffffu, corr != 1.f)) {
#pragma unroll 1
        for (int c = 0; c < HD; c += 32) {
          uint32_t o[32];
          tmem_ld32(tO + lanes + c, o);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
          tmem_st32(tO + lanes + c, o);
        }
      }
      const float mm = m > -INFINITY ? m : 0.f;  // a row that sees nothing so far
      float ps[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        x[c] = ex2_approx(fmaf(x[c], sl2, -mm));
        ps[c & 3] += x[c];
      }
      l += (ps[0] + ps[1]) + (ps[2] + ps[3]);
      uint32_t w[NC / 2];
#pragma unroll
      for (int c = 0; c < NC / 2; ++c) w[c] = pack2(x[2 * c], x[2 * c + 1]);
#pragma unroll
      for (int c = 0; c < NC / 2; c += 16) tmem_st16(tS + lanes + c, w + c);
      tmem_st_wait();
    };
    for (int j = 0; j < kb.n; ++j) {
      if (!(ok = warp_wait(s_full, j & 1))) break;
      tc_fence_after();
      const int k0 = kb.k0(j), w = kb.width(j);
      const bool masked = !all_visible(q0, kQB, k0, kQB, p.window, p.sinks);
      if (w <= 32) block(std::integral_constant<int, 32>{}, true, k0, j);
      else block(std::integral_constant<int, 128>{}, masked, k0, j);
      tc_fence_before();
      mbar_arrive(p_full);
    }
    if (ok && warp_wait(o_full, 0)) {
      tc_fence_after();
      const float inv = 1.f / l;
      const int64_t t = (int64_t)b * p.S + i;
      const bool live = i < p.S;
#pragma unroll 1
      for (int c = 0; c < HD; c += 32) {
        uint32_t o[32];
        tmem_ld32(tO + lanes + c, o);
        tmem_ld_wait();
        if (live) {
          float y[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = __uint_as_float(o[e]) * inv;
          __nv_bfloat16* dst = p.o + t * p.ldo + (int64_t)h * HD + c;
#pragma unroll
          for (int e = 0; e < 32; e += 8)
            *reinterpret_cast<uint4*>(dst + e) = make_uint4(pack2(y[e], y[e + 1]), pack2(y[e + 2], y[e + 3]),
                                                            pack2(y[e + 4], y[e + 5]), pack2(y[e + 6], y[e + 7]));
          if (p.o32) {
            float* d32 = p.o32 + (t * p.hq + h) * HD + c;
#pragma unroll
            for (int e = 0; e < 32; e += 4) *reinterpret_cast<float4*>(d32 + e) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
          }
        }
      }
      if (live) p.lse[t * p.hq + h] = (m + log2f(l)) * kLn2;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tS, 256);
  }
}

// Columns [part HD / 4, part HD / 4 + HD / 4) of a gradient row and their rotary partners HD / 2 further, part
// 0 or 1: x * scale with the rotary embedding of position pos undone.
template <int HD>
__device__ __forceinline__ void store_grad(__nv_bfloat16* dst, const float (&lo)[HD / 4], const float (&hi)[HD / 4],
                                           const AttnBwdArgs& p, int pos, int part) {
  constexpr int HALF = HD / 2, Q4 = HD / 4;
#pragma unroll
  for (int c0 = 0; c0 < Q4; c0 += 8) {
    const int c = part * Q4 + c0;
    float y1[8], y2[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y1[e] = lo[c0 + e] * p.scale;
      y2[e] = hi[c0 + e] * p.scale;
      if (p.rope_cos) {
        const float cs = p.rope_cos[(int64_t)pos * HALF + c + e], sn = p.rope_sin[(int64_t)pos * HALF + c + e];
        const float a = y1[e] * cs + y2[e] * sn;
        y2[e] = y2[e] * cs - y1[e] * sn;
        y1[e] = a;
      }
    }
    *reinterpret_cast<uint4*>(dst + c) = make_uint4(pack2(y1[0], y1[1]), pack2(y1[2], y1[3]), pack2(y1[4], y1[5]), pack2(y1[6], y1[7]));
    *reinterpret_cast<uint4*>(dst + c + HALF) =
        make_uint4(pack2(y2[0], y2[1]), pack2(y2[2], y2[3]), pack2(y2[4], y2[5]), pack2(y2[6], y2[7]));
  }
}
// N consecutive TMEM columns of this thread's row
template <int N>
__device__ __forceinline__ void tmem_row(float (&x)[N], uint32_t addr) {
  if constexpr (N % 32 == 0) {
#pragma unroll
    for (int c = 0; c < N; c += 32) tmem_ld32(addr + c, *reinterpret_cast<uint32_t(*)[32]>(x + c));
  } else {
    static_assert(N == 16, "HD / 4");
    uint32_t* r = reinterpret_cast<uint32_t*>(x);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
  }
  tmem_ld_wait();
}

// What the dK / dV kernel reads of a query: its lse in units of log2 (infinity behind the sequence, which
// makes its P zero) and D. [B, hq, S rounded up to 128], in front of the scratch.
__host__ __device__ __forceinline__ int64_t stat_row(int b, int h, int hq, int S) { return ((int64_t)b * hq + h) * up(S, kQB); }

// ---------------------------------------------------------------------------------- dQ
// One CTA per query tile of one head, 320 threads: warp 0 TMA (Q and dO once, three K and two V tiles
// in flight), warp 1 the MMAs, warps 2-9 two threads a query row (half the columns of a block each).
// S has two TMEM buffers: while the threads turn S, dP of block j into dS (bf16, over their own columns
// of S j), the tensor cores form dQ += dS K of j - 1, S of j + 1 and dP of j + 1.
template <int HD>
struct DqCfg {
  static constexpr uint32_t CH = kQB * 128;
  static constexpr uint32_t TILE = (HD / 64) * CH;
  static constexpr int NK = 3, NV = 2;
  static constexpr uint32_t SMEM = (2 + NK + NV) * TILE + 1024 + 256 + kQB * 4;
};

template <int HD>
__global__ void __launch_bounds__(320, 1)
k_window_dq(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmO,
            const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
            const __grid_constant__ CUtensorMap tmK16, const __grid_constant__ CUtensorMap tmV16, const WinBwdArgs p) {
  using C = DqCfg<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *sQ = smem, *sO = smem + C::TILE, *sK = smem + 2 * C::TILE, *sV = sK + C::NK * C::TILE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sV + C::NV * C::TILE);
  uint64_t *q_full = bars, *dp_full = bars + 1, *ds_full = bars + 2, *done = bars + 3, *s_full = bars + 4;  // [2]
  uint64_t *k_full = bars + 6, *k_empty = k_full + C::NK, *v_full = k_empty + C::NK, *v_empty = v_full + C::NV;
  constexpr int kBars = 6 + 2 * C::NK + 2 * C::NV;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kBars);
  float* sD = reinterpret_cast<float*>(bars + kBars + 1);  // [128]

  const int nq = (p.S + kQB - 1) / kQB;
  const int h = blockIdx.x % p.hq, u = blockIdx.x / p.hq;
  const int b = u / nq, q0 = (nq - 1 - u % nq) * kQB;
  const int kvh = h / (p.hq / p.hkv);
  const Blocks kb(q0, p.S, p.window, p.sinks);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kBars; ++i) mbar_init(bars + i, bars + i == ds_full ? 256 : 1);
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmO);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot, tP = tmem + 256, tQ = tmem + 384;  // S in columns 0 and 128
  pdl_wait();
  pdl_trigger();

  if (warp == 0) {
    if (elect_one()) {
      mbar_arrive_expect_tx(q_full, 2 * C::TILE);
      load_tile<HD>(sQ, C::CH, &tmQ, q_full, h * HD, q0, b);
      load_tile<HD>(sO, C::CH, &tmO, q_full, h * HD, q0, b);
    }
    __syncwarp();
    bool ok = true;
    for (int j = 0; j < kb.n && ok; ++j) {
      const int k0 = kb.k0(j), w = kb.width(j);
      for (int kv = 0; kv < 2; ++kv) {
        const int ns = kv ? C::NV : C::NK, s = j % ns;
        if (j >= ns && !(ok = warp_wait((kv ? v_empty : k_empty) + s, (j / ns - 1) & 1))) break;
        if (elect_one())
          load_keys<HD>((kv ? sV : sK) + s * C::TILE, C::CH, kv ? &tmV : &tmK, kv ? &tmV16 : &tmK16,
                        (kv ? v_full : k_full) + s, kvh * HD, k0, w, b);
        __syncwarp();
      }
    }
  } else if (warp == 1) {
    constexpr uint32_t idQ = umma_idesc_bf16(128, HD, 0, 1);
    bool ok = warp_wait(q_full, 0);
    const auto scores = [&](int j) {  // S_j = Q K_j^T
      if (!(ok = ok && warp_wait(&k_full[j % C::NK], (j / C::NK) & 1))) return;
      tc_fence_after();
      if (elect_one()) {
        mma_ss<HD>(tmem + (j & 1) * 128, umma_desc(smem_u32(sQ), 16, 1024), C::CH,
                   umma_desc(smem_u32(sK + j % C::NK * C::TILE), 16, 1024), C::CH, umma_idesc_bf16(128, kb.width(j), 0, 0));
        umma_commit(&s_full[j & 1]);
      }
      __syncwarp();
    };
    const auto dprobs = [&](int j) {  // dP_j = dO V_j^T
      if (!(ok = ok && warp_wait(&v_full[j % C::NV], (j / C::NV) & 1))) return;
      tc_fence_after();
      if (elect_one()) {
        mma_ss<HD>(tP, umma_desc(smem_u32(sO), 16, 1024), C::CH, umma_desc(smem_u32(sV + j % C::NV * C::TILE), 16, 1024),
                   C::CH, umma_idesc_bf16(128, kb.width(j), 0, 0));
        umma_commit(dp_full);
        umma_commit(&v_empty[j % C::NV]);
      }
      __syncwarp();
    };
    scores(0);
    dprobs(0);
    if (kb.n > 1) scores(1);
    for (int j = 0; j < kb.n && ok; ++j) {
      if (!(ok = warp_wait(ds_full, j & 1))) break;  // dS_j is written, dP_j has been read
      if (j + 1 < kb.n) dprobs(j + 1);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {  // each half of a block's columns holds its own 64 keys' dS
        mma_ts<kQB, 64>(tQ, tmem + (j & 1) * 128, umma_desc(smem_u32(sK + j % C::NK * C::TILE), C::CH, 1024), idQ,
                        kb.width(j), j > 0);
        umma_commit(j + 1 < kb.n ? &k_empty[j % C::NK] : done);
      }
      __syncwarp();
      if (j + 2 < kb.n) scores(j + 2);
    }
  } else {
    const int half = (int)(threadIdx.x - 64) >> 7;
    const int r = (warp & 3) * 32 + lane, i = q0 + r;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const bool live = i < p.S;
    const int64_t t = (int64_t)b * p.S + i;
    const float sl2 = p.scale * kLog2e;
    // D of the tile's rows, from the forward's unrounded o where it was kept: a warp takes 16 rows, HD / 8
    // lanes a row, every load in flight before the first sum
    {
      constexpr int LPR = HD / 8, RPI = 32 / LPR;  // lanes a row, rows a load
      const int w8 = warp - 2, col = lane % LPR * 8;
      uint4 dv[16 / RPI];
      float4 ov[16 / RPI][2];
#pragma unroll
      for (int n = 0; n < 16 / RPI; ++n) {
        const int row = q0 + w8 * 16 + n * RPI + lane / LPR;
        const int64_t tt = (int64_t)b * p.S + row;
        dv[n] = make_uint4(0, 0, 0, 0);
        ov[n][0] = ov[n][1] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (row < p.S) {
          dv[n] = *reinterpret_cast<const uint4*>(p.dout + tt * p.lddo + (int64_t)h * HD + col);
          if (p.o32) {
            const float4* src = reinterpret_cast<const float4*>(p.o32 + (tt * p.hq + h) * HD + col);
            ov[n][0] = src[0];
            ov[n][1] = src[1];
          } else {
            *reinterpret_cast<uint4*>(&ov[n][0]) = *reinterpret_cast<const uint4*>(p.o + tt * p.ldo + (int64_t)h * HD + col);
          }
        }
      }
#pragma unroll
      for (int n = 0; n < 16 / RPI; ++n) {
        const __nv_bfloat16* d8 = reinterpret_cast<const __nv_bfloat16*>(&dv[n]);
        const __nv_bfloat16* o8 = reinterpret_cast<const __nv_bfloat16*>(&ov[n][0]);
        const float* f8 = reinterpret_cast<const float*>(&ov[n][0]);
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += __bfloat162float(d8[e]) * (p.o32 ? f8[e] : __bfloat162float(o8[e]));
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane % LPR == 0) sD[w8 * 16 + n * RPI + lane / LPR] = sum;
      }
    }
    const float lse2 = live ? p.lse[t * p.hq + h] * kLog2e : INFINITY;
    asm volatile("bar.sync 1, 256;" ::: "memory");
    const float D = sD[r];
    if (half == 0) reinterpret_cast<float2*>(p.D)[stat_row(b, h, p.hq, p.S) + i] = make_float2(lse2, D);
    bool ok = true;
    // columns [64 half, 64 half + NC) of a block
    const auto block = [&](auto nc, bool masked, int k0, int j) {
      constexpr int NC = decltype(nc)::value;
      const uint32_t tS = tmem + (j & 1) * 128 + half * 64 + lanes;
      float x[NC], y[NC];
      tmem_row<NC>(x, tS);
#pragma unroll
      for (int c = 0; c < NC; ++c) x[c] = ex2_approx(fmaf(x[c], sl2, -lse2));
      if (masked) {
        const int hi = i - k0 - half * 64, lo = hi - p.window, sc = p.sinks - k0 - half * 64;
#pragma unroll
        for (int c = 0; c < NC; ++c)
          if (c > hi || (c <= lo && c >= sc)) x[c] = 0.f;
      }
      if (!(ok = warp_wait(dp_full, j & 1))) return;
      tc_fence_after();
      tmem_row<NC>(y, tP + half * 64 + lanes);
      uint32_t w[NC / 2];
#pragma unroll
      for (int c = 0; c < NC / 2; ++c) w[c] = pack2(x[2 * c] * (y[2 * c] - D), x[2 * c + 1] * (y[2 * c + 1] - D));
#pragma unroll
      for (int c = 0; c < NC / 2; c += 16) tmem_st16(tS + c, w + c);
      tmem_st_wait();
    };
    for (int j = 0; j < kb.n && ok; ++j) {
      if (!(ok = warp_wait(&s_full[j & 1], (j >> 1) & 1))) break;
      tc_fence_after();
      const int k0 = kb.k0(j), w = kb.width(j);
      if (w > 32) block(std::integral_constant<int, 64>{}, !all_visible(q0, kQB, k0, kQB, p.window, p.sinks), k0, j);
      else if (half == 0) block(std::integral_constant<int, 32>{}, true, k0, j);
      else ok = warp_wait(dp_full, j & 1);
      tc_fence_before();
      mbar_arrive(ds_full);
    }
    if (ok && warp_wait(done, 0)) {
      tc_fence_after();
      float lo[HD / 4], hi[HD / 4];
      tmem_row<HD / 4>(lo, tQ + half * (HD / 4) + lanes);
      tmem_row<HD / 4>(hi, tQ + half * (HD / 4) + HD / 2 + lanes);
      if (live) store_grad<HD>(p.dq + t * p.lddq + (int64_t)h * HD, lo, hi, p, i, half);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------------- dK, dV
// The work of one key tile of a kv head: its group's heads times the 64-row query blocks that see any
// of its keys. It is cut into parts of equal length (n for the tiles that hold sinks, whose queries
// reach to the end of the sequence, n for the others); with one part a CTA stores dK and dV itself,
// else its fp32 sums go to the scratch and k_window_join adds them in order.
struct Split {
  int nkb, nsb;    // key tiles, those that hold sinks
  int near;        // query blocks that see a tile through the window
  int nq;          // query blocks of a sequence
  int ps, pw;      // parts of a tile with sinks, of another
  __host__ __device__ int ctas() const { return nsb * ps + (nkb - nsb) * pw; }  // a sequence and kv head
  __host__ __device__ int blocks(int kb) const {
    const int n = nq - 2 * kb;
    return kb < nsb || n < near ? n : near;
  }
};
// parts whose sums go to the scratch come first in its order, those of the tiles with sinks in front
__host__ __device__ __forceinline__ int64_t joined_parts(const Split& s) {
  return (s.ps > 1 ? (int64_t)s.nsb * s.ps : 0) + (s.pw > 1 ? (int64_t)(s.nkb - s.nsb) * s.pw : 0);
}

template <int HD>
struct DkvCfg {
  static constexpr int QB = 64, NS = 3;                       // rows of a query block, blocks in flight
  static constexpr uint32_t CH = kQB * 128, QCH = QB * 128;  // [128 x 64], [64 x 64] bf16
  static constexpr uint32_t KT = (HD / 64) * CH, QT = (HD / 64) * QCH;
  static constexpr uint32_t STAGE = 2 * QT + QB * 8;  // Q, dO, (lse, D)
  static constexpr uint32_t STEP = (STAGE + 1023) / 1024 * 1024;
  static constexpr uint32_t SMEM = 2 * KT + NS * STEP + 1024 + 256;
  static constexpr uint32_t COLS = 2 * 128 + 2 * HD <= 256 ? 256 : 512;
};

// 320 threads: warp 0 TMA, warp 1 the MMAs, warps 2-9 two threads a key row (half a block's queries each).
//   S^T = K Q^T and dP^T = V dO^T into one of two TMEM buffer pairs; P^T and dS^T as bf16 over the
//   threads' own columns of them, the A operands of dV += P^T dO and dK += dS^T Q (Q and dO read
//   MN-major from the tiles used K-major above). While the threads work on block j, the tensor cores
//   form the sums of j - 1 and the scores of j + 1.
template <int HD>
__global__ void __launch_bounds__(320, 1)
k_window_dkdv(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmO,
              const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const WinBwdArgs p,
              const Split sp, float* __restrict__ parts) {
  using C = DkvCfg<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *sK = smem, *sV = smem + C::KT, *sQ = smem + 2 * C::KT;  // [NS] stages
  uint64_t* bars = reinterpret_cast<uint64_t*>(sQ + C::NS * C::STEP);
  uint64_t *kv_full = bars, *done = bars + 1, *s_full = bars + 2, *t_full = bars + 4, *q_full = bars + 6,
           *q_empty = bars + 6 + C::NS;
  constexpr int kBars = 6 + 2 * C::NS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kBars);

  const int grp = p.hq / p.hkv;
  const int x = (int)blockIdx.x % sp.ctas(), bk = (int)blockIdx.x / sp.ctas();
  const int b = bk / p.hkv, kvh = bk % p.hkv;
  const bool sink = x < sp.nsb * sp.ps;
  const int np = sink ? sp.ps : sp.pw, y = sink ? x : x - sp.nsb * sp.ps;
  const int kb = sink ? y / np : sp.nsb + y / np, part = y % np;
  const int k0 = kb * kQB, nqb = sp.blocks(kb);
  const int64_t total = (int64_t)grp * nqb;
  const int it0 = (int)(total * part / np), n = (int)(total * (part + 1) / np) - it0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // item j of this CTA: its head and first query
  const auto head = [&](int j) { return kvh * grp + (it0 + j) / nqb; };
  const auto query = [&](int j) { return k0 + (it0 + j) % nqb * C::QB; };

  if (threadIdx.x == 0) {
    for (int i = 0; i < kBars; ++i) mbar_init(bars + i, bars + i == t_full || bars + i == t_full + 1 ? 256 : 1);
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmO);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot, tV = tmem + 256, tK = tmem + 256 + HD;  // S^T at 0, 64; dP^T at 128, 192
  pdl_wait();
  pdl_trigger();

  if (n <= 0) {
    // nothing of the work fell to this part
  } else if (warp == 0) {
    if (elect_one()) {
      mbar_arrive_expect_tx(kv_full, 2 * C::KT);
      load_tile<HD>(sK, C::CH, &tmK, kv_full, kvh * HD, k0, b);
      load_tile<HD>(sV, C::CH, &tmV, kv_full, kvh * HD, k0, b);
    }
    __syncwarp();
    for (int j = 0; j < n; ++j) {
      const int s = j % C::NS, h = head(j), q = query(j);
      if (j >= C::NS && !warp_wait(&q_empty[s], (j / C::NS - 1) & 1)) break;
      if (elect_one()) {
        uint8_t* st = sQ + s * C::STEP;
        mbar_arrive_expect_tx(&q_full[s], C::STAGE);
        load_tile<HD>(st, C::QCH, &tmQ, &q_full[s], h * HD, q, b);
        load_tile<HD>(st + C::QT, C::QCH, &tmO, &q_full[s], h * HD, q, b);
        bulk_load(st + 2 * C::QT, reinterpret_cast<const float2*>(p.D) + stat_row(b, h, p.hq, p.S) + q, C::QB * 8,
                  &q_full[s]);
      }
      __syncwarp();
    }
  } else if (warp == 1) {
    constexpr uint32_t idS = umma_idesc_bf16(128, C::QB, 0, 0), idG = umma_idesc_bf16(128, HD, 0, 1);
    bool ok = warp_wait(kv_full, 0);
    for (int j = 0; j < n + 2 && ok; ++j) {
      if (j >= 2) {  // dV += P^T dO, dK += dS^T Q of block j - 2
        const int i = j - 2, st = i & 1;
        if (!(ok = warp_wait(&t_full[st], (i >> 1) & 1))) break;
        tc_fence_after();
        if (elect_one()) {  // the second half of the queries lies 32 columns further
          const uint64_t q = umma_desc(smem_u32(sQ + i % C::NS * C::STEP), C::QCH, 1024);
          mma_ts<C::QB, 32>(tV, tmem + st * 64, at(q, C::QT), idG, C::QB, i > 0);
          mma_ts<C::QB, 32>(tK, tmem + 128 + st * 64, q, idG, C::QB, i > 0);
          umma_commit(i + 1 < n ? &q_empty[i % C::NS] : done);
        }
        __syncwarp();
      }
      if (j < n) {  // S^T_j = K Q_j^T, dP^T_j = V dO_j^T
        const int st = j & 1;
        if (!(ok = warp_wait(&q_full[j % C::NS], (j / C::NS) & 1))) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t q = umma_desc(smem_u32(sQ + j % C::NS * C::STEP), 16, 1024);
          mma_ss<HD>(tmem + st * 64, umma_desc(smem_u32(sK), 16, 1024), C::CH, q, C::QCH, idS);
          mma_ss<HD>(tmem + 128 + st * 64, umma_desc(smem_u32(sV), 16, 1024), C::CH, at(q, C::QT), C::QCH, idS);
          umma_commit(&s_full[st]);
        }
        __syncwarp();
      }
    }
  } else {
    const int half = (int)(threadIdx.x - 64) >> 7;
    const int r = (warp & 3) * 32 + lane, key = k0 + r;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const float sl2 = p.scale * kLog2e;
    bool ok = true;
    for (int j = 0; j < n && ok; ++j) {
      const int st = j & 1, q = query(j) + half * 32;  // this thread's first query
      if (!(ok = warp_wait(&q_full[j % C::NS], (j / C::NS) & 1) && warp_wait(&s_full[st], (j >> 1) & 1))) break;
      tc_fence_after();
      const float4* stat = reinterpret_cast<const float4*>(sQ + (j % C::NS) * C::STEP + 2 * C::QT) + half * 16;
      const uint32_t tS = tmem + st * 64 + half * 32 + lanes, tP = tS + 128;
      float a[32], d[32];
      tmem_ld32(tS, *reinterpret_cast<uint32_t(*)[32]>(a));
      tmem_ld32(tP, *reinterpret_cast<uint32_t(*)[32]>(d));
      tmem_ld_wait();
      const bool masked = !all_visible(query(j), C::QB, k0, kQB, p.window, p.sinks);
      // visible queries of this key: [key, key + window), from key on where it is a sink
      const int lo = key - q, hi = key < p.sinks ? C::QB : lo + p.window;
      uint32_t w[16], u[16];
#pragma unroll
      for (int c = 0; c < 32; c += 2) {
        const float4 s2 = stat[c / 2];  // (lse, D) of two queries
        float p0 = ex2_approx(fmaf(a[c], sl2, -s2.x)), p1 = ex2_approx(fmaf(a[c + 1], sl2, -s2.z));
        if (masked) {
          if (c < lo || c >= hi) p0 = 0.f;
          if (c + 1 < lo || c + 1 >= hi) p1 = 0.f;
        }
        w[c / 2] = pack2(p0, p1);
        u[c / 2] = pack2(p0 * (d[c] - s2.y), p1 * (d[c + 1] - s2.w));
      }
      tmem_st16(tS, w);
      tmem_st16(tP, u);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&t_full[st]);
    }
    if (ok && warp_wait(done, 0)) {
      tc_fence_after();
      if (np == 1) {
        const bool live = key < p.S;
        const int64_t t = (int64_t)b * p.S + key;
        float x0[HD / 4], x1[HD / 4];
        tmem_row<HD / 4>(x0, tK + half * (HD / 4) + lanes);
        tmem_row<HD / 4>(x1, tK + half * (HD / 4) + HD / 2 + lanes);
        if (live) store_grad<HD>(p.dk + t * p.lddk + (int64_t)kvh * HD, x0, x1, p, key, half);
        __nv_bfloat16* dst = p.dv + t * p.lddv + (int64_t)kvh * HD + half * (HD / 2);
#pragma unroll
        for (int c = 0; c < HD / 2; c += 32) {
          float v[32];
          tmem_row<32>(v, tV + half * (HD / 2) + c + lanes);
          if (live) {
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              *reinterpret_cast<uint4*>(dst + c + e) = make_uint4(pack2(v[e], v[e + 1]), pack2(v[e + 2], v[e + 3]),
                                                                  pack2(v[e + 4], v[e + 5]), pack2(v[e + 6], v[e + 7]));
          }
        }
      } else {  // [key row][dK, dV]
        const int64_t at = (int64_t)bk * joined_parts(sp) + (sink || sp.ps == 1 ? y : (int64_t)sp.nsb * sp.ps + y);
        float* dst = parts + (at * kQB + r) * (2 * HD) + half * HD;
#pragma unroll 1
        for (int c = 0; c < HD; c += 32) {
          float v[32];
          tmem_row<32>(v, (half ? tV : tK) + c + lanes);
#pragma unroll
          for (int e = 0; e < 32; e += 4) *reinterpret_cast<float4*>(dst + c + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::COLS);
  }
}

// Adds the parts of a key row in order: a warp a row of dK and dV, its lanes over pairs of columns (c, c + HD / 2).
// Parts without items were not written. Grid: [joined tiles x 16] x [B hkv], 8 rows a CTA.
template <int HD>
__global__ void __launch_bounds__(256) k_window_join(const WinBwdArgs p, const Split sp, const float* __restrict__ parts,
                                                     int kb0) {
  pdl_wait();
  pdl_trigger();
  const int kb = kb0 + (int)blockIdx.x / 16, r = ((int)blockIdx.x % 16) * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int bk = blockIdx.y, b = bk / p.hkv, kvh = bk % p.hkv, key = kb * kQB + r;
  if (key >= p.S) return;
  const bool sink = kb < sp.nsb;
  const int np = sink ? sp.ps : sp.pw;
  const int64_t at = (int64_t)bk * joined_parts(sp) + (sink ? (int64_t)kb * np : (sp.ps > 1 ? (int64_t)sp.nsb * sp.ps : 0) + (int64_t)(kb - sp.nsb) * np);
  const int64_t total = (int64_t)(p.hq / p.hkv) * sp.blocks(kb);
  constexpr int N = HD / 64;  // pairs of columns a lane
  float2 k1[N] = {}, v1[N] = {};
  for (int i = 0; i < np; ++i) {
    if (total * i / np == total * (i + 1) / np) continue;
    const float* src = parts + ((at + i) * kQB + r) * (2 * HD);
#pragma unroll
    for (int c = 0; c < N; ++c) {
      const int o = lane + 32 * c;
      k1[c].x += src[o];
      k1[c].y += src[o + HD / 2];
      v1[c].x += src[HD + o];
      v1[c].y += src[HD + o + HD / 2];
    }
  }
  const int64_t t = (int64_t)b * p.S + key;
#pragma unroll
  for (int c = 0; c < N; ++c) {
    const int o = lane + 32 * c;
    float y1 = k1[c].x * p.scale, y2 = k1[c].y * p.scale;
    if (p.rope_cos) {
      const float cs = p.rope_cos[(int64_t)key * (HD / 2) + o], sn = p.rope_sin[(int64_t)key * (HD / 2) + o];
      const float z = y1 * cs + y2 * sn;
      y2 = y2 * cs - y1 * sn;
      y1 = z;
    }
    __nv_bfloat16* dk = p.dk + t * p.lddk + (int64_t)kvh * HD;
    __nv_bfloat16* dv = p.dv + t * p.lddv + (int64_t)kvh * HD;
    dk[o] = __float2bfloat16_rn(y1);
    dk[o + HD / 2] = __float2bfloat16_rn(y2);
    dv[o] = __float2bfloat16_rn(v1[c].x);
    dv[o + HD / 2] = __float2bfloat16_rn(v1[c].y);
  }
}

// How the dK / dV work is cut: the parts of a tile are chosen for the fewest rounds of a B200's SMs times
// what a round takes, a CTA costing about 6 blocks besides its own (start, tiles of K and V, stores).
Split plan_split(int64_t T, int S, int hq, int hkv, int window, int sinks) {
  constexpr int sms = 148;
  const int64_t B = T / S;
  const int grp = hq / hkv;
  Split s;
  s.nkb = (S + kQB - 1) / kQB;
  s.nsb = (int)(((int64_t)std::min(sinks, S) + kQB - 1) / kQB);
  s.nq = (S + 63) / 64;
  s.near = (int)std::min<int64_t>(s.nq, ((int64_t)kQB - 2 + std::min(window, S)) / 64 + 1);
  const int64_t tw = (int64_t)grp * s.near, ts = (int64_t)grp * s.nq;
  int64_t best = INT64_MAX;
  s.ps = s.pw = 1;
  for (int n = 1; n <= 16 && (n == 1 || tw / n >= 4); ++n) {
    const int64_t len = (tw + n - 1) / n;
    const int64_t ps = std::min<int64_t>((ts + len - 1) / len, 4096);
    const int64_t ctas = B * hkv * (s.nsb * ps + (int64_t)(s.nkb - s.nsb) * n);
    const int64_t cost = ((ctas + sms - 1) / sms) * (len + 6);
    if (cost < best) {
      best = cost;
      s.ps = (int)ps;
      s.pw = n;
    }
  }
  return s;
}

// 3D map of a [B, S, cols] bf16 tensor with row stride ld: boxes of `rows` rows x 64 columns, 128-byte swizzle,
// zeros outside of a sequence
bool make_map3(CUtensorMap* m, const void* base, int64_t B, int64_t S, int64_t cols, int64_t ld, int rows) {
  const auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)S, (cuuint64_t)B};
  const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)(S * ld) * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)rows, 1}, es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename K>
cudaError_t allow_smem(K* kernel, uint32_t bytes, std::atomic<unsigned long long>& done) {
  if (done_on_device(done)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) mark_done_on_device(done);
  return e;
}

template <int HD>
cudaError_t launch_fwd(const WinArgs& a, cudaStream_t s) {
  using C = FwdCfg<HD>;
  const int64_t B = a.T / a.S, cq = (int64_t)a.hq * HD, ck = (int64_t)a.hkv * HD;
  CUtensorMap q, k, v, k16, v16;
  if (!make_map3(&q, a.q, B, a.S, cq, a.ldq, kQB) || !make_map3(&k, a.k, B, a.S, ck, a.ldk, kQB) ||
      !make_map3(&v, a.v, B, a.S, ck, a.ldv, kQB) || !make_map3(&k16, a.k, B, a.S, ck, a.ldk, 16) ||
      !make_map3(&v16, a.v, B, a.S, ck, a.ldv, 16))
    return cudaErrorInvalidValue;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem(k_window_fwd<HD>, C::SMEM, done);
  if (e != cudaSuccess) return e;
  const int64_t tiles = B * a.hq * ((a.S + kQB - 1) / kQB);
  return launch_k(k_window_fwd<HD>, dim3((unsigned)tiles), dim3(192), C::SMEM, s, 0, q, k, v, k16, v16, a);
}

template <int HD>
cudaError_t launch_bwd(const WinBwdArgs& a, cudaStream_t s) {
  using Q = DqCfg<HD>;
  using K = DkvCfg<HD>;
  const int64_t B = a.T / a.S, cq = (int64_t)a.hq * HD, ck = (int64_t)a.hkv * HD;
  CUtensorMap q, o, k, v, k16, v16, q64, o64;
  if (!make_map3(&q, a.q, B, a.S, cq, a.ldq, kQB) || !make_map3(&o, a.dout, B, a.S, cq, a.lddo, kQB) ||
      !make_map3(&k, a.k, B, a.S, ck, a.ldk, kQB) || !make_map3(&v, a.v, B, a.S, ck, a.ldv, kQB) ||
      !make_map3(&k16, a.k, B, a.S, ck, a.ldk, 16) || !make_map3(&v16, a.v, B, a.S, ck, a.ldv, 16) ||
      !make_map3(&q64, a.q, B, a.S, cq, a.ldq, K::QB) || !make_map3(&o64, a.dout, B, a.S, cq, a.lddo, K::QB))
    return cudaErrorInvalidValue;
  static std::atomic<unsigned long long> done_q{0}, done_k{0};
  cudaError_t e = allow_smem(k_window_dq<HD>, Q::SMEM, done_q);
  if (e == cudaSuccess) e = allow_smem(k_window_dkdv<HD>, K::SMEM, done_k);
  if (e != cudaSuccess) return e;
  const int64_t tiles = B * a.hq * ((a.S + kQB - 1) / kQB);
  e = launch_k(k_window_dq<HD>, dim3((unsigned)tiles), dim3(320), Q::SMEM, s, 0, q, o, k, v, k16, v16, a);
  note_launch(1);
  if (e != cudaSuccess) return e;
  const Split sp = plan_split(a.T, a.S, a.hq, a.hkv, a.window, a.sinks);
  float* parts = a.D + 2 * B * a.hq * up(a.S, kQB);
  e = launch_k(k_window_dkdv<HD>, dim3((unsigned)(B * a.hkv * sp.ctas())), dim3(320), K::SMEM, s, 0, q64, o64, k, v, a, sp,
               parts);
  note_launch(1);
  if (e != cudaSuccess || joined_parts(sp) == 0) return e;
  const int kb0 = sp.nsb > 0 && sp.ps > 1 ? 0 : sp.nsb, kb1 = sp.pw > 1 ? sp.nkb : sp.nsb;
  e = launch_k(k_window_join<HD>, dim3((unsigned)((kb1 - kb0) * 16), (unsigned)(B * a.hkv)), dim3(256), 0, s, 0, a, sp,
               static_cast<const float*>(parts), kb0);
  note_launch(1);
  return e;
}

}  // namespace

bool window_shape_ok(int64_t T, int S, int hq, int hkv, int hd, int window, int sinks) {
  return (hd == 64 || hd == 128) && hq > 0 && hkv > 0 && hq % hkv == 0 && S > 0 && T > 0 && T % S == 0 &&
         T <= INT32_MAX && T * hq <= INT32_MAX && T / S * hkv <= 65535 && window >= 1 && sinks >= 0;
}

int64_t window_scratch(int64_t T, int S, int hq, int hkv, int hd, int window, int sinks) {
  const Split sp = plan_split(T, S, hq, hkv, std::min(window, S), std::min(sinks, S));
  return T / S * (2 * (int64_t)hq * up(S, kQB) + hkv * joined_parts(sp) * kQB * 2 * hd);
}

cudaError_t window_fwd(WinArgs a, cudaStream_t s) {
  if (!window_shape_ok(a.T, a.S, a.hq, a.hkv, a.hd, a.window, a.sinks)) return cudaErrorInvalidValue;
  a.window = std::min(a.window, a.S);
  a.sinks = std::min(a.sinks, a.S);
  const cudaError_t e = a.hd == 128 ? launch_fwd<128>(a, s) : launch_fwd<64>(a, s);
  note_launch(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t window_bwd(WinBwdArgs a, cudaStream_t s) {
  if (!window_shape_ok(a.T, a.S, a.hq, a.hkv, a.hd, a.window, a.sinks)) return cudaErrorInvalidValue;
  a.window = std::min(a.window, a.S);
  a.sinks = std::min(a.sinks, a.S);
  const cudaError_t e = a.hd == 128 ? launch_bwd<128>(a, s) : launch_bwd<64>(a, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace lst
