// Causal GQA attention with a sliding window and sinks: key j of a sequence is visible to its query
// i when j <= i and (i - j < window or j < sinks).
//   s_ij = q_i . k_j / sqrt(hd),  P = softmax of s over the visible keys,  o_i = sum_j P_ij v_j,
//   lse_i = log sum_j exp s_ij;
//   D_i = do_i . o_i,  dS_ij = P_ij (do_i . v_j - D_i),
//   dq_i = sum_j dS_ij k_j / sqrt(hd),  dk_j = sum_{h, i} dS_ij q_i / sqrt(hd),  dv_j = sum_{h, i} P_ij do_i,
// the last two over the query heads h that share the kv head.
//
// Three kernels on tcgen05 (bf16 operands, fp32 in TMEM), each walking only the tiles that hold a
// visible pair: the forward, dQ (which forms D first), and dK / dV, whose work is cut into equal shares; a
// fourth adds the parts of what was cut.
// Tiles come by 3D TMA maps (column, row of the sequence, sequence): rows behind a sequence read as
// zeros, never as the next sequence. D is formed from the unrounded o where the caller has it (AttnArgs::o32,
// AttnBwdArgs::o32), else from the bf16 one. Operands of products are bf16: q, k, v, dout as given, dS and the
// backward's P rounded (half a step of 2^-8 relative each, independent of the output's own rounding), the
// forward's P rounded too or held in two bf16 parts (WinArgs::parts). Scores, lse, sums and products are fp32.
#include "common.cuh"
#include "sync.cuh"
#include "pdl.cuh"
#include "ex2.cuh"
#include "gemm.cuh"
#include "window.cuh"

#include <algorithm>
#include <cudaTypedefs.h>

namespace lst {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn();  // gemm.cu

namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kQB = 128;  // rows of a tile in TMEM: queries (forward, dQ) or keys (dK, dV)

// Two fp32 values as one operand of the packed instructions.
__device__ __forceinline__ uint64_t f2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack(uint64_t v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// 2^x of a pair. (Every other pair by a polynomial on the FMA pipe, to spare the exponential unit, made the backward
// of 8192 tokens 2 % longer and that of 4 x 512 tokens 1.5 % shorter.)
__device__ __forceinline__ void ex2_pair(uint64_t x, float& r0, float& r1) {
  unpack(x, r0, r1);
  r0 = ex2_approx(r0);
  r1 = ex2_approx(r1);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// A shared-memory matrix descriptor with its 32-bit halves apart: only the low one, which holds the
// address, differs between the tiles and steps of a product.
struct Desc {
  uint32_t lo, hi;
};
__device__ __forceinline__ Desc make_desc(uint32_t saddr, uint32_t lbo_bytes, uint32_t sbo_bytes) {
  const uint64_t d = umma_desc(saddr, lbo_bytes, sbo_bytes);
  return {(uint32_t)d, (uint32_t)(d >> 32)};
}
__device__ __forceinline__ Desc at(Desc d, uint32_t bytes) { return {d.lo + (bytes >> 4), d.hi}; }
// D (+)= A B with A [128, 16] bf16 in TMEM (two values a column, row = lane) and B by descriptor
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, Desc b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 x, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], x, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// the same with A by descriptor
__device__ __forceinline__ void umma_ss(uint32_t d, Desc a, Desc b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "mov.b64 x, {%1, %2};\n\t"
      "mov.b64 y, {%3, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, p;\n\t}" ::"r"(d),
      "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// x, the same in every lane, as a value that the compiler too knows to be the same
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
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

// Wait of a whole warp; false (for all of it) once it ran out. Not unrolled: there are many of them, and the
// kernels' code has to stay in the instruction cache (dQ with 111 KB of code took 3000 clocks a block).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  bool done = false;
#pragma unroll 1
  for (uint32_t i = 0; i < kSpinLimit && !done; ++i) done = __all_sync(0xffffffffu, mbar_try_wait(bar, parity));
  if (!done) dev_fail(DEV_ERR_MBAR_TIMEOUT);
  return done;
}

// the same for two barriers
__device__ __forceinline__ bool warp_wait2(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb) {
  bool done = false;
#pragma unroll 1
  for (uint32_t i = 0; i < kSpinLimit && !done; ++i) {
    const bool x = mbar_try_wait(a, pa), y = mbar_try_wait(b, pb);
    done = __all_sync(0xffffffffu, x && y);
  }
  if (!done) dev_fail(DEV_ERR_MBAR_TIMEOUT);
  return done;
}

__host__ __device__ __forceinline__ int up(int a, int b) { return (a + b - 1) / b * b; }

// The key blocks that the queries [q0, q0 + 128) of a sequence see, in order: sinks in front of the
// window's first block, then the window's blocks. A block starts at a multiple of KB; its width is a
// multiple of 16 that covers its last visible key.
template <int kKB>
struct Blocks {
  int nsink, n, jb0, front, end;
  __device__ __forceinline__ Blocks(int q0, int S, int window, int sinks) {
    jb0 = max(0, q0 - window + 1) / kKB;
    front = min(sinks, jb0 * kKB);  // sinks that the window's blocks do not hold
    nsink = (front + kKB - 1) / kKB;
    end = min(S, q0 + kQB);
    n = nsink + (end + kKB - 1) / kKB - jb0;
  }
  __device__ __forceinline__ int k0(int j) const { return (j < nsink ? j : jb0 + j - nsink) * kKB; }
  __device__ __forceinline__ int width(int j) const {
    const int left = (j < nsink ? front : end) - k0(j);
    return left >= kKB ? kKB : up(left, 16);
  }
};
__device__ __forceinline__ uint64_t bits_below(int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1; }
// Bit c: query i sees key k0 + c, c < 64.
__device__ __forceinline__ uint64_t visible_keys(int i, int k0, int window, int sinks) {
  return bits_below(i - k0 + 1) & (~bits_below(i - window + 1 - k0) | bits_below(sinks - k0));
}
// Bit c: key j is seen by query q0 + c, c < 64.
__device__ __forceinline__ uint64_t visible_queries(int j, int q0, int window, int sinks) {
  return ~bits_below(j - q0) & (j < sinks ? ~0ull : bits_below(j + window - q0));
}
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

// w rows of a key tile (w a multiple of 16), in one box of KB rows where they are more than 32
template <int HD, int KB>
__device__ __forceinline__ void load_keys(uint8_t* dst, uint32_t chunk, const CUtensorMap* m, const CUtensorMap* m16,
                                          uint64_t* bar, int col, int row, int w, int b) {
  mbar_arrive_expect_tx(bar, (uint32_t)(w <= 32 ? w : KB) * 2 * HD);
  if (w <= 32) {
    for (int r = 0; r < w; r += 16) load_tile<HD>(dst + r * 128, chunk, m16, bar, col, row + r, b);
  } else {
    load_tile<HD>(dst, chunk, m, bar, col, row, b);
  }
}
// A bf16 row (32 packed words of 64 columns) into its place of a swizzled [rows x 64] tile
__device__ __forceinline__ void stage_row(uint8_t* tile, int row, const uint32_t* w) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    *reinterpret_cast<uint4*>(tile + row * 128 + ((i ^ (row & 7)) * 16)) =
        make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* m, const void* src, int32_t x, int32_t y, int32_t z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
               : "memory");
}
// Until this thread's TMA stores have read their shared memory.
__device__ __forceinline__ void tma_store_wait() {
  asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group.read 0;" ::: "memory");
}
// Fetches a tile into L2 for a CTA to come.
template <int HD>
__device__ __forceinline__ void prefetch_tile(const CUtensorMap* m, int col, int row, int b) {
#pragma unroll
  for (int c = 0; c < HD / 64; ++c)
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global [%0, {%1, %2, %3}];" ::"l"(reinterpret_cast<uint64_t>(m)),
                 "r"(col + c * 64), "r"(row), "r"(b)
                 : "memory");
}
// D = A B^T over HD columns, A in TMEM (HD / 2 columns), B K-major in chunks of 64 columns
template <int HD>
__device__ __forceinline__ void mma_tt(uint32_t d, uint32_t a, Desc bb, uint32_t bchunk, uint32_t id) {
#pragma unroll
  for (int kk = 0; kk < HD / 16; ++kk) umma_ts(d, a + kk * 8, at(bb, (kk >> 2) * bchunk + (kk & 3) * 32), id, kk != 0);
}
// D = A B^T over HD columns, both K-major in chunks of 64 columns
template <int HD>
__device__ __forceinline__ void mma_ss(uint32_t d, Desc a, uint32_t achunk, Desc bb, uint32_t bchunk, uint32_t id) {
#pragma unroll
  for (int kk = 0; kk < HD / 16; ++kk)
    umma_ss(d, at(a, (kk >> 2) * achunk + (kk & 3) * 32), at(bb, (kk >> 2) * bchunk + (kk & 3) * 32), id, kk != 0);
}
// D (+)= A B over w <= N rows of B (MN-major, 128-byte rows): A bf16 in TMEM, 16 rows of B every 8 columns; with HALF,
// each HALF rows HALF columns behind the last ones
template <int N, int HALF>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, Desc bb, uint32_t id, int w, bool add) {
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
// Query tile x of those of `heads` heads (of all sequences): the sequences' last tiles (the longest) first, the heads
// of a tile next to each other.
struct QueryTile {
  int h, b, q0;
  __device__ __forceinline__ QueryTile(int x, int hq, int heads, int S) {
    const int q = x / heads, u = x - q * heads;
    b = u / hq;
    h = u - b * hq;
    q0 = ((S + kQB - 1) / kQB - 1 - q) * kQB;
  }
};
// The tiles of CTA c of n in its order: c, 2 n - 1 - c, 2 n + c, ...: back and forth, so that no CTA gets the longer tile
// in every round. (The backward of 4 sequences of 512 tokens takes 57.4 us so, 60.4 with every n-th tile of the
// sequences one behind the other.)
struct TileWalk : QueryTile {
  int x, round;
  __device__ __forceinline__ TileWalk(int hq, int heads, int S) : QueryTile(blockIdx.x, hq, heads, S), x(blockIdx.x), round(0) {}
  __device__ __forceinline__ int after() const {
    const int n = gridDim.x, c = blockIdx.x;
    return (round + 1) * n + (round & 1 ? c : n - 1 - c);
  }
  __device__ __forceinline__ void next(int hq, int heads, int S) {
    x = after();
    ++round;
    static_cast<QueryTile&>(*this) = QueryTile(x, hq, heads, S);
  }
};

// One CTA per query tile of one head, two CTAs an SM, so that a CTA's start and end hide behind the
// other's blocks. 192 threads: warp 0 TMA (two K and two V blocks of 64 keys in flight), warp 1 issues
// the MMAs, warps 2-5 one thread a query row.
//   S = Q K^T into one of two TMEM buffers; P = 2^(S' - m) as bf16 over S itself, the A operand of O += P V.
// While a row's thread works on block j, the tensor cores form P V of j - 1 and S of j + 1.
// The reference m of a row moves only when a block's maximum exceeds it by 2^8; O is then rescaled in
// TMEM, once P V of j - 1 has been added. The tile of O leaves through Q's shared memory by TMA.
// Bound by the hand-over between MMAs and row threads: 16384 tokens, 32 heads of 128 over 8, window 1024, 4 sinks
// take 288 us, 0.55 of the matrix rate that a large product reaches, the tensor pipe 50 % active (an S of N = 64
// takes 48 clocks an MMA where 32 would do: both operands come from shared memory); 4 x 512 tokens 17.7 us, 20 %
// active: 512 CTAs of 2 to 7 blocks, each with a start and an end. (Persistent CTAs with the next tile's Q and K
// under this one's end took 292 us against 287, and 18.0 us against 18.4. Blocks of 128 keys with one buffer of S,
// whose MMAs read Q half as often: 324 us, with two threads a row 336.)
template <int HD>
struct FwdCfg {
  static constexpr int KB = 64;  // keys of a block
  static constexpr uint32_t CH = kQB * 128, KCH = KB * 128;  // [128 x 64], [64 x 64] bf16
  static constexpr uint32_t TILE = (HD / 64) * CH, KT = (HD / 64) * KCH;
  static constexpr uint32_t SMEM = TILE + 4 * KT + 1024 + 256;
};

// PARTS 2: what the rounding of P to bf16 leaves goes behind it as a second bf16 value and takes a product of its own,
// so that 16 bits of P count (the causal kernel's fp16 has 11, at the price of v's range). Where only the output's
// 8 bits matter, as in a call of the kernel by itself, one part is enough: 16384 tokens as above take 366 us in two
// parts against 293 in one, 4 x 512 19.6 against 17.8. The engine's steps take two, which
// their copies hide: with one, a window would cost a stack of layers bits that the causal kernel keeps.
template <int HD, int PARTS>
__global__ void __launch_bounds__(192, 2)
k_window_fwd(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
             const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmK16,
             const __grid_constant__ CUtensorMap tmV16, const __grid_constant__ CUtensorMap tmO, const WinArgs p,
             const int ahead) {
  using C = FwdCfg<HD>;
  constexpr int kKB = C::KB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *sQ = smem, *sK = smem + C::TILE, *sV = sK + 2 * C::KT;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sV + 2 * C::KT);
  uint64_t *q_full = bars, *o_full = bars + 1, *k_full = bars + 2, *v_full = bars + 4, *k_empty = bars + 6,
           *v_empty = bars + 8, *s_full = bars + 10, *p_full = bars + 12;  // [2] from k_full on
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 14);

  const QueryTile tile(blockIdx.x, p.hq, p.heads, p.S);
  const int h = tile.h, b = tile.b, q0 = tile.q0;
  const int kvh = h / (p.hq / p.hkv);
  const Blocks<kKB> kb(q0, p.S, p.window, p.sinks);
  const int warp = (int)uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 14; ++i) mbar_init(bars + i, i >= 12 ? 128 : 1);
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmO);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tS = uniform(*tmem_slot), tO = tS + 128;
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
      if (j == 2 && blockIdx.x + ahead < gridDim.x && elect_one()) {
        const QueryTile next(blockIdx.x + ahead, p.hq, p.heads, p.S);
        prefetch_tile<HD>(&tmQ, next.h * HD, next.q0, next.b);
      }
      const int k0 = kb.k0(j), w = kb.width(j), s = j & 1;
      for (int kv = 0; kv < 2; ++kv) {
        if (j >= 2 && !(ok = warp_wait((kv ? v_empty : k_empty) + s, ((j >> 1) - 1) & 1))) break;
        if (elect_one())
          load_keys<HD, kKB>((kv ? sV : sK) + s * C::KT, C::KCH, kv ? &tmV : &tmK, kv ? &tmV16 : &tmK16,
                        (kv ? v_full : k_full) + s, kvh * HD, k0, w, b);
        __syncwarp();
      }
    }
  } else if (warp == 1) {
    constexpr uint32_t idO = umma_idesc_bf16(128, HD, 0, 1);
    bool ok = warp_wait(q_full, 0);
    const auto scores = [&](int j) {  // S_j = Q K_j^T
      const int s = j & 1;
      if (!(ok = ok && warp_wait(k_full + s, (j >> 1) & 1))) return;
      tc_fence_after();
      if (elect_one()) {
        mma_ss<HD>(tS + s * kKB, make_desc(smem_u32(sQ), 16, 1024), C::CH, make_desc(smem_u32(sK + s * C::KT), 16, 1024),
                   C::KCH, umma_idesc_bf16(128, kb.width(j), 0, 0));
        umma_commit(s_full + s);
        umma_commit(k_empty + s);
      }
      __syncwarp();
    };
    scores(0);
    if (kb.n > 1) scores(1);
    for (int j = 0; j < kb.n && ok; ++j) {
      const int s = j & 1;
      if (!(ok = warp_wait(v_full + s, (j >> 1) & 1) && warp_wait(p_full + s, (j >> 1) & 1))) break;
      tc_fence_after();
      if (elect_one()) {  // O += P_j V_j
        const Desc v = make_desc(smem_u32(sV + s * C::KT), C::KCH, 1024);
        mma_ts<kKB, 0>(tO, tS + s * kKB, v, idO, kb.width(j), j > 0);
        if (PARTS == 2) mma_ts<kKB, 0>(tO, tS + s * kKB + kKB / 2, v, idO, kb.width(j), true);
        umma_commit(j + 1 < kb.n ? v_empty + s : o_full);
      }
      __syncwarp();
      if (j + 2 < kb.n) scores(j + 2);
    }
  } else {
    const int r = (warp & 3) * 32 + lane, i = q0 + r;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const float sl2 = p.scale * kLog2e;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < kb.n && ok; ++j) {
      if (!(ok = warp_wait(s_full + (j & 1), (j >> 1) & 1))) break;
      tc_fence_after();
      const int k0 = kb.k0(j);
      const uint32_t tX = tS + (j & 1) * kKB + lanes;
      float x[kKB];
      tmem_row<kKB>(x, tX);
      if (!all_visible(q0, kQB, k0, kKB, p.window, p.sinks)) {  // also what lies behind a narrower block
        const uint64_t vis = visible_keys(i, k0, p.window, p.sinks);
        const uint32_t bits[2] = {(uint32_t)vis, (uint32_t)(vis >> 32)};
#pragma unroll
        for (int c = 0; c < kKB; ++c)
          if (!(bits[c / 32] >> (c % 32) & 1)) x[c] = -INFINITY;
      }
      float pm[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
      for (int c = 4; c < kKB - 4; c += 8) {
#pragma unroll
        for (int e = 0; e < 4; ++e) pm[e] = max3(pm[e], x[c + 2 * e], x[c + 2 * e + 1]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) pm[e] = fmaxf(pm[e], x[kKB - 4 + e]);
      const float bm = fmaxf(max3(pm[0], pm[1], pm[2]), pm[3]) * sl2;
      float corr = 1.f;
      if (bm > m + 8.f) {
        corr = ex2_approx(m - bm);  // 0 where nothing was visible before
        m = bm;
        l *= corr;
      }
      if (j > 0 && __any_sync(0xffffffffu, corr != 1.f)) {
        if (!(ok = warp_wait(v_empty + ((j - 1) & 1), ((j - 1) >> 1) & 1))) break;  // P V of j - 1 has been added
        tc_fence_after();
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
      uint64_t ps[2] = {0, 0};
      uint32_t w[PARTS * kKB / 2];
      const uint64_t sl = f2(sl2, sl2), mn = f2(-mm, -mm);
#pragma unroll
      for (int c = 0; c < kKB / 2; ++c) {
        float a0, a1;
        ex2_pair(fma2(f2(x[2 * c], x[2 * c + 1]), sl, mn), a0, a1);
        ps[c & 1] = add2(ps[c & 1], f2(a0, a1));
        w[c] = pack2(a0, a1);
        if constexpr (PARTS == 2) {  // what the rounding leaves, exact in fp32
          unpack(fma2(f2(__uint_as_float(w[c] << 16), __uint_as_float(w[c] & 0xffff0000u)), f2(-1.f, -1.f), f2(a0, a1)), a0, a1);
          w[kKB / 2 + c] = pack2(a0, a1);
        }
      }
      float l0, l1;
      unpack(add2(ps[0], ps[1]), l0, l1);
      l += l0 + l1;
#pragma unroll
      for (int c = 0; c < PARTS * kKB / 2; c += 16) tmem_st16(tX + c, w + c);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(p_full + (j & 1));
    }
    ok = ok && warp_wait(o_full, 0);
    if (ok) {
      tc_fence_after();
      const float inv = 1.f / l;
      const int64_t t = (int64_t)b * p.S + i;
      if (i < p.S) p.lse[t * p.hq + h] = (m + log2f(l)) * kLn2;
#pragma unroll 1
      for (int c = 0; c < HD; c += 64) {
        float y[64];
        uint32_t w[32];
        tmem_ld32(tO + lanes + c, *reinterpret_cast<uint32_t(*)[32]>(y));
        tmem_ld32(tO + lanes + c + 32, *reinterpret_cast<uint32_t(*)[32]>(y + 32));
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 64; ++e) y[e] *= inv;
#pragma unroll
        for (int e = 0; e < 32; ++e) w[e] = pack2(y[2 * e], y[2 * e + 1]);
        stage_row(sQ + c / 64 * C::CH, r, w);
        if (p.o32 && i < p.S) {  // for the backward's D
          float4* dst = reinterpret_cast<float4*>(p.o32 + (t * p.hq + h) * HD + c);
#pragma unroll
          for (int e = 0; e < 16; ++e) dst[e] = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
        }
        __syncwarp();
      }
      fence_proxy_async();
    }
    asm volatile("bar.sync 1, 128;" ::: "memory");
    if (warp == 2 && ok && elect_one()) {
#pragma unroll
      for (int c = 0; c < HD / 64; ++c) tma_store_3d(&tmO, sQ + c * C::CH, h * HD + c * 64, q0, b);
      tma_store_wait();
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
// 0 or 1: x * scale with the rotary embedding of position pos undone, as bf16 into the row's place of a
// swizzled tile (chunks of 64 columns).
template <int HD>
__device__ __forceinline__ void stage_grad(uint8_t* tile, uint32_t chunk, int row, float (&lo)[HD / 4], float (&hi)[HD / 4],
                                           const AttnBwdArgs& p, int pos, int part) {
  constexpr int HALF = HD / 2, Q4 = HD / 4;
#pragma unroll
  for (int e = 0; e < Q4; ++e) {
    lo[e] *= p.scale;
    hi[e] *= p.scale;
  }
  if (p.rope_cos && pos < p.S) {
    const float4* ct = reinterpret_cast<const float4*>(p.rope_cos + (int64_t)pos * HALF + part * Q4);
    const float4* st = reinterpret_cast<const float4*>(p.rope_sin + (int64_t)pos * HALF + part * Q4);
#pragma unroll
    for (int e = 0; e < Q4; e += 4) {
      const float4 c4 = ct[e / 4], s4 = st[e / 4];
      const float cs[4] = {c4.x, c4.y, c4.z, c4.w}, sn[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float a = lo[e + u] * cs[u] + hi[e + u] * sn[u];
        hi[e + u] = hi[e + u] * cs[u] - lo[e + u] * sn[u];
        lo[e + u] = a;
      }
    }
  }
  const auto put = [&](int col, const float* y) {
    *reinterpret_cast<uint4*>(tile + col / 64 * chunk + row * 128 + ((col % 64 / 8) ^ (row & 7)) * 16) =
        make_uint4(pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]), pack2(y[6], y[7]));
  };
#pragma unroll
  for (int e = 0; e < Q4; e += 8) {
    put(part * Q4 + e, lo + e);
    put(part * Q4 + e + HALF, hi + e);
  }
}
// What the dK / dV kernel reads of a query: its lse in units of log2 (infinity behind the sequence, which
// makes its P zero) and D. Two rows of S rounded up to 128 for each sequence and head, in front of the scratch.
__host__ __device__ __forceinline__ int64_t stat_row(int b, int h, int hq, int S) {
  return ((int64_t)b * hq + h) * 2 * up(S, kQB);
}

// ---------------------------------------------------------------------------------- dQ
// Persistent CTAs, one an SM, taking the query tiles in turn; 320 threads: warp 0 TMA, warp 1 the MMAs, warps 2-9 two
// threads a query row (half of a block's columns each); the next tile's Q, dO and o and up to three K
// blocks and one V block of 128 keys are in flight.
// Q and dO are copied into TMEM first and serve as the A operands from there: read from shared memory for
// every block they took its whole bandwidth (128 bytes a clock: with K, V, their loads and dS K 1800
// clocks a block, where the tensor cores take 1540), and their place is free for the next tile's. o, which
// only D needs, passes through K's ring.
// S of block j + 1 is issued once the threads have read S of j; dS goes over dP (bf16, the A operand of dQ += dS K),
// and dP of j + 1 is issued in one run with that product, under the exponentials of j + 1. (Blocks of 64 keys with
// two buffers of each took 2060 clocks for 64 keys: at N = 64 the issue of an MMA takes longer than its 32 clocks.)
// A tile's end overlaps the next one's start: Q and dO of the next tile go to TMEM before dQ leaves it, so that
// the first products run under dQ's way out (by TMA, from shared memory).
// Bound by the chain dS -> dQ, dP -> dS of a block (about 2100 clocks, of which the tensor cores work 1540): 8192
// tokens, 32 heads of 128 over 8, window 1024, 4 sinks take 204 us, the tensor pipe 55 % active; 4 x 512 tokens 28 us.
template <int HD>
struct DqCfg {
  static constexpr int KB = 128, NK = 3;  // keys of a block, blocks of K in flight
  static constexpr uint32_t CH = kQB * 128;
  static constexpr uint32_t TILE = (HD / 64) * CH;
  static constexpr uint32_t SMEM = 7 * TILE + 256 + 4 * kQB * 4;
};

// O32: D from the unrounded o (told apart for the registers: with the choice made in the kernel, calls without it took
// 1 % longer).
template <int HD, bool O32>
__global__ void __launch_bounds__(320, 1)
k_window_dq(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmO,
            const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
            const __grid_constant__ CUtensorMap tmK16, const __grid_constant__ CUtensorMap tmV16,
            const __grid_constant__ CUtensorMap tmDq, const __grid_constant__ CUtensorMap tmFo, const WinBwdArgs p,
            const int tiles) {
  using C = DqCfg<HD>;
  constexpr int kKB = C::KB;
  extern __shared__ __align__(1024) uint8_t smem_tiles[];  // no room to round up: its start is aligned
  if (smem_u32(smem_tiles) & 1023) {  // for every thread alike
    dev_fail(DEV_ERR_BAD_INDEX);
    return;
  }
  // Q, dO, K and o [NK], V, dQ on its way out
  uint8_t *sQ = smem_tiles, *sO = sQ + C::TILE, *sK = sO + C::TILE, *sV = sK + C::NK * C::TILE, *sG = sV + C::TILE;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sG + C::TILE);
  uint64_t *a_full = bars, *s_free = bars + 1, *ds_full = bars + 2;  // of all 256 row threads
  uint64_t *q_full = bars + 3, *s_full = bars + 4, *dp_full = bars + 5, *done = bars + 6, *v_full = bars + 7,
           *v_empty = bars + 8, *k_full = bars + 9, *k_empty = k_full + C::NK;
  constexpr int kBars = 9 + 2 * C::NK;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kBars);
  float* sD = reinterpret_cast<float*>(bars + kBars + 1);  // [2][2][128]: of a tile, the halves of D
  const int grp = p.hq / p.hkv;
  const int warp = (int)uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kBars; ++i) mbar_init(bars + i, i < 3 ? 256 : 1);
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmO);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmDq);
    tma_prefetch_desc(&tmFo);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Q and dO (64 columns each), S, dP, dQ
  const uint32_t tmem = uniform(*tmem_slot), tA = tmem, tS = tmem + 128, tP = tmem + 256, tQ = tmem + 384;
  pdl_wait();
  pdl_trigger();

  // it counts the CTA's tiles, jj its blocks: barrier phases run on over the tiles. K's ring holds o of a tile
  // and then its blocks; slot and par: its next entry and the parity of that entry's phase.
  bool ok = true;
  int it = 0, jj = 0, slot = 0;
  uint32_t par = 0;
  const auto advance = [&](int n) {
    slot += n;
    while (slot >= C::NK) {
      slot -= C::NK;
      par ^= 1;
    }
  };
  TileWalk tile(p.hq, p.heads, p.S);
  if (warp == 0) {
    int entry = 0;
    for (; tile.x < tiles && ok; ++it, tile.next(p.hq, p.heads, p.S)) {
      const Blocks<kKB> kb(tile.q0, p.S, p.window, p.sinks);
      const int kvh = tile.h / grp;
      if (it > 0 && !(ok = warp_wait(a_full, (it - 1) & 1))) break;  // the last tile's have been copied
      if (elect_one()) {
        mbar_arrive_expect_tx(q_full, 2 * C::TILE);
        load_tile<HD>(sQ, C::CH, &tmQ, q_full, tile.h * HD, tile.q0, tile.b);
        load_tile<HD>(sO, C::CH, &tmO, q_full, tile.h * HD, tile.q0, tile.b);
      }
      __syncwarp();
      for (int j = -1; j < kb.n; ++j, ++entry, advance(1)) {  // -1: o
        if (entry >= C::NK && !(ok = warp_wait(k_empty + slot, par ^ 1))) break;
        if (elect_one()) {
          if (O32 && j < 0) {
            mbar_arrive(k_full + slot);
          } else if (j < 0) {
            mbar_arrive_expect_tx(k_full + slot, C::TILE);
            load_tile<HD>(sK + slot * C::TILE, C::CH, &tmFo, k_full + slot, tile.h * HD, tile.q0, tile.b);
          } else {
            load_keys<HD, kKB>(sK + slot * C::TILE, C::CH, &tmK, &tmK16, k_full + slot, kvh * HD, kb.k0(j), kb.width(j), tile.b);
          }
        }
        __syncwarp();
        if (j < 0) continue;
        if (jj >= 1 && !(ok = warp_wait(v_empty, (jj - 1) & 1))) break;
        if (elect_one()) load_keys<HD, kKB>(sV, C::CH, &tmV, &tmV16, v_full, kvh * HD, kb.k0(j), kb.width(j), tile.b);
        __syncwarp();
        ++jj;
      }
    }
  } else if (warp == 1) {
    constexpr uint32_t idQ = umma_idesc_bf16(128, HD, 0, 1);
    const Desc kk = make_desc(smem_u32(sK), 16, 1024), km = make_desc(smem_u32(sK), C::CH, 1024);  // K- and MN-major
    const Desc vk = make_desc(smem_u32(sV), 16, 1024);
    const auto scores = [&](int w) {  // S = Q K^T
      mma_tt<HD>(tS, tA, at(kk, slot * C::TILE), C::CH, umma_idesc_bf16(128, w, 0, 0));
      umma_commit(s_full);
    };
    const auto dprobs = [&](int w) {  // dP = dO V^T
      mma_tt<HD>(tP, tA + 64, vk, C::CH, umma_idesc_bf16(128, w, 0, 0));
      umma_commit(dp_full);
      umma_commit(v_empty);
    };
    for (; tile.x < tiles && ok; ++it, tile.next(p.hq, p.heads, p.S)) {
      const Blocks<kKB> kb(tile.q0, p.S, p.window, p.sinks);
      advance(1);
      if (!(ok = warp_wait(a_full, it & 1) && warp_wait(k_full + slot, par))) break;
      tc_fence_after();
      int w = kb.width(0);
      if (elect_one()) scores(w);
      __syncwarp();
      if (!(ok = warp_wait(v_full, jj & 1))) break;
      tc_fence_after();
      if (elect_one()) dprobs(w);
      __syncwarp();
      for (int j = 0; j < kb.n; ++j, ++jj) {
        const bool more = j + 1 < kb.n;
        const int next = more ? kb.width(j + 1) : 0, cur = slot;
        advance(1);
        if (more) {
          if (!(ok = warp_wait2(s_free, jj & 1, k_full + slot, par))) break;
          tc_fence_after();
          if (elect_one()) scores(next);
          __syncwarp();
        }
        // dS is written; with a tile's first block its threads have also read the last tile's dQ
        if (!(ok = more ? warp_wait2(v_full, (jj + 1) & 1, ds_full, jj & 1) : warp_wait(ds_full, jj & 1))) break;
        tc_fence_after();
        if (elect_one()) {  // each half of a block's columns holds its own 64 keys' dS
          mma_ts<kKB, 64>(tQ, tP, at(km, cur * C::TILE), idQ, w, j > 0);
          umma_commit(k_empty + cur);
          if (more) dprobs(next);
          else umma_commit(done);
        }
        __syncwarp();
        w = next;
      }
    }
  } else {
    const int g = (int)(threadIdx.x - 64) >> 7;  // half of the columns
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tX = tS + g * 64 + lanes, tY = tP + g * 64 + lanes;
    const float sl2 = p.scale * kLog2e;
    const uint64_t sl = f2(sl2, sl2);
    const auto load_lse = [&] {
      return tile.q0 + r < p.S ? p.lse[((int64_t)tile.b * p.S + tile.q0 + r) * p.hq + tile.h] : INFINITY;
    };
    // the first four warps copy Q's rows of tile `n` into TMEM, the others dO's; each of them forms D = dO . o over
    // half of the columns, o unrounded where it is given: the rounding of o takes dO . (o - bf16 o) from D, and dq
    // then has that times the row's mean key (keys and values with offsets of 4: the q adapter's gradients were off by
    // 0.19 of their largest value, instead of 0.004)
    const auto copy = [&](int n) {
      if (!warp_wait2(q_full, n & 1, k_full + slot, par)) return false;
      const auto row = [&](const uint8_t* t, int e) {  // columns [8 e, 8 e + 8)
        return reinterpret_cast<const uint4*>(t + e / 8 * C::CH + r * 128 + ((e % 8) ^ (r & 7)) * 16);
      };
#pragma unroll
      for (int c = 0; c < HD / 64; ++c) {
        uint32_t w[32];
#pragma unroll
        for (int e = 0; e < 8; ++e) *reinterpret_cast<uint4*>(w + 4 * e) = *row(g ? sO : sQ, 8 * c + e);
        tmem_st32(tA + g * 64 + c * 32 + lanes, w);
      }
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
      const auto dot = [&](int e, const float2 (&o)[4]) {  // over columns [8 e, 8 e + 8) of this half
        const uint4 d4 = *row(sO, g * (HD / 16) + e);
        const uint32_t d[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float2 d2 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(d + u));
          sum[u] = fmaf(d2.x, o[u].x, fmaf(d2.y, o[u].y, sum[u]));
        }
      };
      if constexpr (!O32) {
#pragma unroll
        for (int e = 0; e < HD / 16; ++e) {
          const uint4 o4 = *row(sK + slot * C::TILE, g * (HD / 16) + e);
          const uint32_t w[4] = {o4.x, o4.y, o4.z, o4.w};
          float2 o[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) o[u] = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(w + u));
          dot(e, o);
        }
      } else {
        const int64_t t = (int64_t)tile.b * p.S + min(tile.q0 + r, p.S - 1);
        const float4* src = reinterpret_cast<const float4*>(p.o32 + (t * p.hq + tile.h) * HD + g * (HD / 2));
#pragma unroll
        for (int e = 0; e < HD / 16; ++e) {
          const float4 a = src[2 * e], b = src[2 * e + 1];
          dot(e, {make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y), make_float2(b.z, b.w)});
        }
      }
      sD[((n & 1) * 2 + g) * kQB + r] = tile.q0 + r < p.S ? (sum[0] + sum[1]) + (sum[2] + sum[3]) : 0.f;
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(a_full);
      return true;
    };
    float lse = load_lse();
    // a wait that runs out is shared at the next barrier, which every warp reaches
    ok = sync_all(1, 256, copy(0));
    if (ok && warp == 2 && elect_one()) mbar_arrive(k_empty + slot);
    for (bool another = true; another && ok; ++it) {
      const int q0 = tile.q0, h = tile.h, b = tile.b, i = q0 + r;
      const Blocks<kKB> kb(q0, p.S, p.window, p.sinks);
      another = tile.after() < tiles;
      const float D = sD[(it & 1) * 2 * kQB + r] + sD[((it & 1) * 2 + 1) * kQB + r], lse2 = lse * kLog2e;
      const uint64_t ln = f2(-lse2, -lse2), Dn = f2(-D, -D);
      p.D[stat_row(b, h, p.hq, p.S) + g * up(p.S, kQB) + i] = g ? D : lse2;
      if (another) {
        tile.next(p.hq, p.heads, p.S);
        lse = load_lse();  // under this tile
      }
      for (int j = 0; j < kb.n; ++j, ++jj) {  // columns [64 g, 64 g + 64) of each block
        if (!(ok = warp_wait(s_full, jj & 1))) break;
        tc_fence_after();
        const int k0 = kb.k0(j);
        float a[64], y[64];
        uint32_t w[32];
        tmem_row<64>(a, tX);
        tc_fence_before();
        mbar_arrive(s_free);
#pragma unroll
        for (int c = 0; c < 32; ++c) ex2_pair(fma2(f2(a[2 * c], a[2 * c + 1]), sl, ln), a[2 * c], a[2 * c + 1]);
        if (!all_visible(q0, kQB, k0, kKB, p.window, p.sinks)) {  // also what lies behind a narrower block
          const uint64_t vis = visible_keys(i, k0 + g * 64, p.window, p.sinks);
          const uint32_t bits[2] = {(uint32_t)vis, (uint32_t)(vis >> 32)};
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (!(bits[c / 32] >> (c % 32) & 1)) a[c] = 0.f;
        }
        if (!(ok = warp_wait(dp_full, jj & 1))) break;
        tc_fence_after();
        tmem_row<64>(y, tY);
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          float d0, d1;
          unpack(mul2(f2(a[2 * c], a[2 * c + 1]), add2(f2(y[2 * c], y[2 * c + 1]), Dn)), d0, d1);
          w[c] = pack2(d0, d1);
        }
        tmem_st16(tY, w);
        tmem_st16(tY + 16, w + 16);
        tmem_st_wait();
        tc_fence_before();
        if (warp == 2 && j + 1 == kb.n) tma_store_wait();  // the last tile's dQ has left sG; `done` tells the others
        mbar_arrive(ds_full);
      }
      advance(kb.n + 1);  // o of the next tile
      if (ok && another) ok = copy(it + 1);
      if ((ok = ok && warp_wait(done, it & 1))) {
        tc_fence_after();
        float lo[HD / 4], hi[HD / 4];
        tmem_row<HD / 4>(lo, tQ + g * (HD / 4) + lanes);
        tmem_row<HD / 4>(hi, tQ + g * (HD / 4) + HD / 2 + lanes);
        stage_grad<HD>(sG, C::CH, r, lo, hi, p, i, g);
        fence_proxy_async();
      }
      if (!(ok = sync_all(1, 256, ok))) break;
      if (warp == 2 && elect_one()) {
        if (another) mbar_arrive(k_empty + slot);
#pragma unroll
        for (int c = 0; c < HD / 64; ++c) tma_store_3d(&tmDq, sG + c * C::CH, h * HD + c * 64, q0, b);
      }
      __syncwarp();
    }
    if (warp == 2) tma_store_wait();
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
// An item is 128 keys of a kv head against 128 queries of one of its heads; the items of a key tile lie by head, by
// query block. The tiles lie in a row, by sequence and kv head (a unit), those that hold sinks, whose queries
// reach to the sequence's end, behind all others. Of the row's front each CTA takes every ctas-th tile whole, so
// that the CTAs at work are on neighbouring tiles, which share most of Q and dO (with neighbouring tiles in one
// CTA instead, 685 MB came from HBM for 9472 tokens rather than 196, and the kernel took 10 % longer); the rest
// is cut, at fixed places, to make the CTAs' work equal. What a tile costs besides its items (K, V, the
// stores) counts as kSeg items in front of them, which also moves cuts next to a tile's border onto the
// border (with 1 item 2048 tokens, 32 heads of 128 over 8, window 512 take 85.4 us instead of 81.0, 1024 tokens, window
// 1024, 47.6 instead of 45.8; with 4 items 81.3 and 46.2, and 2 x 512, window 256, 37.8 instead of 37.1). The sums of a cut tile's parts go to the scratch as fp32, where k_window_join adds them in order.
constexpr int kSms = 148, kSeg = 2;
struct Split {
  int nkb, nsb;  // key tiles of a sequence, those that hold sinks
  int near;      // query blocks that see a tile through the window
  int grp;       // heads of a kv head
  int plain;     // tiles without sinks, of all units
  int ctas, rounds;  // each CTA's whole tiles
  // CTA c's share of the rest: from place off[c] of tile[c] to place off[c + 1] of tile[c + 1]
  int tile[kSms + 1], off[kSms + 1];
  __host__ __device__ int blocks(int kb) const {  // query blocks that see a key tile
    const int n = nkb - kb;
    return kb < nsb || n < near ? n : near;
  }
  __host__ __device__ void locate(int t, int& bk, int& kb) const {  // unit and key tile of the row's tile t
    const int n = t < plain ? nkb - nsb : nsb, u = t < plain ? t : t - plain;
    bk = u / n;
    kb = u % n + (t < plain ? nsb : 0);
  }
  __host__ __device__ bool cut(int c) const { return off[c] > kSeg; }  // border c lies inside of tile[c]'s items
};
// A CTA's tiles: items [i0, i1) of key tile kb of unit bk, seen by nqb query blocks.
struct Share {
  int round, t;  // the next round, or tile of the cut rest
  int bk, kb, nqb, i0, i1;
  __device__ __forceinline__ Share() : round(0), t(-1) {}
  __device__ __forceinline__ bool next(const Split& sp) {
    const int c = blockIdx.x;
    if (round < sp.rounds) {
      sp.locate(c + sp.ctas * round++, bk, kb);
      nqb = sp.blocks(kb);
      i0 = 0;
      i1 = sp.grp * nqb;
      return true;
    }
    if (t < 0) t = sp.tile[c];
    while (t <= sp.tile[c + 1]) {
      const bool head = t == sp.tile[c], tail = t == sp.tile[c + 1];
      if (tail && !sp.cut(c + 1)) break;
      sp.locate(t++, bk, kb);
      nqb = sp.blocks(kb);
      i0 = head ? max(sp.off[c] - kSeg, 0) : 0;
      i1 = tail ? sp.off[c + 1] - kSeg : sp.grp * nqb;
      if (i1 > i0) return true;
    }
    return false;
  }
  __device__ __forceinline__ bool all(const Split& sp) const { return i1 - i0 == sp.grp * nqb; }
};

// Where columns [col, col + 4) of dK (dv 0) or dV (dv 1) of CTA c's part lie in the scratch, in units of 4
// floats: those of a tile's 128 rows one behind the other, as the threads that own a row each store them.
// A CTA has at most two parts: the end of a tile (slot 0) and the start of another (slot 1).
template <int HD>
__device__ __forceinline__ int64_t part_at(int c, int slot, int dv, int col) {
  return (((int64_t)c * 2 + slot) * 2 + dv) * (HD / 4 * kQB) + col / 4 * kQB;
}

template <int HD>
struct DkvCfg {
  static constexpr int QB = 128, NQ = 3, NO = 2;  // rows of a query block, blocks of Q and of dO in flight
  static constexpr uint32_t CH = kQB * 128;      // [128 x 64] bf16
  static constexpr uint32_t TILE = (HD / 64) * CH;
  static constexpr uint32_t SMEM = (2 + NQ + NO) * TILE + (NQ + NO) * QB * 4 + 256;
};

// 320 threads: warp 0 TMA, warp 1 the MMAs, warps 2-9 two threads a key row (half a block's queries each).
//   S^T = K Q^T, P^T = 2^(S' - lse'), dP^T = V dO^T, dS^T = P^T (dP^T - D),
//   dV += P^T dO, dK += dS^T Q with P^T and dS^T, as bf16 side by side over dP^T in TMEM, as A operands
// (Q and dO read MN-major from the tiles used K-major for the scores). With dV, dK and both scores TMEM is
// full; with K, V, three blocks of Q and two of dO shared memory is, too. P waits in registers for dP, so that S
// of j + 1 is issued once the threads have read S of j; dV and dK of j and dP of j + 1 are issued in one run, since
// the tensor cores' queue is short and a wait in between leaves them idle.
// (P over S makes the next S wait for dV: the backward of 8192 tokens took 518 us against 511. P in shared memory
// leaves room for two blocks of Q only, whose loads then are the chain: 545 against 501. Blocks of 64 queries
// with two buffers of each: 4000 clocks for 128 queries, as at N = 64 an MMA takes 48 clocks for 32.)
// Bound by the chain dS -> dV, dK, dP -> dS (about 2900 clocks an item, of which the tensor cores work 2050): 8192
// tokens, 32 heads of 128 over 8, window 1024, 4 sinks take 245 us, the tensor pipe 68 % active; 4 x 512 tokens
// 34 us, the longest CTA 16 items, the mean 8.6.
template <int HD>
__global__ void __launch_bounds__(320, 1)
k_window_dkdv(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmO,
              const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
              const __grid_constant__ CUtensorMap tmDk, const __grid_constant__ CUtensorMap tmDv, const WinBwdArgs p,
              const __grid_constant__ Split sp, float* __restrict__ parts) {
  using C = DkvCfg<HD>;
  extern __shared__ __align__(1024) uint8_t smem_tiles[];  // no room to round up: its start is aligned
  if (smem_u32(smem_tiles) & 1023) {  // for every thread alike
    dev_fail(DEV_ERR_BAD_INDEX);
    return;
  }
  uint8_t *sK = smem_tiles, *sV = sK + C::TILE, *sQ = sV + C::TILE, *sO = sQ + C::NQ * C::TILE;  // sQ [NQ], sO [NO]
  float *sL = reinterpret_cast<float*>(sO + C::NO * C::TILE), *sD = sL + C::NQ * C::QB;          // lse [NQ], D [NO]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sD + C::NO * C::QB);
  uint64_t *ds_full = bars, *s_free = bars + 1;  // of all 256 row threads
  uint64_t *kv_full = bars + 2, *kv_free = bars + 3, *done = bars + 4, *s_full = bars + 5, *dp_full = bars + 6,
           *q_full = bars + 7, *q_empty = q_full + C::NQ, *o_full = q_empty + C::NQ, *o_empty = o_full + C::NO;
  constexpr int kBars = 7 + 2 * C::NQ + 2 * C::NO;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kBars);
  const int warp = (int)uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kBars; ++i) mbar_init(bars + i, i < 2 ? 256 : 1);
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmO);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmDk);
    tma_prefetch_desc(&tmDv);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot), tS = tmem, tP = tmem + 128, tV = tmem + 256, tK = tmem + 384;
  Share my;
  pdl_wait();
  pdl_trigger();

  // seg counts the CTA's tiles, jj its items: barrier phases run on over the tiles
  int jj = 0;
  bool ok = true;
  if (warp == 0) {
    for (int seg = 0; ok && my.next(sp); ++seg) {
      const int b = my.bk / p.hkv, kvh = my.bk % p.hkv, k0 = my.kb * kQB;
      int h = kvh * sp.grp + my.i0 / my.nqb, qb = my.i0 % my.nqb;
      for (int j = my.i0; j < my.i1; ++j, ++jj) {
        const int s = jj % C::NQ, t = jj % C::NO, q = k0 + qb * C::QB;
        const float* stat = p.D + stat_row(b, h, p.hq, p.S) + q;
        if (jj >= C::NQ && !(ok = warp_wait(&q_empty[s], (jj / C::NQ - 1) & 1))) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&q_full[s], C::TILE + C::QB * 4);
          load_tile<HD>(sQ + s * C::TILE, C::CH, &tmQ, &q_full[s], h * HD, q, b);
          bulk_load(sL + s * C::QB, stat, C::QB * 4, &q_full[s]);
        }
        __syncwarp();
        if (j == my.i0) {
          if (seg > 0 && !(ok = warp_wait(kv_free, (seg - 1) & 1))) break;
          if (elect_one()) {
            mbar_arrive_expect_tx(kv_full, 2 * C::TILE);
            load_tile<HD>(sK, C::CH, &tmK, kv_full, kvh * HD, k0, b);
            load_tile<HD>(sV, C::CH, &tmV, kv_full, kvh * HD, k0, b);
          }
          __syncwarp();
        }
        if (jj >= C::NO && !(ok = warp_wait(&o_empty[t], (jj / C::NO - 1) & 1))) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&o_full[t], C::TILE + C::QB * 4);
          load_tile<HD>(sO + t * C::TILE, C::CH, &tmO, &o_full[t], h * HD, q, b);
          bulk_load(sD + t * C::QB, stat + up(p.S, kQB), C::QB * 4, &o_full[t]);
        }
        __syncwarp();
        if (++qb == my.nqb) {
          qb = 0;
          ++h;
        }
      }
    }
  } else if (warp == 1) {
    constexpr uint32_t idS = umma_idesc_bf16(128, C::QB, 0, 0), idG = umma_idesc_bf16(128, HD, 0, 1);
    const Desc dK = make_desc(smem_u32(sK), 16, 1024), dV = make_desc(smem_u32(sV), 16, 1024);
    const Desc qk = make_desc(smem_u32(sQ), 16, 1024), qm = make_desc(smem_u32(sQ), C::CH, 1024);  // K- and MN-major
    const Desc ok_ = make_desc(smem_u32(sO), 16, 1024), om = make_desc(smem_u32(sO), C::CH, 1024);
    // the next slots of the rings of Q and dO and the parities of their phases
    int sq = 0, so = 0;
    uint32_t pq = 0, po = 0;
    const auto scores = [&] {  // S^T = K Q^T
      mma_ss<HD>(tS, dK, C::CH, at(qk, sq * C::TILE), C::CH, idS);
      umma_commit(s_full);
    };
    const auto dprobs = [&] {  // dP^T = V dO^T
      mma_ss<HD>(tP, dV, C::CH, at(ok_, so * C::TILE), C::CH, idS);
      umma_commit(dp_full);
    };
    for (int seg = 0; ok && my.next(sp); ++seg) {
      if (!(ok = warp_wait2(kv_full, seg & 1, &q_full[sq], pq))) break;
      tc_fence_after();
      if (elect_one()) scores();
      __syncwarp();
      if (!(ok = warp_wait(&o_full[so], po))) break;
      tc_fence_after();
      if (elect_one()) dprobs();
      __syncwarp();
      bool add = false;
      for (int n = my.i1 - my.i0; n > 0; --n, ++jj) {
        const int q0 = sq, o0 = so;
        if (++sq == C::NQ) {
          sq = 0;
          pq ^= 1;
        }
        if (++so == C::NO) {
          so = 0;
          po ^= 1;
        }
        if (n > 1) {
          if (!(ok = warp_wait2(s_free, jj & 1, &q_full[sq], pq))) break;
          tc_fence_after();
          if (elect_one()) scores();
          __syncwarp();
        }
        // dS and P are written; with a tile's first item its threads have also read the last tile's dV and dK
        if (!(ok = n > 1 ? warp_wait2(&o_full[so], po, ds_full, jj & 1) : warp_wait(ds_full, jj & 1))) break;
        tc_fence_after();
        if (elect_one()) {
          mma_ts<C::QB, 32>(tV, tP + 16, at(om, o0 * C::TILE), idG, C::QB, add);
          umma_commit(&o_empty[o0]);
          mma_ts<C::QB, 32>(tK, tP, at(qm, q0 * C::TILE), idG, C::QB, add);
          umma_commit(&q_empty[q0]);
          if (n > 1) dprobs();
          else umma_commit(done);
        }
        __syncwarp();
        add = true;
      }
    }
  } else {
    const int half = (int)(threadIdx.x - 64) >> 7;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tX = tS + half * 64 + lanes, tY = tP + half * 64 + lanes;
    const uint64_t sl = f2(p.scale * kLog2e, p.scale * kLog2e);
    for (int seg = 0; ok && my.next(sp); ++seg) {
      const int k0 = my.kb * kQB, key = k0 + r;
      int qb = my.i0 % my.nqb;
      for (int j = my.i0; j < my.i1; ++j, ++jj) {
        const int q = k0 + qb * C::QB;
        if (!(ok = warp_wait(&q_full[jj % C::NQ], (jj / C::NQ) & 1) && warp_wait(s_full, jj & 1))) break;
        tc_fence_after();
        // lse and D of this thread's 64 queries
        const float4* lse = reinterpret_cast<const float4*>(sL + jj % C::NQ * C::QB) + half * 16;
        const float4* del = reinterpret_cast<const float4*>(sD + jj % C::NO * C::QB) + half * 16;
        float x[64];
        tmem_row<64>(x, tX);
        tc_fence_before();
        mbar_arrive(s_free);
#pragma unroll
        for (int c = 0; c < 64; c += 4) {
          const float4 l4 = lse[c / 4];
          ex2_pair(fma2(f2(x[c], x[c + 1]), sl, f2(-l4.x, -l4.y)), x[c], x[c + 1]);
          ex2_pair(fma2(f2(x[c + 2], x[c + 3]), sl, f2(-l4.z, -l4.w)), x[c + 2], x[c + 3]);
        }
        if (!all_visible(q, C::QB, k0, kQB, p.window, p.sinks)) {
          const uint64_t vis = visible_queries(key, q + half * 64, p.window, p.sinks);
          const uint32_t bits[2] = {(uint32_t)vis, (uint32_t)(vis >> 32)};
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (!(bits[c / 32] >> (c % 32) & 1)) x[c] = 0.f;
        }
        if (!(ok = warp_wait(&o_full[jj % C::NO], (jj / C::NO) & 1) && warp_wait(dp_full, jj & 1))) break;
        tc_fence_after();
#pragma unroll
        for (int g = 0; g < 64; g += 32) {  // 32 queries' dP make room for 16 columns of dS and 16 of P
          float y[32];
          uint32_t w[32];
          tmem_row<32>(y, tY + g);
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            const float4 d4 = del[(g + c) / 4];
            const float* v = x + g + c;
            float a0, a1, a2, a3;
            unpack(mul2(f2(v[0], v[1]), add2(f2(y[c], y[c + 1]), f2(-d4.x, -d4.y))), a0, a1);
            unpack(mul2(f2(v[2], v[3]), add2(f2(y[c + 2], y[c + 3]), f2(-d4.z, -d4.w))), a2, a3);
            w[c / 2] = pack2(a0, a1);
            w[c / 2 + 1] = pack2(a2, a3);
            w[16 + c / 2] = pack2(v[0], v[1]);
            w[16 + c / 2 + 1] = pack2(v[2], v[3]);
          }
          tmem_st32(tY + g, w);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(ds_full);
        if (++qb == my.nqb) qb = 0;
      }
      const bool all = my.all(sp);
      // a wait that runs out is shared at the barrier below, which every warp reaches
      if ((ok = ok && warp_wait(done, seg & 1))) {
        tc_fence_after();
        if (!all && warp == 2 && elect_one()) mbar_arrive(kv_free);
        if (all) {  // K's and V's shared memory takes the tiles of dK and dV
          float x0[HD / 4], x1[HD / 4];
          tmem_row<HD / 4>(x0, tK + half * (HD / 4) + lanes);
          tmem_row<HD / 4>(x1, tK + half * (HD / 4) + HD / 2 + lanes);
          stage_grad<HD>(sK, C::CH, r, x0, x1, p, key, half);
          if (HD == 128 || half == 0) {
            float v[64];
            uint32_t w[32];
            tmem_row<64>(v, tV + half * 64 + lanes);
#pragma unroll
            for (int e = 0; e < 32; ++e) w[e] = pack2(v[2 * e], v[2 * e + 1]);
            stage_row(sV + half * C::CH, r, w);
          }
          fence_proxy_async();
        } else {
          float4* dst = reinterpret_cast<float4*>(parts) + part_at<HD>(blockIdx.x, my.i0 == 0, half, 0) + r;
#pragma unroll 1
          for (int c = 0; c < HD; c += 32) {
            float v[32];
            tmem_row<32>(v, (half ? tV : tK) + c + lanes);
#pragma unroll
            for (int e = 0; e < 8; ++e) dst[(c / 4 + e) * kQB] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
          }
        }
      }
      if (!(ok = sync_all(1, 256, ok))) break;
      if (all && warp == 2 && elect_one()) {
        const int b = my.bk / p.hkv, kvh = my.bk % p.hkv;
#pragma unroll
        for (int c = 0; c < HD / 64; ++c) {
          tma_store_3d(&tmDk, sK + c * C::CH, kvh * HD + c * 64, k0, b);
          tma_store_3d(&tmDv, sV + c * C::CH, kvh * HD + c * 64, k0, b);
        }
        tma_store_wait();
        mbar_arrive(kv_free);
      }
      __syncwarp();
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

// Adds the parts of a cut tile in order: a warp takes 32 rows, 8 columns of dK or dV and their 8 rotary partners.
// Grid: HD / 16 CTAs for each border between two shares; the first one that cuts a tile stands for it. Bound by the
// parts' way through L2: 16 us for 147 cuts of 128 KB each side, read cold.
template <int HD>
__global__ void __launch_bounds__(256) k_window_join(const WinBwdArgs p, const __grid_constant__ Split sp,
                                                     const float* __restrict__ parts) {
  const int cut = 1 + (int)blockIdx.x / (HD / 16), o = (int)blockIdx.x % (HD / 16) * 8, warp = threadIdx.x >> 5;
  const int dv = warp >> 2, r = (warp & 3) * 32 + (threadIdx.x & 31);
  pdl_wait();
  pdl_trigger();
  if (!sp.cut(cut) || (sp.tile[cut - 1] == sp.tile[cut] && sp.cut(cut - 1))) return;
  int bk, kb;
  sp.locate(sp.tile[cut], bk, kb);
  const int b = bk / p.hkv, kvh = bk % p.hkv, key = kb * kQB + r;
  if (key >= p.S) return;
  float lo[8] = {}, hi[8] = {};
  for (int c = cut - 1; c < cut || (c < sp.ctas && sp.tile[c] == sp.tile[cut]); ++c) {
    if (c >= cut && sp.tile[c + 1] == sp.tile[c] && sp.off[c + 1] == sp.off[c]) continue;  // an empty share
    const float4* src = reinterpret_cast<const float4*>(parts) + part_at<HD>(c, c < cut, dv, o) + r;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float4 x = src[e * kQB], y = src[(HD / 8 + e) * kQB];
      lo[4 * e] += x.x, lo[4 * e + 1] += x.y, lo[4 * e + 2] += x.z, lo[4 * e + 3] += x.w;
      hi[4 * e] += y.x, hi[4 * e + 1] += y.y, hi[4 * e + 2] += y.z, hi[4 * e + 3] += y.w;
    }
  }
  if (!dv) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      lo[e] *= p.scale;
      hi[e] *= p.scale;
      if (p.rope_cos) {
        const int64_t t = (int64_t)key * (HD / 2) + o + e;
        const float cs = p.rope_cos[t], sn = p.rope_sin[t], z = lo[e] * cs + hi[e] * sn;
        hi[e] = hi[e] * cs - lo[e] * sn;
        lo[e] = z;
      }
    }
  }
  __nv_bfloat16* out = (dv ? p.dv : p.dk) + ((int64_t)b * p.S + key) * (dv ? p.lddv : p.lddk) + (int64_t)kvh * HD + o;
  *reinterpret_cast<uint4*>(out) = make_uint4(pack2(lo[0], lo[1]), pack2(lo[2], lo[3]), pack2(lo[4], lo[5]), pack2(lo[6], lo[7]));
  *reinterpret_cast<uint4*>(out + HD / 2) = make_uint4(pack2(hi[0], hi[1]), pack2(hi[2], hi[3]), pack2(hi[4], hi[5]), pack2(hi[6], hi[7]));
}

// How the dK / dV work is dealt out. As many rounds of whole tiles as leave no CTA with more than its share; where
// the tiles are as few as the SMs, a CTA each, if the longest of them takes no longer than equal shares and the
// stores and the kernel that join them (about kJoin items). Backward in whole tiles and in shares, by how many items the
// longest tile is above an equal share: 4, 8 x 256 tokens, 36 us against 45; 8, 4 x 512, 52.5 against 57.0; 9, 2048
// tokens, 8 heads each of its own, 51.1 against 53.3; 12, 300 tokens, 30.5 against 27.5; 13, 2 x 512, 42.5 against 37.0.
constexpr int kJoin = 10;
Split make_split(int64_t T, int S, int hq, int hkv, int window, int sinks) {
  const int64_t units = T / S * hkv;
  Split s;
  s.nkb = (S + kQB - 1) / kQB;
  s.nsb = (int)(((int64_t)std::min(sinks, S) + kQB - 1) / kQB);
  s.near = (int)std::min<int64_t>(s.nkb, ((int64_t)kQB - 2 + std::min(window, S)) / kQB + 1);
  s.grp = hq / hkv;
  s.plain = (int)(units * (s.nkb - s.nsb));
  const int tiles = (int)(units * s.nkb);
  const auto cost = [&](int t) {
    int bk, kb;
    s.locate(t, bk, kb);
    return (int64_t)s.grp * s.blocks(kb) + kSeg;
  };
  int64_t total = 0;
  for (int kb = 0; kb < s.nkb; ++kb) total += units * ((int64_t)s.grp * s.blocks(kb) + kSeg);
  const int64_t items = total - (int64_t)kSeg * tiles;
  s.ctas = (int)std::min<int64_t>(kSms, std::max<int64_t>(1, items / 2));
  s.rounds = 0;
  if (tiles <= kSms && (int64_t)s.grp * s.blocks(0) + kSeg <= total / s.ctas + kJoin) {
    s.ctas = tiles;
    s.rounds = 1;
  }
  int64_t own[kSms] = {};  // whole tiles of each CTA
  if (s.rounds == 0) {
    for (int64_t t = 0; t + s.ctas <= s.plain; t += s.ctas, ++s.rounds) {
      bool fits = true;
      for (int c = 0; c < s.ctas; ++c) fits = fits && own[c] + cost((int)t + c) <= total / s.ctas;
      if (!fits) break;
      for (int c = 0; c < s.ctas; ++c) own[c] += cost((int)t + c);
    }
  } else {
    for (int c = 0; c < s.ctas; ++c) own[c] = cost(c);
  }
  int t = s.rounds * s.ctas;
  int64_t at = 0;  // place in tile t
  for (int c = 0; c <= s.ctas; ++c) {
    while (t < tiles && (c == s.ctas || at >= cost(t))) at -= cost(t++);
    s.tile[c] = t;
    s.off[c] = t < tiles ? (int)at : 0;
    if (c < s.ctas) at += std::max<int64_t>(0, total * (c + 1) / s.ctas - total * c / s.ctas - own[c]);
  }
  return s;
}
// The same, kept for a thread's next call: a model's layers ask for the same sizes.
const Split& plan_split(int64_t T, int S, int hq, int hkv, int window, int sinks) {
  struct Key {
    int64_t T;
    int S, hq, hkv, window, sinks;
  };
  static thread_local Key last{0, 0, 0, 0, 0, 0};
  static thread_local Split split;
  if (last.T != T || last.S != S || last.hq != hq || last.hkv != hkv || last.window != window || last.sinks != sinks) {
    split = make_split(T, S, hq, hkv, window, sinks);
    last = Key{T, S, hq, hkv, window, sinks};
  }
  return split;
}
// parts that go to the scratch
int64_t split_parts(const Split& s) {
  for (int c = 1; c < s.ctas; ++c)
    if (s.cut(c)) return 2 * (int64_t)s.ctas;
  return 0;
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

template <int HD, int PARTS>
cudaError_t launch_fwd(const WinArgs& a, cudaStream_t s) {
  using C = FwdCfg<HD>;
  const int64_t B = a.T / a.S, cq = (int64_t)a.hq * HD, ck = (int64_t)a.hkv * HD;
  CUtensorMap q, k, v, k16, v16, o;
  if (!make_map3(&q, a.q, B, a.S, cq, a.ldq, kQB) || !make_map3(&k, a.k, B, a.S, ck, a.ldk, C::KB) ||
      !make_map3(&v, a.v, B, a.S, ck, a.ldv, C::KB) || !make_map3(&k16, a.k, B, a.S, ck, a.ldk, 16) ||
      !make_map3(&v16, a.v, B, a.S, ck, a.ldv, 16) || !make_map3(&o, a.o, B, a.S, cq, a.ldo, kQB))
    return cudaErrorInvalidValue;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem(k_window_fwd<HD, PARTS>, C::SMEM, done);
  if (e != cudaSuccess) return e;
  const int64_t tiles = B * a.hq * ((a.S + kQB - 1) / kQB);
  return launch_k(k_window_fwd<HD, PARTS>, dim3((unsigned)tiles), dim3(192), C::SMEM, s, 0, q, k, v, k16, v16, o, a,
                  2 * device_sm_count());
}

template <int HD>
cudaError_t launch_bwd(const WinBwdArgs& a, cudaStream_t s) {
  using Q = DqCfg<HD>;
  using K = DkvCfg<HD>;
  const int64_t B = a.T / a.S, cq = (int64_t)a.hq * HD, ck = (int64_t)a.hkv * HD;
  CUtensorMap q, o, k, v, k16, v16, dq, dk, dv, fo;
  if (!make_map3(&q, a.q, B, a.S, cq, a.ldq, kQB) || !make_map3(&o, a.dout, B, a.S, cq, a.lddo, kQB) ||
      !make_map3(&k, a.k, B, a.S, ck, a.ldk, Q::KB) || !make_map3(&v, a.v, B, a.S, ck, a.ldv, Q::KB) ||
      !make_map3(&k16, a.k, B, a.S, ck, a.ldk, 16) || !make_map3(&v16, a.v, B, a.S, ck, a.ldv, 16) ||
      !make_map3(&dq, a.dq, B, a.S, cq, a.lddq, kQB) || !make_map3(&fo, a.o, B, a.S, cq, a.ldo, kQB) ||
      !make_map3(&dk, a.dk, B, a.S, ck, a.lddk, kQB) ||
      !make_map3(&dv, a.dv, B, a.S, ck, a.lddv, kQB))
    return cudaErrorInvalidValue;
  static std::atomic<unsigned long long> done_q[2] = {{0}, {0}}, done_k{0};
  const auto dq_kernel = a.o32 ? k_window_dq<HD, true> : k_window_dq<HD, false>;
  cudaError_t e = allow_smem(dq_kernel, Q::SMEM, done_q[a.o32 != nullptr]);
  if (e == cudaSuccess) e = allow_smem(k_window_dkdv<HD>, K::SMEM, done_k);
  if (e != cudaSuccess) return e;
  const int tiles = (int)(B * a.hq * ((a.S + kQB - 1) / kQB));
  e = launch_k(dq_kernel, dim3((unsigned)std::min(tiles, device_sm_count())), dim3(320), Q::SMEM, s, 0, q, o, k, v, k16,
               v16, dq, fo, a, tiles);
  note_launch(1);
  if (e != cudaSuccess) return e;
  const Split& sp = plan_split(a.T, a.S, a.hq, a.hkv, a.window, a.sinks);
  float* parts = a.D + 2 * B * a.hq * up(a.S, kQB);
  e = launch_k(k_window_dkdv<HD>, dim3((unsigned)sp.ctas), dim3(320), K::SMEM, s, 0, q, o, k, v, dk, dv, a, sp,
               parts);
  note_launch(1);
  if (e != cudaSuccess || split_parts(sp) == 0) return e;
  e = launch_k(k_window_join<HD>, dim3((unsigned)(sp.ctas - 1) * (HD / 16)), dim3(256), 0, s, 0, a, sp, static_cast<const float*>(parts));
  note_launch(1);
  return e;
}

}  // namespace

bool window_shape_ok(int64_t T, int S, int hq, int hkv, int hd, int window, int sinks) {
  return (hd == 64 || hd == 128) && hq > 0 && hkv > 0 && hq % hkv == 0 && S > 0 && T > 0 && T % S == 0 &&
         S <= (1 << 30) && T <= INT32_MAX && T * hq <= INT32_MAX && T / S * hkv <= 65535 && window >= 1 && sinks >= 0;
}

int64_t window_scratch(int64_t T, int S, int hq, int hkv, int hd, int window, int sinks) {
  const Split& sp = plan_split(T, S, hq, hkv, std::min(window, S), std::min(sinks, S));
  return T / S * 2 * hq * up(S, kQB) + split_parts(sp) * kQB * 2 * hd;
}

cudaError_t window_fwd(WinArgs a, cudaStream_t s) {
  if (!window_shape_ok(a.T, a.S, a.hq, a.hkv, a.hd, a.window, a.sinks)) return cudaErrorInvalidValue;
  a.window = std::min(a.window, a.S);
  a.sinks = std::min(a.sinks, a.S);
  a.heads = (int)(a.T / a.S) * a.hq;
  const cudaError_t e = a.parts == 2 ? (a.hd == 128 ? launch_fwd<128, 2>(a, s) : launch_fwd<64, 2>(a, s))
                                     : (a.hd == 128 ? launch_fwd<128, 1>(a, s) : launch_fwd<64, 1>(a, s));
  note_launch(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t window_bwd(WinBwdArgs a, cudaStream_t s) {
  if (!window_shape_ok(a.T, a.S, a.hq, a.hkv, a.hd, a.window, a.sinks)) return cudaErrorInvalidValue;
  a.window = std::min(a.window, a.S);
  a.sinks = std::min(a.sinks, a.S);
  a.heads = (int)(a.T / a.S) * a.hq;
  const cudaError_t e = a.hd == 128 ? launch_bwd<128>(a, s) : launch_bwd<64>(a, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace lst
