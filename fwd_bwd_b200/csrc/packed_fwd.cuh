// packed_fwd.cuh -- 16-bit softmax attention over packed sequences with grouped heads, forward.
//
//   z_ij = tau q_i . k_j over the keys j of i's sequence (j <= i when causal)
//   O_i = sum_j softmax(z_i)_j v_j,  LSE_i = log sum_j exp(z_ij)
//
// Tiles: a sequence of n tokens is cut into ceil(n / 128) tiles FROM ITS END, so only its
// first tile is ragged, and query and key tiles share one alignment (the causal diagonal is the
// diagonal of a tile).  The tiles are loaded through 4-D tensor maps (channel, row, token, head)
// whose row and token axes have the same stride: the ragged tile starts at a negative row, which
// the TMA unit reads as zeros, so no row of a neighbouring sequence ever enters shared memory
// and non-finite values cannot leak through a product with a zero probability.
//
// attn_fwd_kernel (d = 128), per CTA: two query tiles that share their keys: two heads of one group
// (an even number of query heads per key head), else two neighbouring tiles of one head.
//   warps 0-3, 4-7  softmax of tile 0 / 1, one query row per thread
//   warp 8          TMA producer: the query tiles, then K and V tiles through a ring
//   warp 9          MMA issuer: S = Q K^T (operands in shared memory), O += P V (P in TMEM)
//   warps 10-11     idle (they complete the warpgroup that gives its registers away)
// TMEM: S of tile g at 128 g (P overwrites its first 64 columns, two 16-bit values each), O of
// tile g at 256 + 128 g, accumulated there over all keys.
// The tensor core alternates between the tiles: while tile 0's softmax runs, it multiplies tile
// 1's P V and Q K^T.  S of the next key tile is issued after P V of this one, so its arrival
// also tells the softmax warps that O is up to date.
//
// attn_fwd64_kernel (d = 64), per CTA: one query tile, keys in runs of 64, a quarter of an SM's TMEM,
// registers and shared memory: the products of d = 64 are short and the softmax is a chain of
// latencies, so four CTAs share an SM and hide each other's, first loads and last stores included.
//   warps 0-3  softmax, one query row per thread;  warp 4  TMA and MMA issue
// TMEM: S at 0 (P over its first 32 columns), O at 64.  One thread issues everything: once P of a
// run has arrived, the run's Q K^T and the last run's P V are complete, so their K and V
// buffers are free without further barriers.
//
// Both: the running maximum that P is taken against is raised (and O rescaled in TMEM) only when
// a row's maximum grows by more than 2^8: P then stays below 256, exact in the final division
// by the row sum, and most key tiles leave O untouched.
// A row that sees a score of NaN or +inf is NaN in O and LSE: the maximum keeps NaN, and the row's
// exponentials, sum and rescaled O are NaN from that tile on.
// Rounding: P (in half precision times 2^7, kFwdShift) to the tensors' type for P V (the sum l uses
// the unrounded P); O once at the end.
// A quarter of the exponentials runs on the FMA pipe (32 heads of 128, prompts of 4099 to 8 tokens:
// 222 us, 224 us with an eighth, 225 us with none; d = 64, images: 38 us against 39 us).
//
// Measured (B200, kernel time; causal, 2 products counted over the visible scores):
//   d = 128, 16384 tokens, 32 / 8 heads, bf16                1627 us, 1352 TFLOP/s
//   d = 128, 4 x 8192, 16 heads                               851 us, 1293 TFLOP/s
//   d = 64, 8 x 2048, 16 heads                                111 us,  620 TFLOP/s
// (cuBLAS bf16: 1614 TFLOP/s for a moment, 1368 under the power cap, which the first two reach
// after some milliseconds: 1871 us in a loop.)  Bound: d = 128 by the chain S -> softmax -> P V of
// two tiles that take turns (tensor pipe 58% active, special-function unit 45%); d = 64 by the
// exponentials and the instructions around them (issue 50%, special-function unit 49%, tensor
// pipe 31%), with a fixed 28 us for setting up and storing 2048 CTAs, partly hidden by the four to
// an SM.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stddef.h>
#include <stdint.h>

#include <type_traits>

#include "ptx.cuh"
#include "rowops.cuh"

namespace sage {
namespace packed {

constexpr int BT = 128;  // tokens per tile

// One tile of a sequence (or the later of two neighbouring tiles).
struct Item {
  int start;  // first row of the sequence
  int len;    // tokens of the sequence
  int tile;   // tile index, 0 = the ragged one
  int seq;    // sequence index
};

__host__ __device__ __forceinline__ int tiles_of(const Item& it) {
  return static_cast<int>((static_cast<int64_t>(it.len) + BT - 1) / BT);
}

// The grid's order: the heads in chunks, within a chunk the items in list order (most work
// first), within an item the chunk's heads.  A chunk is sized so that what its CTAs read over and
// over (keys and values, or queries and gradients) stays in L2.
struct Grid {
  const Item* items;
  int n_items, heads, chunk;
};
__device__ __forceinline__ Item grid_at(const Grid& g, int& head) {
  const int64_t per = static_cast<int64_t>(g.n_items) * g.chunk;
  const int c = static_cast<int>(blockIdx.x / per);
  const int rest = static_cast<int>(blockIdx.x - c * per);
  const int n = min(g.chunk, g.heads - c * g.chunk);
  head = c * g.chunk + rest % n;
  return g.items[rest / n];
}

struct Out {
  char* ptr;
  int64_t ts, hs;  // elements
};

// Row and token coordinates of the t-th run of R rows in the 4-D maps.
struct TileAt {
  int row, token;
};
template <int R>
__device__ __forceinline__ TileAt tile_at(const Item& it, int t) {
  const int first = t * R - (tiles_of(it) * BT - it.len);  // negative: padding
  TileAt a;
  a.row = min(first, 0);
  a.token = it.start + max(first, 0);
  return a;
}
// Index within the sequence of row r of the t-th run of R rows (negative: padding).
template <int R = BT>
__device__ __forceinline__ int row_index(const Item& it, int t, int r) {
  return t * R - tiles_of(it) * BT + it.len + r;
}

// Loads tile t of N rows by boxes of BOX rows x 64 channels (128-byte swizzled rows; the tile's
// 64-channel parts follow each other).
template <typename T, int D, int BOX, int N>
__device__ __forceinline__ void load_tile(T* dst, const CUtensorMap* map, const Item& it, int t,
                                          int head, uint64_t* bar) {
#pragma unroll
  for (int s = 0; s < N / BOX; ++s) {
    const TileAt at = tile_at<BOX>(it, t * (N / BOX) + s);
#pragma unroll
    for (int b = 0; b < D / 64; ++b)
      tma_load_4d(dst + b * N * 64 + s * BOX * 64, map, b * 64, at.row, at.token, head, bar);
  }
}

// Operand descriptors of a tile: the K-major form (K = 16 channels per step) and the MN-major form
// (channels as N, 16 rows of the tile as K per step).  A step adds a constant to the address
// field (16-byte units), so the issuing thread spends one addition per instruction.
__device__ __forceinline__ uint64_t desc_k(const void* tile) {
  return smem_desc(smem_u32(tile), 16, 1024, kSwizzle128B);
}
template <int N>  // rows of the tile
__device__ __forceinline__ uint64_t desc_mn(const void* tile) {
  return smem_desc(smem_u32(tile), N * 128, 1024, kSwizzle128B);
}
template <int N>
__host__ __device__ constexpr uint32_t step_k(int kk) {
  return ((kk >> 2) * (N * 128) + (kk & 3) * 32) >> 4;
}
__host__ __device__ constexpr uint32_t step_mn(int kk) { return (kk * 16 * 128) >> 4; }

// D = A B^T over D channels, K-major tiles of 128 and N rows.  (These are for a whole warp.)
template <int D, int N>
__device__ __forceinline__ void mma_rows(uint32_t leader, uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc) {
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk)
    mma_f16_warp(leader, d_tmem, a + step_k<BT>(kk), b + step_k<N>(kk), idesc, kk > 0 ? 1u : 0u);
}
// D (+)= A B over 64 rows of tile B, A in 32 TMEM columns.
__device__ __forceinline__ void mma_sum_half(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem, uint64_t b,
                                             uint32_t idesc, bool start) {
#pragma unroll
  for (int kk = 0; kk < 4; ++kk)
    mma_f16_ts_warp(leader, d_tmem, a_tmem + 8 * kk, b + step_mn(kk), idesc, kk > 0 || !start ? 1u : 0u);
}

// The same over 32 rows.
__device__ __forceinline__ void mma_sum_quarter(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem,
                                                uint64_t b, uint32_t idesc, bool start) {
#pragma unroll
  for (int kk = 0; kk < 2; ++kk)
    mma_f16_ts_warp(leader, d_tmem, a_tmem + 8 * kk, b + step_mn(kk), idesc,
                    kk > 0 || !start ? 1u : 0u);
}

// Position in a ring of N buffers, and the parity of the buffer's current round.
template <int N>
struct Ring {
  int slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      parity ^= 1;
    }
  }
};

// 2^z for a pair as in exp2_poly2, for z <= 127 or NaN.  Below 2^-126 the exponent field runs out at
// -127 and the result is off by up to 2^-127; -inf gives 2^-149, zero in 16 bits.  NaN passes the
// clamp and the polynomial, and the exponent's addition makes it the largest float, infinity in 16
// bits: with P that is not finite, neither are the sums it enters.
__device__ __forceinline__ float2 exp2_fma2(float2 z) {
  constexpr float kC0 = 1.0000001192092896f, kC1 = 0.6931469440460205f,
                  kC2 = 0.24022120237350464f, kC3 = 0.05550713092088699f,
                  kC4 = 0.009675540961325169f, kC5 = 0.0013276472454890609f;
  const float2 zc = make_float2(fmax_nan(z.x, -127.0f), fmax_nan(z.y, -127.0f));
  const float2 t = __fadd2_rn(zc, make_float2(kMagic, kMagic));
  const float2 j = __fadd2_rn(t, make_float2(-kMagic, -kMagic));
  const float2 f = __ffma2_rn(j, make_float2(-1.0f, -1.0f), zc);
  float2 q = __ffma2_rn(make_float2(kC5, kC5), f, make_float2(kC4, kC4));
  q = __ffma2_rn(q, f, make_float2(kC3, kC3));
  q = __ffma2_rn(q, f, make_float2(kC2, kC2));
  q = __ffma2_rn(q, f, make_float2(kC1, kC1));
  q = __ffma2_rn(q, f, make_float2(kC0, kC0));
  return make_float2(__uint_as_float(__float_as_uint(q.x) + (__float_as_uint(t.x) << 23)),
                     __uint_as_float(__float_as_uint(q.y) + (__float_as_uint(t.y) << 23)));
}

// log2 of the factor that the forward's P (and with it l and O) carries: half precision's normal
// numbers end at 2^-14, so P, at most 2^8, is taken times 2^7: weights down to 2^-21 of the row's
// largest keep all bits.
template <typename T>
constexpr float kFwdShift = std::is_same<T, __half>::value ? 7.0f : 0.0f;

// What the scores of a row are shifted by: -m; 0 while no key weighs anything (m = -inf), so that
// -inf stays -inf; NaN for a maximum of +inf, whose row has no softmax.  P's factor comes on top.
template <typename T>
__device__ __forceinline__ float neg_max(float m) {
  return kFwdShift<T> + (m == -INFINITY ? 0.0f : fmaf(m, 0.0f, -m));
}

// Pairs whose exponentials run on the FMA pipe.
__device__ __forceinline__ constexpr bool poly_pair(int i) { return (i & 3) == 3; }

namespace fwd {

constexpr int kThreads = 384;
constexpr int kProducerWarp = 8, kMmaWarp = 9;
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 216, kOtherRegs = 72;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs,
              "register split exceeds the launch allocation");
constexpr uint32_t kColO = 256;
template <typename T, int D>
struct Smem {
  static_assert(D == 128, "two tiles of d = 128 fill TMEM; d = 64 has its own kernel");
  static constexpr int NST = 5;  // K / V tiles in flight
  alignas(1024) T q[2][BT * D];
  alignas(1024) T kv[NST][BT * D];
  uint64_t q_full, full[NST], empty[NST], s_full[2], p_full[2][2], o_full;
  uint32_t tmem_base;
  int abort;
};

template <typename T, int D>
constexpr size_t smem_bytes() {
  return sizeof(Smem<T, D>) + 1024;
}
static_assert(smem_bytes<__half, 128>() <= 232448, "shared memory exceeds the limit");

struct Args {
  Grid grid;   // heads: CTAs per item
  Out o;
  float* lse;  // [Hq][T]
  int64_t T;
  int group;        // query heads per key head
  int causal;
  float scale_log2;  // softmax_scale log2(e)
  // The walk over a tile's keys may be cut into `splits` parts: the grid then has splits x heads, and
  // a part's unnormalized O goes to part [splits][tokens][Hq][D], its row maxima (log2 units) and
  // sums to stats [splits][tokens][Hq][2].
  int splits, heads;
  float* part;
  float2* stats;
  int64_t tokens;
};

// A row's results: the output and LSE, or this part's share of them.  y: 32 channels from cc on of
// the accumulated O.
template <typename T, bool PARTS>
struct RowOut {
  T* out;
  float* part;
  float inv_l;
  __device__ __forceinline__ void store32(const uint32_t (&y)[32], int cc) const {
#pragma unroll
    for (int e = 0; e < 32; e += 8) {
      float f[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(y[e + k]) * inv_l;
      if (!PARTS) {
        *reinterpret_cast<uint4*>(out + cc + e) = pack8<T>(f);
      } else {
        *reinterpret_cast<float4*>(part + cc + e) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4*>(part + cc + e + 4) = make_float4(f[4], f[5], f[6], f[7]);
      }
    }
  }
};
template <typename T, int D, bool PARTS>
__device__ __forceinline__ RowOut<T, PARTS> row_out(const Args& a, int64_t row, int head, int split,
                                             float m, float l) {
  RowOut<T, PARTS> r;
  r.out = reinterpret_cast<T*>(a.o.ptr) + row * a.o.ts + head * a.o.hs;
  if (!PARTS) {
    r.part = nullptr;
    r.inv_l = 1.0f / l;
    a.lse[head * a.T + row] = (m + log2f(l)) * 0.69314718055994531f;
  } else {
    const int64_t at = (split * a.tokens + row) * a.heads + head;
    r.part = a.part + at * D;
    r.inv_l = 1.0f;
    a.stats[at] = make_float2(m, l);
  }
  return r;
}

// Output and LSE from the parts, in their order: 8 channels of a row per thread.
template <typename T, int D>
__global__ void __launch_bounds__(256) merge_kernel(const Args a) {
  const int64_t n = a.tokens * a.heads * (D / 8);
  const int64_t v = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (v >= n) return;
  const int64_t vec = v / (D / 8), row = vec / a.heads;
  const int head = static_cast<int>(vec - row * a.heads);
  const int c0 = 8 * static_cast<int>(v - vec * (D / 8));
  float m = -INFINITY;
  for (int s = 0; s < a.splits; ++s) m = fmaxf(m, a.stats[s * a.tokens * a.heads + vec].x);
  const float shift = m == -INFINITY ? 0.0f : m;
  float f[8] = {}, l = 0.0f;
  for (int s = 0; s < a.splits; ++s) {
    const float2 t = a.stats[s * a.tokens * a.heads + vec];
    if (t.y == 0.0f) continue;  // a part without keys has written no O
    const float w = exp2f(t.x - shift);
    l = fmaf(t.y, w, l);
    const float4* p =
        reinterpret_cast<const float4*>(a.part + (s * a.tokens * a.heads + vec) * D + c0);
    const float4 x = __ldcs(p), y = __ldcs(p + 1);
    f[0] = fmaf(x.x, w, f[0]);
    f[1] = fmaf(x.y, w, f[1]);
    f[2] = fmaf(x.z, w, f[2]);
    f[3] = fmaf(x.w, w, f[3]);
    f[4] = fmaf(y.x, w, f[4]);
    f[5] = fmaf(y.y, w, f[5]);
    f[6] = fmaf(y.z, w, f[6]);
    f[7] = fmaf(y.w, w, f[7]);
  }
  const float inv_l = 1.0f / l;
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] *= inv_l;
  *reinterpret_cast<uint4*>(reinterpret_cast<T*>(a.o.ptr) + row * a.o.ts + head * a.o.hs + c0) =
      pack8<T>(f);
  if (c0 == 0) a.lse[head * a.T + row] = (m + log2f(l)) * 0.69314718055994531f;
}

// HEADS: the CTA's tiles are two heads of one group; otherwise tiles `tile` and `tile - 1` of one
// head (the second absent when tile = 0).
// PARTS: the walks are cut into parts (Args::splits > 1).
template <typename T, int D, bool HEADS, bool PARTS>
__global__ void __launch_bounds__(kThreads, 1)
    attn_fwd_kernel(const __grid_constant__ CUtensorMap tm_q,
                    const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const Args a) {
  extern __shared__ uint8_t smem_raw[];
  using SM = Smem<T, D>;
  SM& sm = *reinterpret_cast<SM*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  constexpr int NST = SM::NST;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int splits = PARTS ? a.splits : 1;
  int grid_head;
  const Item it = grid_at(a.grid, grid_head);
  const int hg = grid_head / splits, split = grid_head - hg * splits;
  const int head0 = HEADS ? 2 * hg : hg;
  const int kv_head = head0 / a.group;
  const bool two = HEADS || it.tile > 0;
  auto tile_of = [&](int g) { return HEADS ? it.tile : it.tile - g; };
  auto keys_of = [&](int g) { return a.causal ? tile_of(g) + 1 : tiles_of(it); };
  // key tiles of this part, for tile 0 (the most) and tile 1: from .. from + n - 1
  const int all = keys_of(0);
  const int from = static_cast<int>(static_cast<int64_t>(all) * split / splits);
  const int to = static_cast<int>(static_cast<int64_t>(all) * (split + 1) / splits);
  const int n0 = to - from;
  const int n1 = two ? max(0, min(keys_of(1), to) - from) : 0;

  if (threadIdx.x == 0) {
    sm.abort = device_aborted() ? 1 : 0;
    mbar_init(&sm.q_full, 1);
    for (int s = 0; s < NST; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(&sm.s_full[g], 1);
      mbar_init(&sm.p_full[g][0], 4);
      mbar_init(&sm.p_full[g][1], 4);
    }
    mbar_init(&sm.o_full, 1);
    fence_barrier_init();
  }
  __syncthreads();
  if (sm.abort) return;
  if (warp == kMmaWarp) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kOtherRegs));
    if (warp == kProducerWarp) {
      if (lane == 0 && (!PARTS || n0 > 0)) {
        mbar_arrive_expect_tx(&sm.q_full, (two ? 2 : 1) * BT * D * 2);
        load_tile<T, D, D, BT>(sm.q[0], &tm_q, it, tile_of(0), head0, &sm.q_full);
        if (two)
          load_tile<T, D, D, BT>(sm.q[1], &tm_q, it, tile_of(1), HEADS ? head0 + 1 : head0,
                                 &sm.q_full);
        Ring<NST> ring;
        for (int i = 0; i < 2 * n0; ++i, ring.next()) {  // K0 K1 V0 K2 V1 ... V(n0 - 1)
          const int st = ring.slot;
          const bool v = i == 2 * n0 - 1 || (i > 0 && (i & 1) == 0);
          const int j = v ? (i == 2 * n0 - 1 ? n0 - 1 : i / 2 - 1) : (i + 1) / 2;
          if (i >= NST) mbar_wait(&sm.empty[st], ring.parity ^ 1, 301);
          mbar_arrive_expect_tx(&sm.full[st], BT * D * 2);
          load_tile<T, D, D, BT>(sm.kv[st], v ? &tm_v : &tm_k, it, from + j, kv_head,
                                 &sm.full[st]);
        }
      }
      __syncwarp();
    } else if (warp == kMmaWarp) {
      if (!PARTS || n0 > 0) {
        const uint32_t leader = elect_one(), tmem = uniform(sm.tmem_base);
        constexpr uint32_t kFmt = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
        constexpr uint32_t id_s = instr_desc(1, kFmt, kFmt, false, false, BT, BT);
        constexpr uint32_t id_o = instr_desc(1, kFmt, kFmt, false, true, BT, D);
        const uint64_t q_desc[2] = {desc_k(sm.q[0]), desc_k(sm.q[1])};
        auto scores = [&](int g, uint64_t k_desc) {  // S_g = Q_g K^T
          mma_rows<D, BT>(leader, tmem + 128 * g, q_desc[g], k_desc, id_s);
          mma_commit_warp(leader, &sm.s_full[g]);
        };
        auto values = [&](int g, uint64_t v_desc, int j) {  // O_g += P_g V
          // in halves of the keys, so that the first runs during the second's exponentials
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            mbar_wait(&sm.p_full[g][h], j & 1, 312);
            tc_fence_after();
            mma_sum_half(leader, tmem + kColO + D * g, tmem + 128 * g + 32 * h, v_desc + step_mn(4 * h),
                         id_o, j == 0 && h == 0);
          }
        };
        Ring<NST> ring;  // tiles in their order: K_0, then K_(j + 1) and V_j
        mbar_wait(&sm.q_full, 0, 310);
        mbar_wait(&sm.full[0], 0, 311);
        tc_fence_after();
        scores(0, desc_k(sm.kv[0]));
        if (n1 > 0) scores(1, desc_k(sm.kv[0]));
        mma_commit_warp(leader, &sm.empty[0]);
        ring.next();
        for (int j = 0; j < n0; ++j) {
          const bool more = j + 1 < n0;
          const int k_slot = ring.slot;
          const uint64_t k_desc = desc_k(sm.kv[k_slot]);
          if (more) {
            mbar_wait(&sm.full[k_slot], ring.parity, 311);
            ring.next();
          }
          const int v_slot = ring.slot;
          const uint64_t v_desc = desc_mn<BT>(sm.kv[v_slot]);
          mbar_wait(&sm.full[v_slot], ring.parity, 311);
          ring.next();
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const int n = g == 0 ? n0 : n1;
            if (j >= n) continue;
            values(g, v_desc, j);
            if (j + 1 < n) scores(g, k_desc);
          }
          mma_commit_warp(leader, &sm.empty[v_slot]);
          if (more) mma_commit_warp(leader, &sm.empty[k_slot]);
        }
        mma_commit_warp(leader, &sm.o_full);
      }
      __syncwarp();
    }
    tc_fence_before();
    named_barrier_sync(15, kThreads);
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kSoftmaxRegs));
    const int g = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = tmem + (((warp & 3) * 32u) << 16);
    const uint32_t s_at = lane_base + 128 * g, o_at = lane_base + kColO + D * g;
    const int n = g == 0 ? n0 : n1;
    const int tile = tile_of(g);
    const int i = row_index(it, tile, r);
    const float c = a.scale_log2;
    float m = -INFINITY, l = 0.0f;

    auto block = [&](int j, auto masked) {
      constexpr bool MASK = decltype(masked)::value;
      mbar_wait(&sm.s_full[g], j & 1, 320);
      tc_fence_after();
      uint32_t x[4][32];
#pragma unroll
      for (int q = 0; q < 4; ++q) tmem_ld32(s_at + 32 * q, x[q]);
      tmem_ld_wait_regs32(x[0]);
      tie32(x[1]);
      tie32(x[2]);
      tie32(x[3]);
      if (MASK) {
        // key index within the sequence must be >= 0 (the ragged first tile) and, when causal,
        // not above the row's
        const int lo = -row_index(it, from + j, 0);
        const int hi = a.causal ? i - row_index(it, from + j, 0) : BT - 1;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (32 * q + e < lo || 32 * q + e > hi) x[q][e] = 0xff800000u;  // -inf
      }
      float mx[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        mx[q] = fmax_nan(__uint_as_float(x[q][0]), __uint_as_float(x[q][1]));
#pragma unroll
        for (int e = 2; e < 32; e += 2)
          mx[q] = fmax3_nan(mx[q], __uint_as_float(x[q][e]), __uint_as_float(x[q][e + 1]));
      }
      const float top = fmax_nan(fmax3_nan(mx[0], mx[1], mx[2]), mx[3]) * c;
      // always on the first tile with a visible key, and from the first NaN on
      const bool grow = !(top <= m + 8.0f);
      if (__any_sync(0xffffffffu, grow)) {
        const float mn = grow ? top : m;
        const float alpha = grow ? ex2_approx(m - mn) : 1.0f;
        m = mn;
        l *= alpha;
        if (j > 0) {
#pragma unroll
          for (int cc = 0; cc < D; cc += 32) {
            uint32_t y[32];
            tmem_ld32(o_at + cc, y);
            tmem_ld_wait_regs32(y);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              y[e] = __float_as_uint(__uint_as_float(y[e]) * alpha);
            tmem_st32(o_at + cc, y);
          }
        }
      }
      const float neg = neg_max<T>(m);
      const float2 c2 = make_float2(c, c), n2 = make_float2(neg, neg);
      float2 sum = make_float2(0.0f, 0.0f), sum2 = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        // three passes over 64 columns, so that independent operations follow each other
        float2 z[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          const int q = 2 * hh + (k >> 4), e = 2 * (k & 15);
          z[k] = __ffma2_rn(
              make_float2(__uint_as_float(x[q][e]), __uint_as_float(x[q][e + 1])), c2, n2);
        }
#pragma unroll
        for (int k = 0; k < 32; ++k)
          z[k] = !MASK && poly_pair(k) ? exp2_fma2(z[k])
                                       : make_float2(ex2_approx(z[k].x), ex2_approx(z[k].y));
        uint32_t w[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          if (k & 1)
            sum2 = __fadd2_rn(sum2, z[k]);
          else
            sum = __fadd2_rn(sum, z[k]);
          w[k] = Cvt<T>::pack2(z[k].x, z[k].y);
        }
        tmem_st32(s_at + 32 * hh, w);
        tmem_st_wait();  // of O too, where it was rescaled
        tc_fence_before();
        mbar_arrive_warp(&sm.p_full[g][hh], lane);
      }
      l += (sum.x + sum.y) + (sum2.x + sum2.y);
    };
    const bool ragged = tiles_of(it) * BT != it.len;
    for (int j = 0; j < n; ++j) {
      if ((from + j == 0 && ragged) || (a.causal && from + j == tile))
        block(j, std::true_type{});
      else
        block(j, std::false_type{});
    }
    RowOut<T, PARTS> res = {};
    if (!PARTS || n0 > 0) mbar_wait(&sm.o_full, 0, 321);
    tc_fence_after();
    if (i >= 0 && (g == 0 || two)) {
      const int64_t row = static_cast<int64_t>(it.start) + i;
      res = row_out<T, D, PARTS>(a, row, HEADS ? head0 + g : head0, split, m - kFwdShift<T>, l);
    }
    if (n > 0) {
#pragma unroll
      for (int cc = 0; cc < D; cc += 32) {
        uint32_t y[32];
        tmem_ld32(o_at + cc, y);
        tmem_ld_wait_regs32(y);
        if (i >= 0) res.store32(y, cc);
      }
    }
    tc_fence_before();
    named_barrier_sync(15, kThreads);
  }
}

// ---- d = 64 ---------------------------------------------------------------------------------
constexpr int kThreads64 = 160;
constexpr int kIssueWarp64 = 4;

template <typename T>
struct Smem64 {
  alignas(1024) T q[BT * 64];
  alignas(1024) T k[2][64 * 64], v[2][64 * 64];  // even and odd runs
  uint64_t q_full, k_full[2], v_full[2], s_full, p_full, o_full;
  uint32_t tmem_base;
  int abort;
};
template <typename T>
constexpr size_t smem64_bytes() {
  return sizeof(Smem64<T>) + 1024;
}
static_assert(4 * (smem64_bytes<__half>() + 1024) <= 233472,
              "shared memory of four CTAs exceeds the limit");

template <typename T, bool PARTS>
__global__ void __launch_bounds__(kThreads64, 4)
    attn_fwd64_kernel(const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const Args a) {
  constexpr int D = 64, BN = 64;
  extern __shared__ uint8_t smem_raw[];
  using SM = Smem64<T>;
  SM& sm = *reinterpret_cast<SM*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  constexpr uint32_t kColO64 = 64;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int splits = PARTS ? a.splits : 1;
  int grid_head;
  const Item it = grid_at(a.grid, grid_head);
  const int head = grid_head / splits, split = grid_head - head * splits;
  const int kv_head = head / a.group;
  const int tiles = tiles_of(it), pad = tiles * BT - it.len;
  const int ragged = pad / BN;  // first run of keys: one that is all padding is left out
  const int runs = (a.causal ? it.tile + 1 : tiles) * (BT / BN) - ragged;
  // this part's runs
  const int from = static_cast<int>(static_cast<int64_t>(runs) * split / splits);
  const int n = static_cast<int>(static_cast<int64_t>(runs) * (split + 1) / splits) - from;
  const int first = ragged + from;

  if (threadIdx.x == 0) {
    sm.abort = device_aborted() ? 1 : 0;
    mbar_init(&sm.q_full, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.k_full[s], 1);
      mbar_init(&sm.v_full[s], 1);
    }
    mbar_init(&sm.s_full, 1);
    mbar_init(&sm.p_full, 4);
    mbar_init(&sm.o_full, 1);
    fence_barrier_init();
  }
  __syncthreads();
  if (sm.abort) return;
  if (warp == kIssueWarp64) {
    tmem_alloc(&sm.tmem_base, 128);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;

  if (warp == kIssueWarp64) {
    if (!PARTS || n > 0) {
      const uint32_t leader = elect_one(), tmem = uniform(sm.tmem_base);
      constexpr uint32_t kFmt = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
      constexpr uint32_t id_s = instr_desc(1, kFmt, kFmt, false, false, BT, BN);
      constexpr uint32_t id_o = instr_desc(1, kFmt, kFmt, false, true, BT, D);
      auto load = [&](T* dst, const CUtensorMap* map, int j, uint64_t* bar) {
        if (j >= n || !leader) return;
        mbar_arrive_expect_tx(bar, BN * D * 2);
        load_tile<T, D, BN, BN>(dst, map, it, first + j, kv_head, bar);
      };
      if (leader) {
        mbar_arrive_expect_tx(&sm.q_full, BT * D * 2);
        load_tile<T, D, BN, BT>(sm.q, &tm_q, it, it.tile, head, &sm.q_full);
      }
      __syncwarp();
      load(sm.k[0], &tm_k, 0, &sm.k_full[0]);
      load(sm.v[0], &tm_v, 0, &sm.v_full[0]);
      load(sm.k[1], &tm_k, 1, &sm.k_full[1]);
      const uint64_t q_desc = desc_k(sm.q);
      const uint64_t k_desc[2] = {desc_k(sm.k[0]), desc_k(sm.k[1])};
      const uint64_t v_desc[2] = {desc_mn<BN>(sm.v[0]), desc_mn<BN>(sm.v[1])};
      mbar_wait(&sm.q_full, 0, 340);
      mbar_wait(&sm.k_full[0], 0, 341);
      tc_fence_after();
      mma_rows<D, BN>(leader, tmem, q_desc, k_desc[0], id_s);
      mma_commit_warp(leader, &sm.s_full);
      for (int j = 0; j < n; ++j) {
        const int b = j & 1, nb = b ^ 1;
        const uint32_t parity = (j >> 1) & 1;
        mbar_wait(&sm.v_full[b], parity, 342);
        if (j + 1 < n) mbar_wait(&sm.k_full[nb], ((j + 1) >> 1) & 1, 341);
        mbar_wait(&sm.p_full, j & 1, 343);
        tc_fence_after();
        mma_sum_half(leader, tmem + kColO64, tmem, v_desc[b], id_o, j == 0);  // O += P V
        if (j + 1 < n) {
          mma_rows<D, BN>(leader, tmem, q_desc, k_desc[nb], id_s);
          mma_commit_warp(leader, &sm.s_full);
        } else {
          mma_commit_warp(leader, &sm.o_full);
        }
        // P of run j has arrived: S of run j and P V of run j - 1 are complete
        load(sm.v[nb], &tm_v, j + 1, &sm.v_full[nb]);
        load(sm.k[b], &tm_k, j + 2, &sm.k_full[b]);
      }
    }
    __syncwarp();
    tc_fence_before();
    named_barrier_sync(15, kThreads64);
    tc_fence_after();
    tmem_dealloc(tmem, 128);
  } else {
    const int r = threadIdx.x;
    const uint32_t lane_base = tmem + ((warp * 32u) << 16);
    const uint32_t o_at = lane_base + kColO64;
    const int i = row_index(it, it.tile, r);
    const float c = a.scale_log2;
    float m = -INFINITY, l = 0.0f;

    auto block = [&](int j, auto masked) {
      constexpr bool MASK = decltype(masked)::value;
      mbar_wait(&sm.s_full, j & 1, 350);
      tc_fence_after();
      uint32_t x[2][32];
      tmem_ld32(lane_base, x[0]);
      tmem_ld32(lane_base + 32, x[1]);
      tmem_ld_wait_regs32(x[0]);
      tie32(x[1]);
      if (MASK) {
        // key index within the sequence >= 0 (ragged first run) and, when causal, not above i
        const int key0 = row_index<BN>(it, first + j, 0);
        const int lo = -key0, hi = a.causal ? i - key0 : BN;
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (32 * q + e < lo || 32 * q + e > hi) x[q][e] = 0xff800000u;  // -inf
      }
      float mx[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t* y = &x[q >> 1][16 * (q & 1)];
        mx[q] = fmax_nan(__uint_as_float(y[0]), __uint_as_float(y[1]));
#pragma unroll
        for (int e = 2; e < 16; e += 2)
          mx[q] = fmax3_nan(mx[q], __uint_as_float(y[e]), __uint_as_float(y[e + 1]));
      }
      const float top = fmax_nan(fmax3_nan(mx[0], mx[1], mx[2]), mx[3]) * c;
      // always on the first run with a visible key, and from the first NaN on
      const bool grow = !(top <= m + 8.0f);
      if (__any_sync(0xffffffffu, grow)) {
        const float mn = grow ? top : m;
        const float alpha = grow ? ex2_approx(m - mn) : 1.0f;
        m = mn;
        l *= alpha;
        if (j > 0) {  // O is up to date: S of this run was issued after P V of the last
#pragma unroll 1
          for (int cc = 0; cc < D; cc += 8) {  // few registers: x is live
            uint32_t y[8], none[8] = {};
            tmem_ld8(o_at + cc, y);
            tmem_ld_wait_regs8(y, none);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              y[e] = __float_as_uint(__uint_as_float(y[e]) * alpha);
            tmem_st8(o_at + cc, y);
          }
        }
      }
      const float neg = neg_max<T>(m);
      const float2 c2 = make_float2(c, c), n2 = make_float2(neg, neg);
      float2 sum = make_float2(0.0f, 0.0f), sum2 = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t w[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float2 z = __ffma2_rn(
              make_float2(__uint_as_float(x[q][2 * k]), __uint_as_float(x[q][2 * k + 1])), c2, n2);
          const float2 p = !MASK && poly_pair(k) ? exp2_fma2(z)
                                                 : make_float2(ex2_approx(z.x), ex2_approx(z.y));
          if (k & 1)
            sum2 = __fadd2_rn(sum2, p);
          else
            sum = __fadd2_rn(sum, p);
          w[k] = Cvt<T>::pack2(p.x, p.y);
        }
        tmem_st16(lane_base + 16 * q, w);
      }
      tmem_st_wait();  // of O too, where it was rescaled
      tc_fence_before();
      mbar_arrive_warp(&sm.p_full, lane);
      l += (sum.x + sum.y) + (sum2.x + sum2.y);
    };
    for (int j = 0; j < n; ++j) {
      if ((first + j == ragged && pad > 0) || (a.causal && first + j >= it.tile * (BT / BN)))
        block(j, std::true_type{});
      else
        block(j, std::false_type{});
    }
    if (!PARTS || n > 0) mbar_wait(&sm.o_full, 0, 352);
    tc_fence_after();
    RowOut<T, PARTS> res = {};
    if (i >= 0) res = row_out<T, D, PARTS>(a, static_cast<int64_t>(it.start) + i, head, split, m - kFwdShift<T>, l);
    if (!PARTS || n > 0) {
#pragma unroll
      for (int cc = 0; cc < D; cc += 32) {
        uint32_t y[32];
        tmem_ld32(o_at + cc, y);
        tmem_ld_wait_regs32(y);
        if (i >= 0) res.store32(y, cc);
      }
    }
    tc_fence_before();
    named_barrier_sync(15, kThreads64);
  }
}

}  // namespace fwd
}  // namespace packed
}  // namespace sage
