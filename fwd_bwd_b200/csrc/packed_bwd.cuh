// packed_bwd.cuh -- backward of the 16-bit attention over packed sequences with grouped heads.
//
//   P_ij = exp(tau q_i . k_j - LSE_i), D_i = dO_i . O_i, dS_ij = P_ij (dO_i . v_j - D_i)
//   dV_j = sum_{h,i} P_ij dO_i,  dK_j = tau sum_{h,i} dS_ij q_i,  dQ_i = tau sum_j dS_ij k_j
// (h over the query heads that share j's key head).  Tiles and tensor maps as in the forward.
//
// Two kernels after the row pass that forms D, each recomputing S and dP for its own direction:
//   * dq_kernel: one CTA per (query tile, query head), walking the key tiles: dQ += dS K;
//   * dkv_kernel: one CTA per (key tile, key head), walking the query tiles of every head of the
//     group.  It works on transposed tiles (rows = keys), so P^T and dS^T go from registers to
//     TMEM as the A operands of dV += P^T dO and dK += dS^T Q, and dV, dK stay in TMEM.
// Seven products where one fused pass would need five, but a gradient is summed by one CTA: no
// atomics, no float32 accumulator in HBM, no finishing pass, the same bits every run, and grouped
// heads cost nothing extra.  Only where walks are cut into parts (few heads, long walks) do several
// CTAs share a sum: each part's float32 sums go to the workspace, for every token of the batch, and
// join_kernel adds them in the parts' order: the same bits every run there too.
//
// Both work on blocks of 128 rows x D columns (the walked side in runs of D rows).  d = 128 fills
// TMEM and shared memory: one CTA per SM.  d = 64 takes half of both, so two CTAs share an SM and
// hide each other's latencies, their first loads and last stores included.
// A thread holds 64 columns of a row: warps 0-3 (d = 128: 0-7, the second four with the second
// half of the columns) compute; then follow the TMA producer, the MMA issuer, a warp that brings
// the query rows' LSE and D to shared memory (dkv_kernel), and an idle one that completes the
// warpgroup, which gives registers to the computing ones.
//
// D_i: the row pass takes it from the stored, rounded o.  That rounding weighs most in rows of few
// keys (|o| ~ |v|), so rows of a sequence's first tile get it from P and dP instead: dq_kernel
// walks their at most 128 keys twice, first for D_i = sum_j P_ij dP_ij, which dkv_kernel then
// uses too.  (bf16, 1024-token documents: dQ and dK off by 0.24% of their norm, not 0.26%; their
// two unavoidable roundings make 0.235%.)
//
// Measured (B200, kernel time; causal; dq_kernel's 3 products and dkv_kernel's 4 counted over the
// visible scores):
//   d = 128, 4 x 8192, 16 heads, bf16    dQ 1277 us, 1291 TFLOP/s   dK/dV 1527 us, 1440 TFLOP/s
//   d = 64, 8 x 2048, 16 heads           dQ  134 us,  772 TFLOP/s   dK/dV  171 us,  804 TFLOP/s
// Bound: d = 128 by the chain of products and exponentials of one tile (tensor pipe 52% and 64%
// active) and, in longer runs, by the power cap; d = 64 by the chains of two CTAs (36%, 38%).
//
// Rounding: P and dS to the tensors' type for their products; sums in float32; outputs once.
// Half precision: P is multiplied by 2^14 before it is rounded, and dS by the power of two that
// puts the bound 2 max |dO_i| max |v_j| of |dP - D| (over the finite rows of the sequence and key
// head) at 2^15 or just below: small values keep their bits, nothing overflows, and the factors
// are taken out of the float32 sums exactly.
#pragma once

#include "packed_fwd.cuh"

namespace sage {
namespace packed {
namespace bwd {

template <int D>
struct Cfg {
  static constexpr int BN = D;                   // rows of the walked side per step
  static constexpr int kWG = BN / 64;            // computing warpgroups
  static constexpr int kCompute = 128 * kWG;
  static constexpr int kThreads = kCompute + 128;
  static constexpr int kProducerWarp = 4 * kWG, kMmaWarp = kProducerWarp + 1,
                       kRowWarp = kProducerWarp + 2;
  static constexpr int kCtas = D == 64 ? 2 : 1;  // per SM
  static constexpr int kLaunchRegs = D == 64 ? 128 : 168;
  static constexpr int kComputeRegs = D == 64 ? 184 : 216, kOtherRegs = 72;
  static constexpr int kTmem = 4 * D;            // columns
  static_assert(kCompute * kComputeRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs,
                "register split exceeds the launch allocation");
};
constexpr float kLog2e = 1.4426950408889634f;

template <typename T>
struct Scaling {
  static constexpr bool kOn = false;
  static constexpr float kPShift = 0.0f;  // log2 of P's factor
};
template <>
struct Scaling<__half> {
  static constexpr bool kOn = true;
  static constexpr float kPShift = 14.0f;
};

// ---- row pass: D_i = dO_i . O_i; half precision also the largest |dO_i|^2 and |v_j|^2 ---------
struct RowArgs {
  Out o, dout, v;        // inputs
  const Item* items;
  float* dvec;           // [Hq][T]
  uint32_t* norms;       // [sequences][Hkv][2]: bits of max |dO|^2, max |v|^2, finite (zeroed before)
  int64_t T;
  int tiles, Hq, Hkv, group;
};

constexpr int kRowKernelThreads = 256;

// One CTA per (tile, query head); with NORMS, then per (tile, key head) for v.
template <typename T, int D, bool NORMS>
__global__ void __launch_bounds__(kRowKernelThreads) row_kernel(const RowArgs a) {
  constexpr int LPR = D / 8, ROWS = kRowKernelThreads / LPR, STEPS = BT / ROWS;
  const int64_t n_q = static_cast<int64_t>(a.tiles) * a.Hq;
  const bool on_v = NORMS && blockIdx.x >= n_q;
  const int64_t at = on_v ? blockIdx.x - n_q : blockIdx.x;
  const int H = on_v ? a.Hkv : a.Hq;
  const Item it = a.items[at / H];
  const int head = static_cast<int>(at % H);
  const int l = threadIdx.x % LPR, r0 = threadIdx.x / LPR;
  const uint32_t mask = ((1u << LPR) - 1u) << ((threadIdx.x & 31) - l);
  const Out& x = on_v ? a.v : a.dout;
  uint4 xr[STEPS], yr[STEPS];
  float dot[STEPS];
  float most = 0.0f;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int i = row_index(it, it.tile, r0 + s * ROWS);
    xr[s] = yr[s] = make_uint4(0, 0, 0, 0);
    if (i < 0) continue;
    const int64_t row = static_cast<int64_t>(it.start) + i;
    xr[s] = *reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(x.ptr) + row * x.ts +
                                            head * x.hs + 8 * l);
    if (!on_v)
      yr[s] = *reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.o.ptr) + row * a.o.ts +
                                              head * a.o.hs + 8 * l);
  }
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    float f[8], g[8];
    Cvt<T>::load8(xr[s], f);
    Cvt<T>::load8(yr[s], g);
    float p = 0.0f, q = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      p = fmaf(f[e], g[e], p);
      if (NORMS) q = fmaf(f[e], f[e], q);
    }
    dot[s] = row_sum<LPR>(p, mask);
    if (NORMS) {
      q = row_sum<LPR>(q, mask);
      // what is not finite says nothing: the rows that see it have no finite gradient anyhow
      if (q > most && q < INFINITY) most = q;
    }
    const int i = row_index(it, it.tile, r0 + s * ROWS);
    if (!on_v && l == 0 && i >= 0) a.dvec[head * a.T + it.start + i] = dot[s];
  }
  if (NORMS) {
    // float bits of non-negative values order like unsigned integers, and a maximum does not depend
    // on the order
    uint32_t m = __float_as_uint(most);
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) {
      const int kv = on_v ? head : head / a.group;
      atomicMax(&a.norms[(static_cast<int64_t>(it.seq) * a.Hkv + kv) * 2 + (on_v ? 1 : 0)], m);
    }
  }
}

// The factor of dS (a power of two) from the two norms; 1 where one is zero.
__device__ __forceinline__ float ds_factor(const uint32_t* norms) {
  const float b = 2.0f * sqrtf(__uint_as_float(norms[0])) * sqrtf(__uint_as_float(norms[1]));
  if (!(b > 0.0f)) return 1.0f;  // at most 2^40 otherwise
  int e = 14 - ilogbf(b);  // b 2^e in [2^14, 2^15)
  e = max(-60, min(60, e));
  return scalbnf(1.0f, e);
}

// D (+)= A B over the 64 WG rows of tile B, A in TMEM: 32 columns from every 64th.
template <int WG>
__device__ __forceinline__ void mma_sum(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem, uint64_t b,
                                        uint32_t idesc, bool start) {
#pragma unroll
  for (int h = 0; h < WG; ++h)
    mma_sum_half(leader, d_tmem, a_tmem + 64 * h, b + step_mn(4 * h), idesc, start && h == 0);
}

struct Args {
  Grid grid;          // heads: query heads (dq_kernel), key heads (dkv_kernel)
  const float* lse;   // [Hq][T]
  float* dvec;        // [Hq][T]
  const uint32_t* norms;
  Out out[2];         // dq_kernel: dq; dkv_kernel: dv, dk
  int64_t T;
  int group, kv_heads;
  int causal;
  float scale_log2, tau;
  // A CTA's walk may be cut into `splits` parts: the grid then has splits x heads, and the parts go
  // to part, [splits][tokens][query heads][D] (dq_kernel) or [splits][2 (dV, dK)][tokens][kv_heads][D]
  int splits;
  float* part;
  int64_t tokens;
};

// P (times 2^shift) of 32 columns from the scores x, in place: z = x c + offset(e).
// MASK: columns for which hidden(e) holds are zero.  POLY: a quarter of the exponentials on the
// FMA pipe (dkv_kernel: 1563 us against 1588 us without; dq_kernel: 1297 us against 1311 us with).
template <bool MASK, bool POLY, typename Offset, typename Hidden>
__device__ __forceinline__ void probabilities(uint32_t (&x)[32], float c, Offset offset,
                                              Hidden hidden) {
  const float2 c2 = make_float2(c, c);
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    float2 z = __ffma2_rn(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), c2,
                          offset(e));
    float2 p;
    if (MASK) {
      if (hidden(e)) z.x = -INFINITY;
      if (hidden(e + 1)) z.y = -INFINITY;
      p = make_float2(ex2_approx(z.x), ex2_approx(z.y));
    } else if (POLY && poly_pair(e >> 1)) {
      p = exp2_fma2(z);
    } else {
      p = make_float2(ex2_approx(z.x), ex2_approx(z.y));
    }
    x[e] = __float_as_uint(p.x);
    x[e + 1] = __float_as_uint(p.y);
  }
}
template <typename T>
__device__ __forceinline__ void pack32(const uint32_t (&x)[32], uint32_t (&w)[16]) {
#pragma unroll
  for (int e = 0; e < 16; ++e)
    w[e] = Cvt<T>::pack2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
}
// Two neighbouring values of a shared-memory vector, four of which are loaded together.
__device__ __forceinline__ float2 pair_of(const float4& v, int e) {
  return (e & 2) ? make_float2(v.z, v.w) : make_float2(v.x, v.y);
}

// 32 sums of a row, scaled, to the output or, in float32, to a part (zeros for one without steps).
template <typename T, bool PARTS>
__device__ __forceinline__ void store32(const uint32_t (&y)[32], bool any, float scale, T* dst,
                                        float* part) {
#pragma unroll
  for (int e = 0; e < 32; e += 8) {
    float f[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = any ? __uint_as_float(y[e + k]) * scale : 0.0f;
    if (!PARTS) {
      *reinterpret_cast<uint4*>(dst + e) = pack8<T>(f);
    } else {
      *reinterpret_cast<float4*>(part + e) = make_float4(f[0], f[1], f[2], f[3]);
      *reinterpret_cast<float4*>(part + e + 4) = make_float4(f[4], f[5], f[6], f[7]);
    }
  }
}

// ---- dK and dV ------------------------------------------------------------------------------
template <typename T, int D>
struct DkvSmem {
  static constexpr int BN = Cfg<D>::BN;
  static constexpr int NST = D == 128 ? 4 : 6;  // Q / dO runs in flight
  alignas(1024) T k[BT * D];
  alignas(1024) T v[BT * D];
  alignas(1024) T ring[NST][BN * D];
  // of the query rows, negated: LSE log2 e - P's shift (-inf for padding: P = 0), and D
  alignas(16) float neg_lse[2][BN];
  alignas(16) float neg_d[2][BN];
  uint64_t kv_full, full[NST], empty[NST], vec_full[2], vec_empty[2];
  uint64_t s_full, dp_full, p_ready[2], ds_ready, done;
  uint32_t tmem_base;
  int abort;
};
template <typename T, int D>
constexpr size_t dkv_smem_bytes() {
  return sizeof(DkvSmem<T, D>) + 1024;
}
static_assert(dkv_smem_bytes<__half, 128>() <= 232448 && dkv_smem_bytes<__half, 64>() <= 115712,
              "shared memory exceeds the limit");

// PARTS: the walks are cut into parts (Args::splits > 1); apart, because the others' code would
// lose 4% to it.
template <typename T, int D, bool PARTS>
__global__ void __launch_bounds__(Cfg<D>::kThreads, Cfg<D>::kCtas)
    dkv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
               const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
               const Args a) {
  extern __shared__ uint8_t smem_raw[];
  using SM = DkvSmem<T, D>;
  using C = Cfg<D>;
  SM& sm = *reinterpret_cast<SM*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  constexpr int NST = SM::NST, BN = C::BN;
  // TMEM columns: S^T (then P^T), dP^T (then dS^T), dV, dK.  P^T and dS^T of column half h start at
  // 64 h of their block, over columns that only the same warps have read.
  constexpr uint32_t kColDP = BN, kColDV = 2 * BN, kColDK = 2 * BN + D;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int splits = PARTS ? a.splits : 1;
  int grid_head;
  const Item it = grid_at(a.grid, grid_head);
  const int kv_head = grid_head / splits, split = grid_head - kv_head * splits;
  const int tiles = tiles_of(it);
  // under a causal mask the list's order (most work first) is by query tile: mirrored for keys
  const int kt = a.causal ? tiles - 1 - it.tile : it.tile;
  const int runs = tiles * (BT / BN), pad = tiles * BT - it.len;
  // first run of query rows that sees these keys and is not all padding
  const int diag = kt * (BT / BN);
  const int first = max(a.causal ? diag : 0, pad / BN);
  // this part's steps of the walk over every head's runs
  const int walk = (runs - first) * a.group;
  const int n_from = static_cast<int>(static_cast<int64_t>(walk) * split / splits);
  const int n_all =
      static_cast<int>(static_cast<int64_t>(walk) * (split + 1) / splits) - n_from;
  // the steps' (query head, run of query rows), in order
  struct Walk {
    int head, run, first, runs;
    __device__ __forceinline__ void next() {
      if (++run == runs) {
        run = first;
        ++head;
      }
    }
  };
  const Walk begin = {kv_head * a.group + n_from / (runs - first), first + n_from % (runs - first),
                      first, runs};

  if (threadIdx.x == 0) {
    sm.abort = device_aborted() ? 1 : 0;
    mbar_init(&sm.kv_full, 1);
    for (int s = 0; s < NST; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.vec_full[s], 1);
      mbar_init(&sm.vec_empty[s], C::kCompute / 32);
    }
    mbar_init(&sm.s_full, 1);
    mbar_init(&sm.dp_full, 1);
    mbar_init(&sm.p_ready[0], C::kCompute / 32);
    mbar_init(&sm.p_ready[1], C::kCompute / 32);
    mbar_init(&sm.ds_ready, C::kCompute / 32);
    mbar_init(&sm.done, 1);
    fence_barrier_init();
  }
  __syncthreads();
  if (sm.abort) return;
  if (warp == C::kMmaWarp) {
    tmem_alloc(&sm.tmem_base, C::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;

  if (warp >= C::kProducerWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(C::kOtherRegs));
    if (warp == C::kProducerWarp) {
      if (lane == 0 && (!PARTS || n_all > 0)) {
        mbar_arrive_expect_tx(&sm.kv_full, 2 * BT * D * 2);
        load_tile<T, D, BN, BT>(sm.k, &tm_k, it, kt, kv_head, &sm.kv_full);
        load_tile<T, D, BN, BT>(sm.v, &tm_v, it, kt, kv_head, &sm.kv_full);
        Ring<NST> ring;
        Walk at = begin;
        for (int n = 0; n < n_all; ++n, at.next()) {  // Q0 dO0 Q1 dO1 ...
#pragma unroll
          for (int w = 0; w < 2; ++w, ring.next()) {
            const int st = ring.slot;
            if (2 * n + w >= NST) mbar_wait(&sm.empty[st], ring.parity ^ 1, 401);
            mbar_arrive_expect_tx(&sm.full[st], BN * D * 2);
            load_tile<T, D, BN, BN>(sm.ring[st], w ? &tm_do : &tm_q, it, at.run, at.head,
                                    &sm.full[st]);
          }
        }
      }
      __syncwarp();
    } else if (warp == C::kRowWarp) {
      Walk at = begin;
      for (int n = 0; n < n_all; ++n, at.next()) {
        const int b = n & 1;
        if (n >= 2) mbar_wait(&sm.vec_empty[b], ((n >> 1) - 1) & 1, 402);
        const int64_t base = at.head * a.T + it.start;
#pragma unroll
        for (int r = lane; r < BN; r += 32) {
          const int i = row_index<BN>(it, at.run, r);
          sm.neg_lse[b][r] =
              i >= 0 ? fmaf(a.lse[base + i], -kLog2e, Scaling<T>::kPShift) : -INFINITY;
          sm.neg_d[b][r] = i >= 0 ? -a.dvec[base + i] : 0.0f;
        }
        mbar_arrive_warp(&sm.vec_full[b], lane);
      }
      __syncwarp();
    } else if (warp == C::kMmaWarp) {
      if ((!PARTS || n_all > 0)) {
        const uint32_t leader = elect_one(), tmem = uniform(sm.tmem_base);
        constexpr uint32_t kFmt = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
        constexpr uint32_t id_s = instr_desc(1, kFmt, kFmt, false, false, BT, BN);
        constexpr uint32_t id_g = instr_desc(1, kFmt, kFmt, false, true, BT, D);
        const uint64_t k_desc = desc_k(sm.k), v_desc = desc_k(sm.v);
        auto product = [&](uint32_t col, uint64_t rows, const Ring<NST>& at, uint64_t* bar) {
          mbar_wait(&sm.full[at.slot], at.parity, 411);
          tc_fence_after();
          mma_rows<D, BN>(leader, tmem + col, rows, desc_k(sm.ring[at.slot]), id_s);
          mma_commit_warp(leader, bar);
        };
        Ring<NST> q_at, do_at;  // of Q_n and dO_n
        do_at.next();
        mbar_wait(&sm.kv_full, 0, 410);
        product(0, k_desc, q_at, &sm.s_full);
        product(kColDP, v_desc, do_at, &sm.dp_full);
        for (int n = 0; n < n_all; ++n) {
          const bool more = n + 1 < n_all;
          const int q_slot = q_at.slot, do_slot = do_at.slot;
          q_at.next();
          q_at.next();
          do_at.next();
          do_at.next();
          // dV += P^T dO, by quarters of 32 query rows (d = 64: halves): the first of every half
          const uint64_t do_desc = desc_mn<BN>(sm.ring[do_slot]);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            mbar_wait(&sm.p_ready[h], n & 1, 412);
            tc_fence_after();
#pragma unroll
            for (int w = 0; w < C::kWG; ++w)
              mma_sum_quarter(leader, tmem + kColDV, tmem + 64 * w + 16 * h,
                              do_desc + step_mn(4 * w + 2 * h), id_g, n == 0 && w == 0 && h == 0);
          }
          mma_commit_warp(leader, &sm.empty[do_slot]);
          if (more) product(0, k_desc, q_at, &sm.s_full);
          mbar_wait(&sm.ds_ready, n & 1, 413);
          tc_fence_after();
          // dK += dS^T Q
          mma_sum<C::kWG>(leader, tmem + kColDK, tmem + kColDP, desc_mn<BN>(sm.ring[q_slot]), id_g, n == 0);
          mma_commit_warp(leader, &sm.empty[q_slot]);
          if (more) product(kColDP, v_desc, do_at, &sm.dp_full);
        }
        mma_commit_warp(leader, &sm.done);
      }
      __syncwarp();
    }
    tc_fence_before();
    named_barrier_sync(15, C::kThreads);
    tc_fence_after();
    if (warp == C::kMmaWarp) tmem_dealloc(tmem, C::kTmem);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(C::kComputeRegs));
    const int half = warp >> 2;
    const int r = (warp & 3) * 32 + lane;  // key row of the tile
    const uint32_t lane_base = tmem + (((warp & 3) * 32u) << 16);
    const uint32_t s_at = lane_base + 64 * half, dp_at = s_at + kColDP;
    const float c = a.scale_log2;
    float factor = 1.0f;  // dS's factor over P's
    if (Scaling<T>::kOn)
      factor = ds_factor(a.norms + (static_cast<int64_t>(it.seq) * a.kv_heads + kv_head) * 2);
    const float f_ds = factor * exp2f(-Scaling<T>::kPShift);

    auto step = [&](int n, int run, auto masked) {
      constexpr bool MASK = decltype(masked)::value;
      const int b = n & 1;
      uint32_t x[2][32];
      mbar_wait(&sm.vec_full[b], (n >> 1) & 1, 420);
      mbar_wait(&sm.s_full, n & 1, 421);
      tc_fence_after();
      tmem_ld32(s_at, x[0]);
      tmem_ld32(s_at + 32, x[1]);
      tmem_ld_wait_regs32(x[0]);
      tie32(x[1]);
      // query row before the key's own position: hidden (the diagonal of a causal mask)
      const int hidden = r - (run - diag) * BN - 64 * half;  // columns below it
      // in halves, so that dV's products with the first run during the second's exponentials
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float4 off[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          off[k] = *reinterpret_cast<const float4*>(&sm.neg_lse[b][64 * half + 32 * h + 4 * k]);
        probabilities<MASK, true>(
            x[h], c, [&](int e) { return pair_of(off[e >> 2], e); },
            [&](int e) { return 32 * h + e < hidden; });
        uint32_t w[16];
        pack32<T>(x[h], w);
        tmem_st16(s_at + 16 * h, w);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive_warp(&sm.p_ready[h], lane);
      }
      // dS = P (dP - D)
      mbar_wait(&sm.dp_full, n & 1, 422);
      tc_fence_after();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t y[32], w[16];
        tmem_ld32(dp_at + 32 * h, y);
        float4 off[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          off[k] = *reinterpret_cast<const float4*>(&sm.neg_d[b][64 * half + 32 * h + 4 * k]);
        tmem_ld_wait_regs32(y);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float2 p = make_float2(__uint_as_float(x[h][2 * e]), __uint_as_float(x[h][2 * e + 1]));
          if (Scaling<T>::kOn) p = __fmul2_rn(p, make_float2(f_ds, f_ds));
          const float2 t =
              __fadd2_rn(make_float2(__uint_as_float(y[2 * e]), __uint_as_float(y[2 * e + 1])),
                         pair_of(off[e >> 1], 2 * e));
          const float2 s = __fmul2_rn(p, t);
          w[e] = Cvt<T>::pack2(s.x, s.y);
        }
        tmem_st16(dp_at + 16 * h, w);
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive_warp(&sm.ds_ready, lane);
      mbar_arrive_warp(&sm.vec_empty[b], lane);
    };
    Walk at = begin;
    for (int n = 0; n < n_all; ++n, at.next()) {
      if (a.causal && at.run < diag + BT / BN)
        step(n, at.run, std::true_type{});
      else
        step(n, at.run, std::false_type{});
    }
    if ((!PARTS || n_all > 0)) mbar_wait(&sm.done, 0, 423);
    tc_fence_after();
    // dV and dK: by a warpgroup each, or one after the other
    const int i = row_index(it, kt, r);
    const int64_t row = static_cast<int64_t>(it.start) + i;
#pragma unroll
    for (int w = 0; w < 2 / C::kWG; ++w) {
      const int which = C::kWG == 2 ? half : w;
      const uint32_t g_at = lane_base + (which == 0 ? kColDV : kColDK);
      const float scale = which == 0 ? exp2f(-Scaling<T>::kPShift) : a.tau / factor;
      const Out& out = a.out[which];
      T* dst = reinterpret_cast<T*>(out.ptr) + row * out.ts + kv_head * out.hs;
      float* part = PARTS
                        ? a.part + (((split * 2 + which) * a.tokens + row) * a.kv_heads + kv_head) * D
                        : nullptr;
#pragma unroll
      for (int cc = 0; cc < D; cc += 32) {
        uint32_t y[32];
        tmem_ld32(g_at + cc, y);
        tmem_ld_wait_regs32(y);
        if (i >= 0) store32<T, PARTS>(y, (!PARTS || n_all > 0), scale, dst + cc, PARTS ? part + cc : nullptr);
      }
    }
    tc_fence_before();
    named_barrier_sync(15, C::kThreads);
  }
}

// Outputs from the parts, added in their order: 8 channels per thread.
struct JoinArgs {
  const float* part;  // [splits][count][tokens][heads][D]
  Out out[2];
  int64_t tokens;
  int heads, splits, count;
};
template <typename T, int D>
__global__ void __launch_bounds__(256) join_kernel(const JoinArgs a) {
  const int64_t n = a.tokens * a.heads * (D / 8);
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (at >= a.count * n) return;
  const int which = at >= n ? 1 : 0;
  const int64_t v = at - which * n;  // vector of 8 channels
  float f[8] = {};
  for (int s = 0; s < a.splits; ++s) {
    const float4* p =
        reinterpret_cast<const float4*>(a.part + ((s * a.count + which) * n + v) * 8);
    const float4 x = __ldcs(p), y = __ldcs(p + 1);
    f[0] += x.x;
    f[1] += x.y;
    f[2] += x.z;
    f[3] += x.w;
    f[4] += y.x;
    f[5] += y.y;
    f[6] += y.z;
    f[7] += y.w;
  }
  const int64_t vec = v / (D / 8), row = vec / a.heads;
  const int head = static_cast<int>(vec - row * a.heads);
  const Out& out = a.out[which];
  *reinterpret_cast<uint4*>(reinterpret_cast<T*>(out.ptr) + row * out.ts + head * out.hs +
                            8 * (v - vec * (D / 8))) = pack8<T>(f);
}

// ---- dQ -------------------------------------------------------------------------------------
template <typename T, int D>
struct DqSmem {
  static constexpr int BN = Cfg<D>::BN;
  static constexpr int NST = D == 128 ? 5 : 8;  // K / V runs in flight
  alignas(1024) T q[BT * D];
  alignas(1024) T dout[BT * D];
  alignas(1024) T ring[NST][BN * D];
  float dot[2][BT];  // halves of D, where the row pass's is replaced
  uint64_t q_full, full[NST], empty[NST], s_full[2], dp_full, dp_free, ds_ready[2], done;
  uint32_t tmem_base;
  int abort;
};
template <typename T, int D>
constexpr size_t dq_smem_bytes() {
  return sizeof(DqSmem<T, D>) + 1024;
}
static_assert(dq_smem_bytes<__half, 128>() <= 232448 && dq_smem_bytes<__half, 64>() <= 115712,
              "shared memory exceeds the limit");

template <typename T, int D, bool PARTS>
__global__ void __launch_bounds__(Cfg<D>::kThreads, Cfg<D>::kCtas)
    dq_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
              const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
              const Args a) {
  extern __shared__ uint8_t smem_raw[];
  using SM = DqSmem<T, D>;
  using C = Cfg<D>;
  SM& sm = *reinterpret_cast<SM*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  constexpr int NST = SM::NST, BN = C::BN;
  // TMEM columns: two S blocks (dS overwrites the one it came from), dP, dQ
  constexpr uint32_t kColDP = 2 * BN, kColDQ = 3 * BN;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int splits = PARTS ? a.splits : 1;
  int grid_head;
  const Item it = grid_at(a.grid, grid_head);
  const int head = grid_head / splits, split = grid_head - head * splits;
  const int kv_head = head / a.group;
  const int tiles = tiles_of(it), pad = tiles * BT - it.len;
  // the steps' runs of keys: first .. first + runs - 1, in a sequence's first tile (or only one)
  // twice, the first `pre` steps for D
  const int first = pad / BN;
  const int runs = (a.causal ? it.tile + 1 : tiles) * (BT / BN) - first;
  const bool twice = runs * BN <= BT;
  // this part's: the walks that are made twice are short and stay whole, in part 0
  const int from = twice ? 0 : static_cast<int>(static_cast<int64_t>(runs) * split / splits);
  const int to = twice ? (split == 0 ? runs : 0)
                       : static_cast<int>(static_cast<int64_t>(runs) * (split + 1) / splits);
  const int pre = twice ? to : 0;
  const int n_all = pre + to - from;
  auto run_of = [&](int n) { return first + from + (n < pre ? n : n - pre); };

  if (threadIdx.x == 0) {
    sm.abort = device_aborted() ? 1 : 0;
    mbar_init(&sm.q_full, 1);
    for (int s = 0; s < NST; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    mbar_init(&sm.s_full[0], 1);
    mbar_init(&sm.s_full[1], 1);
    mbar_init(&sm.dp_full, 1);
    mbar_init(&sm.dp_free, C::kCompute / 32);
    // two, because dP of the next run is issued before this one's dS is waited for
    mbar_init(&sm.ds_ready[0], C::kCompute / 32);
    mbar_init(&sm.ds_ready[1], C::kCompute / 32);
    mbar_init(&sm.done, 1);
    fence_barrier_init();
  }
  __syncthreads();
  if (sm.abort) return;
  if (warp == C::kMmaWarp) {
    tmem_alloc(&sm.tmem_base, C::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;

  if (warp >= C::kProducerWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(C::kOtherRegs));
    if (warp == C::kProducerWarp) {
      if (lane == 0 && (!PARTS || n_all > 0)) {
        mbar_arrive_expect_tx(&sm.q_full, 2 * BT * D * 2);
        load_tile<T, D, BN, BT>(sm.q, &tm_q, it, it.tile, head, &sm.q_full);
        load_tile<T, D, BN, BT>(sm.dout, &tm_do, it, it.tile, head, &sm.q_full);
        Ring<NST> ring;
        for (int n = 0; n < n_all; ++n) {  // K0 V0 K1 V1 ...
#pragma unroll
          for (int w = 0; w < 2; ++w, ring.next()) {
            const int st = ring.slot;
            if (2 * n + w >= NST) mbar_wait(&sm.empty[st], ring.parity ^ 1, 501);
            mbar_arrive_expect_tx(&sm.full[st], BN * D * 2);
            load_tile<T, D, BN, BN>(sm.ring[st], w ? &tm_v : &tm_k, it, run_of(n), kv_head,
                                    &sm.full[st]);
          }
        }
      }
      __syncwarp();
    } else if (warp == C::kMmaWarp) {
      if ((!PARTS || n_all > 0)) {
        const uint32_t leader = elect_one(), tmem = uniform(sm.tmem_base);
        constexpr uint32_t kFmt = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
        constexpr uint32_t id_s = instr_desc(1, kFmt, kFmt, false, false, BT, BN);
        constexpr uint32_t id_g = instr_desc(1, kFmt, kFmt, false, true, BT, D);
        const uint64_t q_desc = desc_k(sm.q), do_desc = desc_k(sm.dout);
        auto product = [&](uint32_t col, uint64_t rows, const Ring<NST>& at, uint64_t* bar) {
          mbar_wait(&sm.full[at.slot], at.parity, 511);
          tc_fence_after();
          mma_rows<D, BN>(leader, tmem + col, rows, desc_k(sm.ring[at.slot]), id_s);
          mma_commit_warp(leader, bar);
        };
        Ring<NST> s_at, v_at, k_at;  // K of the next S, V of the next dP, K of the next dQ
        v_at.next();
        mbar_wait(&sm.q_full, 0, 510);
        product(0, q_desc, s_at, &sm.s_full[0]);
        product(kColDP, do_desc, v_at, &sm.dp_full);
        mma_commit_warp(leader, &sm.empty[v_at.slot]);
        s_at.next();
        s_at.next();
        v_at.next();
        v_at.next();
        if (n_all > 1) {
          product(BN, q_desc, s_at, &sm.s_full[1]);
          s_at.next();
          s_at.next();
        }
        for (int n = 0; n < n_all; ++n) {
          if (n + 1 < n_all) {  // dP of the next run once this one's has been read
            mbar_wait(&sm.dp_free, n & 1, 512);
            product(kColDP, do_desc, v_at, &sm.dp_full);
            mma_commit_warp(leader, &sm.empty[v_at.slot]);
            v_at.next();
            v_at.next();
          }
          mbar_wait(&sm.ds_ready[n & 1], (n >> 1) & 1, 513);
          tc_fence_after();
          // dQ += dS K
          if (n >= pre)
            mma_sum<C::kWG>(leader, tmem + kColDQ, tmem + BN * (n & 1), desc_mn<BN>(sm.ring[k_at.slot]),
                            id_g, n == pre);
          mma_commit_warp(leader, &sm.empty[k_at.slot]);
          k_at.next();
          k_at.next();
          if (n + 2 < n_all) {
            product(BN * (n & 1), q_desc, s_at, &sm.s_full[n & 1]);
            s_at.next();
            s_at.next();
          }
        }
        mma_commit_warp(leader, &sm.done);
      }
      __syncwarp();
    }
    tc_fence_before();
    named_barrier_sync(15, C::kThreads);
    tc_fence_after();
    if (warp == C::kMmaWarp) tmem_dealloc(tmem, C::kTmem);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(C::kComputeRegs));
    const int half = warp >> 2;
    const int r = (warp & 3) * 32 + lane;  // query row of the tile
    const uint32_t lane_base = tmem + (((warp & 3) * 32u) << 16);
    const int i = row_index(it, it.tile, r);
    const int64_t row = static_cast<int64_t>(it.start) + i;
    // padding rows: P = exp2(-inf) = 0
    const float neg_shift =
        i >= 0 ? fmaf(a.lse[head * a.T + row], -kLog2e, Scaling<T>::kPShift) : -INFINITY;
    float dvec = i >= 0 && !twice ? a.dvec[head * a.T + row] : 0.0f;
    const float c = a.scale_log2;
    float factor = 1.0f;
    if (Scaling<T>::kOn)
      factor = ds_factor(
          a.norms + (static_cast<int64_t>(it.seq) * a.kv_heads + kv_head) * 2);
    const float f_ds = factor * exp2f(-Scaling<T>::kPShift);

    const int keys0 = row_index<BN>(it, first + from, 64 * half);
    auto step = [&](int n, int key0, auto masked) {
      constexpr bool MASK = decltype(masked)::value;
      const uint32_t s_at = lane_base + BN * (n & 1) + 64 * half;
      const uint32_t dp_at = lane_base + kColDP + 64 * half;
      uint32_t x[2][32];
      mbar_wait(&sm.s_full[n & 1], (n >> 1) & 1, 520);
      tc_fence_after();
      tmem_ld32(s_at, x[0]);
      tmem_ld32(s_at + 32, x[1]);
      tmem_ld_wait_regs32(x[0]);
      tie32(x[1]);
      const int last = a.causal ? i : 0x7fffffff;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        probabilities<MASK, false>(
            x[h], c, [&](int) { return make_float2(neg_shift, neg_shift); },
            [&](int e) { return key0 + 32 * h + e < 0 || key0 + 32 * h + e > last; });
      mbar_wait(&sm.dp_full, n & 1, 521);
      tc_fence_after();
      if (n < pre) {  // D += P dP
        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t y[32];
          tmem_ld32(dp_at + 32 * h, y);
          tmem_ld_wait_regs32(y);
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            sum = __ffma2_rn(make_float2(__uint_as_float(x[h][e]), __uint_as_float(x[h][e + 1])),
                             make_float2(__uint_as_float(y[e]), __uint_as_float(y[e + 1])), sum);
        }
        tc_fence_before();
        mbar_arrive_warp(&sm.dp_free, lane);
        mbar_arrive_warp(&sm.ds_ready[n & 1], lane);
        dvec += (sum.x + sum.y) * exp2f(-Scaling<T>::kPShift);
        if (n == pre - 1) {
          if (C::kWG == 2) {
            sm.dot[half][r] = dvec;
            named_barrier_sync(1, C::kCompute);
            dvec = sm.dot[0][r] + sm.dot[1][r];
          }
          if (half == 0 && i >= 0) a.dvec[head * a.T + row] = dvec;
        }
        return;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t y[32], w[16];
        tmem_ld32(dp_at + 32 * h, y);
        tmem_ld_wait_regs32(y);
        if (h == 1) {
          tc_fence_before();
          mbar_arrive_warp(&sm.dp_free, lane);
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float2 p = make_float2(__uint_as_float(x[h][2 * e]), __uint_as_float(x[h][2 * e + 1]));
          if (Scaling<T>::kOn) p = __fmul2_rn(p, make_float2(f_ds, f_ds));
          const float2 t =
              __fadd2_rn(make_float2(__uint_as_float(y[2 * e]), __uint_as_float(y[2 * e + 1])),
                         make_float2(-dvec, -dvec));
          const float2 s = __fmul2_rn(p, t);
          w[e] = Cvt<T>::pack2(s.x, s.y);
        }
        tmem_st16(s_at + 16 * h, w);
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive_warp(&sm.ds_ready[n & 1], lane);
    };
    // runs that need a mask, from this part's first: the ragged first and the causal diagonal
    const int ragged = from == 0 && pad > 0 ? 0 : -1;
    const int diag = a.causal ? it.tile * (BT / BN) - first - from : 0x7fffffff;
    for (int n = 0, run = 0; n < n_all; ++n) {
      if (run == ragged || run >= diag)
        step(n, keys0 + run * BN, std::true_type{});
      else
        step(n, keys0 + run * BN, std::false_type{});
      if (++run == to - from) run = 0;  // the second time
    }
    if ((!PARTS || n_all > 0)) mbar_wait(&sm.done, 0, 522);
    tc_fence_after();
    // a warpgroup stores its part of the channels
    const float scale = a.tau / factor;
    T* dst = reinterpret_cast<T*>(a.out[0].ptr) + row * a.out[0].ts + head * a.out[0].hs;
    float* part = PARTS
                      ? a.part + ((split * a.tokens + row) * (a.grid.heads / splits) + head) * D
                      : nullptr;
#pragma unroll
    for (int k0 = 0; k0 < D / C::kWG; k0 += 32) {
      const int cc = half * (D / C::kWG) + k0;
      uint32_t y[32];
      tmem_ld32(lane_base + kColDQ + cc, y);
      tmem_ld_wait_regs32(y);
      if (i >= 0) store32<T, PARTS>(y, (!PARTS || n_all > 0), scale, dst + cc, PARTS ? part + cc : nullptr);
    }
    tc_fence_before();
    named_barrier_sync(15, C::kThreads);
  }
}

}  // namespace bwd
}  // namespace packed
}  // namespace sage
