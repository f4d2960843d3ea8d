// qk_rope.cuh -- QK-norm (RMSNorm over the head dimension, with a gain) and the rotation by
// the token's position in one pass over q and k, forward and backward.
//
//   forward:   xhat = x inv, inv = 1 / sqrt(mean x^2 + eps); y = R (xhat gain)
//   backward:  g = R^T dy; dgain += g xhat; gx = g gain; dx = inv (gx - xhat mean(gx xhat))
//
// Bound: HBM (the forward moves 4 bytes per element, the backward 6).  Layout: a row of d
// channels is held by d/8 lanes, each with two groups of 4 channels (two 8-byte loads): the two
// halves of the same 4 pairs, so the rotation needs no exchange between lanes and a lane needs
// 4 sines and cosines.  Such a group of lanes walks the heads of one token, because the angles
// depend on the token only, a few rows at a time so that their loads and their row sums overlap.
// The blocks are split between q and k by their heads (a warp never works on both).
// The backward reads two rows and keeps more per row in registers, so too few bytes would be in
// flight; each of its threads copies its own channels kAhead rows ahead into shared memory that
// only it reads (no barrier: its own copy groups order it).
//
// Measured (B200): 262144 tokens, 20 heads of 128: forward 459 us (5.8 TB/s), backward 836 us (4.8
// TB/s, against 875 us with rows loaded to registers where they are used); 16384 tokens, 32 heads
// of 64: 30 us and 46 us; a copy runs at 6.5 TB/s.  What keeps the backward from that is latency:
// 125 registers leave 16 warps to an SM, and neither the issue slots (60%) nor DRAM (60%) are full.
//
// Angles: frequency i as F_i = inv_freq_i / (2 pi) * 2^64 modulo 2^64, so position * F_i
// modulo 2^64 is the angle's fraction of a turn, with all full turns dropped exactly.  F_i is rounded
// to a whole number, which moves the angle by 2 pi |position| 2^-65: 2^-31 at position 2^31, 2^-22 at
// 2^40.  The top 32 bits, a signed fraction of a half turn, become a float angle in [-pi, pi]
// (three roundings of 2^-24 pi), whose fast sine and cosine are within 2^-21: 2^-20 in all (they
// multiply values that are rounded to 2^-9 or 2^-11 afterwards).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <type_traits>

#include "ptx.cuh"
#include "rowops.cuh"

namespace sage {
namespace rope {

constexpr int kThreads = 256;
constexpr int kMaxAxes = 4;
constexpr int kAhead = 4;  // rows, backward
constexpr size_t kBwdSmem = static_cast<size_t>(kAhead) * 4 * kThreads * 8;

struct Rows {
  char* ptr;
  int64_t bs, ts, hs;  // elements
};

struct Args {
  Rows x[2];    // raw q, k
  Rows g[2];    // backward: gradients of the outputs
  Rows y[2];    // forward: outputs; backward: gradients of q, k
  const float* gain[2];
  const void* pos;
  float* partial;  // backward: [blocks][D] sums of dgain, or null
  int64_t pos_as, pos_bs;
  uint64_t freq[64];
  int bound[kMaxAxes - 1];  // first pair of axes 1, 2, 3
  int tokens, N;
  int blocks_q;                 // blocks that work on q; the others work on k
  int heads[2];
  int chunks[2], per_chunk[2];  // the heads of a token are cut into `chunks` of per_chunk
  int rotary, pos64, norm;
  float eps;
};

// The 8 channels of a lane as 4 pairs (a, b), two pairs per packed operation.
struct Pairs {
  float2 a[2], b[2];
};

// u: the lane's first 4 channels, v: its second 4.  INTER: pairs are neighbouring channels;
// otherwise channel e of u with channel e of v.
template <typename T, bool INTER>
__device__ __forceinline__ Pairs unpack(const uint2& u, const uint2& v) {
  float f[8];
  Cvt<T>::load8(make_uint4(u.x, u.y, v.x, v.y), f);
  Pairs p;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    p.a[i] = INTER ? make_float2(f[4 * i], f[4 * i + 2]) : make_float2(f[2 * i], f[2 * i + 1]);
    p.b[i] = INTER ? make_float2(f[4 * i + 1], f[4 * i + 3])
                   : make_float2(f[4 + 2 * i], f[5 + 2 * i]);
  }
  return p;
}
template <typename T, bool INTER>
__device__ __forceinline__ void pack(const Pairs& p, uint2& u, uint2& v) {
  if (INTER) {
    u = make_uint2(Cvt<T>::pack2(p.a[0].x, p.b[0].x), Cvt<T>::pack2(p.a[0].y, p.b[0].y));
    v = make_uint2(Cvt<T>::pack2(p.a[1].x, p.b[1].x), Cvt<T>::pack2(p.a[1].y, p.b[1].y));
  } else {
    u = make_uint2(Cvt<T>::pack2(p.a[0].x, p.a[0].y), Cvt<T>::pack2(p.a[1].x, p.a[1].y));
    v = make_uint2(Cvt<T>::pack2(p.b[0].x, p.b[0].y), Cvt<T>::pack2(p.b[1].x, p.b[1].y));
  }
}

template <typename T, int D, bool INTER, bool BWD>
__global__ void __launch_bounds__(kThreads, BWD ? 2 : 3)
    qk_rope_kernel(const __grid_constant__ Args a) {
  constexpr int LPR = D / 8;              // lanes per row
  constexpr int GROUPS = kThreads / LPR;  // groups of lanes per block
  constexpr int UN = BWD ? 2 : 4;  // rows at a time
  const int lane = threadIdx.x & 31;
  const int l = lane % LPR;               // lane within the row
  const uint32_t mask = ((1u << LPR) - 1u) << (lane - l);
  const int half = a.rotary >> 1;
  // first channels of the lane's two groups
  const bool rot = INTER ? 8 * l < a.rotary : 4 * l < half;
  int cu, cv;
  if (INTER) {
    cu = 8 * l;
    cv = cu + 4;
  } else if (rot) {
    cu = 4 * l;
    cv = cu + half;
  } else {
    cu = a.rotary + 8 * (l - half / 4);
    cv = cu + 4;
  }
  const int dv = cv - cu;
  extern __shared__ uint2 rope_smem[];  // backward: [kAhead][4][kThreads], then the sums
  uint2* ring = rope_smem + threadIdx.x;
  Pairs dgain, gain;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    dgain.a[i] = dgain.b[i] = make_float2(0.0f, 0.0f);
    gain.a[i] = gain.b[i] = make_float2(1.0f, 1.0f);
  }
  const int w = static_cast<int>(blockIdx.x) >= a.blocks_q ? 1 : 0;
  const int block = blockIdx.x - (w ? a.blocks_q : 0);
  const int blocks = w ? gridDim.x - a.blocks_q : a.blocks_q;
  const int chunks = a.chunks[w], per_chunk = a.per_chunk[w], H = a.heads[w];
  if (a.gain[w]) {
    const float4 u = __ldg(reinterpret_cast<const float4*>(a.gain[w] + cu));
    const float4 v = __ldg(reinterpret_cast<const float4*>(a.gain[w] + cv));
    if (INTER) {
      gain.a[0] = make_float2(u.x, u.z);
      gain.b[0] = make_float2(u.y, u.w);
      gain.a[1] = make_float2(v.x, v.z);
      gain.b[1] = make_float2(v.y, v.w);
    } else {
      gain.a[0] = make_float2(u.x, u.y);
      gain.a[1] = make_float2(u.z, u.w);
      gain.b[0] = make_float2(v.x, v.y);
      gain.b[1] = make_float2(v.z, v.w);
    }
  }
  const int64_t xs = a.x[w].hs, gs = a.g[w].hs, ys = a.y[w].hs;

  // a block's unit: GROUPS tokens, one chunk of their heads; neighbouring blocks take the same
  // tokens' chunks
  const int tiles = (a.tokens + GROUPS - 1) / GROUPS;
  const int64_t units = static_cast<int64_t>(tiles) * chunks;
  for (int64_t unit = block; unit < units; unit += blocks) {
    const int tile = static_cast<int>(unit / chunks);
    const int lo = static_cast<int>(unit - static_cast<int64_t>(tile) * chunks) * per_chunk;
    const int hi = min(H, lo + per_chunk);
    const int token = tile * GROUPS + threadIdx.x / LPR;
    if (token >= a.tokens) continue;
    const int b = token < a.N ? 0 : token / a.N, n = token - b * a.N;
    auto row_at = [&](const Rows& r) {
      return reinterpret_cast<T*>(r.ptr) + b * r.bs + static_cast<int64_t>(n) * r.ts +
             static_cast<int64_t>(lo) * r.hs + cu;
    };
    const T* xp = row_at(a.x[w]);
    const T* gp = BWD ? row_at(a.g[w]) : nullptr;
    T* yp = row_at(a.y[w]);
    int64_t at[4];  // the positions of the lane's pairs
    if (rot) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = 4 * l + e;
        const int axis = (i >= a.bound[0]) + (i >= a.bound[1]) + (i >= a.bound[2]);
        const int64_t from = axis * a.pos_as + b * a.pos_bs + n;
        at[e] = a.pos64 ? __ldg(static_cast<const long long*>(a.pos) + from)
                        : __ldg(static_cast<const int32_t*>(a.pos) + from);
      }
    }
    float2 cs[2], sn[2], ns[2];
    bool fresh = rot;  // the angles are still to be computed: after the first rows' loads
    auto angles = [&]() {
      float s[4], c[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int32_t top =
            static_cast<int32_t>((static_cast<uint64_t>(at[e]) * a.freq[4 * l + e]) >> 32);
        __sincosf(static_cast<float>(top) * 1.4629180792671596e-9f, &s[e], &c[e]);  // pi 2^-31
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        cs[i] = make_float2(c[2 * i], c[2 * i + 1]);
        sn[i] = make_float2(s[2 * i], s[2 * i + 1]);
        ns[i] = make_float2(-sn[i].x, -sn[i].y);
      }
      fresh = false;
    };
    int h = lo;
    int slot = 0, next = lo;  // backward: of row h in the ring; next row to copy
    auto copy = [&](int s) {
      if (next < hi) {
        uint2* at_s = ring + s * 4 * kThreads;
        copy_async8(at_s, xp);
        copy_async8(at_s + kThreads, xp + dv);
        copy_async8(at_s + 2 * kThreads, gp);
        copy_async8(at_s + 3 * kThreads, gp + dv);
        xp += xs;
        gp += gs;
        ++next;
      }
      copy_async_commit();  // a group per row, empty ones too: the waits count groups
    };
    if (BWD)
#pragma unroll
      for (int s = 0; s < kAhead; ++s) copy(s);
    // R rows from h on
    auto rows = [&](auto count) {
      constexpr int R = decltype(count)::value;
      uint2 xu[R], xv[R], gu[R], gv[R];
      if (BWD) copy_async_wait<kAhead - R>();
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (BWD) {
          const uint2* at_s = ring + ((slot + i) % kAhead) * 4 * kThreads;
          xu[i] = at_s[0];
          xv[i] = at_s[kThreads];
          gu[i] = at_s[2 * kThreads];
          gv[i] = at_s[3 * kThreads];
        } else {
          xu[i] = __ldcs(reinterpret_cast<const uint2*>(xp));
          xv[i] = __ldcs(reinterpret_cast<const uint2*>(xp + dv));
          xp += xs;
        }
      }
      if (fresh) angles();
      if (!BWD) {
        float inv[R];
        if (a.norm) {
#pragma unroll
          for (int i = 0; i < R; ++i) {
            const Pairs x = unpack<T, INTER>(xu[i], xv[i]);
            float2 ss = __fmul2_rn(x.a[0], x.a[0]);
            ss = __ffma2_rn(x.b[0], x.b[0], ss);
            ss = __ffma2_rn(x.a[1], x.a[1], ss);
            ss = __ffma2_rn(x.b[1], x.b[1], ss);
            inv[i] = ss.x + ss.y;
          }
#pragma unroll
          for (int o = LPR / 2; o >= 1; o >>= 1)
#pragma unroll
            for (int i = 0; i < R; ++i) inv[i] += __shfl_xor_sync(mask, inv[i], o);
#pragma unroll
          for (int i = 0; i < R; ++i) inv[i] = rsqrtf(fmaf(inv[i], 1.0f / D, a.eps));
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
          Pairs x = unpack<T, INTER>(xu[i], xv[i]);
          if (a.norm) {
            const float2 inv2 = make_float2(inv[i], inv[i]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              x.a[k] = __fmul2_rn(__fmul2_rn(x.a[k], inv2), gain.a[k]);
              x.b[k] = __fmul2_rn(__fmul2_rn(x.b[k], inv2), gain.b[k]);
            }
          }
          if (rot) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float2 p = x.a[k], q = x.b[k];
              x.a[k] = __ffma2_rn(p, cs[k], __fmul2_rn(q, ns[k]));
              x.b[k] = __ffma2_rn(q, cs[k], __fmul2_rn(p, sn[k]));
            }
          }
          uint2 u, v;
          pack<T, INTER>(x, u, v);
          *reinterpret_cast<uint2*>(yp) = u;
          *reinterpret_cast<uint2*>(yp + dv) = v;
          yp += ys;
        }
      } else {
        Pairs g[R];
        float2 sums[R];  // of x^2 and of gx x: xhat = x inv, inv known only after them
#pragma unroll
        for (int i = 0; i < R; ++i) {
          g[i] = unpack<T, INTER>(gu[i], gv[i]);
          if (rot) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float2 p = g[i].a[k], q = g[i].b[k];
              g[i].a[k] = __ffma2_rn(p, cs[k], __fmul2_rn(q, sn[k]));
              g[i].b[k] = __ffma2_rn(q, cs[k], __fmul2_rn(p, ns[k]));
            }
          }
          if (a.norm) {
            const Pairs x = unpack<T, INTER>(xu[i], xv[i]);
            float2 ss = make_float2(0.0f, 0.0f), dot = ss;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              ss = __ffma2_rn(x.a[k], x.a[k], __ffma2_rn(x.b[k], x.b[k], ss));
              dot = __ffma2_rn(__fmul2_rn(g[i].a[k], gain.a[k]), x.a[k], dot);
              dot = __ffma2_rn(__fmul2_rn(g[i].b[k], gain.b[k]), x.b[k], dot);
            }
            sums[i] = make_float2(ss.x + ss.y, dot.x + dot.y);
          }
        }
        if (a.norm) {
#pragma unroll
          for (int o = LPR / 2; o >= 1; o >>= 1)
#pragma unroll
            for (int i = 0; i < R; ++i)
              sums[i] = __fadd2_rn(sums[i], make_float2(__shfl_xor_sync(mask, sums[i].x, o),
                                                        __shfl_xor_sync(mask, sums[i].y, o)));
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
          if (a.norm) {
            Pairs x = unpack<T, INTER>(xu[i], xv[i]);
            const float inv = rsqrtf(fmaf(sums[i].x, 1.0f / D, a.eps));
            // xhat mean(gx xhat) = xhat * (mean(gx x) inv)
            const float mean = sums[i].y * (1.0f / D) * inv;
            const float2 inv2 = make_float2(inv, inv), neg2 = make_float2(-mean, -mean);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              x.a[k] = __fmul2_rn(x.a[k], inv2);
              x.b[k] = __fmul2_rn(x.b[k], inv2);
              dgain.a[k] = __ffma2_rn(g[i].a[k], x.a[k], dgain.a[k]);
              dgain.b[k] = __ffma2_rn(g[i].b[k], x.b[k], dgain.b[k]);
              g[i].a[k] = __fmul2_rn(
                  __ffma2_rn(x.a[k], neg2, __fmul2_rn(g[i].a[k], gain.a[k])), inv2);
              g[i].b[k] = __fmul2_rn(
                  __ffma2_rn(x.b[k], neg2, __fmul2_rn(g[i].b[k], gain.b[k])), inv2);
            }
          }
          uint2 u, v;
          pack<T, INTER>(g[i], u, v);
          *reinterpret_cast<uint2*>(yp) = u;
          *reinterpret_cast<uint2*>(yp + dv) = v;
          yp += ys;
        }
      }
      h += R;
      if (BWD) {  // these rows have been used: their places are free
#pragma unroll
        for (int i = 0; i < R; ++i) copy((slot + i) % kAhead);
        slot = (slot + R) % kAhead;
      }
    };
    while (h + UN <= hi) rows(std::integral_constant<int, UN>{});
    while (h < hi) rows(std::integral_constant<int, 1>{});
  }
  if constexpr (BWD) {
    copy_async_wait<0>();
    if (a.partial == nullptr) return;
    // the block's sums, groups in order
    __syncthreads();  // every thread has read its rows
    float(*red)[D] = reinterpret_cast<float(*)[D]>(rope_smem);
    float* row = red[threadIdx.x / LPR];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 p = dgain.a[i], q = dgain.b[i];
      if (INTER) {
        float* at = row + (i == 0 ? cu : cv);
        at[0] = p.x;
        at[1] = q.x;
        at[2] = p.y;
        at[3] = q.y;
      } else {
        row[cu + 2 * i] = p.x;
        row[cu + 2 * i + 1] = p.y;
        row[cv + 2 * i] = q.x;
        row[cv + 2 * i + 1] = q.y;
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += kThreads) {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < GROUPS; ++i) sum += red[i][c];
      a.partial[static_cast<size_t>(blockIdx.x) * D + c] = sum;
    }
  }
}

// dgain from the blocks' partial sums (the first blocks_q are q's): 32 channels per block, 32
// threads per channel each sum every 32nd partial, then a tree, all in a fixed order.
template <int D>
__global__ void __launch_bounds__(1024)
    dgain_kernel(const float* partial, int blocks_q, int blocks, float* dgain_q, float* dgain_k) {
  __shared__ float red[32][33];
  const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
  const bool on_k = blockIdx.x >= D / 32;
  const int col = (blockIdx.x % (D / 32)) * 32;
  const int end = on_k ? blocks : blocks_q;
  float sum = 0.0f;
  for (int i = (on_k ? blocks_q : 0) + r; i < end; i += 32)
    sum += partial[static_cast<size_t>(i) * D + col + c];
  red[r][c] = sum;
  __syncthreads();
  // transposed: warp r now holds channel r
  float v = red[c][r];
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (c == 0) (on_k ? dgain_k : dgain_q)[col + r] = v;
}

}  // namespace rope
}  // namespace sage
