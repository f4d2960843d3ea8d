// qk_rope.cuh -- QK-norm (RMSNorm over the head dimension, with a gain) and the rotation by
// the token's position in one pass over q and k, forward and backward.
//
//   forward:   xhat = x inv, inv = 1 / sqrt(mean x^2 + eps); y = R (xhat gain)
//   backward:  g = R^T dy; dgain += g xhat; gx = g gain; dx = inv (gx - xhat mean(gx xhat))
//
// Bound: HBM (about 10 flops per byte-pair moved; the forward moves 4 bytes per element, the
// backward 6).  Layout: a row of d channels is held by d/8 lanes (one 16-byte load each), and
// such a group of lanes walks the heads of one token, because the rotation's angles depend on
// the token only: its 8 sines and cosines per lane are computed once per token and used for
// every head of the group's chunk.
//
// Angles: frequency i as F_i = inv_freq_i / (2 pi) * 2^64 modulo 2^64, so position * F_i
// modulo 2^64 is the angle's fraction of a turn, with all full turns dropped exactly: the same
// accuracy at position 2^31 as at 1.  Its top 32 bits, read as a signed fraction of a half turn,
// go to sincospif in float32 (angle error below 2^-23).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "ptx.cuh"
#include "rowops.cuh"

namespace sage {
namespace rope {

constexpr int kThreads = 256;
constexpr int kMaxAxes = 4;

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
  float* partial;  // backward: [blocks][2][D] sums of dgain, or null
  int64_t pos_as, pos_bs;
  uint64_t freq[64];
  int bound[kMaxAxes - 1];  // first pair of axes 1, 2, 3
  int tokens, N, Hq, Hkv;
  int chunks, per_chunk;  // the heads of a token are cut into `chunks` of per_chunk
  int rotary, interleaved, n_axes, pos64, norm;
  float eps;
};

// Angle data of one lane: the cosine and (signed) sine of its 8 channels' pairs.
template <int D>
struct Turn {
  float c[8], s[8];
  bool rot;  // the lane's channels are rotated

  // y = R v (SIGN = 1) or R^T v (SIGN = -1) of the lane's 8 channels.  partner: lane that
  // holds the other channels of the pairs (half-split), or this lane itself.
  template <int SIGN>
  __device__ __forceinline__ void apply(float (&v)[8], bool interleaved, int partner,
                                        uint32_t mask) const {
    if (interleaved) {
      if (!rot) return;
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float a = v[e], b = v[e + 1];
        v[e] = fmaf(a, c[e], SIGN * b * s[e]);
        v[e + 1] = fmaf(b, c[e], SIGN * a * s[e + 1]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float o = __shfl_sync(mask, v[e], partner);
        if (rot) v[e] = fmaf(v[e], c[e], SIGN * o * s[e]);
      }
    }
  }
};

template <typename T, int D, bool BWD>
__global__ void __launch_bounds__(kThreads, BWD ? 2 : 4)
    qk_rope_kernel(const __grid_constant__ Args a) {
  constexpr int LPR = D / 8;             // lanes per row
  constexpr int GROUPS = kThreads / LPR; // groups of lanes per block
  __shared__ uint64_t freq[64];
  __shared__ float red[BWD ? GROUPS : 1][BWD ? D : 1];
  for (int i = threadIdx.x; i < 64; i += kThreads) freq[i] = a.freq[i];
  __syncthreads();

  const int lane = threadIdx.x & 31;
  const int l = lane % LPR;          // lane within the row
  const int base = lane - l;         // first lane of the row
  const uint32_t mask = LPR == 32 ? 0xffffffffu : ((1u << LPR) - 1u) << base;
  const int half = a.rotary >> 1;
  const int c0 = 8 * l;              // first channel of the lane
  const bool rot = c0 < a.rotary;
  int partner = lane, pair0 = 0;
  float sign = 1.0f;
  if (a.interleaved) {
    pair0 = c0 >> 1;
  } else if (rot) {
    const bool upper = c0 >= half;
    partner = upper ? lane - half / 8 : lane + half / 8;
    pair0 = upper ? c0 - half : c0;
    sign = upper ? 1.0f : -1.0f;  // y_lo = lo c - hi s, y_hi = hi c + lo s
  }
  float gain[2][8];
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int e = 0; e < 8; ++e) gain[w][e] = a.gain[w] ? a.gain[w][c0 + e] : 1.0f;
  float dgain[2][8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dgain[0][e] = dgain[1][e] = 0.0f;

  const int64_t units = static_cast<int64_t>(a.tokens) * a.chunks;
  const int64_t step = static_cast<int64_t>(gridDim.x) * GROUPS;
  const int H = a.Hq + a.Hkv;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * GROUPS + threadIdx.x / LPR; u < units;
       u += step) {
    const int token = static_cast<int>(u / a.chunks);
    const int chunk = static_cast<int>(u - static_cast<int64_t>(token) * a.chunks);
    const int b = token / a.N, n = token - b * a.N;
    Turn<D> t;
    t.rot = rot;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      t.c[e] = 1.0f;
      t.s[e] = 0.0f;
    }
    if (rot) {
      uint64_t p[kMaxAxes];
#pragma unroll
      for (int ax = 0; ax < kMaxAxes; ++ax) {
        if (ax >= a.n_axes) {
          p[ax] = 0;
          continue;
        }
        const int64_t at = ax * a.pos_as + b * a.pos_bs + n;
        p[ax] = a.pos64 ? static_cast<uint64_t>(static_cast<const int64_t*>(a.pos)[at])
                        : static_cast<uint64_t>(
                              static_cast<int64_t>(static_cast<const int32_t*>(a.pos)[at]));
      }
      auto angle = [&](int i, float& s, float& c) {
        uint64_t pp = p[0];
        if (i >= a.bound[0]) pp = p[1];
        if (i >= a.bound[1]) pp = p[2];
        if (i >= a.bound[2]) pp = p[3];
        const int32_t top = static_cast<int32_t>((pp * freq[i]) >> 32);
        sincospif(static_cast<float>(top) * 4.656612873077393e-10f, &s, &c);  // 2^-31
      };
      if (a.interleaved) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          float s, c;
          angle(pair0 + (e >> 1), s, c);
          t.c[e] = t.c[e + 1] = c;
          t.s[e] = -s;
          t.s[e + 1] = s;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float s, c;
          angle(pair0 + e, s, c);
          t.c[e] = c;
          t.s[e] = sign * s;
        }
      }
    }
    const int h_end = min(H, (chunk + 1) * a.per_chunk);
    // one tensor after the other: a chunk may hold heads of both
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int first = w == 0 ? 0 : a.Hq;
      const int lo = max(chunk * a.per_chunk, first) - first;
      const int hi = min(h_end, w == 0 ? a.Hq : H) - first;
      const T* xp = reinterpret_cast<const T*>(a.x[w].ptr) + b * a.x[w].bs +
                    static_cast<int64_t>(n) * a.x[w].ts + c0;
      const T* gp = BWD ? reinterpret_cast<const T*>(a.g[w].ptr) + b * a.g[w].bs +
                              static_cast<int64_t>(n) * a.g[w].ts + c0
                        : nullptr;
      T* yp = reinterpret_cast<T*>(a.y[w].ptr) + b * a.y[w].bs +
              static_cast<int64_t>(n) * a.y[w].ts + c0;
      constexpr int UN = BWD ? 2 : 4;  // rows in flight per group
      for (int h0 = lo; h0 < hi; h0 += UN) {
        uint4 xr[UN], gr[UN];
#pragma unroll
        for (int i = 0; i < UN; ++i) {
          const int h = min(h0 + i, hi - 1);
          xr[i] = __ldcs(reinterpret_cast<const uint4*>(xp + h * a.x[w].hs));
          if (BWD) gr[i] = __ldcs(reinterpret_cast<const uint4*>(gp + h * a.g[w].hs));
        }
#pragma unroll
        for (int i = 0; i < UN; ++i) {
          if (h0 + i >= hi) break;
          float x[8];
          Cvt<T>::load8(xr[i], x);
          float inv = 1.0f;
          if (a.norm) {
            float ss = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
            inv = 1.0f / sqrtf(row_sum<LPR>(ss, mask) * (1.0f / D) + a.eps);
          }
          if (!BWD) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= inv * gain[w][e];
            t.template apply<1>(x, a.interleaved, partner, mask);
            *reinterpret_cast<uint4*>(yp + (h0 + i) * a.y[w].hs) = pack8<T>(x);
          } else {
            float g[8];
            Cvt<T>::load8(gr[i], g);
            t.template apply<-1>(g, a.interleaved, partner, mask);
            if (a.norm) {
              float dot = 0.0f;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                x[e] *= inv;
                dgain[w][e] = fmaf(g[e], x[e], dgain[w][e]);
                g[e] *= gain[w][e];
                dot = fmaf(g[e], x[e], dot);
              }
              dot = row_sum<LPR>(dot, mask) * (1.0f / D);
#pragma unroll
              for (int e = 0; e < 8; ++e) g[e] = inv * fmaf(-x[e], dot, g[e]);
            }
            *reinterpret_cast<uint4*>(yp + (h0 + i) * a.y[w].hs) = pack8<T>(g);
          }
        }
      }
    }
  }
  if constexpr (BWD) {
    if (a.partial == nullptr) return;
    // the block's sums, groups in order
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 8; ++e) red[threadIdx.x / LPR][c0 + e] = dgain[w][e];
      __syncthreads();
      for (int c = threadIdx.x; c < D; c += kThreads) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) sum += red[i][c];
        a.partial[(static_cast<size_t>(blockIdx.x) * 2 + w) * D + c] = sum;
      }
    }
  }
}

// dgain from the blocks' partial sums: 32 channels per block, 32 threads per channel each
// sum every 32nd partial, then a tree, all in a fixed order.
template <int D>
__global__ void __launch_bounds__(1024)
    dgain_kernel(const float* partial, int blocks, float* dgain_q, float* dgain_k) {
  __shared__ float red[32][33];
  const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + c;  // column of [2][D]
  float sum = 0.0f;
  for (int i = r; i < blocks; i += 32) sum += partial[static_cast<size_t>(i) * 2 * D + col];
  red[r][c] = sum;
  __syncthreads();
  // transposed: warp r now holds channel r
  float v = red[c][r];
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (c == 0) {
    const int out = blockIdx.x * 32 + r;
    if (out < D) dgain_q[out] = v;
    else dgain_k[out - D] = v;
  }
}

}  // namespace rope
}  // namespace sage
