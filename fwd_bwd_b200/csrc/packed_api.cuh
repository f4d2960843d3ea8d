// packed_api.cuh -- host side of include/sage_packed.h: argument checks, the packed plan, tensor
// maps and launches.  Included once, by sage_api.cu (one translation unit).
#pragma once

#include <algorithm>
#include <atomic>
#include <new>
#include <vector>

#include "packed_bwd.cuh"
#include "packed_fwd.cuh"
#include "qk_rope.cuh"
#include "sage_packed.h"

namespace {

using sage::packed::Item;

int check_rows(const sage_rows* r, int64_t batches, int64_t tokens, int heads, int d, bool out) {
  if (!r || !r->ptr) return SAGE_ERR_INVALID_ARG;
  if (!aligned16(r->ptr)) return SAGE_ERR_ALIGNMENT;
  const int64_t n[3] = {batches, tokens, heads};
  const int64_t s[3] = {r->batch_stride, r->token_stride, r->head_stride};
  constexpr int64_t kMost = int64_t{1} << 38;  // elements; byte strides stay below 2^40
  for (int i = 0; i < 3; ++i) {
    if (n[i] == 1) continue;  // the stride of a single entry is never used
    if (s[i] < d || s[i] > kMost) return SAGE_ERR_INVALID_ARG;
    if (s[i] % 8 != 0) return SAGE_ERR_ALIGNMENT;
  }
  if (out) {  // no two vectors of an output may overlap: sorted by stride, each axis must clear
              // the extent of the ones inside it
    int order[3] = {0, 1, 2};
    std::sort(order, order + 3, [&](int x, int y) { return s[x] < s[y]; });
    int64_t extent = d;
    for (int i : order) {
      if (n[i] == 1) continue;
      if (s[i] < extent) return SAGE_ERR_INVALID_ARG;
      extent += s[i] * (n[i] - 1);
    }
  }
  return SAGE_OK;
}

// ---- QK-norm and rotary positions ---------------------------------------------------------
int check_rope(const sage_rope_params* p) {
  if (!p || p->B <= 0 || p->N <= 0 || p->Hq <= 0 || p->Hkv <= 0) return SAGE_ERR_INVALID_ARG;
  if (p->dtype != SAGE_FP16 && p->dtype != SAGE_BF16) return SAGE_ERR_INVALID_ARG;
  if (p->d != 64 && p->d != 128) return SAGE_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(p->B) * p->N >= (int64_t{1} << 31) - 64 || p->Hq > 65536 ||
      p->Hkv > 65536)
    return SAGE_ERR_UNSUPPORTED;
  if ((p->norm != 0 && p->norm != 1) || (p->interleaved != 0 && p->interleaved != 1))
    return SAGE_ERR_INVALID_ARG;
  if (!(p->eps >= 0.0f) || !std::isfinite(p->eps)) return SAGE_ERR_INVALID_ARG;
  if (p->rotary_dim < 0 || p->rotary_dim > p->d) return SAGE_ERR_INVALID_ARG;
  if (p->rotary_dim % 16 != 0) return SAGE_ERR_UNSUPPORTED;
  if (p->rotary_dim > 0) {
    if (!p->inv_freq || (p->pos_bits != 32 && p->pos_bits != 64)) return SAGE_ERR_INVALID_ARG;
    if (p->n_axes < 1 || p->n_axes > sage::rope::kMaxAxes) return SAGE_ERR_INVALID_ARG;
    int64_t sum = 0;
    for (int i = 0; i < p->n_axes; ++i) {
      if (p->sections[i] <= 0) return SAGE_ERR_INVALID_ARG;
      sum += p->sections[i];
    }
    if (sum != p->rotary_dim / 2) return SAGE_ERR_INVALID_ARG;
    for (int i = 0; i < p->rotary_dim / 2; ++i)
      if (!std::isfinite(p->inv_freq[i])) return SAGE_ERR_INVALID_ARG;
    if (p->pos_axis_stride < 0 || p->pos_batch_stride < 0) return SAGE_ERR_INVALID_ARG;
  }
  return SAGE_OK;
}

// inv_freq / (2 pi) as a fraction of a turn per position, in units of 2^-64 turns.
uint64_t turn_fraction(double inv_freq) {
  const long double turns = static_cast<long double>(inv_freq) /
                            6.283185307179586476925286766559005768L;
  const long double frac = turns - std::floor(turns);  // [0, 1]
  const long double scaled = frac * 18446744073709551616.0L;
  return scaled >= 18446744073709551615.0L ? 0 : static_cast<uint64_t>(scaled + 0.5L);
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return n;
}

// Blocks of the gradient kernel at most (two per SM of a 148-SM device): their partial sums of
// the gains' gradients are added up by one small kernel.
constexpr int kRopeBwdBlocks = 296;

sage::rope::Rows rope_rows(const sage_rows* r) {
  return {static_cast<char*>(r->ptr), r->batch_stride, r->token_stride, r->head_stride};
}

void rope_args(const sage_rope_params* p, const sage_rows* q, const sage_rows* k,
               const sage_rows* yq, const sage_rows* yk, const float* gain_q,
               const float* gain_k, const void* pos, sage::rope::Args* a) {
  std::memset(a, 0, sizeof(*a));
  a->x[0] = rope_rows(q);
  a->x[1] = rope_rows(k);
  a->y[0] = rope_rows(yq);
  a->y[1] = rope_rows(yk);
  a->gain[0] = gain_q;
  a->gain[1] = gain_k;
  a->pos = pos;
  a->tokens = p->B * p->N;
  a->N = p->N;
  a->heads[0] = p->Hq;
  a->heads[1] = p->Hkv;
  a->rotary = p->rotary_dim;
  a->norm = p->norm;
  a->eps = p->eps;
  for (int& b : a->bound) b = 64;  // beyond the last pair
  if (p->rotary_dim > 0) {
    a->pos64 = p->pos_bits == 64;
    a->pos_as = p->pos_axis_stride;
    a->pos_bs = p->pos_batch_stride;
    for (int i = 0; i < p->rotary_dim / 2; ++i) a->freq[i] = turn_fraction(p->inv_freq[i]);
    for (int i = 0, at = 0; i + 1 < p->n_axes; ++i) a->bound[i] = at += p->sections[i];
  }
  // Heads of a token per lane group: all of a tensor's when there are many times more tokens than
  // groups on the device (the angles are then computed once per token), fewer otherwise; a
  // multiple of the rows computed together.
  const int64_t want = 2 * 148 * 1024 / (p->d / 8);  // two rounds of lane groups
  const int64_t chunks = std::max<int64_t>(1, (want + a->tokens - 1) / a->tokens);
  for (int w = 0; w < 2; ++w) {
    const int H = a->heads[w];
    const int per = static_cast<int>(std::max<int64_t>(1, (p->Hq + p->Hkv) / chunks));
    a->per_chunk[w] = std::min(H, per >= 4 ? per / 4 * 4 : per);
    if (chunks == 1) a->per_chunk[w] = H;
    a->chunks[w] = (H + a->per_chunk[w] - 1) / a->per_chunk[w];
  }
}

template <typename T, int D, bool INTER, bool BWD>
int run_rope(sage::rope::Args* a, float* dgain_q, float* dgain_k, cudaStream_t st) {
  const int groups = sage::rope::kThreads / (D / 8);
  const int sms = sm_count();
  if (sms == 0) return SAGE_ERR_CUDA;
  const int most = BWD ? std::min(kRopeBwdBlocks, 2 * sms) : 3 * sms;  // resident at once
  // q and k share them by their heads, and a token's angles and addresses at some rows' cost
  constexpr int kUnitCost = 2;
  const int64_t cost[2] = {a->heads[0] + kUnitCost * a->chunks[0],
                           a->heads[1] + kUnitCost * a->chunks[1]};
  const int64_t tiles = (a->tokens + groups - 1) / groups;
  const int64_t share = most * cost[0] / (cost[0] + cost[1]);
  const int for_q = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(share, most - 1)));
  a->blocks_q = static_cast<int>(std::min<int64_t>(tiles * a->chunks[0], for_q));
  const int blocks =
      a->blocks_q + static_cast<int>(std::min<int64_t>(tiles * a->chunks[1], most - for_q));
  auto kern = sage::rope::qk_rope_kernel<T, D, INTER, BWD>;
  const size_t smem = BWD ? sage::rope::kBwdSmem : 0;
  if (BWD && set_smem(kern, smem) != SAGE_OK) return SAGE_ERR_CUDA;
  kern<<<blocks, sage::rope::kThreads, smem, st>>>(*a);
  if (BWD && a->partial)
    sage::rope::dgain_kernel<D><<<2 * D / 32, 1024, 0, st>>>(a->partial, a->blocks_q, blocks,
                                                                 dgain_q, dgain_k);
  return launch_status();
}

template <bool BWD, typename T, int D>
int run_rope(const sage_rope_params* p, sage::rope::Args* a, float* dgain_q, float* dgain_k,
             cudaStream_t st) {
  return p->interleaved ? run_rope<T, D, true, BWD>(a, dgain_q, dgain_k, st)
                        : run_rope<T, D, false, BWD>(a, dgain_q, dgain_k, st);
}
template <bool BWD>
int launch_rope(const sage_rope_params* p, sage::rope::Args* a, float* dgain_q, float* dgain_k,
                cudaStream_t st) {
  const bool bf = p->dtype == SAGE_BF16;
  if (p->d == 128)
    return bf ? run_rope<BWD, __nv_bfloat16, 128>(p, a, dgain_q, dgain_k, st)
              : run_rope<BWD, __half, 128>(p, a, dgain_q, dgain_k, st);
  return bf ? run_rope<BWD, __nv_bfloat16, 64>(p, a, dgain_q, dgain_k, st)
            : run_rope<BWD, __half, 64>(p, a, dgain_q, dgain_k, st);
}

// ---- packed plan --------------------------------------------------------------------------
// Four lists of Items, each largest work first: query / key tiles under a causal mask (the
// work of query tile t is t + 1 key tiles; key tile tiles - 1 - t has the same), the same without
// (every tile of a sequence works over all of its tiles), then pairs of neighbouring tiles
// (named by the later one, cut from the sequence's end) in the same two orders.
bool plan_counts(const int* lengths, int n, sage_packed_info* info) {
  if (!lengths || n < 1) return false;
  int64_t tokens = 0, tiles = 0, pairs = 0, causal = 0, full = 0;
  int longest = 0;
  for (int i = 0; i < n; ++i) {
    if (lengths[i] < 0) return false;
    tokens += lengths[i];
    if (tokens >= (int64_t{1} << 31) - sage::packed::BT) return false;
    const int64_t t = (static_cast<int64_t>(lengths[i]) + sage::packed::BT - 1) / sage::packed::BT;
    tiles += t;
    pairs += (t + 1) / 2;
    causal += t * (t + 1) / 2;
    full += t * t;
    longest = std::max(longest, lengths[i]);
  }
  info->sequences = n;
  info->tiles = static_cast<int>(tiles);
  info->pairs = static_cast<int>(pairs);
  info->longest = longest;
  info->tokens = tokens;
  info->causal_steps = causal;
  info->full_steps = full;
  return true;
}

size_t plan_bytes(const sage_packed_info& i) {
  return sizeof(Item) * 2 * (static_cast<size_t>(i.tiles) + i.pairs) + sizeof(Item);
}
const Item* plan_list(const void* plan, const sage_packed_info* i, bool causal, bool pairs) {
  const Item* p = static_cast<const Item*>(plan);
  if (pairs) return p + 2 * static_cast<size_t>(i->tiles) + (causal ? 0 : i->pairs);
  return p + (causal ? 0 : i->tiles);
}

int check_packed(const sage_packed_params* p, const sage_packed_info* info, const void* plan) {
  if (!p || !info || !plan) return SAGE_ERR_INVALID_ARG;
  if (p->T <= 0 || p->Hq <= 0 || p->Hkv <= 0 || p->Hq % p->Hkv != 0) return SAGE_ERR_INVALID_ARG;
  if (p->dtype != SAGE_FP16 && p->dtype != SAGE_BF16) return SAGE_ERR_INVALID_ARG;
  if (p->causal != 0 && p->causal != 1) return SAGE_ERR_INVALID_ARG;
  if (!std::isfinite(p->softmax_scale)) return SAGE_ERR_INVALID_ARG;
  if (p->d != 64 && p->d != 128) return SAGE_ERR_UNSUPPORTED;
  if (p->T >= (int64_t{1} << 31) || p->Hq > 65536) return SAGE_ERR_UNSUPPORTED;
  if (info->sequences < 1 || info->tiles < 0 || info->pairs < 0 || info->pairs > info->tiles ||
      info->tokens < 0 || info->tokens > p->T)
    return SAGE_ERR_INVALID_ARG;
  // CTAs of the largest grids
  if (static_cast<int64_t>(info->tiles) * 8 * (static_cast<int64_t>(p->Hq) + p->Hkv) >=
      (int64_t{1} << 31))
    return SAGE_ERR_UNSUPPORTED;
  if (!aligned16(plan)) return SAGE_ERR_ALIGNMENT;
  return SAGE_OK;
}

float packed_tau(const sage_packed_params* p) {
  return p->softmax_scale > 0.0f ? p->softmax_scale
                                 : 1.0f / std::sqrt(static_cast<float>(p->d));
}

// 4-D map (channel, row of a tile, token, head) of 16-bit rows: the row and the token axis have
// the same stride, so a box that starts at a negative row reads zeros there.  The box is 64
// channels x d rows (rows of 128 bytes, swizzled).
bool make_tile_map(CUtensorMap* m, const sage_rows* r, const sage_packed_params* p, int heads) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t ts = p->T > 1 ? r->token_stride : p->d;
  const cuuint64_t hs = heads > 1 ? r->head_stride : p->d;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(p->d), sage::packed::BT,
                        static_cast<cuuint64_t>(p->T), static_cast<cuuint64_t>(heads)};
  cuuint64_t strides[3] = {ts * 2, ts * 2, hs * 2};
  cuuint32_t box[4] = {64, static_cast<cuuint32_t>(p->d), 1, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  auto encode = [&] {
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, r->ptr, dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult s = encode();
  if (s == CUDA_ERROR_INVALID_CONTEXT || s == CUDA_ERROR_NOT_INITIALIZED) {
    // a host thread that has made no runtime call yet (autograd's, say) has no current context:
    // bind the one of its current device
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess) return false;
    s = encode();
  }
  return s == CUDA_SUCCESS;
}

sage::packed::Out packed_out(const sage_rows* r) {
  return {static_cast<char*>(r->ptr), r->token_stride, r->head_stride};
}

// REGS: the launch allocation that the kernel's register split (setmaxnreg) is sized for; 0: none.
template <auto KERN, int REGS, typename... A>
int launch_packed(int64_t grid, int threads, size_t smem, cudaStream_t st, const A&... args) {
  if (set_smem(KERN, smem) != SAGE_OK) return SAGE_ERR_CUDA;
  if (REGS != 0) {
    // a property of the compiled kernel: asked for once
    static std::atomic<int> regs{0};
    int r = regs.load(std::memory_order_relaxed);
    if (r <= 0) regs.store(r = launch_regs(KERN), std::memory_order_relaxed);
    if (r != REGS) return SAGE_ERR_UNSUPPORTED;
  }
  KERN<<<static_cast<unsigned>(grid), threads, smem, st>>>(args...);
  return launch_status();
}

// Heads per chunk of the grid (packed::Grid) when the CTAs of one head read bytes_per_head over
// and over: as many as kChunkBytes holds, so that they stay in L2 (B200, 16 heads, 4 x 8192 tokens,
// d = 128: forward 1023 -> 933 us, dK/dV 1951 -> 1685 us, dQ 1649 -> 1365 us against all heads at
// once); but at least so many that a chunk keeps the device busy for longer than its longest
// item takes, because the last chunk's long items start late (16384 tokens in documents of
// 5021 to 2, 4 key heads, dK/dV: 330 us in one chunk, 442 us in four).
constexpr int64_t kChunkBytes = 40 << 20;  // of the 126 MB L2
// What is this small in all is taken in one chunk: a second one ends the first with a tail and no
// longer pays by its hits. One chunk against chunks of 40 MB (forward, dQ, dK/dV, us):
//   d = 64, 2048 tokens x 8:   50 MB  89, 106, 144 / 105, 114, 151;  67 MB 112, 135, 176 / 114, 138, 180;
//                             84 MB 140, 168, 220 / 138, 169, 224; 101 MB 170, 203, 272 / 176, 204, 280
//   d = 128, 4096 tokens x 2:  50 MB 104, 143, 168 / 130, 163, 178;  75 MB 143, 218, 251 / 145, 214, 249;
//                             84 MB 160, 243, 282 / 158, 235, 272; 101 MB 192, 300, 349 / 201, 281, 331
constexpr int64_t kAllBytes = 80 << 20;
int grid_chunk(const sage_packed_params* p, const sage_packed_info* info, int heads,
               int64_t bytes_per_head) {
  const int64_t fit = heads * bytes_per_head <= kAllBytes
                          ? heads
                          : kChunkBytes / std::max<int64_t>(bytes_per_head, 1);
  const int64_t tiles = (static_cast<int64_t>(info->longest) + 127) / 128;  // the longest item
  const int64_t steps = std::max<int64_t>(p->causal ? info->causal_steps : info->full_steps, 1);
  const int64_t busy = (3 * 148 * tiles / 2 + steps - 1) / steps;  // 1.5 x the longest item
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(heads, std::max(fit, busy))));
}

// Parts that a kernel's walks are cut into.  A CTA walks all the tiles its own tile meets; with few
// heads that leaves SMs idle or one long walk at the end.  Cut when the longest walk (steps) is
// twice the device's share of all of them or more, into parts of eight steps at least, eight parts
// at most (each costs 8 bytes of traffic per element of the output, and the joining kernel 4 to 10
// us).  Whole / cut, us with the joining kernel:
//   8192 tokens, 1 head of 128:   forward 99 / 36 + 7, dQ 76 / 32 + 5, dK/dV 88 / 41 + 7
//   2048 tokens, 32 heads on one key head of 128: dK/dV 621 / 94 + 4
//   4096 tokens, heads of 128, forward: 4 heads (longest 4.5 x the share) 57 / 38 + 7; 8 heads (2.2 x)
//     58 / 50 + 10; cut from the share on: 12 heads (1.5 x) 61 / 92 + 20, 16 heads (1.1 x) 67 / 95 + 20
int walk_splits(int64_t longest, int64_t all, int places) {
  const int64_t share = std::max<int64_t>(1, all / places);
  return static_cast<int>(std::max<int64_t>(
      1, std::min<int64_t>({longest / share, longest / 8, 8})));
}
int64_t all_steps(const sage_packed_params* p, const sage_packed_info* info) {
  return (p->causal ? info->causal_steps : info->full_steps) * p->Hq;
}
int64_t longest_tiles(const sage_packed_info* info) {
  return (static_cast<int64_t>(info->longest) + 127) / 128;
}
// Forward: d = 128 takes two tiles per CTA, d = 64 four CTAs per SM, the backward two.
int fwd_splits(const sage_packed_params* p, const sage_packed_info* info) {
  const bool wide = p->d == 128;
  return walk_splits(longest_tiles(info), all_steps(p, info) / (wide ? 2 : 1),
                     148 * (wide ? 1 : 4));
}
int dq_splits(const sage_packed_params* p, const sage_packed_info* info) {
  return walk_splits(longest_tiles(info), all_steps(p, info),
                     148 * (p->d == 64 ? 2 : 1));
}
int dkv_splits(const sage_packed_params* p, const sage_packed_info* info) {
  return walk_splits(longest_tiles(info) * (p->Hq / p->Hkv), all_steps(p, info),
                     148 * (p->d == 64 ? 2 : 1));
}

// Forward workspace, with parts: O [splits][tokens][Hq][d], then maxima and sums.
struct FwdWs {
  int splits;
  size_t stats, total;
};
FwdWs fwd_ws(const sage_packed_params* p, const sage_packed_info* info) {
  FwdWs w = {fwd_splits(p, info), 0, 0};
  if (w.splits > 1) {
    const size_t rows = static_cast<size_t>(w.splits) * info->tokens * p->Hq;
    w.stats = align_up(rows * p->d * 4);
    w.total = align_up(w.stats + rows * 8);
  }
  return w;
}

template <typename T, int D>
int run_packed_fwd(const sage_packed_params* p, const sage_packed_info* info, const void* plan,
                   const sage_rows* q, const sage_rows* k, const sage_rows* v, const sage_rows* o,
                   float* lse, void* ws, cudaStream_t st) {
  namespace F = sage::packed::fwd;
  CUtensorMap tq, tk, tv;
  if (!make_tile_map(&tq, q, p, p->Hq) || !make_tile_map(&tk, k, p, p->Hkv) ||
      !make_tile_map(&tv, v, p, p->Hkv))
    return SAGE_ERR_CUDA;
  F::Args a;
  a.group = p->Hq / p->Hkv;
  a.o = packed_out(o);
  a.lse = lse;
  a.T = p->T;
  a.causal = p->causal;
  a.scale_log2 = packed_tau(p) * 1.4426950408889634f;
  const FwdWs w = fwd_ws(p, info);
  a.splits = w.splits;
  a.heads = p->Hq;
  a.part = static_cast<float*>(ws);
  a.stats = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + w.stats);
  a.tokens = info->tokens;
  const int64_t kv_bytes = info->tokens * D * 2 * 2;
  int s;
  if constexpr (D == 64) {
    const int ctas = p->Hq * w.splits;  // per item
    a.grid = {plan_list(plan, info, p->causal, false), info->tiles, ctas,
              grid_chunk(p, info, ctas, kv_bytes / a.group / w.splits)};
    const int64_t grid = static_cast<int64_t>(info->tiles) * ctas;
    const size_t smem = F::smem64_bytes<T>();
    s = w.splits > 1 ? launch_packed<F::attn_fwd64_kernel<T, true>, 0>(grid, F::kThreads64, smem, st,
                                                                       tq, tk, tv, a)
                     : launch_packed<F::attn_fwd64_kernel<T, false>, 0>(grid, F::kThreads64, smem,
                                                                        st, tq, tk, tv, a);
  } else {
    const bool heads = a.group % 2 == 0;
    const int ctas = (heads ? p->Hq / 2 : p->Hq) * w.splits;  // per item
    a.grid = {plan_list(plan, info, p->causal, !heads), heads ? info->tiles : info->pairs, ctas,
              grid_chunk(p, info, ctas, kv_bytes / (heads ? a.group / 2 : a.group) / w.splits)};
    const int64_t grid = static_cast<int64_t>(a.grid.n_items) * ctas;
    const size_t smem = F::smem_bytes<T, D>();
    auto launch = [&](auto by_heads, auto parts) {
      return launch_packed<
          F::attn_fwd_kernel<T, D, decltype(by_heads)::value, decltype(parts)::value>,
          F::kLaunchRegs>(grid, F::kThreads, smem, st, tq, tk, tv, a);
    };
    using Yes = std::true_type;
    using No = std::false_type;
    s = heads ? (w.splits > 1 ? launch(Yes{}, Yes{}) : launch(Yes{}, No{}))
              : (w.splits > 1 ? launch(No{}, Yes{}) : launch(No{}, No{}));
  }
  if (s != SAGE_OK || w.splits == 1) return s;
  const int64_t vectors = info->tokens * p->Hq * (D / 8);
  F::merge_kernel<T, D><<<static_cast<unsigned>((vectors + 255) / 256), 256, 0, st>>>(a);
  return launch_status();
}

// Workspace: D [Hq][T]; in half precision the norms [sequences][Hkv][2]; the parts of dQ, then (in
// their place) those of dV and dK.
struct PackedWs {
  int dq_splits, dkv_splits;
  size_t norms, norms_bytes, part, total;
};
PackedWs packed_ws(const sage_packed_params* p, const sage_packed_info* info) {
  PackedWs w;
  w.norms = align_up(static_cast<size_t>(p->Hq) * p->T * 4);
  w.norms_bytes =
      p->dtype == SAGE_FP16 ? static_cast<size_t>(info->sequences) * p->Hkv * 2 * 4 : 0;
  w.part = align_up(w.norms + w.norms_bytes);
  w.dq_splits = dq_splits(p, info);
  w.dkv_splits = dkv_splits(p, info);
  const size_t row = static_cast<size_t>(info->tokens) * p->d * 4;
  w.total = align_up(
      w.part + row * std::max(w.dq_splits > 1 ? static_cast<size_t>(w.dq_splits) * p->Hq : 0,
                              w.dkv_splits > 1 ? static_cast<size_t>(w.dkv_splits) * 2 * p->Hkv
                                               : 0));
  return w;
}

template <typename T, int D>
int run_packed_bwd(const sage_packed_params* p, const sage_packed_info* info, const void* plan,
                   const sage_rows* q, const sage_rows* k, const sage_rows* v, const sage_rows* o,
                   const float* lse, const sage_rows* dout, const sage_rows* dq,
                   const sage_rows* dk, const sage_rows* dv, void* ws, cudaStream_t st) {
  namespace B = sage::packed::bwd;
  constexpr bool kNorms = B::Scaling<T>::kOn;
  CUtensorMap tq, tk, tv, tdo;
  if (!make_tile_map(&tq, q, p, p->Hq) || !make_tile_map(&tk, k, p, p->Hkv) ||
      !make_tile_map(&tv, v, p, p->Hkv) || !make_tile_map(&tdo, dout, p, p->Hq))
    return SAGE_ERR_CUDA;
  const PackedWs w = packed_ws(p, info);
  B::RowArgs r;
  r.o = packed_out(o);
  r.dout = packed_out(dout);
  r.v = packed_out(v);
  r.items = plan_list(plan, info, p->causal, false);
  r.dvec = static_cast<float*>(ws);
  r.norms = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(ws) + w.norms);
  r.T = p->T;
  r.tiles = info->tiles;
  r.Hq = p->Hq;
  r.Hkv = p->Hkv;
  r.group = p->Hq / p->Hkv;
  if (kNorms && cudaMemsetAsync(r.norms, 0, w.norms_bytes, st) != cudaSuccess)
    return SAGE_ERR_CUDA;
  const int64_t row_ctas =
      static_cast<int64_t>(info->tiles) * (p->Hq + (kNorms ? p->Hkv : 0));
  B::row_kernel<T, D, kNorms>
      <<<static_cast<unsigned>(row_ctas), B::kRowKernelThreads, 0, st>>>(r);
  int s = launch_status();
  if (s != SAGE_OK) return s;
  B::Args a;
  a.lse = lse;
  a.dvec = r.dvec;
  a.norms = r.norms;
  a.T = p->T;
  a.group = r.group;
  a.kv_heads = p->Hkv;
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + w.part);
  a.tokens = info->tokens;
  a.causal = p->causal;
  a.tau = packed_tau(p);
  a.scale_log2 = a.tau * 1.4426950408889634f;
  const int64_t pair_bytes = info->tokens * D * 2 * 2;  // two tensors of one head
  auto join = [&](int heads, int count) {
    B::JoinArgs j = {a.part, {a.out[0], a.out[1]}, info->tokens, heads, a.splits, count};
    const int64_t vectors = count * info->tokens * heads * (D / 8);
    B::join_kernel<T, D><<<static_cast<unsigned>((vectors + 255) / 256), 256, 0, st>>>(j);
    return launch_status();
  };
  // dq_kernel first: it refines D for dkv_kernel
  a.splits = w.dq_splits;
  int heads = p->Hq * a.splits;
  a.grid = {r.items, info->tiles, heads,
            grid_chunk(p, info, heads, pair_bytes / r.group / a.splits)};
  a.out[0] = a.out[1] = packed_out(dq);
  s = a.splits > 1
          ? launch_packed<B::dq_kernel<T, D, true>, B::Cfg<D>::kLaunchRegs>(
                static_cast<int64_t>(info->tiles) * heads, B::Cfg<D>::kThreads,
                B::dq_smem_bytes<T, D>(), st, tq, tk, tv, tdo, a)
          : launch_packed<B::dq_kernel<T, D, false>, B::Cfg<D>::kLaunchRegs>(
                static_cast<int64_t>(info->tiles) * heads, B::Cfg<D>::kThreads,
                B::dq_smem_bytes<T, D>(), st, tq, tk, tv, tdo, a);
  if (s == SAGE_OK && a.splits > 1) s = join(p->Hq, 1);
  if (s != SAGE_OK) return s;
  a.splits = w.dkv_splits;
  heads = p->Hkv * a.splits;
  a.grid = {r.items, info->tiles, heads,
            grid_chunk(p, info, heads, pair_bytes * r.group / a.splits)};
  a.out[0] = packed_out(dv);
  a.out[1] = packed_out(dk);
  s = a.splits > 1
          ? launch_packed<B::dkv_kernel<T, D, true>, B::Cfg<D>::kLaunchRegs>(
                static_cast<int64_t>(info->tiles) * heads, B::Cfg<D>::kThreads,
                B::dkv_smem_bytes<T, D>(), st, tq, tk, tv, tdo, a)
          : launch_packed<B::dkv_kernel<T, D, false>, B::Cfg<D>::kLaunchRegs>(
                static_cast<int64_t>(info->tiles) * heads, B::Cfg<D>::kThreads,
                B::dkv_smem_bytes<T, D>(), st, tq, tk, tv, tdo, a);
  if (s == SAGE_OK && a.splits > 1) s = join(p->Hkv, 2);
  return s;
}

}  // namespace

extern "C" {

int sage_qk_norm_rope_fwd(const sage_rope_params* p, const sage_rows* q, const sage_rows* k,
                          const float* gain_q, const float* gain_k, const void* pos,
                          const sage_rows* q_out, const sage_rows* k_out, void* stream) {
  int s = check_rope(p);
  if (s != SAGE_OK) return s;
  const sage_rows* rows[4] = {q, k, q_out, k_out};
  for (int i = 0; i < 4; ++i)
    if ((s = check_rows(rows[i], p->B, p->N, i % 2 ? p->Hkv : p->Hq, p->d, i >= 2)) != SAGE_OK)
      return s;
  if (p->rotary_dim > 0 && !pos) return SAGE_ERR_INVALID_ARG;
  if (!p->norm && (gain_q || gain_k)) return SAGE_ERR_INVALID_ARG;
  if (!aligned16(gain_q) || !aligned16(gain_k)) return SAGE_ERR_ALIGNMENT;
  sage::rope::Args a;
  rope_args(p, q, k, q_out, k_out, gain_q, gain_k, pos, &a);
  return launch_rope<false>(p, &a, nullptr, nullptr, reinterpret_cast<cudaStream_t>(stream));
}

size_t sage_qk_norm_rope_workspace_bytes(const sage_rope_params* p) {
  if (check_rope(p) != SAGE_OK) return 0;
  return align_up(static_cast<size_t>(kRopeBwdBlocks) * p->d * 4);
}

int sage_qk_norm_rope_bwd(const sage_rope_params* p, const sage_rows* q, const sage_rows* k,
                          const float* gain_q, const float* gain_k, const void* pos,
                          const sage_rows* dq_out, const sage_rows* dk_out, const sage_rows* dq,
                          const sage_rows* dk, float* dgain_q, float* dgain_k, void* workspace,
                          size_t workspace_bytes, void* stream) {
  int s = check_rope(p);
  if (s != SAGE_OK) return s;
  const sage_rows* rows[6] = {q, k, dq_out, dk_out, dq, dk};
  for (int i = 0; i < 6; ++i)
    if ((s = check_rows(rows[i], p->B, p->N, i % 2 ? p->Hkv : p->Hq, p->d, i >= 4)) != SAGE_OK)
      return s;
  if (p->rotary_dim > 0 && !pos) return SAGE_ERR_INVALID_ARG;
  if (!p->norm && (gain_q || gain_k || dgain_q || dgain_k)) return SAGE_ERR_INVALID_ARG;
  if ((dgain_q == nullptr) != (dgain_k == nullptr)) return SAGE_ERR_INVALID_ARG;
  if (!aligned16(gain_q) || !aligned16(gain_k)) return SAGE_ERR_ALIGNMENT;
  if (dgain_q) {
    if (!workspace || workspace_bytes < sage_qk_norm_rope_workspace_bytes(p))
      return SAGE_ERR_WORKSPACE;
    if (!aligned16(workspace)) return SAGE_ERR_ALIGNMENT;
  }
  sage::rope::Args a;
  rope_args(p, q, k, dq, dk, gain_q, gain_k, pos, &a);
  a.g[0] = rope_rows(dq_out);
  a.g[1] = rope_rows(dk_out);
  a.partial = dgain_q ? static_cast<float*>(workspace) : nullptr;
  return launch_rope<true>(p, &a, dgain_q, dgain_k, reinterpret_cast<cudaStream_t>(stream));
}

size_t sage_packed_plan_bytes(const int* lengths, int sequences) {
  sage_packed_info info;
  return plan_counts(lengths, sequences, &info) ? plan_bytes(info) : 0;
}

int sage_packed_plan_fill(const int* lengths, int sequences, void* host_plan, size_t bytes,
                          sage_packed_info* info) {
  sage_packed_info in;
  if (!host_plan || !info || !plan_counts(lengths, sequences, &in)) return SAGE_ERR_INVALID_ARG;
  if (bytes < plan_bytes(in)) return SAGE_ERR_WORKSPACE;
  try {
    // counting sort by descending work, sequences in order within one amount of work
    const int most = (in.longest + sage::packed::BT - 1) / sage::packed::BT;
    Item* out = static_cast<Item*>(host_plan);
    std::memset(out, 0, plan_bytes(in));
    for (int list = 0; list < 4; ++list) {
      const bool pairs = list >= 2, causal = list % 2 == 0;
      const int count = pairs ? in.pairs : in.tiles;
      std::vector<int> at(static_cast<size_t>(most) + 2, 0);  // at[most - work]: next place
      for (int pass = 0; pass < 2; ++pass) {
        for (int i = 0, start = 0; i < sequences; start += lengths[i], ++i) {
          const int tiles = static_cast<int>(
              (static_cast<int64_t>(lengths[i]) + sage::packed::BT - 1) / sage::packed::BT);
          for (int t = tiles - 1; t >= 0; t -= pairs ? 2 : 1) {
            const int slot = most - (causal ? t + 1 : tiles);
            if (pass == 0)
              ++at[slot + 1];
            else
              out[at[slot]++] = Item{start, lengths[i], t, i};
          }
        }
        if (pass == 0)
          for (int w = 0; w <= most; ++w) at[w + 1] += at[w];
      }
      out += count;
    }
  } catch (const std::bad_alloc&) {
    return SAGE_ERR_WORKSPACE;
  }
  *info = in;
  return SAGE_OK;
}

size_t sage_packed_attn_fwd_workspace_bytes(const sage_packed_params* p,
                                            const sage_packed_info* info) {
  alignas(16) static const char some[16] = {};
  if (check_packed(p, info, some) != SAGE_OK) return 0;
  return fwd_ws(p, info).total;
}

int sage_packed_attn_fwd(const sage_packed_params* p, const sage_packed_info* info,
                         const void* plan, const sage_rows* q, const sage_rows* k,
                         const sage_rows* v, const sage_rows* o, float* lse, void* workspace,
                         size_t workspace_bytes, void* stream) {
  int s = check_packed(p, info, plan);
  if (s != SAGE_OK) return s;
  const sage_rows* rows[4] = {q, k, v, o};
  for (int i = 0; i < 4; ++i)
    if ((s = check_rows(rows[i], 1, p->T, i == 1 || i == 2 ? p->Hkv : p->Hq, p->d, i == 3)) !=
        SAGE_OK)
      return s;
  if (!lse) return SAGE_ERR_INVALID_ARG;
  if (info->tiles == 0) return SAGE_OK;  // only empty sequences: nothing to write
  const size_t need = fwd_ws(p, info).total;
  if (need > 0 && (!workspace || workspace_bytes < need)) return SAGE_ERR_WORKSPACE;
  if (!aligned16(workspace)) return SAGE_ERR_ALIGNMENT;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool bf = p->dtype == SAGE_BF16;
  if (p->d == 128)
    return bf ? run_packed_fwd<__nv_bfloat16, 128>(p, info, plan, q, k, v, o, lse, workspace, st)
              : run_packed_fwd<__half, 128>(p, info, plan, q, k, v, o, lse, workspace, st);
  return bf ? run_packed_fwd<__nv_bfloat16, 64>(p, info, plan, q, k, v, o, lse, workspace, st)
            : run_packed_fwd<__half, 64>(p, info, plan, q, k, v, o, lse, workspace, st);
}

size_t sage_packed_attn_bwd_workspace_bytes(const sage_packed_params* p,
                                            const sage_packed_info* info) {
  alignas(16) static const char some[16] = {};
  if (check_packed(p, info, some) != SAGE_OK) return 0;
  return packed_ws(p, info).total;
}

int sage_packed_attn_bwd(const sage_packed_params* p, const sage_packed_info* info,
                         const void* plan, const sage_rows* q, const sage_rows* k,
                         const sage_rows* v, const sage_rows* o, const float* lse,
                         const sage_rows* dout, const sage_rows* dq, const sage_rows* dk,
                         const sage_rows* dv, void* workspace, size_t workspace_bytes,
                         void* stream) {
  int s = check_packed(p, info, plan);
  if (s != SAGE_OK) return s;
  const sage_rows* rows[8] = {q, o, dout, dq, k, v, dk, dv};
  for (int i = 0; i < 8; ++i)
    if ((s = check_rows(rows[i], 1, p->T, i >= 4 ? p->Hkv : p->Hq, p->d,
                        i == 3 || i >= 6)) != SAGE_OK)
      return s;
  if (!lse) return SAGE_ERR_INVALID_ARG;
  if (info->tiles == 0) return SAGE_OK;
  if (!workspace || workspace_bytes < packed_ws(p, info).total) return SAGE_ERR_WORKSPACE;
  if (!aligned16(workspace)) return SAGE_ERR_ALIGNMENT;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool bf = p->dtype == SAGE_BF16;
  if (p->d == 128)
    return bf ? run_packed_bwd<__nv_bfloat16, 128>(p, info, plan, q, k, v, o, lse, dout, dq, dk,
                                                   dv, workspace, st)
              : run_packed_bwd<__half, 128>(p, info, plan, q, k, v, o, lse, dout, dq, dk, dv,
                                            workspace, st);
  return bf ? run_packed_bwd<__nv_bfloat16, 64>(p, info, plan, q, k, v, o, lse, dout, dq, dk, dv,
                                                workspace, st)
            : run_packed_bwd<__half, 64>(p, info, plan, q, k, v, o, lse, dout, dq, dk, dv,
                                         workspace, st);
}

}  // extern "C"
