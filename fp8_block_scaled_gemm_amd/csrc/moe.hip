// Expert routing and the expert row layout for gfx950: from the router's logits to the rows that the
// grouped GEMMs read (contiguous and masked forms) and back to the tokens, with the gradients.
//
//   route       logits (T, E) -> the K experts of each token and their weights
//   layout      experts of the tokens -> a row for each (token, place), m_indices, counts
//   dispatch    token rows -> expert rows, copied or quantized (FP8 per 128 columns, int8 per row)
//   combine     expert rows -> weighted sum per token
//
// Every result is deterministic: ranks follow the order of (token, place), sums a fixed order.
#include "rows.hpp"

namespace dg {

// ---------------------------------------------------------------------------
// Routing.
// ---------------------------------------------------------------------------
constexpr int kRouteWaves = 4;          // tokens per workgroup, one wave each
constexpr int kRouteMaxExperts = 1024;  // 16 per lane
constexpr int kRouteMaxTopK = 64;       // one lane per chosen expert

struct RouteParams {
  const void* logits;
  int64_t ld;
  const float* bias;
  int tokens, experts, top_k;
  int groups, group_size, topk_groups, group_top;
  uint32_t group_magic;   // ceil(2^20 / group_size): e * magic >> 20 = e / group_size for e < 1024
  int lanes_per_group;    // 64 / (groups rounded up to a power of two)
  int renorm;
  float scale;
  int32_t* ids;
  float* weights;
};

// LDS written by some lanes of a wave and read by others: nothing moves across (no instruction).
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Unsigned key of a choice value that orders like the value (-0 as +0); 0 stands for "not available".
__device__ __forceinline__ uint32_t choice_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// One wave per token; lane l holds experts l, l + 64, ... (coalesced reads).  What bounds it is the vector
// unit: ~690 instructions a token for 256 experts, 8 groups and 8 choices, against 1 KB read (16384 tokens:
// 18.6 us; plain softmax 11.0; one token 4.2, a launch and two memory latencies).  So each lane
// sorts its C experts once by (choice, lower index first), and a round of the top-k takes the maximum of
// the lanes' heads, and pops one lane.
template <class T, int C, bool SOFTMAX>
__global__ __launch_bounds__(64 * kRouteWaves) void route_kernel(RouteParams p) {
  constexpr float kOff = -__builtin_inff();
  __shared__ float s_value[kRouteWaves][64 * C];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t token = (int64_t)blockIdx.x * kRouteWaves + wave;
  if (token >= p.tokens) return;   // wave-uniform; no workgroup barrier below
  const T* row = static_cast<const T*>(p.logits) + token * p.ld;

  // every lane loads (an absent expert from the last one), so the loads are in flight together
  float x[C], bias[C];
#pragma unroll
  for (int c = 0; c < C; ++c) x[c] = widen(row[64 * c + lane < p.experts ? 64 * c + lane : p.experts - 1]);
#pragma unroll
  for (int c = 0; c < C; ++c) bias[c] = 0.0f;
  if (p.bias != nullptr) {
#pragma unroll
    for (int c = 0; c < C; ++c) bias[c] = p.bias[64 * c + lane < p.experts ? 64 * c + lane : p.experts - 1];
  }
  // a NaN logit: not chosen, and every weight of the token is NaN
  bool nan = false;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (64 * c + lane >= p.experts) x[c] = kOff;
    nan |= x[c] != x[c];
    x[c] = x[c] != x[c] ? kOff : x[c];
  }
  // the softmax's maximum and sum, where a probability itself is needed
  const bool by_logit = SOFTMAX && p.bias == nullptr && !(p.groups > 1 && p.group_top > 1);
  float top = kOff, total = 1.0f;
  if (SOFTMAX && (!by_logit || !p.renorm)) {
#pragma unroll
    for (int c = 0; c < C; ++c) top = fmaxf(top, x[c]);
    top = wave_max(top);
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) sum += x[c] == kOff ? 0.0f : expf(x[c] - top);
    total = wave_sum(sum);
  }
  float value[C];
  if (by_logit) {
#pragma unroll
    for (int c = 0; c < C; ++c) value[c] = x[c];
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float v = (SOFTMAX ? expf(x[c] - top) / total : sigmoid(x[c])) + bias[c];
      const bool off = x[c] == kOff;
      nan |= !off && v != v;
      value[c] = off || v != v ? kOff : v;
    }
  }

  if (p.groups > 1) {
    // lanes_per_group lanes find the two best values of each group, then every group counts the
    // groups ahead of it (higher value, or equal and lower index)
    float* s_val = s_value[wave];
#pragma unroll
    for (int c = 0; c < C; ++c) s_val[64 * c + lane] = value[c];
    wave_lds_fence();
    const int lpg = p.lanes_per_group;
    const int mine = lane / lpg, sub = lane - mine * lpg;
    float t1 = kOff, t2 = kOff;
    if (mine < p.groups) {
      for (int i = sub; i < p.group_size; i += lpg) {
        const float v = s_val[mine * p.group_size + i];
        t2 = __builtin_amdgcn_fmed3f(t1, t2, v);   // t2 <= t1: the second best of the three
        t1 = fmaxf(t1, v);
      }
    }
    for (int sh = 1; sh < lpg; sh *= 2) {
      const float o1 = __shfl_xor(t1, sh), o2 = __shfl_xor(t2, sh);
      t2 = fmaxf(fminf(t1, o1), fmaxf(t2, o2));
      t1 = fmaxf(t1, o1);
    }
    const float sum = p.group_top > 1 && t2 != kOff ? t1 + t2 : t1;
    const uint32_t key = t1 == kOff || mine >= p.groups ? 0u : choice_key(sum);
    // lane (group, sub) compares its group with groups sub, sub + lpg, ...; the group's lanes' votes add up
    int ahead = 0;
    const uint64_t own = ((lpg < 64 ? 1ull << lpg : 0ull) - 1) << (mine * lpg);
    for (int g0 = 0; g0 < p.groups; g0 += lpg) {
      const int g = g0 + sub;
      const uint32_t other = __shfl(key, (g * lpg) & 63);
      ahead += __popcll(__ballot(g < p.groups && (other > key || (other == key && g < mine))) & own);
    }
    const uint64_t kept = __ballot(ahead < p.topk_groups);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t g = ((uint32_t)(64 * c + lane) * p.group_magic) >> 20;
      if (!((kept >> ((g * lpg) & 63)) & 1)) value[c] = kOff;
    }
  }

  // (key, ~expert) pairs, the lane's best first: a sorting network of neighbour exchanges
  uint32_t key[C], inv[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    key[c] = value[c] == kOff ? 0u : choice_key(value[c]);
    inv[c] = ~(uint32_t)(64 * c + lane);
  }
#pragma unroll
  for (int i = 1; i < C; ++i) {
#pragma unroll
    for (int j = i; j > 0; --j) {
      // (of equal keys the earlier one has the lower index already: insertion keeps their order)
      // (copies: a conditional of array elements would select the element's address)
      const uint32_t ka = key[j - 1], kb = key[j], ia = inv[j - 1], ib = inv[j];
      const bool swap = kb > ka;
      key[j - 1] = swap ? kb : ka;
      key[j] = swap ? ka : kb;
      inv[j - 1] = swap ? ib : ia;
      inv[j] = swap ? ia : ib;
    }
  }

  // top_k rounds over the lanes' heads; lane j keeps the j-th choice
  int id = -1;
  for (int j = 0; j < p.top_k; ++j) {
    const uint32_t best = wave_max_u32(key[0]);
    if (best == 0u) break;   // wave-uniform: no available expert is left
    uint64_t has = __ballot(key[0] == best);
    if (has & (has - 1)) {   // wave-uniform: a tie goes to the lowest index
      const uint32_t low = wave_max_u32(key[0] == best ? inv[0] : 0u);
      has = __ballot(key[0] == best && inv[0] == low);
    }
    const int owner = __builtin_ctzll(has);
    const int pick = ~__builtin_amdgcn_readlane((int)inv[0], owner);
    const bool pop = lane == owner;
#pragma unroll
    for (int c = 0; c + 1 < C; ++c) {
      const uint32_t ka = key[c], kb = key[c + 1], ia = inv[c], ib = inv[c + 1];
      key[c] = pop ? kb : ka;
      inv[c] = pop ? ib : ia;
    }
    const uint32_t last = key[C - 1];
    key[C - 1] = pop ? 0u : last;
    id = lane == j ? pick : id;
  }

  const float xk = id >= 0 ? widen(row[id]) : kOff;
  float s;
  if (!SOFTMAX) {
    s = id >= 0 ? sigmoid(xk) : 0.0f;
  } else if (p.renorm) {
    // over the chosen alone: relative to their own maximum, so that their sum does not underflow
    const float m = wave_max(xk);
    s = id >= 0 ? expf(xk - m) : 0.0f;
  } else {
    s = id >= 0 ? expf(xk - top) / total : 0.0f;
  }
  float w = s;
  if (p.renorm) {
    const float sum = wave_sum(s);
    w = sum == 0.0f ? 0.0f : s / sum;
  }
  w *= p.scale;
  if (__ballot(nan) != 0) w = id >= 0 ? __builtin_nanf("") : 0.0f;
  if (lane < p.top_k) {
    p.ids[token * p.top_k + lane] = id;
    p.weights[token * p.top_k + lane] = w;
  }
}

struct RouteGradParams {
  const float* dweights;
  const void* logits;
  int64_t ld;
  const int32_t* ids;
  int tokens, experts, top_k;
  int softmax, renorm;
  float scale;
  void* dlogits;
  int64_t ld_out;
};

// One wave per token.  The experts' choice is held fixed; only the softmax without renormalisation
// needs the whole row of logits, every other form the K chosen ones:
//   s = sigmoid(x) or exp(x - max), r = s / sum s, w = scale r:  dx = scale r (g - sum r g) [(1 - s) for sigmoid]
//   w = scale s:  dx = scale g s (1 - s) for sigmoid; for softmax over the row, dx_e = p_e (u_e - sum p u), u = scale g.
// Every element of the row is written (zeros where nothing was chosen), which bounds it: 16384 x 256 fp32
// 9.5 us, 1.8 TB/s in these sizes' few microseconds; the full softmax 12.4.
template <class T, int C>
__global__ __launch_bounds__(64 * kRouteWaves) void route_grad_kernel(RouteGradParams p) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t token = (int64_t)blockIdx.x * kRouteWaves + wave;
  if (token >= p.tokens) return;
  const T* row = static_cast<const T*>(p.logits) + token * p.ld;
  T* out = static_cast<T*>(p.dlogits) + token * p.ld_out;

  int id = lane < p.top_k ? p.ids[token * p.top_k + lane] : -1;
  if (id >= p.experts) id = -1;
  const float g = id >= 0 ? p.dweights[token * p.top_k + lane] : 0.0f;
  const float xk = id >= 0 ? widen(row[id]) : -__builtin_inff();

  float d = 0.0f;   // dL/dx of this lane's chosen expert
  float x[C], top = -__builtin_inff(), total = 1.0f, dot = 0.0f;
  const bool full = p.softmax && !p.renorm;
  if (full) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int e = 64 * c + lane;
      x[c] = e < p.experts ? widen(row[e]) : -__builtin_inff();
      top = fmaxf(top, x[c]);
    }
    top = wave_max(top);
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      x[c] = x[c] == -__builtin_inff() ? 0.0f : expf(x[c] - top);
      sum += x[c];
    }
    total = wave_sum(sum);
    if (total == 0.0f) total = 1.0f;   // a row without an available expert
    const float pk = id >= 0 ? expf(xk - top) / total : 0.0f;
    const float u = p.scale * g;
    dot = wave_sum(pk * u);
    d = pk * (u - dot);
  } else {
    const float m = p.softmax ? wave_max(xk) : 0.0f;
    const float s = id < 0 ? 0.0f : p.softmax ? expf(xk - m) : sigmoid(xk);
    if (p.renorm) {
      const float sum = wave_sum(s);
      const float r = sum == 0.0f ? 0.0f : s / sum;
      const float u = p.scale * r * (g - wave_sum(r * g));   // scale r (g - sum r g) = s dL/ds
      d = p.softmax ? u : u * (1.0f - s);
    } else {
      d = p.scale * g * s * (1.0f - s);
    }
  }
  float v[C];
#pragma unroll
  for (int c = 0; c < C; ++c) v[c] = full ? -(x[c] / total) * dot : 0.0f;
  for (int j = 0; j < p.top_k; ++j) {
    const int e = __builtin_amdgcn_readlane(id, j);
    const float de = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(d), j));
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (e == 64 * c + lane) v[c] = de;
  }
#pragma unroll
  for (int c = 0; c < C; ++c)
    if (64 * c + lane < p.experts) out[64 * c + lane] = narrow<T>(v[c]);
}


template <class T, bool SOFTMAX>
static const void* route_fn(int experts) {
  void (*fn)(RouteParams) = experts <= 64    ? route_kernel<T, 1, SOFTMAX>
                            : experts <= 128 ? route_kernel<T, 2, SOFTMAX>
                            : experts <= 256 ? route_kernel<T, 4, SOFTMAX>
                            : experts <= 512 ? route_kernel<T, 8, SOFTMAX>
                                             : route_kernel<T, 16, SOFTMAX>;
  return reinterpret_cast<const void*>(fn);
}
template <class T>
static const void* route_fn(int experts, bool softmax) {
  return softmax ? route_fn<T, true>(experts) : route_fn<T, false>(experts);
}
template <class T>
static const void* route_grad_fn(int experts) {
  void (*fn)(RouteGradParams) = experts <= 64    ? route_grad_kernel<T, 1>
                                : experts <= 128 ? route_grad_kernel<T, 2>
                                : experts <= 256 ? route_grad_kernel<T, 4>
                                : experts <= 512 ? route_grad_kernel<T, 8>
                                                 : route_grad_kernel<T, 16>;
  return reinterpret_cast<const void*>(fn);
}

static int launched(const void* fn, dim3 grid, dim3 block, void** args, hipStream_t stream, const char* what) {
  if ((uint64_t)grid.x * block.x > 0xffffffffull || grid.y > 65535u)
    return set_error(kUnsupported, "%s: shape too large for the launch grid", what);
  const hipError_t e = hipLaunchKernel(fn, grid, block, args, 0, stream);
  return e == hipSuccess ? kOk : set_error(kHip, "%s launch: %s", what, hipGetErrorString(e));
}

int launch_route(const void* logits, int dtype, int64_t ld, const float* bias, int64_t tokens, int experts, int top_k,
                 int groups, int topk_groups, int group_top, bool softmax, bool renorm, float scale, int32_t* ids,
                 float* weights, hipStream_t stream) {
  RouteParams p{};
  p.logits = logits; p.ld = ld; p.bias = bias;
  p.tokens = (int)tokens; p.experts = experts; p.top_k = top_k;
  p.groups = groups; p.group_size = experts / groups; p.topk_groups = topk_groups; p.group_top = group_top;
  p.group_magic = ((1u << 20) + (uint32_t)p.group_size - 1) / (uint32_t)p.group_size;
  int pow2 = 1;
  while (pow2 < groups) pow2 *= 2;
  p.lanes_per_group = 64 / pow2;
  p.renorm = renorm; p.scale = scale;
  p.ids = ids; p.weights = weights;
  const void* fn = dtype == kF32 ? route_fn<float>(experts, softmax) : dtype == kBf16 ? route_fn<Bf16>(experts, softmax)
                                                                                     : route_fn<_Float16>(experts, softmax);
  void* args[] = {&p};
  return launched(fn, dim3((unsigned)((tokens + kRouteWaves - 1) / kRouteWaves)), dim3(64 * kRouteWaves), args, stream,
                  "moe_route");
}

int launch_route_grad(const float* dweights, const void* logits, int dtype, int64_t ld, const int32_t* ids,
                      int64_t tokens, int experts, int top_k, bool softmax, bool renorm, float scale, void* dlogits,
                      int64_t ld_out, hipStream_t stream) {
  RouteGradParams p{};
  p.dweights = dweights; p.logits = logits; p.ld = ld; p.ids = ids;
  p.tokens = (int)tokens; p.experts = experts; p.top_k = top_k;
  p.softmax = softmax; p.renorm = renorm; p.scale = scale;
  p.dlogits = dlogits; p.ld_out = ld_out;
  const void* fn = dtype == kF32 ? route_grad_fn<float>(experts) : dtype == kBf16 ? route_grad_fn<Bf16>(experts)
                                                                                 : route_grad_fn<_Float16>(experts);
  void* args[] = {&p};
  return launched(fn, dim3((unsigned)((tokens + kRouteWaves - 1) / kRouteWaves)), dim3(64 * kRouteWaves), args, stream,
                  "moe_route_grad");
}

// ---------------------------------------------------------------------------
// Layout: a stable counting sort of the (token, place) entries by expert.
//
// Nothing here is more than a few KB; what counts is the latency of the steps.  A wave takes 64 entries at
// a time: one ballot per bit of the expert index tells every lane which lanes have its expert, so the
// expert's first lane adds their number to the wave's own counter in LDS without an atomic, and a lane's
// rank is the counter's old value plus the earlier lanes of its expert - in the entries' order.
// Up to kLayOnce entries are counted by every workgroup for itself, in one launch; more are counted by a
// launch of their own, a chunk a workgroup, whose histograms every workgroup of the second then adds up
// (2048 entries into 256 experts: 8.8 us in one launch, 9.5 in two; 4096: 13.8 and 9.4).
// ---------------------------------------------------------------------------
constexpr int kLayThreads = 512;
constexpr int kLayWaves = kLayThreads / 64;
constexpr int kLayOnce = 2048;
constexpr int kLayChunk = 1024;      // least entries per workgroup where there is more than one
constexpr int kLayMostChunks = 256;  // every workgroup reads all their histograms

struct LayoutParams {
  const int32_t* ids;
  int n;                 // entries: tokens * top_k
  int experts;
  int rows_per_expert;   // 0: the contiguous layout
  int align;             // row alignment of the contiguous layout
  int rows_total;
  int chunk, blocks;     // entries per chunk, chunks
  int32_t* rows;
  int32_t* sources;
  int32_t* m_indices;
  int32_t* counts;
  int32_t* hist;         // (chunks, experts), with more than one chunk
};

// Entries [begin, end) in order, split over the waves; f(entry, expert or -1, rank of the entry among the
// wave's earlier entries of its expert + the counter's start).  s_next: the wave's own (experts) counters.
template <class F>
__device__ __forceinline__ void for_entries(const LayoutParams& p, int begin, int end, int* s_next, F f) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int per_wave = ((end - begin + kLayWaves - 1) / kLayWaves + 63) & ~63;
  // (differences, not sums: an index near 2^31 must not wrap)
  const int w0 = end - begin > wave * per_wave ? begin + wave * per_wave : end;
  const int w1 = end - w0 > per_wave ? w0 + per_wave : end;
  for (int i0 = w0; i0 < w1; i0 = w1 - i0 > 64 ? i0 + 64 : w1) {
    const int i = i0 + lane;
    int e = w1 - i0 > lane ? p.ids[i] : -1;
    if ((uint32_t)e >= (uint32_t)p.experts) e = -1;
    uint64_t same = __ballot(e >= 0);
    for (int bit = 1; bit < p.experts; bit *= 2) {
      const uint64_t set = __ballot((e & bit) != 0);   // (a lane without an expert is masked out of `same`)
      same &= (e & bit) ? set : ~set;
    }
    const int earlier = __popcll(same & ((1ull << lane) - 1));
    const int next = s_next[e >= 0 ? e : 0];
    wave_lds_fence();
    if (e >= 0 && earlier == 0) s_next[e] = next + __popcll(same);
    wave_lds_fence();
    if (w1 - i0 > lane) f(i, e, next + earlier);
  }
}

// s_hist[wave][expert]: the entries [begin, end) of each wave, by expert.
__device__ __forceinline__ void count_entries(const LayoutParams& p, int begin, int end, int* s_hist) {
  for (int i = threadIdx.x; i < kLayWaves * p.experts; i += kLayThreads) s_hist[i] = 0;
  __syncthreads();
  for_entries(p, begin, end, s_hist + (threadIdx.x >> 6) * p.experts, [](int, int, int) {});
  __syncthreads();
}

__global__ __launch_bounds__(kLayThreads) void layout_count_kernel(LayoutParams p) {
  extern __shared__ int s_hist[];
  const int begin = blockIdx.x * p.chunk;
  count_entries(p, begin, p.n - begin < p.chunk ? p.n : begin + p.chunk, s_hist);
  for (int e = threadIdx.x; e < p.experts; e += kLayThreads) {
    int sum = 0;
    for (int w = 0; w < kLayWaves; ++w) sum += s_hist[w * p.experts + e];
    p.hist[(int64_t)blockIdx.x * p.experts + e] = sum;
  }
}

__global__ __launch_bounds__(kLayThreads) void layout_place_kernel(LayoutParams p) {
  extern __shared__ int smem[];
  int* s_hist = smem;                             // (waves, experts): counts, then next ranks
  int* s_start = smem + kLayWaves * p.experts;    // (experts + 1): first row of each expert
  int* s_count = s_start + p.experts + 1;         // (experts): entries of each expert
  __shared__ int s_scan[kLayWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int block = blockIdx.x;
  // this workgroup's chunk (with one chunk every workgroup counts it and the first one places it)
  const int chunk = p.blocks == 1 ? 0 : block;
  const int begin = chunk < p.blocks ? chunk * p.chunk : p.n;
  const int end = p.n - begin < p.chunk ? p.n : begin + p.chunk;
  count_entries(p, begin, end, s_hist);

  // ranks: entries of the expert in earlier chunks, then in this chunk's earlier waves
  for (int e = tid; e < p.experts; e += kLayThreads) {
    int before = 0, all = 0;
    if (p.blocks > 1) {
#pragma unroll 16
      for (int b = 0; b < p.blocks; ++b) {
        const int c = p.hist[(int64_t)b * p.experts + e];
        before += b < chunk ? c : 0;
        all += c;
      }
    }
    int here = 0;
#pragma unroll
    for (int w = 0; w < kLayWaves; ++w) {
      const int c = s_hist[w * p.experts + e];
      s_hist[w * p.experts + e] = before + here;
      here += c;
    }
    if (p.blocks == 1) all = here;
    s_count[e] = all;
    if (block == 0) p.counts[e] = all;
  }
  __syncthreads();
  // first rows: an exclusive scan of the aligned counts (each thread two experts), or a fixed pitch
  if (p.rows_per_expert) {
    for (int e = tid; e <= p.experts; e += kLayThreads) s_start[e] = e * p.rows_per_expert;
  } else {
    const int e0 = 2 * tid;
    const int c0 = e0 < p.experts ? (s_count[e0] + p.align - 1) / p.align * p.align : 0;
    const int c1 = e0 + 1 < p.experts ? (s_count[e0 + 1] + p.align - 1) / p.align * p.align : 0;
    int run = c0 + c1;
    for (int sh = 1; sh < 64; sh *= 2) {
      const int o = __shfl_up(run, sh);
      if (lane >= sh) run += o;
    }
    if (lane == 63) s_scan[wave] = run;
    __syncthreads();
    int base = 0;
    for (int w = 0; w < wave; ++w) base += s_scan[w];
    const int excl = base + run - c0 - c1;
    if (e0 <= p.experts) s_start[e0] = excl;
    if (e0 + 1 <= p.experts) s_start[e0 + 1] = excl + c0;
    if (tid == kLayThreads - 1) s_start[p.experts] = base + run;   // also where no thread's pair reaches it
  }
  __syncthreads();

  if (p.blocks > 1 || block == 0)
    for_entries(p, begin, end, s_hist + wave * p.experts, [&](int i, int e, int rank) {
      const bool fits = e >= 0 && (p.rows_per_expert == 0 || rank < p.rows_per_expert);
      const int row = fits ? s_start[e] + rank : -1;
      p.rows[i] = row;
      if (fits) p.sources[row] = i;
    });

  // every row's expert, and -1 for the rows that no entry fills (a row or two a thread)
  const int used = s_start[p.experts];
  for (uint32_t at = block * kLayThreads + tid; at < (uint32_t)p.rows_total; at += gridDim.x * kLayThreads) {
    const int r = (int)at;
    int lo = 0, hi = p.experts;   // s_start[lo] <= r < s_start[hi]
    if (r < used) {
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_start[mid] <= r) lo = mid;
        else hi = mid;
      }
    }
    if (p.m_indices != nullptr) p.m_indices[r] = r < used ? lo : -1;
    if (r >= used || r - s_start[lo] >= s_count[lo]) p.sources[r] = -1;
  }
}

static int64_t layout_chunk(int64_t n) {
  if (n <= kLayOnce) return kLayOnce;
  const int64_t even = (n + kLayMostChunks - 1) / kLayMostChunks;
  return even <= kLayChunk ? kLayChunk : (even + kLayThreads - 1) / kLayThreads * kLayThreads;
}
static int layout_blocks(int64_t n) { return n <= kLayOnce ? 1 : (int)((n + layout_chunk(n) - 1) / layout_chunk(n)); }

size_t moe_layout_workspace_size(int64_t n, int64_t experts) {
  const int b = layout_blocks(n);
  return b > 1 ? (size_t)b * (size_t)experts * 4 : 0;
}

int launch_moe_layout(const int32_t* ids, int64_t n, int experts, int64_t rows_per_expert, int align,
                      int64_t rows_total, int32_t* rows, int32_t* sources, int32_t* m_indices, int32_t* counts,
                      void* ws, hipStream_t stream) {
  LayoutParams p{};
  p.ids = ids; p.n = (int)n; p.experts = experts;
  p.rows_per_expert = (int)rows_per_expert; p.align = align; p.rows_total = (int)rows_total;
  p.blocks = layout_blocks(n);
  p.chunk = (int)layout_chunk(n);
  p.rows = rows; p.sources = sources; p.m_indices = m_indices; p.counts = counts;
  p.hist = static_cast<int32_t*>(ws);
  const size_t lds = (size_t)kLayWaves * experts * 4;
  if (p.blocks > 1) {
    hipLaunchKernelGGL(layout_count_kernel, dim3(p.blocks), dim3(kLayThreads), lds, stream, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return set_error(kHip, "moe_layout launch: %s", hipGetErrorString(e));
  }
  // workgroups: a chunk each, and enough to write the rows' arrays
  int64_t grid = (rows_total + kLayThreads - 1) / kLayThreads;
  if (grid > 128) grid = 128;
  if (grid < p.blocks) grid = p.blocks;
  hipLaunchKernelGGL(layout_place_kernel, dim3((unsigned)(grid < 1 ? 1 : grid)), dim3(kLayThreads),
                     lds + (2 * (size_t)experts + 1) * 4, stream, p);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? kOk : set_error(kHip, "moe_layout launch: %s", hipGetErrorString(e));
}

// ---------------------------------------------------------------------------
// Dispatch: each token's row is read (and quantized) once and written to its K expert rows.
// ---------------------------------------------------------------------------
enum Form : int { kCopy = 0, kFp8 = 1, kInt8 = 2 };
constexpr int kRowThreads = 256;
constexpr int kPadRows = 16;   // rows per padding workgroup
constexpr int kNarrowRow = 1024;   // rows up to this long are a wave's, longer ones a workgroup's

struct DispatchParams {
  const void* x;
  const int32_t* rows;
  const int32_t* sources;
  const int32_t* m_indices;   // contiguous layout: padding rows are zeroed; NULL: masked layout
  int tokens, top_k, hidden;
  int rows_total, rows_per_expert;
  void* q;
  float* s;
  int64_t ld_s;
  float* s_tmp;               // FP8: token-major scales (tokens, K groups), or NULL: stored to their places at once
};

// Row of a (token, place) entry, or -1: entries without a row, and anything a caller's array holds
// that is not a row of the layout.
__device__ __forceinline__ int row_at(const int32_t* rows, int k, int rows_total) {
  const int r = rows[k];
  return (uint32_t)r < (uint32_t)rows_total ? r : -1;
}

// Where row's scales of K group kb lie (FP8: K-group-major per matrix, as the GEMMs read them).
__device__ __forceinline__ int64_t fp8_scale_at(const DispatchParams& p, int row, int kb, int kbc) {
  if (p.rows_per_expert == 0) return (int64_t)kb * p.ld_s + row;
  const int g = row / p.rows_per_expert;
  return ((int64_t)g * kbc + kb) * p.ld_s + (row - g * p.rows_per_expert);
}

// Zero the padding rows among [row0, row0 + kPadRows): rows of an expert that no entry fills.
template <class T, int FORM>
__device__ __forceinline__ void zero_padding(const DispatchParams& p, int row0) {
  const int lane = threadIdx.x & 63;
  const int r = row0 + lane;
  uint64_t pad = __ballot(lane < kPadRows && r < p.rows_total && p.sources[r < p.rows_total ? r : 0] < 0 &&
                          p.m_indices[r < p.rows_total ? r : 0] >= 0);
  const int kbc = (p.hidden + kGroup - 1) / kGroup;
  constexpr int kSize = FORM == kCopy ? (int)sizeof(T) : 1;
  const int pieces = p.hidden * kSize / 16;
  while (pad != 0) {   // the same mask in every wave
    const int row = row0 + __builtin_ctzll(pad);
    pad &= pad - 1;
    u32x4_t* dst = reinterpret_cast<u32x4_t*>(static_cast<uint8_t*>(p.q) + (int64_t)row * p.hidden * kSize);
    for (int i = threadIdx.x; i < pieces; i += kRowThreads) dst[i] = u32x4_t{0u, 0u, 0u, 0u};
    if constexpr (FORM == kInt8) {
      if (threadIdx.x == 0) p.s[row] = 1.0f;
    } else if constexpr (FORM == kFp8) {
      if (p.s_tmp == nullptr)   // (else scale_rows_kernel writes them)
        for (int kb = threadIdx.x; kb < kbc; kb += kRowThreads) p.s[fp8_scale_at(p, row, kb, kbc)] = 1.0f;
    }
  }
}

// LT lanes hold a token's row (16 elements each at a time): a wave per token, four tokens a workgroup, for
// rows of up to 1024 elements (16384 tokens of 256: 29 us with a workgroup each), else the workgroup.
// FP8 scales lie K-group-major, so a row's are ld_s apart, each in a cache line of its own that 31 other
// rows share: with many of them the kernel writes them token-major into s_tmp and scale_rows_kernel moves
// them (4096 tokens x 8 of 7168: 72 us, 84 with the scattered stores).
template <class T, int FORM, int LT>
__global__ __launch_bounds__(kRowThreads) void dispatch_kernel(DispatchParams p) {
  constexpr int kTokens = kRowThreads / LT;
  __shared__ uint32_t s_max[kRowThreads / 64];
  const int tid = threadIdx.x;
  const int blocks = (p.tokens + kTokens - 1) / kTokens;
  if ((int)blockIdx.x >= blocks) {
    zero_padding<T, FORM>(p, ((int)blockIdx.x - blocks) * kPadRows);
    return;
  }
  // (wave-uniform: LT is a whole number of waves)
  const int token = blockIdx.x * kTokens + __builtin_amdgcn_readfirstlane(tid / LT);
  const int lane = tid % LT;
  if (token >= p.tokens) return;   // only where a wave holds a token: no barrier below
  const T* src = static_cast<const T*>(p.x) + (int64_t)token * p.hidden;
  const int32_t* rows = p.rows + (int64_t)token * p.top_k;

  if constexpr (FORM == kCopy) {
    T* out = static_cast<T*>(p.q);
    for (int i = 8 * lane; i < p.hidden; i += 8 * LT) {
      const Raw8<T> v = load8(src + i);
      for (int k = 0; k < p.top_k; ++k) {
        const int row = row_at(rows, k, p.rows_total);
        if (row >= 0) store8(out + (int64_t)row * p.hidden + i, v);
      }
    }
  } else if constexpr (FORM == kInt8) {
    uint8_t* out = static_cast<uint8_t*>(p.q);
    // a lane's first 16 elements stay in registers; those of longer rows are read again, from the caches
    Raw8<T> held[2];
    uint32_t amax = 0;
    auto largest = [&](const Raw8<T> (&r)[2]) {
      float v[16];
      widen8(r[0], v);
      widen8(r[1], v + 8);
#pragma unroll
      for (int u = 0; u < 16; ++u) amax = umax(amax, abs_bits(v[u]));
    };
    if (16 * lane < p.hidden) {
      held[0] = load8(src + 16 * lane);
      held[1] = load8(src + 16 * lane + 8);
      largest(held);
    }
    for (int i = 16 * (lane + LT); i < p.hidden; i += 16 * LT) {
      const Raw8<T> r[2] = {load8(src + i), load8(src + i + 8)};
      largest(r);
    }
    amax = wave_max_u32(amax);
    if constexpr (LT > 64) {
      if ((tid & 63) == 0) s_max[tid >> 6] = amax;
      __syncthreads();
      amax = umax(umax(s_max[0], s_max[1]), umax(s_max[2], s_max[3]));
    }
    const float s = int8_scale(amax);
    auto encode = [&](const Raw8<T> (&r)[2], int i) {
      float v[16];
      widen8(r[0], v);
      widen8(r[1], v + 8);
      const u32x4_t codes = {pack4_int8(v, s), pack4_int8(v + 4, s), pack4_int8(v + 8, s), pack4_int8(v + 12, s)};
      for (int k = 0; k < p.top_k; ++k) {
        const int row = row_at(rows, k, p.rows_total);
        if (row >= 0) *reinterpret_cast<u32x4_t*>(out + (int64_t)row * p.hidden + i) = codes;
      }
    };
    if (16 * lane < p.hidden) encode(held, 16 * lane);
    for (int i = 16 * (lane + LT); i < p.hidden; i += 16 * LT) {
      const Raw8<T> r[2] = {load8(src + i), load8(src + i + 8)};
      encode(r, i);
    }
    if (lane < p.top_k) {
      const int row = row_at(rows, lane, p.rows_total);
      if (row >= 0) p.s[row] = s;
    }
  } else {
    // 8 lanes hold one 128-wide group, 16 elements each (hidden % 16 == 0: a lane's are all present
    // or all absent; absent ones count as zeros)
    uint8_t* out = static_cast<uint8_t*>(p.q);
    const int kbc = (p.hidden + kGroup - 1) / kGroup;
    const int padded = kbc * kGroup;
    for (int i = 16 * lane; i < padded; i += 16 * LT) {
      const bool there = i < p.hidden;
      float v[16];
      widen8(load8(src + (there ? i : 0)), v);
      widen8(load8(src + (there ? i + 8 : 0)), v + 8);
      // the quantizer's maximum: a NaN takes no part unless the group holds nothing else
      float amax = fabsf(v[0]);
#pragma unroll
      for (int u = 1; u < 16; ++u) amax = fmaxf(amax, fabsf(v[u]));
      amax = max8(there ? amax : 0.0f);
      const float s = amax == 0.0f ? 1.0f : amax / kE4M3Max;
      u32x4_t codes;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        codes[u] = pack4_e4m3(clamp448(v[4 * u] / s), clamp448(v[4 * u + 1] / s), clamp448(v[4 * u + 2] / s),
                              clamp448(v[4 * u + 3] / s));
      if (p.s_tmp != nullptr && (lane & 7) == 0) p.s_tmp[(int64_t)token * kbc + i / kGroup] = s;
      for (int k = 0; k < p.top_k; ++k) {
        const int row = row_at(rows, k, p.rows_total);
        if (row < 0) continue;
        if (there) *reinterpret_cast<u32x4_t*>(out + (int64_t)row * p.hidden + i) = codes;
        if (p.s_tmp == nullptr && (lane & 7) == 0) p.s[fp8_scale_at(p, row, i / kGroup, kbc)] = s;
      }
    }
  }
}

// FP8 scales of 64 rows x 64 K groups from s_tmp (token-major) to their K-group-major places, through LDS.
constexpr int kScaleTile = 64;

__global__ __launch_bounds__(256) void scale_rows_kernel(DispatchParams p) {
  __shared__ float s_tile[kScaleTile][kScaleTile + 1];
  __shared__ int s_src[kScaleTile];
  const int kbc = (p.hidden + kGroup - 1) / kGroup;
  const int row0 = blockIdx.x * kScaleTile, kb0 = blockIdx.y * kScaleTile;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (wave == 0) {
    const int r = row0 + lane;
    const int src = r < p.rows_total ? p.sources[r] : -1;
    const bool pad = r < p.rows_total && src < 0 && p.m_indices != nullptr && p.m_indices[r] >= 0;
    // the row's token; -2: a padding row (scales 1); -1: not written (an entry past the tokens included)
    s_src[lane] = pad ? -2 : src >= 0 && src < (int64_t)p.tokens * p.top_k ? src / p.top_k : -1;
  }
  __syncthreads();
  float v[kScaleTile / 4];   // every lane loads, all of a wave's rows in flight together
  const int col = kb0 + lane < kbc ? kb0 + lane : kb0;
#pragma unroll
  for (int u = 0; u < kScaleTile / 4; ++u) {
    const int token = s_src[wave + 4 * u];
    v[u] = p.s_tmp[(int64_t)(token >= 0 ? token : 0) * kbc + col];
    v[u] = token >= 0 ? v[u] : 1.0f;
  }
#pragma unroll
  for (int u = 0; u < kScaleTile / 4; ++u) s_tile[lane][wave + 4 * u] = v[u];
  __syncthreads();
  const bool write = s_src[lane] != -1;
  for (int kb = wave; kb < kScaleTile && kb0 + kb < kbc; kb += 4)
    if (write) p.s[fp8_scale_at(p, row0 + lane, kb0 + kb, kbc)] = s_tile[kb][lane];
}

// Scales past which the second launch pays (2048 tokens x 8 of 2048, 256 K scales: 12.7 us scattered, 14.0 in
// two launches; 2048 x 8 of 7168, 0.9 M: 36.6 and 32.4; 4096 x 8 of 7168, 1.8 M: 84 and 72).
constexpr int64_t kScatterScales = 512 * 1024;

size_t moe_dispatch_fp8_workspace_size(int64_t tokens, int64_t top_k, int64_t hidden) {
  const int64_t kbc = (hidden + kGroup - 1) / kGroup;
  return tokens * top_k * kbc > kScatterScales ? (size_t)(tokens * kbc) * 4 : 0;
}

template <int FORM, int LT>
static const void* dispatch_fn(int dtype) {
  void (*fn)(DispatchParams) = dtype == kF32    ? dispatch_kernel<float, FORM, LT>
                               : dtype == kBf16 ? dispatch_kernel<Bf16, FORM, LT>
                                                : dispatch_kernel<_Float16, FORM, LT>;
  return reinterpret_cast<const void*>(fn);
}

template <int FORM>
static int launch_dispatch_form(DispatchParams p, int dtype, hipStream_t stream) {
  const int64_t pad = p.m_indices != nullptr ? (p.rows_total + kPadRows - 1) / kPadRows : 0;
  const bool narrow_rows = p.hidden <= kNarrowRow;
  const int64_t blocks = narrow_rows ? ((int64_t)p.tokens + 3) / 4 : p.tokens;
  if (blocks + pad == 0) return kOk;
  void* args[] = {&p};
  const int r = launched(narrow_rows ? dispatch_fn<FORM, 64>(dtype) : dispatch_fn<FORM, 256>(dtype),
                         dim3((unsigned)(blocks + pad)), dim3(kRowThreads), args, stream, "moe_dispatch");
  if (r != kOk || p.s_tmp == nullptr) return r;
  const int kbc = (p.hidden + kGroup - 1) / kGroup;
  return launched(reinterpret_cast<const void*>(scale_rows_kernel),
                  dim3((unsigned)((p.rows_total + kScaleTile - 1) / kScaleTile), (unsigned)((kbc + kScaleTile - 1) / kScaleTile)),
                  dim3(256), args, stream, "moe_dispatch_fp8 scales");
}

int launch_moe_dispatch(int form, const void* x, int dtype, const int32_t* rows, const int32_t* sources,
                        const int32_t* m_indices, int64_t tokens, int top_k, int64_t hidden, int64_t rows_total,
                        int64_t rows_per_expert, void* q, float* s, int64_t ld_s, float* s_tmp, hipStream_t stream) {
  DispatchParams p{};
  p.x = x; p.rows = rows; p.sources = sources; p.m_indices = m_indices;
  p.tokens = (int)tokens; p.top_k = top_k; p.hidden = (int)hidden;
  p.rows_total = (int)rows_total; p.rows_per_expert = (int)rows_per_expert;
  p.q = q; p.s = s; p.ld_s = ld_s; p.s_tmp = s_tmp;
  switch (form) {
    case kFp8: return launch_dispatch_form<kFp8>(p, dtype, stream);
    case kInt8: return launch_dispatch_form<kInt8>(p, dtype, stream);
    default: return launch_dispatch_form<kCopy>(p, dtype, stream);
  }
}

// ---------------------------------------------------------------------------
// Combine: y[t] = sum over k of w[t, k] * rows[row(t, k)], in fp32, in the order of k.
//
// It reads K rows for one written: bound by memory reads.  4096 tokens x 8 rows of 7168 bf16: 91 us, 5.8 TB/s;
// 16384 x 2 of 1024: 20.2 us, 5.0 TB/s (a large copy reaches 5.1, a large read 6 to 7; calls back to back in a
// graph, other rows each time).
// ---------------------------------------------------------------------------
constexpr int kCombThreads = 128;
constexpr int kCombBatch = 8;   // expert rows whose loads are in flight together

// Rows that the last-level cache cannot hold are read with nontemporal loads (4096 tokens x 8 of 7168 bf16, 470 MB:
// combine 109.5 us, 95.8 with them; 2048 x 8 of 7168, 235 MB: 40.6 and 48.3 when the rows are there).
constexpr int64_t kCacheBytes = 256 << 20;

struct CombineParams {
  const void* out;
  const int32_t* rows;
  const float* weights;   // NULL: 1
  int tokens, top_k, hidden;
  int rows_total;
  int pieces, slab;       // workgroups of a row, tokens of a grid row
  void* y;
};

// B rows' loads are in flight together.  They are unconditional (a branch around a load makes it wait for
// the ones before it: 4093 tokens x 6 of 2048, 33.3 us, 29.9 without): a place without a row reads the
// token's first one again, or the output's row.
template <class T, int B, bool NT>
__global__ __launch_bounds__(kCombThreads) void combine_kernel(CombineParams p) {
  // a row's pieces by neighbouring workgroups, so that memory sees whole rows (4093 x 6 of 2048 29.7 us, 24.7 so)
  const int in_slab = blockIdx.x / p.pieces;
  const int token = blockIdx.y * p.slab + in_slab;
  const int i = 8 * ((blockIdx.x - in_slab * p.pieces) * kCombThreads + threadIdx.x);
  if (token >= p.tokens || i >= p.hidden) return;
  const int32_t* rows = p.rows + (int64_t)token * p.top_k;
  const float* w = p.weights != nullptr ? p.weights + (int64_t)token * p.top_k : nullptr;
  const T* out = static_cast<const T*>(p.out);
  T* y = static_cast<T*>(p.y) + (int64_t)token * p.hidden;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int k0 = 0; k0 < p.top_k; k0 += B) {
    Raw8<T> v[B];
    int row[B];
#pragma unroll
    for (int u = 0; u < B; ++u) row[u] = k0 + u < p.top_k ? row_at(rows, k0 + u, p.rows_total) : -1;
    const T* spare = row[0] >= 0 ? out + (int64_t)row[0] * p.hidden : y;
#pragma unroll
    for (int u = 0; u < B; ++u) v[u] = load8<NT>((row[u] >= 0 ? out + (int64_t)row[u] * p.hidden : spare) + i);
#pragma unroll
    for (int u = 0; u < B; ++u) {
      if (row[u] >= 0) {
        float f[8];
        widen8(v[u], f);
        const float wk = w != nullptr ? w[k0 + u] : 1.0f;
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[c] = __builtin_fmaf(wk, f[c], acc[c]);
      }
    }
  }
  store8(y + i, narrow8<T>(acc));
}

template <int B, bool NT>
static const void* combine_fn(int dtype) {
  void (*fn)(CombineParams) = dtype == kF32    ? combine_kernel<float, B, NT>
                              : dtype == kBf16 ? combine_kernel<Bf16, B, NT>
                                               : combine_kernel<_Float16, B, NT>;
  return reinterpret_cast<const void*>(fn);
}
template <bool NT>
static const void* combine_fn(int dtype, int top_k) {
  return top_k <= 2 ? combine_fn<2, NT>(dtype) : top_k <= 4 ? combine_fn<4, NT>(dtype) : combine_fn<kCombBatch, NT>(dtype);
}

int launch_moe_combine(const void* out, int dtype, const int32_t* rows, const float* weights, int64_t tokens, int top_k,
                       int64_t hidden, int64_t rows_total, void* y, hipStream_t stream) {
  CombineParams p{};
  p.rows_total = (int)rows_total;
  p.out = out; p.rows = rows; p.weights = weights;
  p.tokens = (int)tokens; p.top_k = top_k; p.hidden = (int)hidden; p.y = y;
  p.pieces = (int)((hidden + 8 * kCombThreads - 1) / (8 * kCombThreads));
  const int64_t most = (1 << 24) / p.pieces, slab = tokens < most ? tokens : most;
  p.slab = (int)slab;
  const bool nontemporal = tokens * top_k * hidden * (dtype == kF32 ? 4 : 2) > kCacheBytes;
  void* args[] = {&p};
  return launched(nontemporal ? combine_fn<true>(dtype, top_k) : combine_fn<false>(dtype, top_k),
                  dim3((unsigned)(slab * p.pieces), (unsigned)((tokens + slab - 1) / slab)),
                  dim3(kCombThreads), args, stream, "moe_combine");
}

// Gradient of the weighted combine: dout[row(t, k)] = w[t, k] dy[t] (padding rows 0) and
// dw[t, k] = <dy[t], out[row(t, k)]>; a token a wave or a workgroup, as in dispatch (16384 tokens x 2 of 1024
// bf16: 58.9 us with a workgroup each, 35.2 with a wave).  Bound by memory, half of it writes: that call moves
// 4.8 TB/s, 4096 x 8 of 7168 (218 us) 4.6 without counting the padding rows' zeros.
struct CombineGradParams {
  DispatchParams pad;    // q = dout; for the padding rows
  const void* dy;
  const void* out;
  const float* weights;
  void* dout;
  float* dweights;
};

template <class T, int LT, bool NT>
__global__ __launch_bounds__(kRowThreads) void combine_grad_kernel(CombineGradParams p) {
  constexpr int kTokens = kRowThreads / LT;
  __shared__ float s_sum[kRowThreads / 64][64];
  const int tid = threadIdx.x, lane = tid % LT, wave_lane = tid & 63, wave = tid >> 6;
  const int blocks = (p.pad.tokens + kTokens - 1) / kTokens;
  if ((int)blockIdx.x >= blocks) {
    zero_padding<T, kCopy>(p.pad, ((int)blockIdx.x - blocks) * kPadRows);
    return;
  }
  const int token = blockIdx.x * kTokens + __builtin_amdgcn_readfirstlane(tid / LT);
  const int top_k = p.pad.top_k, hidden = p.pad.hidden;
  if (token >= p.pad.tokens) return;   // only where a wave holds a token: no barrier below
  // lane k holds place k's row and weight: one load each, where one by one they would wait for each other
  const int at = wave_lane < top_k ? wave_lane : 0;
  const int rows = wave_lane < top_k ? row_at(p.pad.rows + (int64_t)token * top_k, at, p.pad.rows_total) : -1;
  const float weights = p.weights[(int64_t)token * top_k + at];
  const T* dy = static_cast<const T*>(p.dy) + (int64_t)token * hidden;
  const T* out = static_cast<const T*>(p.out);
  T* dout = static_cast<T*>(p.dout);
  float mine = 0.f;   // place wave_lane's sum over this wave's elements; 0 where the entry has no row
  for (int k0 = 0; k0 < top_k; k0 += kCombBatch) {
    float sum[kCombBatch], wk[kCombBatch];
    int row[kCombBatch];
#pragma unroll
    for (int u = 0; u < kCombBatch; ++u) {
      sum[u] = 0.f;
      row[u] = __builtin_amdgcn_readlane(rows, k0 + u);   // (k0 + u < 64; -1 past top_k)
      wk[u] = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(weights), k0 + u));
    }
    for (int i = 8 * lane; i < hidden; i += 8 * LT) {
      float g[8];
      const Raw8<T> dg = load8(dy + i);
      Raw8<T> v[kCombBatch];
#pragma unroll
      for (int u = 0; u < kCombBatch; ++u)
        if (row[u] >= 0) v[u] = load8<NT>(out + (int64_t)row[u] * hidden + i);
      widen8(dg, g);
#pragma unroll
      for (int u = 0; u < kCombBatch; ++u) {
        if (row[u] < 0) continue;   // wave-uniform
        float f[8], d[8];
        widen8(v[u], f);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          sum[u] = __builtin_fmaf(g[c], f[c], sum[u]);
          d[c] = wk[u] * g[c];
        }
        store8(dout + (int64_t)row[u] * hidden + i, narrow8<T>(d));
      }
    }
#pragma unroll
    for (int u = 0; u < kCombBatch; ++u) {
      if (row[u] < 0) continue;
      const float s = wave_sum(sum[u]);
      mine = wave_lane == k0 + u ? s : mine;
    }
  }
  if constexpr (LT > 64) {
    s_sum[wave][wave_lane] = mine;
    __syncthreads();
    mine = ((s_sum[0][wave_lane] + s_sum[1][wave_lane]) + s_sum[2][wave_lane]) + s_sum[3][wave_lane];
  }
  if (lane < top_k) p.dweights[(int64_t)token * top_k + lane] = mine;   // (top_k <= 64: lane is wave_lane)
}

template <int LT, bool NT>
static const void* combine_grad_fn(int dtype) {
  void (*fn)(CombineGradParams) = dtype == kF32    ? combine_grad_kernel<float, LT, NT>
                                  : dtype == kBf16 ? combine_grad_kernel<Bf16, LT, NT>
                                                   : combine_grad_kernel<_Float16, LT, NT>;
  return reinterpret_cast<const void*>(fn);
}
template <int LT>
static const void* combine_grad_fn(int dtype, bool nontemporal) {
  return nontemporal ? combine_grad_fn<LT, true>(dtype) : combine_grad_fn<LT, false>(dtype);
}

int launch_moe_combine_grad(const void* dy, const void* out, int dtype, const int32_t* rows, const int32_t* sources,
                            const int32_t* m_indices, const float* weights, int64_t tokens, int top_k, int64_t hidden,
                            int64_t rows_total, void* dout, float* dweights, hipStream_t stream) {
  CombineGradParams p{};
  p.pad.rows = rows; p.pad.sources = sources; p.pad.m_indices = m_indices;
  p.pad.tokens = (int)tokens; p.pad.top_k = top_k; p.pad.hidden = (int)hidden;
  p.pad.rows_total = (int)rows_total; p.pad.q = dout;
  p.dy = dy; p.out = out; p.weights = weights; p.dout = dout; p.dweights = dweights;
  const bool nontemporal = 2 * tokens * top_k * hidden * (dtype == kF32 ? 4 : 2) > kCacheBytes;   // rows and their gradients
  const int64_t pad = m_indices != nullptr ? (rows_total + kPadRows - 1) / kPadRows : 0;
  const bool narrow_rows = hidden <= kNarrowRow;
  const int64_t blocks = narrow_rows ? (tokens + 3) / 4 : tokens;
  if (blocks + pad == 0) return kOk;
  void* args[] = {&p};
  return launched(narrow_rows ? combine_grad_fn<64>(dtype, nontemporal) : combine_grad_fn<256>(dtype, nontemporal), dim3((unsigned)(blocks + pad)),
                  dim3(kRowThreads), args, stream, "moe_combine_grad");
}

}  // namespace dg
