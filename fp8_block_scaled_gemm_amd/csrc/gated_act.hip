// The activation and product of a gated feed-forward block on projections that exist already, h = act(g) u from rows
// (g | u) of 2n values, and the backward pass, dg = dh u act'(g) and du = dh act(g).  Arithmetic in fp32.  Bound by memory,
// but for the gradient in FP8.
#include "gated.hpp"
#include "rows.hpp"

namespace dg {

// Which rows are computed: all; those before masked_m[row / rows_per_group] of their group; or those whose m_indices is
// not negative.
struct RowMask {
  const int32_t* m_indices;
  const int32_t* masked_m;
  int64_t rows_per_group;
  // (group, row in it) of a row: of the masked layout, or all one group.  Rows are below 2^31.
  __device__ __forceinline__ void split(int64_t row, int& group, int& in_group) const {
    group = masked_m != nullptr ? (int)((uint32_t)row / (uint32_t)rows_per_group) : 0;
    in_group = (int)row - group * (int)rows_per_group;
  }
  __device__ __forceinline__ bool skips(int64_t row, int group, int in_group) const {
    if (masked_m != nullptr) return in_group >= masked_m[group];
    return m_indices != nullptr && m_indices[row] < 0;
  }
};

struct GatedActParams {
  const void* pre;
  void* h;            // or its codes
  float* scales;
  int64_t ld_s;
  int64_t rows;
  int n;
  RowMask mask;
};

template <int ACT>
__device__ __forceinline__ void gated_values(const float* g, const float* u, float* h) {
#pragma unroll
  for (int c = 0; c < 8; ++c) h[c] = act_value<ACT>(g[c]) * u[c];
}

constexpr int kActThreads = 256;

// h in the type of pre, or E4M3 codes with a scale per 128: 16 lanes a group of 128, 16 rows a workgroup, G groups of a
// row each, whose loads are in flight together (8192 x 2048 bf16 to FP8 15.1 us, 84 MB at 5.6 TB/s; 32 groups of 256 rows
// with half of them in use 10 us).
template <class T, int ACT, bool FP8, int G>
__global__ __launch_bounds__(kActThreads) void gated_act_kernel(GatedActParams p) {
  const int lane = threadIdx.x & 15;
  const int64_t row = ((int64_t)blockIdx.y + (int64_t)gridDim.y * blockIdx.z) * (kActThreads / 16) + (threadIdx.x >> 4);
  int group, in_group;
  p.mask.split(row, group, in_group);
  if (row >= p.rows || p.mask.skips(row, group, in_group)) return;   // uniform over the 16 lanes
  const int col0 = blockIdx.x * (G * kGroup) + 8 * lane;
  const T* src = static_cast<const T*>(p.pre) + row * 2 * p.n;
  Raw8<T> g[G], u[G];
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const int col = col0 + i * kGroup < p.n ? col0 + i * kGroup : 0;   // (an absent piece loads the first one)
    g[i] = load8(src + col);
    u[i] = load8(src + p.n + col);
  }
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const int col = col0 + i * kGroup;
    float a[8], b[8], h[8];
    widen8(g[i], a);
    widen8(u[i], b);
    gated_values<ACT>(a, b, h);
    if constexpr (FP8) {
      if (col >= p.n)
#pragma unroll
        for (int c = 0; c < 8; ++c) h[c] = 0.0f;
      const GroupScale s = group16_scale(h);
      if (col < p.n) {
        *reinterpret_cast<u32x2_t*>(static_cast<uint8_t*>(p.h) + row * p.n + col) = pack8_e4m3(h, s);
        if (lane == 0) p.scales[((int64_t)group * ((p.n + kGroup - 1) / kGroup) + col / kGroup) * p.ld_s + in_group] = s.d.s;
      }
    } else if (col < p.n) {
      store8(static_cast<T*>(p.h) + row * p.n + col, narrow8<T>(h));
    }
  }
}

// int8 codes with one scale a row: LT lanes a row (a wave and four rows a workgroup where rows are short: 65536 x 128 bf16
// 28 us, 60 with a workgroup each), HOLD pieces of 8 values a lane held in registers (the rest of a longer row is computed
// twice).  8192 x 2048 bf16: 18 us, 84 MB at 4.7 TB/s.
template <class T, int ACT, int LT, int HOLD>
__global__ __launch_bounds__(LT < kActThreads ? kActThreads : LT) void gated_act_int8_kernel(GatedActParams p) {
  constexpr int kRows = LT < kActThreads ? kActThreads / LT : 1, kWaves = LT / 64;
  __shared__ uint32_t s_max[kWaves];
  const int tid = threadIdx.x % LT;
  const int64_t row = (blockIdx.x + (int64_t)gridDim.x * blockIdx.y) * kRows + __builtin_amdgcn_readfirstlane(threadIdx.x / LT);
  int group, in_group;
  p.mask.split(row, group, in_group);
  if (row >= p.rows || p.mask.skips(row, group, in_group)) return;   // uniform over the row's waves, which share no barrier with another row's
  const T* src = static_cast<const T*>(p.pre) + row * 2 * p.n;
  uint8_t* dst = static_cast<uint8_t*>(p.h) + row * p.n;
  float h[HOLD][8];
  auto values = [&](int col, float* v) {
    float a[8], b[8];
    widen8(load8(src + col), a);
    widen8(load8(src + p.n + col), b);
    gated_values<ACT>(a, b, v);
  };
  uint32_t amax = 0;
  auto largest = [&](const float* v) {
#pragma unroll
    for (int c = 0; c < 8; ++c) amax = umax(amax, abs_bits(v[c]));
  };
#pragma unroll
  for (int i = 0; i < HOLD; ++i) {
    const int col = 8 * (tid + LT * i);
    if (col < p.n) {
      values(col, h[i]);
      largest(h[i]);
    }
  }
  for (int col = 8 * (tid + LT * HOLD); col < p.n; col += 8 * LT) {
    float v[8];
    values(col, v);
    largest(v);
  }
  amax = wave_max_u32(amax);
  if constexpr (kWaves > 1) {
    if ((tid & 63) == 0) s_max[tid >> 6] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) amax = umax(amax, s_max[w]);
  }
  const float s = int8_scale(amax);
  auto put = [&](int col, const float* v) {
    *reinterpret_cast<u32x2_t*>(dst + col) = u32x2_t{pack4_int8(v, s), pack4_int8(v + 4, s)};
  };
#pragma unroll
  for (int i = 0; i < HOLD; ++i) {
    const int col = 8 * (tid + LT * i);
    if (col < p.n) put(col, h[i]);
  }
  for (int col = 8 * (tid + LT * HOLD); col < p.n; col += 8 * LT) {
    float v[8];
    values(col, v);
    put(col, v);
  }
  if (tid == 0) p.scales[row] = s;
}

// (dg | du) in the type of the projections, a piece of 8 columns a lane (8192 x 2048 bf16 25.6 us, 168 MB).
template <class T, int ACT>
__global__ __launch_bounds__(kActThreads) void gated_act_grad_kernel(const T* __restrict__ dh, const T* __restrict__ pre,
                                                                     T* __restrict__ dpre, int64_t pieces, int n) {
  const int per_row = n / 8;
  const int64_t i = (int64_t)blockIdx.x * kActThreads + threadIdx.x;
  if (i >= pieces) return;
  const int64_t row = i / per_row;
  const int col = 8 * (int)(i - row * per_row);
  const int64_t at = row * 2 * n + col;
  const Raw8<T> rg = load8(pre + at), ru = load8(pre + at + n), rd = load8(dh + row * n + col);
  float g[8], u[8], d[8], dg[8], du[8];
  widen8(rg, g);
  widen8(ru, u);
  widen8(rd, d);
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    float value, slope;
    act_both<ACT>(g[c], value, slope);
    dg[c] = d[c] * u[c] * slope;
    du[c] = d[c] * value;
  }
  store8(dpre + at, narrow8<T>(dg));
  store8(dpre + at + n, narrow8<T>(du));
}

// The same gradient in FP8, as the two backward products of the projections read it, and h for the weight gradient of the
// product that follows them:
//   q, s   (rows, 2n), a scale per row and 128 columns       operand of dX = dpre * W
//   qt, st (2n, rows), a scale per column and 128 rows       operand of dW = dpre^T * X
//   ht, hst (n, rows), likewise of h                         operand of dW_out = dY^T * h
// A workgroup takes 128 rows x 128 columns of g, u and dh: a thread 4 consecutive rows of 8 columns.
// A row's 128 columns are the pieces of 16 neighbouring lanes, whose maximum is a row scale; a column's 128 rows are the 32
// threads 16 apart, reduced over the 4 lanes of a wave and then over the 8 waves through LDS.  Codes of columns are
// turned in LDS, one matrix after the other, so that stores are 128-byte runs.  Every input is read once, every output
// written once.  8192 x 2048 bf16: 48 us where a copy of its 185 MB takes 37; the vector instructions, 75 for each g, u and
// dh (22 the activation and its slope, 25 the five codes), are busy for most of it.
struct ActGradFp8Params {
  const void* dh;
  const void* pre;
  uint8_t* q;
  float* s;
  int64_t ld_s;
  uint8_t* qt;
  float* st;
  int64_t ld_st;
  uint8_t* ht;
  float* hst;
  int64_t ld_hst;
  int64_t rows;
  int n;
};

constexpr int kGradThreads = 512;
// Up to this many tiles, half of the CUs, four workgroups share a tile's outputs (rows, the columns of dg, of du, of h), each
// with the activation's arithmetic: 512 x 2048 9.4 us, 15.5 without; 1024 x 2048 14.6, 16.4; 1536 x 2048 18.8, 17.4.
constexpr int64_t kSplitTiles = 128;
constexpr int kTurnPitch = 33;   // dwords of one turned column (128 bytes and one dword, against bank conflicts)

template <class T, int ACT>
__global__ __launch_bounds__(kGradThreads) void gated_act_grad_fp8_kernel(ActGradFp8Params p) {
  __shared__ float s_max[kGradThreads / 64][kGroup];
  __shared__ Divisor s_scale[kGroup];
  __shared__ int s_plain[2];
  __shared__ uint32_t s_turn[kGroup * kTurnPitch];
  const int tid = threadIdx.x, lane = tid & 15, quad = tid >> 4;   // rows 4 quad .. 4 quad + 3 of the tile
  const int col = blockIdx.x * kGroup + 8 * lane;
  const int64_t row0 = (int64_t)blockIdx.y * kGroup, row = row0 + 4 * quad;
  const bool there = row < p.rows;   // rows % 16 == 0: all four or none
  const int parts = gridDim.z > 1 ? 1 << blockIdx.z : 15;   // this workgroup's outputs
  float dg[4][8], du[4][8], h[4][8];
  {
    Raw8<T> rg[4], ru[4], rd[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (there) {
        rg[i] = load8(static_cast<const T*>(p.pre) + (row + i) * 2 * p.n + col);
        ru[i] = load8(static_cast<const T*>(p.pre) + (row + i) * 2 * p.n + p.n + col);
        rd[i] = load8(static_cast<const T*>(p.dh) + (row + i) * p.n + col);
      }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (there) {
        float g[8], u[8], d[8];
        widen8(rg[i], g);
        widen8(ru[i], u);
        widen8(rd[i], d);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          float value, slope;
          act_both<ACT>(g[c], value, slope);
          dg[i][c] = d[c] * u[c] * slope;
          du[i][c] = d[c] * value;
          h[i][c] = value * u[c];
        }
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c) dg[i][c] = du[i][c] = h[i][c] = 0.0f;
      }
    }
  }
  if (p.q != nullptr && (parts & 1)) {
    auto by_rows = [&](const float (*v)[8], int half) {
      v4f scales;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const GroupScale s = group16_scale(v[i]);
        scales[i] = s.d.s;
        if (there)
          *reinterpret_cast<u32x2_t*>(p.q + (row + i) * 2 * p.n + half * p.n + col) = pack8_e4m3(v[i], s);
      }
      if (there && lane == 0)
        *reinterpret_cast<v4f*>(p.s + (int64_t)(half * (p.n / kGroup) + blockIdx.x) * p.ld_s + row) = scales;
    };
    by_rows(dg, 0);
    by_rows(du, 1);
  }
  // columns of one matrix: codes out + (col0 + c) * rows + row0, scales sc + blockIdx.y * ld + col0 + c
  auto by_columns = [&](const float (*v)[8], uint8_t* out, float* sc, int64_t ld, int64_t col0) {
    float m[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      m[c] = fmaxf(fmaxf(fabsf(v[0][c]), fabsf(v[1][c])), fmaxf(fabsf(v[2][c]), fabsf(v[3][c])));
      m[c] = fmaxf(m[c], __shfl_xor(m[c], 16));
      m[c] = fmaxf(m[c], __shfl_xor(m[c], 32));
    }
    if ((tid & 63) < 16) {
#pragma unroll
      for (int c = 0; c < 8; ++c) s_max[tid >> 6][8 * lane + c] = m[c];
    }
    __syncthreads();   // (and the previous matrix's codes are read)
    if (tid < kGroup) {
      float a = 0.0f;   // (a group of nothing but NaN has the scale 1, as in the quantizer of columns)
#pragma unroll
      for (int w = 0; w < kGradThreads / 64; ++w) a = fmaxf(a, s_max[w][tid]);
      const GroupScale s = group_scale(a);
      s_scale[tid] = s.d;
      if ((tid & 63) == 0) s_plain[tid >> 6] = s.plain;
      sc[(int64_t)blockIdx.y * ld + col0 + tid] = s.d.s;
    }
    __syncthreads();
    auto turn = [&](auto plain) {
      constexpr bool P = decltype(plain)::value;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const Divisor d = s_scale[8 * lane + c];
        s_turn[(8 * lane + c) * kTurnPitch + quad] = codes4_e4m3(quotient<P>(v[0][c], d), quotient<P>(v[1][c], d),
                                                                 quotient<P>(v[2][c], d), quotient<P>(v[3][c], d));
      }
    };
    if (s_plain[0] && s_plain[1]) turn(std::true_type{});
    else turn(std::false_type{});
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int piece = tid + kGradThreads * i, c = piece >> 3, at = piece & 7;   // 128 columns x 8 pieces of 16 rows
      const uint32_t* w = s_turn + c * kTurnPitch + 4 * at;
      if (row0 + 16 * at < p.rows)
        *reinterpret_cast<u32x4_t*>(out + (col0 + c) * p.rows + row0 + 16 * at) = u32x4_t{w[0], w[1], w[2], w[3]};
    }
  };
  const int64_t col0 = (int64_t)blockIdx.x * kGroup;
  if (p.qt != nullptr && (parts & 2)) by_columns(dg, p.qt, p.st, p.ld_st, col0);
  if (p.qt != nullptr && (parts & 4)) by_columns(du, p.qt, p.st, p.ld_st, p.n + col0);
  if (p.ht != nullptr && (parts & 8)) by_columns(h, p.ht, p.hst, p.ld_hst, col0);
}

// ---- host ------------------------------------------------------------------------------------------
static int act_launched(const char* what, hipError_t e) {
  return e == hipSuccess ? kOk : set_error(kHip, "%s launch: %s", what, hipGetErrorString(e));
}

template <class T, int ACT>
static int launch_act(int form, GatedActParams p, hipStream_t stream) {
  void* args[] = {&p};
  if (form == 2) {
    const int per_wg = p.n <= 1024 ? 4 : 1;
    const int64_t blocks = (p.rows + per_wg - 1) / per_wg, gx = blocks < kGridRow ? blocks : kGridRow;
    void (*fn)(GatedActParams) = p.n <= 1024   ? gated_act_int8_kernel<T, ACT, 64, 2>
                                 : p.n <= 8192 ? gated_act_int8_kernel<T, ACT, 256, 4> : gated_act_int8_kernel<T, ACT, 512, 4>;
    return act_launched("gated_act_int8", hipLaunchKernel(reinterpret_cast<const void*>(fn),
                                                          dim3((unsigned)gx, (unsigned)((blocks + gx - 1) / gx)),
                                                          dim3(p.n <= 8192 ? kActThreads : 512), args, 0, stream));
  }
  const int groups = (p.n + kGroup - 1) / kGroup;
  const int64_t row_blocks = (p.rows + kActThreads / 16 - 1) / (kActThreads / 16);
  const int64_t gy = row_blocks < 65535 ? row_blocks : 65535, gz = (row_blocks + gy - 1) / gy;
  if (gz > 65535) return set_error(kUnsupported, "gated_act: too many rows for the launch grid");
  const bool wide = row_blocks * ((groups + 1) / 2) >= 1024;   // two groups a lane where the grid stays wide
  void (*fn)(GatedActParams) = form == 1 ? (wide ? gated_act_kernel<T, ACT, true, 2> : gated_act_kernel<T, ACT, true, 1>)
                                         : (wide ? gated_act_kernel<T, ACT, false, 2> : gated_act_kernel<T, ACT, false, 1>);
  const unsigned gx = (unsigned)(wide ? (groups + 1) / 2 : groups);
  return act_launched("gated_act", hipLaunchKernel(reinterpret_cast<const void*>(fn), dim3(gx, (unsigned)gy, (unsigned)gz),
                                                   dim3(kActThreads), args, 0, stream));
}

template <class T>
static int launch_act_of(int act, int form, const GatedActParams& p, hipStream_t stream) {
  return act == kSilu ? launch_act<T, kSilu>(form, p, stream) : launch_act<T, kGelu>(form, p, stream);
}

// form 0: h in the type of pre, 1: E4M3 codes, 2: int8 codes.
int launch_gated_act(int form, const void* pre, int dtype, int act, const int32_t* m_indices, const int32_t* masked_m,
                     int64_t rows_per_group, int64_t rows, int64_t n, void* h, float* scales, int64_t ld_s,
                     hipStream_t stream) {
  GatedActParams p{};
  p.pre = pre;
  p.h = h;
  p.scales = scales;
  p.ld_s = ld_s;
  p.rows = rows;
  p.n = (int)n;
  p.mask = RowMask{m_indices, masked_m, rows_per_group};
  return dtype == kF32 ? launch_act_of<float>(act, form, p, stream)
         : dtype == kBf16 ? launch_act_of<Bf16>(act, form, p, stream) : launch_act_of<_Float16>(act, form, p, stream);
}

template <class T>
static int launch_act_grad(int act, const void* dh, const void* pre, void* dpre, int64_t rows, int64_t n,
                           hipStream_t stream) {
  const int64_t pieces = rows * (n / 8), blocks = (pieces + kActThreads - 1) / kActThreads;
  if (blocks > 0x7fffffffLL / kActThreads) return set_error(kUnsupported, "gated_act_grad: shape too large for the launch grid");
  auto fn = act == kSilu ? gated_act_grad_kernel<T, kSilu> : gated_act_grad_kernel<T, kGelu>;
  hipLaunchKernelGGL(fn, dim3((unsigned)blocks), dim3(kActThreads), 0, stream, static_cast<const T*>(dh),
                     static_cast<const T*>(pre), static_cast<T*>(dpre), pieces, (int)n);
  return act_launched("gated_act_grad", hipGetLastError());
}

int launch_gated_act_grad(const void* dh, const void* pre, int dtype, int act, int64_t rows, int64_t n, void* dpre,
                          hipStream_t stream) {
  return dtype == kF32 ? launch_act_grad<float>(act, dh, pre, dpre, rows, n, stream)
         : dtype == kBf16 ? launch_act_grad<Bf16>(act, dh, pre, dpre, rows, n, stream)
                          : launch_act_grad<_Float16>(act, dh, pre, dpre, rows, n, stream);
}

template <class T>
static const void* act_grad_fp8_fn(int act) {
  void (*fn)(ActGradFp8Params) = act == kSilu ? gated_act_grad_fp8_kernel<T, kSilu> : gated_act_grad_fp8_kernel<T, kGelu>;
  return reinterpret_cast<const void*>(fn);
}

int launch_gated_act_grad_fp8(const void* dh, const void* pre, int dtype, int act, int64_t rows, int64_t n, uint8_t* q,
                              float* s, int64_t ld_s, uint8_t* qt, float* st, int64_t ld_st, uint8_t* ht, float* hst,
                              int64_t ld_hst, hipStream_t stream) {
  const int64_t gy = (rows + kGroup - 1) / kGroup;
  if (gy > 65535) return set_error(kUnsupported, "gated_act_grad_fp8: too many rows for the launch grid");
  ActGradFp8Params p{dh, pre, q, s, ld_s, qt, st, ld_st, ht, hst, ld_hst, rows, (int)n};
  const void* fn = dtype == kF32 ? act_grad_fp8_fn<float>(act) : dtype == kBf16 ? act_grad_fp8_fn<Bf16>(act)
                                                                               : act_grad_fp8_fn<_Float16>(act);
  void* args[] = {&p};
  const unsigned gz = gy * (n / kGroup) <= kSplitTiles ? 4 : 1;
  return act_launched("gated_act_grad_fp8", hipLaunchKernel(fn, dim3((unsigned)(n / kGroup), (unsigned)gy, gz),
                                                            dim3(kGradThreads), args, 0, stream));
}

}  // namespace dg
