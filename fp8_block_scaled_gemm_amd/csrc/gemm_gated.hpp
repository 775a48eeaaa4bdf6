// The epilogue that the kernels of the gated GEMM share.
#pragma once

#include "gated.hpp"
#include "gemm_common.hpp"
#include "rows.hpp"

namespace dg {

constexpr int kGatedPitch = 2 * kGroup + 4;   // floats of a row of projections in LDS: 128 gate, 128 up, against bank conflicts

// A lane's 32 codes of a K block as bf16, which holds every E4M3 value: four operands of eight.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
struct Wide { bf16x8 v[4]; };
__device__ __forceinline__ Wide widen_codes(const v8i& x) {
  Wide w;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    bf16x2 p[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      p[2 * i] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[2 * t + i], 1.0f, false);
      p[2 * i + 1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[2 * t + i], 1.0f, true);
    }
    w.v[t] = bf16x8{p[0][0], p[0][1], p[1][0], p[1][1], p[2][0], p[2][1], p[3][0], p[3][1]};
  }
  return w;
}
// The 16 x 16 products of two such operands over a K block, added to 2^-22 of them.
__device__ __forceinline__ v4f exact_product(const Wide& a, const Wide& b) {
  v4f sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int t = 0; t < 4; ++t) sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[t], b.v[t], sum, 0, 0, 0);
  return sum;
}

// Eight bf16 values (four words) of a row's columns to dst and on, `count` of them there (8, fewer at the row's end,
// none or negative past it).  A row of odd length begins at any 2-byte address: where dst is not 4-byte aligned, 16
// neighbouring lanes shift their values by one, each storing its left neighbour's last one with its first seven.  Called by the
// 16 lanes of a row together.
__device__ __forceinline__ void store_bf16_run(uint16_t* dst, const uint32_t* w, int count, int lane16) {
  struct __attribute__((packed, aligned(4))) Words { uint32_t w[4]; };
  struct __attribute__((packed, aligned(4))) Words3 { uint32_t w[3]; };
  const uint32_t left = dpp_u32<0x111>(w[3]) >> 16;                  // row_shr:1, the lane before
  const int next = (int)dpp_u32<0x101>((uint32_t)(count > 0 ? count : 0));   // row_shl:1, the lane after (0 for the last)
  if (count <= 0) return;
  if (count < 8) {   // the last columns of a row: one by one (the lane before stores its own last value)
    for (int i = 0; i < count; ++i) dst[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    return;
  }
  if ((reinterpret_cast<uintptr_t>(dst) & 2) == 0) {
    *reinterpret_cast<Words*>(dst) = Words{{w[0], w[1], w[2], w[3]}};
    return;
  }
  const uint32_t x1 = (w[0] >> 16) | (w[1] << 16), x2 = (w[1] >> 16) | (w[2] << 16), x3 = (w[2] >> 16) | (w[3] << 16);
  if (lane16 == 0) {
    dst[0] = (uint16_t)w[0];
    *reinterpret_cast<Words3*>(dst + 1) = Words3{{x1, x2, x3}};
  } else {
    *reinterpret_cast<Words*>(dst - 1) = Words{{left | (w[0] << 16), x1, x2, x3}};
  }
  if (next < 8) dst[7] = (uint16_t)(w[3] >> 16);   // no lane after this one stores it
}

// One piece of a row: 8 columns from `col` of the projections g and u -> the projections, h or its codes, by the 16 lanes
// that hold the row's 128 columns of the tile (one scale group).
__device__ __forceinline__ void gated_piece(const GemmParams& p, int64_t out_row, float* scale_at, int col, int lane16,
                                            const float* g, const float* u) {
  const int count = p.n - col < 8 ? p.n - col : 8;
  auto store = [&](uint16_t* dst, const float* v) {
    const uint32_t w[4] = {pack2_bf16_rne(v[0], v[1]), pack2_bf16_rne(v[2], v[3]), pack2_bf16_rne(v[4], v[5]),
                           pack2_bf16_rne(v[6], v[7])};
    if ((p.n & 7) == 0) {   // every run of eight is 16-byte aligned, and there or not there as a whole
      if (count > 0) *reinterpret_cast<u32x4*>(dst) = u32x4{w[0], w[1], w[2], w[3]};
    } else {
      store_bf16_run(dst, w, count, lane16);
    }
  };
  if (p.pre != nullptr) {
    uint16_t* dst = p.pre + out_row * 2 * p.n + col;
    store(dst, g);
    store(dst + p.n, u);
  }
  float h[8];
  if (p.act == kSilu) {
#pragma unroll
    for (int c = 0; c < 8; ++c) h[c] = act_value<kSilu>(g[c]) * u[c];
  } else {
#pragma unroll
    for (int c = 0; c < 8; ++c) h[c] = act_value<kGelu>(g[c]) * u[c];
  }
  if (p.q == nullptr) {
    store(p.d + out_row * p.n + col, h);
    return;
  }
  if (count <= 0)   // columns past n take no part (n % 16 == 0: all eight or none)
#pragma unroll
    for (int c = 0; c < 8; ++c) h[c] = 0.0f;
  const GroupScale s = group16_scale(h);
  if (count > 0) *reinterpret_cast<u32x2_t*>(p.q + out_row * p.n + col) = pack8_e4m3(h, s);
  if (lane16 == 0) *scale_at = s.d.s;
}

// The rows of a tile of 128 columns of h, a loop of few instructions (written out for every fragment, the epilogue is tens
// of KB of code that each CU fetches once per launch: 20 us of a 30 us call).  `dump(c)` puts the projections of chunk c into
// LDS, chunk_rows rows of kGatedPitch floats; `row_of(c, r)` is the matrix's row that row r of it is.  The 16 lanes of
// a row then hold 8 columns each.
template <int NT, int LAYOUT, bool kTwoPass, class Dump, class RowOf>
__device__ __forceinline__ void gated_epilogue(const GemmParams& p, const TileCoord& t, int n0, int chunks, int chunk_rows,
                                               float* lds, Dump&& dump, RowOf&& row_of) {
  const int lane16 = threadIdx.x & 15;
  const int col = n0 + 8 * lane16;
  const int64_t row_base = LAYOUT == kMasked ? (int64_t)t.g * p.m : 0;
  float* scales = p.s + (LAYOUT == kMasked ? (int64_t)t.g * p.s_gstride : 0) + (int64_t)(n0 / kGroup) * p.ld_s;
#pragma unroll 1
  for (int c = 0; c < chunks; ++c) {
    if (row_of(c, 0) >= t.m_valid) break;   // the chunk's first row is its smallest
    __syncthreads();   // every wave is done with what LDS held
    dump(c);
    __syncthreads();
#pragma unroll 1
    for (int r = threadIdx.x >> 4; r < chunk_rows; r += NT / 16) {
      const int row = row_of(c, r);
      if ((kTwoPass && row < t.m_lo) || row >= t.m_valid) continue;   // (uniform over the 16 lanes)
      const float* src = lds + r * kGatedPitch + 8 * lane16;
      float g[8], u[8];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        *reinterpret_cast<v4f*>(g + 4 * i) = *reinterpret_cast<const v4f*>(src + 4 * i);
        *reinterpret_cast<v4f*>(u + 4 * i) = *reinterpret_cast<const v4f*>(src + kGroup + 4 * i);
      }
      gated_piece(p, row_base + row, scales + row, col, lane16, g, u);
    }
  }
}

}  // namespace dg
