// 8-bit integer GEMM for gfx950 (CDNA4): D = (A * B^T) * sa[row] * sb[col], one fp32 scale per token
// (row of A) and per output channel (row of B), in the three forms of the FP8 GEMM: normal,
// contiguous-grouped and masked-grouped.
//
// The sum over K is exact: int8 products accumulate in int32 in the matrix cores
// (v_mfma_i32_16x16x64_i8), whose range holds K <= 131071 products of the largest codes.  The scales
// are applied once, in fp32, in the epilogue, and the result is rounded once to the output's type.
//
//  * MFMA operand A is the weight tile (rows n), operand B the activation tile (rows m): a lane holds
//    4 consecutive n of one row m.
//  * Operand tiles of 128 K bytes go from global memory into LDS by DMA (buffer_load ... lds); row r's
//    16-byte chunk c lies at slot c ^ f(r), f(r) = (r & 7) ^ ((r >> 3) & 1), so a DMA writes whole lines
//    and a fragment read (16 rows, one chunk) touches 16 distinct bank groups.
#include "gemm_common.hpp"
#include "rows.hpp"

namespace dg {

typedef __attribute__((address_space(3))) void lds_void;
typedef int v4i __attribute__((ext_vector_type(4)));

constexpr int kI8Block = 128;   // K bytes of one LDS stage

__device__ __forceinline__ int swz8(int r) { return (r & 7) ^ ((r >> 3) & 1); }

struct I8Params {
  const int8_t* a;
  const float* sa;
  const int8_t* b;
  const float* sb;
  void* d;
  const int32_t* m_indices;
  const int32_t* masked_m;
  int m, n, k;
  int groups;
  int tiles_m, tiles_n;
  int out_dtype;
};

template <int BN_, int BM_, int WN_, int WM_>
struct I8Cfg {
  static constexpr int BN = BN_, BM = BM_, WN = WN_, WM = WM_;
  static constexpr int kWaves = (BN / WN) * (BM / WM);
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int kFragN = WN / 16, kFragM = WM / 16;
  static constexpr int kDma = (BN + BM) / 8;            // DMA instructions of a stage (8 rows each)
  static constexpr int kDmaPerWave = kDma / kWaves;
  static_assert(kDma % kWaves == 0 && (BN / 8) % kWaves == 0, "DMA instructions must split evenly over waves");
};

// Four fp32 results of consecutive columns, rounded to the output's type.
__device__ __forceinline__ void store_out4(void* d, int dtype, int64_t at, const float* v, int count, bool vec) {
  if (dtype == kF32) {
    float* o = static_cast<float*>(d) + at;
    if (vec) *reinterpret_cast<v4f*>(o) = v4f{v[0], v[1], v[2], v[3]};
    else
      for (int i = 0; i < count; ++i) o[i] = v[i];
    return;
  }
  uint32_t lo, hi;
  if (dtype == kBf16) {
    lo = pack2_bf16_rne(v[0], v[1]);
    hi = pack2_bf16_rne(v[2], v[3]);
  } else {
    lo = pack2_f16(v[0], v[1]);
    hi = pack2_f16(v[2], v[3]);
  }
  uint16_t* o = static_cast<uint16_t*>(d) + at;
  if (vec) *reinterpret_cast<u32x2_t*>(o) = u32x2_t{lo, hi};
  else {
    const uint16_t h[4] = {(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi, (uint16_t)(hi >> 16)};
    for (int i = 0; i < count; ++i) o[i] = h[i];
  }
}

template <class C, int LAYOUT>
__global__ __launch_bounds__(C::kThreads) void gemm_int8_kernel(I8Params p) {
  constexpr int kStage = (C::BN + C::BM) * kI8Block;
  __shared__ __attribute__((aligned(1024))) uint8_t st[2][kStage];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g4 = lane >> 4;
  const int wn0 = (wave % (C::BN / C::WN)) * C::WN;
  const int wm0 = (wave / (C::BN / C::WN)) * C::WM;

  int rest = blockIdx.x;
  const int per_group = p.tiles_m * p.tiles_n;
  const int g = rest / per_group;
  rest -= g * per_group;
  const int m0 = (rest % p.tiles_m) * C::BM;
  const int n0 = (rest / p.tiles_m) * C::BN;
  int expert = g, m_valid = p.m;
  if constexpr (LAYOUT == kMasked) {
    const int mv = p.masked_m[g];
    m_valid = mv < 0 ? 0 : mv > p.m ? p.m : mv;
    if (m0 >= m_valid) return;
  }
  if constexpr (LAYOUT == kContiguous) {
    expert = p.m_indices[m0];
    if (expert < 0 || expert >= p.groups) return;
  }
  const int8_t* a = p.a + (LAYOUT == kMasked ? (int64_t)g * p.m * p.k : 0) + (int64_t)m0 * p.k;
  const int8_t* b = p.b + ((int64_t)expert * p.n + n0) * p.k;
  // rows past the edge read zeros (the hardware range check)
  const __amdgpu_buffer_rsrc_t rs_a = make_rsrc(a, (int64_t)(m_valid - m0) * p.k);
  const __amdgpu_buffer_rsrc_t rs_b = make_rsrc(b, (int64_t)(p.n - n0) * p.k);

  const int dma_row = 8 * wave + (lane >> 3);
  const int dma_chunk = ((lane & 7) ^ swz8(dma_row)) << 4;
  auto issue = [&](int kb, int slot) {
    const bool out = kb * kI8Block + dma_chunk >= p.k;   // chunks past K take an out-of-range offset: zeros
#pragma unroll
    for (int u = 0; u < C::kDmaPerWave; ++u) {
      constexpr int kB = C::BN / 8 / C::kWaves;
      const bool is_b = u < kB;
      const int row = dma_row + 8 * C::kWaves * (is_b ? u : u - kB);
      const uint32_t off = out ? 0xFFFFFFF0u : (uint32_t)row * (uint32_t)p.k + (uint32_t)dma_chunk;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(is_b ? rs_b : rs_a,
                                               (lds_void*)(st[slot] + (wave + C::kWaves * u) * 8 * kI8Block), 16, off,
                                               kb * kI8Block, 0, 0);
    }
  };

  v4i acc[C::kFragN][C::kFragM];
#pragma unroll
  for (int i = 0; i < C::kFragN; ++i)
#pragma unroll
    for (int j = 0; j < C::kFragM; ++j) acc[i][j] = v4i{0, 0, 0, 0};

  const int kbc = (p.k + kI8Block - 1) / kI8Block;
  issue(0, 0);
  for (int kb = 0; kb < kbc; ++kb) {
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();   // block kb landed for every wave; every wave is done with the other slot
    if (kb + 1 < kbc) issue(kb + 1, (kb + 1) & 1);
    const uint8_t* sb = st[kb & 1];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      v4i fb[C::kFragM];
#pragma unroll
      for (int j = 0; j < C::kFragM; ++j) {
        const int r = wm0 + 16 * j + l16;
        fb[j] = *reinterpret_cast<const v4i*>(sb + (C::BN + r) * kI8Block + (((4 * s + g4) ^ swz8(r)) << 4));
      }
#pragma unroll
      for (int i = 0; i < C::kFragN; ++i) {
        const int r = wn0 + 16 * i + l16;
        const v4i fa = *reinterpret_cast<const v4i*>(sb + r * kI8Block + (((4 * s + g4) ^ swz8(r)) << 4));
#pragma unroll
        for (int j = 0; j < C::kFragM; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fa, fb[j], acc[i][j], 0, 0, 0);
      }
    }
  }

  const float* sa = p.sa + (LAYOUT == kMasked ? (int64_t)g * p.m : 0);
  const float* sbp = p.sb + (int64_t)expert * p.n;
  const int64_t row_base = LAYOUT == kMasked ? (int64_t)g * p.m : 0;
#pragma unroll
  for (int j = 0; j < C::kFragM; ++j) {
    const int row = m0 + wm0 + 16 * j + l16;
    if (row >= m_valid) continue;
    const float sr = sa[row];
#pragma unroll
    for (int i = 0; i < C::kFragN; ++i) {
      const int col = n0 + wn0 + 16 * i + 4 * g4;
      const int count = p.n - col;
      if (count <= 0) continue;
      float v[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = (float)acc[i][j][r] * (sr * (r < count ? sbp[col + r] : 0.f));
      store_out4(p.d, p.out_dtype, (row_base + row) * p.n + col, v, count < 4 ? count : 4, (p.n & 3) == 0);
    }
  }
}

using I8Tile = I8Cfg<128, 128, 64, 64>;

int launch_quant_int8(const void* x, int dtype, int64_t rows, int64_t k, int8_t* q, float* s, hipStream_t stream);

size_t int8_workspace_size(int64_t, int64_t, int64_t, int64_t, int) { return 0; }

int launch_gemm_int8(int layout, const int8_t* a, const float* sa, const int8_t* b, const float* sb, void* d,
                     int out_dtype, const int32_t* m_indices, const int32_t* masked_m, int64_t groups, int64_t m,
                     int64_t n, int64_t k, void* ws, size_t ws_bytes, hipStream_t stream, int num_cus) {
  (void)ws; (void)ws_bytes; (void)num_cus;
  I8Params p{};
  p.a = a; p.sa = sa; p.b = b; p.sb = sb; p.d = d;
  p.m_indices = m_indices; p.masked_m = masked_m;
  p.m = (int)m; p.n = (int)n; p.k = (int)k;
  p.groups = (int)groups;
  p.tiles_m = (int)((m + I8Tile::BM - 1) / I8Tile::BM);
  p.tiles_n = (int)((n + I8Tile::BN - 1) / I8Tile::BN);
  p.out_dtype = out_dtype;
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n * (layout == kMasked ? groups : 1);
  if (tiles * I8Tile::kThreads > 0xffffffffLL) return set_error(kUnsupported, "int8 gemm: too many output tiles");
  void (*fn)(I8Params) = layout == kMasked ? gemm_int8_kernel<I8Tile, kMasked>
                         : layout == kContiguous ? gemm_int8_kernel<I8Tile, kContiguous>
                                                 : gemm_int8_kernel<I8Tile, kDense>;
  void* args[] = {&p};
  const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(fn), dim3((unsigned)tiles), dim3(I8Tile::kThreads),
                                       args, 0, stream);
  return e == hipSuccess ? kOk : set_error(kHip, "int8 gemm launch: %s", hipGetErrorString(e));
}

// In-call quantization: the counter prefix, the codes, the scales (256-byte pieces).
static size_t align256(size_t v) { return (v + 255) / 256 * 256; }

size_t int8_act_quant_workspace_size(int64_t m, int64_t n, int64_t k, int num_cus) {
  (void)n; (void)num_cus;
  return kCounterBytes + align256((size_t)(m * k)) + align256((size_t)m * 4);
}

int launch_gemm_int8_act_quant(const void* x, int dtype, const int8_t* b, const float* sb, void* d, int out_dtype,
                               int64_t m, int64_t n, int64_t k, void* ws, size_t ws_bytes, hipStream_t stream,
                               int num_cus) {
  (void)ws_bytes;
  int8_t* q = reinterpret_cast<int8_t*>(static_cast<uint8_t*>(ws) + kCounterBytes);
  float* s = reinterpret_cast<float*>(q + align256((size_t)(m * k)));
  const int r = launch_quant_int8(x, dtype, m, k, q, s, stream);
  if (r != kOk) return r;
  return launch_gemm_int8(kDense, q, s, b, sb, d, out_dtype, nullptr, nullptr, 1, m, n, k, nullptr, 0, stream, num_cus);
}

}  // namespace dg
