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
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "gemm_common.hpp"
#include "rows.hpp"

namespace dg {

typedef __attribute__((address_space(3))) void lds_void;
typedef int v4i __attribute__((ext_vector_type(4)));

constexpr int kI8Block = 128;   // K bytes of one LDS stage

// Every lane copies 16 (4) bytes from rsrc + voff + soff into lds + lane * 16 (4); out-of-range offsets
// read zeros.
__device__ __forceinline__ void lds_dma16(__amdgpu_buffer_rsrc_t rsrc, void* lds, uint32_t voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void*)lds, 16, voff, soff, 0, 0);
}
__device__ __forceinline__ void lds_dma4(__amdgpu_buffer_rsrc_t rsrc, void* lds, uint32_t voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void*)lds, 4, voff, soff, 0, 0);
}

__device__ __forceinline__ int swz8(int r) { return (r & 7) ^ ((r >> 3) & 1); }

struct I8Params {
  const int8_t* a;
  const float* sa;
  const int8_t* b;
  const float* sb;
  void* d;
  const int32_t* m_indices;
  const int32_t* masked_m;
  int* ws;               // K-split partials
  unsigned* counters;    // arrival counters, one per split tile
  int m, n, k;           // rows per group, columns, K
  int groups;
  int kb_total;          // ceil(k / 128)
  int tiles_m, tiles_n;
  int splits;            // K splits of every tile (1: none)
  int kb_per_split;
  int out_dtype;
};

// A workgroup tile of BN weight rows x BM activation rows in 8 waves of WN x WM, OCC workgroups per CU.
template <int BN_, int BM_, int WN_, int WM_, int OCC_>
struct I8Cfg {
  static constexpr int BN = BN_, BM = BM_, WN = WN_, WM = WM_, OCC = OCC_;
  static constexpr int kWavesN = BN / WN;
  static constexpr int kWaves = kWavesN * (BM / WM);
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int kFragN = WN / 16, kFragM = WM / 16;
  static constexpr int kStage = (BN + BM) * kI8Block;       // one LDS slot
  static constexpr int kBandsB = BN / 8 / kWaves;           // DMA instructions (8 rows each) per wave: weights,
  static constexpr int kDmaPerWave = (BN + BM) / 8 / kWaves;   // and in all
  static constexpr int kScaleBytes = (BN + BM) * 4;
  static_assert(kWaves == 8 && BN % 64 == 0 && BM % 64 == 0 && kFragN >= 3, "eight waves, at least three fragment rows");
};

// A sum times its two scales: their product rounds first where it is a normal number.  Elsewhere it can have lost
// bits that the result has, or have overflowed beside a zero sum: then the smaller scale comes first (a sum is
// an integer, so sum * scale is no smaller than the scale, and overflows only where the result does as well).
// Three roundings either way; a NaN scale gives NaN.
__device__ __forceinline__ bool is_normal(float v) { return __builtin_amdgcn_classf(v, 0x108); }   // of either sign
__device__ __forceinline__ float scaled_sum(int sum, float sr, float sc) {
  const float both = sr * sc;
  const bool row_first = fabsf(sr) < fabsf(sc);
  const float first = row_first ? sr : sc, second = row_first ? sc : sr;
  return is_normal(both) ? (float)sum * both : (float)sum * first * second;
}
// Scales any two of which have a normal product (or one of exact zero): 0, or from 2^-62 to below 2^63.
__device__ __forceinline__ bool plain_scale(float s) {
  const uint32_t a = abs_bits(s);
  return a == 0u || a - 0x20800000u < 0x3E800000u;
}

// The first `count` (at most 4) of four fp32 results of consecutive columns, rounded to the output's type;
// four are stored together, whatever the row's alignment.
__device__ __forceinline__ void store_out4(void* d, int dtype, int64_t at, const float* v, int count) {
  typedef v4f F32x4 __attribute__((aligned(4)));
  typedef u32x2_t Half4 __attribute__((aligned(2)));
  if (dtype == kF32) {
    float* o = static_cast<float*>(d) + at;
    if (count >= 4) *reinterpret_cast<F32x4*>(o) = v4f{v[0], v[1], v[2], v[3]};
    else
      for (int i = 0; i < count; ++i) o[i] = v[i];
    return;
  }
  const u32x2_t h = dtype == kBf16 ? u32x2_t{pack2_bf16_rne(v[0], v[1]), pack2_bf16_rne(v[2], v[3])}
                                   : u32x2_t{pack2_f16(v[0], v[1]), pack2_f16(v[2], v[3])};
  uint16_t* o = static_cast<uint16_t*>(d) + at;
  if (count >= 4) {
    *reinterpret_cast<Half4*>(o) = h;
  } else {
    const uint32_t w0 = h.x, w1 = h.y;
    if (count > 0) o[0] = (uint16_t)w0;
    if (count > 1) o[1] = (uint16_t)(w0 >> 16);
    if (count > 2) o[2] = (uint16_t)w1;
  }
}

// ---------------------------------------------------------------------------
// Tiles: a persistent grid over (group, m-block, n-block, K split), one workgroup per CU, two LDS slots.
//
// K block tk is multiplied from slot tk & 1.  A wave reads its weight fragments two fragment rows ahead
// of their MFMAs and its activation fragments one block ahead, each as soon as the last row's MFMA has
// consumed its predecessor, so every LDS read has two rows of MFMAs to return, across block boundaries
// too.  Two rows before a block's end every wave has read all it reads of the block's slot and waits for
// its own DMAs of the next block; one barrier makes both hold for all.  Then block tk + 2's DMAs go into
// the freed slot, spread over the MFMAs of the last two rows, and have one block's compute to land.
// The block body has no branch: past the last block the DMAs take out-of-range offsets and write zeros
// that nothing reads.
//
// Bound by the matrix cores: 16384 x 7168 x 16384 runs at 2.65e15 operations/s (1450 us, 1424 to 1482 over several
// cards), 4096 x 4096 x 7168 at 2.45e15 (98 us, one round of 256 tiles: its first loads and its stores are not
// hidden).  The rate depends on the operands' bits (zeros 3.2e15, random codes 2.65e15): power holds the clock, not the
// instruction stream.  32x32x32 products in the place of
// 16x16x64 ones ran at 2.53e15; a 256x128 tile was slower for the grouped forms; the smaller tile serves
// launches that the square one leaves short of work (256 x 4096 x 7168: 21.6 us, split in four).
// ---------------------------------------------------------------------------
template <int V>
using IC = std::integral_constant<int, V>;

template <class C, int LAYOUT>
__global__ __launch_bounds__(C::kThreads, 2 * C::OCC) void gemm_int8_kernel(I8Params p) {
  constexpr int NT = C::kThreads, kFN = C::kFragN, kFM = C::kFragM;
  constexpr int kBarRow = kFN - 2;
  __shared__ __attribute__((aligned(1024))) uint8_t st0[C::kStage];
  __shared__ __attribute__((aligned(1024))) uint8_t st1[C::kStage];
  __shared__ __attribute__((aligned(16))) float s_scale[C::BN + C::BM];   // the tile's column, then row scales
  __shared__ int s_prefix[LAYOUT == kMasked ? 1025 : 1];
  __shared__ int s_scan[LAYOUT == kMasked ? 256 : 1];
  __shared__ int s_flag;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g4 = lane >> 4;
  const int wn0 = (wave % C::kWavesN) * C::WN;
  const int wm0 = (wave / C::kWavesN) * C::WM;

  int total_items;
  if constexpr (LAYOUT == kMasked) {
    masked_item_prefix(p.masked_m, p.groups, p.m, C::BM, p.tiles_n, s_prefix, s_scan);
    total_items = s_prefix[p.groups];
  } else {
    total_items = p.tiles_m * p.tiles_n * p.splits;
  }
  // workgroup b runs on XCD b % 8: each XCD takes a contiguous range of items in every round
  const int grid = gridDim.x;
  int wg = blockIdx.x;
  if ((grid & 7) == 0) wg = (blockIdx.x & 7) * (grid >> 3) + (blockIdx.x >> 3);

  // contiguous layout: a tile whose 128-row blocks name two experts runs once for each
  constexpr bool kTwoPass = LAYOUT == kContiguous && C::BM > kGroup;
  int step = grid, next_pass = 0;
  for (int item = wg, pass = 0; item < total_items; item += step, pass = next_pass) {
    step = grid;
    next_pass = 0;
    const int tile_id = LAYOUT == kDense ? item / p.splits : item;   // only the normal form splits K
    const int split = LAYOUT == kDense ? item - tile_id * p.splits : 0;
    int rest = tile_id;
    int g = 0, mb, nbt, m_lo = 0, m_valid = p.m;
    if constexpr (LAYOUT == kMasked) {
      g = masked_group_of(s_prefix, p.groups, rest);
      rest -= s_prefix[g];
      const int mblocks = (s_prefix[g + 1] - s_prefix[g]) / p.tiles_n;
      mb = rest % mblocks;
      nbt = rest / mblocks;
      const int mv = p.masked_m[g];
      m_valid = mv < 0 ? 0 : mv > p.m ? p.m : mv;
    } else {
      // runs of 8 m-tiles x all n-tiles, m fastest: the items of one XCD's round share their panels in its L2
      constexpr int kRun = 8;
      const int run = rest / (kRun * p.tiles_n);
      const int first_m = run * kRun;
      const int run_m = p.tiles_m - first_m < kRun ? p.tiles_m - first_m : kRun;
      const int in_run = rest - run * (kRun * p.tiles_n);
      mb = first_m + in_run % run_m;
      nbt = in_run / run_m;
    }
    const int m0 = mb * C::BM, n0 = nbt * C::BN;
    int expert = g;
    if constexpr (LAYOUT == kContiguous) {
      expert = p.m_indices[m0];
      if constexpr (kTwoPass) {
        static_assert(C::BM == 2 * kGroup, "a contiguous tile spans one or two 128-row expert blocks");
        const int e1 = m0 + kGroup < p.m ? p.m_indices[m0 + kGroup] : expert;
        if (e1 != expert) {   // uniform
          if (pass == 0) {
            step = 0;   // the same item again, as pass 1
            next_pass = 1;
            m_valid = m0 + kGroup;
          } else {
            expert = e1;
            m_lo = m0 + kGroup;
          }
        }
      }
      if (expert < 0 || expert >= p.groups) continue;   // uniform: an unmapped block
    }
    const int kb_begin = split * p.kb_per_split;
    const int nk = p.kb_total - kb_begin < p.kb_per_split ? p.kb_total - kb_begin : p.kb_per_split;

    const int64_t row_base = LAYOUT == kMasked ? (int64_t)g * p.m : 0;
    // rows past the edge read zeros (the hardware range check)
    const __amdgpu_buffer_rsrc_t rs_a = make_rsrc(p.a + (row_base + m0) * p.k, (int64_t)(m_valid - m0) * p.k);
    const __amdgpu_buffer_rsrc_t rs_b =
        make_rsrc(p.b + ((int64_t)expert * p.n + n0) * p.k, (int64_t)(p.n - n0) * p.k);
    const __amdgpu_buffer_rsrc_t rs_sa = make_rsrc(p.sa + row_base + m0, (int64_t)(m_valid - m0) * 4);
    const __amdgpu_buffer_rsrc_t rs_sb = make_rsrc(p.sb + (int64_t)expert * p.n + n0, (int64_t)(p.n - n0) * 4);

    // DMA instruction d of a wave fills 8 tile rows, weights first; lane i writes row i / 8, slot i % 8,
    // so it loads the logical chunk (i % 8) ^ f(row) (f has period 16 rows: the same for every d)
    const int dma_row = 8 * wave + (lane >> 3);
    const int dma_chunk = ((lane & 7) ^ swz8(dma_row)) << 4;
    const uint32_t dma_off = (uint32_t)dma_row * (uint32_t)p.k + (uint32_t)dma_chunk;
    const uint32_t band_step = (uint32_t)(8 * C::kWaves) * (uint32_t)p.k;
    uint8_t* const slot0 = st1;   // blocks 0, 2, ...: the buffer that the epilogue's strips do not use
    uint8_t* const slot1 = st0;
    struct DmaCtx { uint8_t* sbase; int koff; uint32_t off, out; };
    auto dma_ctx = [&](int tk, auto slot_c, bool valid) {
      DmaCtx c;
      c.sbase = decltype(slot_c)::value == 0 ? slot0 : slot1;
      c.koff = (kb_begin + tk) * kI8Block;
      c.off = dma_off;
      asm volatile("" : "+v"(c.off));   // the bands' offsets are one add each, not registers of their own
      // bitwise, no branch: chunks past K and blocks past the last take an out-of-range offset
      c.out = 0u - ((uint32_t)(!valid) | (uint32_t)(c.koff + dma_chunk >= p.k));
      return c;
    };
    auto dma_one = [&](const DmaCtx& c, int d) {
      const bool is_b = d < C::kBandsB;
      const uint32_t off = c.off + (uint32_t)(is_b ? d : d - C::kBandsB) * band_step;
      lds_dma16(is_b ? rs_b : rs_a, c.sbase + (wave + C::kWaves * d) * 8 * kI8Block, off | (c.out & 0xFFFFFFF0u), c.koff);
    };
    auto issue = [&](int tk, auto slot_c, bool valid) {
      const DmaCtx c = dma_ctx(tk, slot_c, valid);
#pragma unroll
      for (int d = 0; d < C::kDmaPerWave; ++d) dma_one(c, d);
    };

    v4i acc[kFN][kFM];
#pragma unroll
    for (int i = 0; i < kFN; ++i)
#pragma unroll
      for (int j = 0; j < kFM; ++j) acc[i][j] = v4i{0, 0, 0, 0};

    // a fragment: 16 rows x 128 K bytes, as two steps of 64 (logical chunks g4 and 4 + g4 of a lane's row;
    // the second's slot differs in bit 2 only: address ^ 64)
    struct Frag { v4i s[2]; };
    const int lane_off = l16 * kI8Block + ((g4 ^ swz8(l16)) << 4);
    auto read_frag = [&](const uint8_t* sbase, int row) {
      const int off = row * kI8Block + lane_off;
      Frag f;
      f.s[0] = *reinterpret_cast<const v4i*>(sbase + off);
      f.s[1] = *reinterpret_cast<const v4i*>(sbase + (off ^ 64));
      return f;
    };
    // fragment rows [R0, R1) of the block in slot cur.  Row i's weights come from fa[i % 3]; at its start
    // row i + 2's are requested (rows kFN and kFN + 1 are the next block's rows 0 and 1, from slot nxt).
    // In the last row each activation fragment half is replaced by the next block's once used.
    auto rows = [&](auto r0_c, auto r1_c, const uint8_t* cur, const uint8_t* nxt, Frag* fa, Frag* fb, const DmaCtx* dc) {
      constexpr int R0 = decltype(r0_c)::value, R1 = decltype(r1_c)::value;
      constexpr int T = (R1 - R0) * kFM * 2;   // MFMAs; with dc, the stage's DMAs are spread over them
#pragma unroll
      for (int i = R0; i < R1; ++i) {
        __builtin_amdgcn_sched_barrier(0);
        fa[(i + 2) % 3] = i + 2 < kFN ? read_frag(cur, wn0 + 16 * (i + 2)) : read_frag(nxt, wn0 + 16 * (i + 2 - kFN));
#pragma unroll
        for (int q = 0; q < 2 * kFM; ++q) {
          const int s = q / kFM, j = q % kFM;
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fa[i % 3].s[s], fb[j].s[s], acc[i][j], 0, 0, 0);
          if (i == kFN - 1) {
            const int off = (C::BN + wm0 + 16 * j) * kI8Block + lane_off;
            fb[j].s[s] = *reinterpret_cast<const v4i*>(nxt + (s == 0 ? off : off ^ 64));
          }
          if (dc != nullptr) {
            const int t = (i - R0) * 2 * kFM + q;
            const int d0 = t * C::kDmaPerWave / T, d1 = (t + 1) * C::kDmaPerWave / T;
            for (int d = d0; d < d1; ++d) dma_one(*dc, d);
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (R1 == kBarRow) {   // no MFMA of these rows moves below the barrier
#pragma unroll
        for (int i = R0; i < R1; ++i)
#pragma unroll
          for (int j = 0; j < kFM; ++j) asm volatile("" : "+v"(acc[i][j]));
      }
    };
    // the barrier of block tk (slot CUR) and its last two rows; on return fa[0], fa[1] and fb hold the
    // next block's first fragments
    auto bar_tail = [&](int tk, auto cur_c, auto nxt_c, Frag* fa, Frag* fb) {
      const uint8_t* cur = decltype(cur_c)::value == 0 ? slot0 : slot1;
      const uint8_t* nxt = decltype(nxt_c)::value == 0 ? slot0 : slot1;
      __builtin_amdgcn_s_waitcnt(0x0070);   // vmcnt(0), lgkmcnt(0): reads of CUR done, DMAs of tk + 1 landed
      __syncthreads();
      const DmaCtx dc = dma_ctx(tk + 2, cur_c, tk + 2 < nk);
      rows(IC<kBarRow>{}, IC<kFN>{}, cur, nxt, fa, fb, &dc);
      const Frag f0 = fa[kFN % 3], f1 = fa[(kFN + 1) % 3];
      fa[0] = f0;
      fa[1] = f1;
    };

    // Block 0's DMAs go out before the first wait: every wave is past its last read of slot 0, and their
    // latency overlaps the draining of the previous tile's stores.
    issue(0, IC<0>{}, true);
    __builtin_amdgcn_s_waitcnt(0x0070);
    __syncthreads();   // block 0 landed for every wave; every wave is done with the strips and scales
    issue(1, IC<1>{}, nk > 1);
    {   // the tile's scales: 64 a wave (lanes past the edge read zeros)
      const bool col = wave < C::BN / 64;
      const int at = col ? 64 * wave : 64 * wave - C::BN;
      if (64 * wave < C::BN + C::BM)   // wave-uniform
        lds_dma4(col ? rs_sb : rs_sa, s_scale + 64 * wave, (uint32_t)(at + lane) * 4u, 0);
    }
    // A wave whose rows or columns all lie outside the tile's part of the problem (edges, a masked
    // group's count, one half of a two-expert tile) only moves data: its SIMD partner has the matrix
    // core to itself, and a tile of half the rows takes little more than half the time.
    const bool active = m0 + wm0 < m_valid && m0 + wm0 + C::WM > m_lo && n0 + wn0 < p.n;   // wave-uniform
    if (!active) {
      for (int tk = 0; tk < nk; ++tk) {   // the same barriers and DMAs as below
        __builtin_amdgcn_s_waitcnt(0x0070);
        __syncthreads();
        if (tk + 2 < nk) {
          if (tk & 1) issue(tk + 2, IC<1>{}, true);
          else issue(tk + 2, IC<0>{}, true);
        }
      }
    } else {
      Frag fa[3], fb[kFM];
#pragma unroll
      for (int j = 0; j < kFM; ++j) fb[j] = read_frag(slot0, C::BN + wm0 + 16 * j);
      fa[0] = read_frag(slot0, wn0);
      fa[1] = read_frag(slot0, wn0 + 16);
      rows(IC<0>{}, IC<kBarRow>{}, slot0, slot1, fa, fb, nullptr);
      int tk = 0;
      for (; tk + 2 < nk; tk += 2) {
        bar_tail(tk, IC<0>{}, IC<1>{}, fa, fb);
        rows(IC<0>{}, IC<kBarRow>{}, slot1, slot0, fa, fb, nullptr);
        bar_tail(tk + 1, IC<1>{}, IC<0>{}, fa, fb);
        rows(IC<0>{}, IC<kBarRow>{}, slot0, slot1, fa, fb, nullptr);
      }
      bar_tail(tk, IC<0>{}, IC<1>{}, fa, fb);
      if (tk + 1 < nk) {
        rows(IC<0>{}, IC<kBarRow>{}, slot1, slot0, fa, fb, nullptr);
        bar_tail(tk + 1, IC<1>{}, IC<0>{}, fa, fb);
      }
      __builtin_amdgcn_s_waitcnt(0x0070);   // the zero-filling DMAs past the last block
    }

    // ---- K split: the workgroup that arrives last adds the other partials -------------------------
    if (LAYOUT == kDense && p.splits > 1) {
      constexpr int kFrags = kFN * kFM;
      constexpr int kSplitBytes = kFrags * NT * 16;   // [fragment][thread] pieces of 16 bytes
      const __amdgpu_buffer_rsrc_t rs_ws =
          make_rsrc(p.ws + (int64_t)tile_id * p.splits * (kSplitBytes / 4), (int64_t)p.splits * kSplitBytes);
#pragma unroll
      for (int f = 0; f < kFrags; ++f)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[f / kFM][f % kFM]), rs_ws,
                                               split * kSplitBytes + tid * 16 + f * NT * 16, 0, kCpolSc1);
      __builtin_amdgcn_s_waitcnt(0);   // this thread's partials have arrived
      __syncthreads();
      if (tid == 0) {
        const unsigned prev = __hip_atomic_fetch_add(p.counters + tile_id, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        s_flag = prev == (unsigned)(p.splits - 1);
        if (s_flag) __hip_atomic_store(p.counters + tile_id, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      __syncthreads();
      if (!s_flag) continue;
      for (int o = 0; o < p.splits; ++o) {   // integers: any order
        if (o == split) continue;
        constexpr int kBatch = kFrags < 16 ? kFrags : 16;   // loads in flight together
#pragma unroll
        for (int f0 = 0; f0 < kFrags; f0 += kBatch) {
          v4i v[kBatch];
#pragma unroll
          for (int f = 0; f < kBatch; ++f)
            v[f] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(
                                               rs_ws, o * kSplitBytes + tid * 16 + (f0 + f) * NT * 16, 0, kCpolSc1));
#pragma unroll
          for (int f = 0; f < kBatch; ++f) acc[(f0 + f) / kFM][(f0 + f) % kFM] += v[f];
        }
      }
    }

    // ---- epilogue: scale, round, store --------------------------------------------------------------
    __syncthreads();   // every wave is done with the slots; the scales have landed
    // an opaque copy of the lane: the epilogue's addresses are formed here, not kept in registers (256 a
    // wave, most of them sums) across the main loop
    int el = lane;
    asm volatile("" : "+v"(el));
    const int e16 = el & 15, e4 = el >> 4;
    auto scaled = [&](auto plain_c, int i, int j, float* v) {
      const float sr = s_scale[C::BN + wm0 + 16 * j + e16];
      const v4f sc = *reinterpret_cast<const v4f*>(&s_scale[wn0 + 16 * i + 4 * e4]);
#pragma unroll
      for (int r = 0; r < 4; ++r)
        v[r] = decltype(plain_c)::value ? (float)acc[i][j][r] * (sr * sc[r]) : scaled_sum(acc[i][j][r], sr, sc[r]);
    };
    // Through LDS: each wave turns 16 output rows of its tile (fp32: of half its columns at a time) into
    // row pieces of 16 bytes (a fragment's own stores would touch 16 rows of 32 or 64 bytes each).
    auto store_rows = [&](auto size_c, auto plain_c) {
      constexpr int kSize = decltype(size_c)::value;   // bytes of an element
      constexpr int kParts = kSize / 2, kCols = C::WN / kParts;
      constexpr int kPitch = kCols * kSize + 16;
      constexpr int kPiecesRow = kCols * kSize / 16, kPiecesLane = 16 * kPiecesRow / 64;
      static_assert(C::kWaves * 16 * kPitch <= C::kStage && kFN % kParts == 0, "the strips fit in one slot");
      uint8_t* strip = st0 + wave * (16 * kPitch);
#pragma unroll
      for (int part = 0; part < kParts; ++part) {
#pragma unroll
        for (int j = 0; j < kFM; ++j) {
#pragma unroll
          for (int i0 = 0; i0 < kFN / kParts; ++i0) {
            // (one fragment at a time: interleaved, the cases' operands spill)
            if constexpr (!decltype(plain_c)::value) __builtin_amdgcn_sched_barrier(0);
            float v[4];
            scaled(plain_c, part * (kFN / kParts) + i0, j, v);
            uint8_t* at = strip + e16 * kPitch + (16 * i0 + 4 * e4) * kSize;
            if constexpr (kSize == 4) *reinterpret_cast<v4f*>(at) = v4f{v[0], v[1], v[2], v[3]};
            else if (p.out_dtype == kBf16)
              *reinterpret_cast<u32x2_t*>(at) = u32x2_t{pack2_bf16_rne(v[0], v[1]), pack2_bf16_rne(v[2], v[3])};
            else *reinterpret_cast<u32x2_t*>(at) = u32x2_t{pack2_f16(v[0], v[1]), pack2_f16(v[2], v[3])};
          }
          // the wave reads back what its own lanes wrote (its LDS operations complete in order)
          uint8_t* out = static_cast<uint8_t*>(p.d);
          const int row0 = m0 + wm0 + 16 * j, col0 = n0 + wn0 + part * kCols;
          using E = std::conditional_t<kSize == 4, uint32_t, uint16_t>;
          typedef u32x4 Piece __attribute__((aligned(2)));   // rows need no alignment past their elements'
          constexpr int kElems = 16 / kSize;
#pragma unroll
          for (int u = 0; u < kPiecesLane; ++u) {
            const int c = el + 64 * u;
            const int row = c / kPiecesRow, cc = c % kPiecesRow;
            const uint8_t* from = strip + row * kPitch + cc * 16;
            const int mrow = row0 + row, ncol = col0 + cc * kElems;
            if ((kTwoPass && mrow < m_lo) || mrow >= m_valid || ncol >= p.n) continue;
            E* to = reinterpret_cast<E*>(out) + (row_base + mrow) * p.n + ncol;
            if (ncol + kElems <= p.n) *reinterpret_cast<Piece*>(to) = *reinterpret_cast<const u32x4*>(from);
            else   // the N edge inside a piece
              for (int e = 0; e < p.n - ncol; ++e) to[e] = reinterpret_cast<const E*>(from)[e];
          }
        }
      }
    };
    // Scales of ordinary size need none of scaled_sum's cases (8192 x 8192 x 512 57.5 us, 61.8 with them for every
    // tile); the results are the same bits.
    bool odd = false;
#pragma unroll
    for (int at = 0; at < C::WN; at += 64) odd |= !plain_scale(s_scale[wn0 + at + el]);
    odd |= !plain_scale(s_scale[C::BN + wm0 + el % C::WM]);
    static_assert(C::WN % 64 == 0 && C::WM <= 64, "a lane looks at every scale of the wave");
    if (__ballot(odd) != 0) {   // wave-uniform
      if (p.out_dtype == kF32) store_rows(IC<4>{}, IC<0>{});
      else store_rows(IC<2>{}, IC<0>{});
    } else if (p.out_dtype == kF32) {
      store_rows(IC<4>{}, IC<1>{});
    } else {
      store_rows(IC<2>{}, IC<1>{});
    }
  }
}

// ---------------------------------------------------------------------------
// Few rows: the weights are streamed once from memory, and that is what bounds the kernels.  Two of them, both
// multiplying straight from the registers that memory filled; the waves of a workgroup (and S workgroups of
// one tile) split K.  Rows past the edges take out-of-range addresses and cost no traffic.  The waves' int32
// partials are added in LDS, the S partials of a tile go through the workspace to the workgroup that arrives
// last; integers, so no order changes the result.
//  * direct: one or two unquantized rows, which every workgroup quantizes for itself while its first weights
//    are on the way (1 x 4096 x 7168: 8.6 us, 3.4 TB/s of weights; 1 x 24576 x 7168: 30.3 us, 5.8 TB/s).
//  * staged: the activations pass through LDS (16 x 24576 x 7168: 29.0 us, 6.1 TB/s of weights; 64 rows 40.3,
//    4.4 TB/s; 64 x 4096 x 7168: 13.0 us).
//
// A load of weights takes whole lines of 8 rows, lane (l16, g4) the 16 bytes 16 g4 + 64 (l16 / 8) of row
// l16 % 8; two such loads (rows 0-7, rows 8-15) become two products' operands by exchanging half rows of
// lanes, one move across lanes (row_ror:8) per register.  Half lines of 16 rows, which need no exchange, stream
// at 4.0 TB/s where whole ones reach 5.9 (7168 x 16384, nothing but the loads).  Up to 32 rows the loads are
// nontemporal, as a model's weights come from memory (16 x 7168 x 16384: 23.3 us, 25.4 without; where the
// last-level cache holds them 21.7 and 20.4; more rows only lose by it, 128 x 4096 x 7168 18.0 and 20.2).
// ---------------------------------------------------------------------------
struct I8FewParams {
  const int8_t* a;        // codes, or (with X) the unquantized activations
  const float* sa;
  const int8_t* b;
  const float* sb;
  void* d;
  const int32_t* masked_m;
  int m, n, k;
  int strips, mtiles;     // tiles of a group: ceil(n / 16R) x ceil(m / 16J)
  int splits;
  int block0;             // the launch's first (tile, split) pair: under a CU cap a call is several launches
  int all_chunks, chunks;   // of K, and of one split
  int out_dtype;
  int* ws;
  unsigned* counters;
};

// The in-kernel quantizer's limits: rows, and the K that its threads hold in registers.
constexpr int kFewFusedRows = 2;
constexpr int kFewFusedK = 16384;

struct FewTile { int g, split, id, m0, n0, m_valid; };

// Block -> (group, tile, split).  The m-tiles of one strip and split are 8 blocks apart, so that they
// run on one XCD, whose L2 then serves the strip's weights to the second; m_valid = 0 past the last.
template <int BN, int BM>
__device__ __forceinline__ FewTile few_tile(const I8FewParams& p) {
  FewTile t;
  const int units = p.strips * p.splits;
  const int per_group = ((units + 7) & ~7) * p.mtiles;
  const int block = p.block0 + blockIdx.x;
  t.g = block / per_group;
  const int rest = block - t.g * per_group;
  const int run = rest / (8 * p.mtiles), in_run = rest - run * (8 * p.mtiles);
  const int mtile = in_run >> 3;
  const int unit = 8 * run + (in_run & 7);
  const int strip = unit / p.splits;
  t.split = unit - strip * p.splits;
  t.id = (t.g * p.strips + strip) * p.mtiles + mtile;
  t.m0 = mtile * BM;
  t.n0 = strip * BN;
  t.m_valid = p.m;
  if (p.masked_m != nullptr) {
    const int mv = p.masked_m[t.g];
    t.m_valid = mv < 0 ? 0 : mv > p.m ? p.m : mv;
  }
  if (unit >= units) t.m_valid = 0;
  return t;
}

// The two loads' halves exchanged: w[h] holds K bytes 64 h + 16 g4 .. + 15 of the line, of row l16.
constexpr int kNontemporal = 2;

__device__ __forceinline__ void exchange_halves(const v4i (&x)[2], v4i (&w)[2]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int x0 = x[0][c], x1 = x[1][c];
    w[0][c] = __builtin_amdgcn_update_dpp(x0, x1, 0x128, 0xf, 0xc, false);   // lanes 8-15 of each row: x1 of 8 before
    w[1][c] = __builtin_amdgcn_update_dpp(x1, x0, 0x128, 0xf, 0x3, false);   // lanes 0-7: x0 of 8 after
  }
}

// The workgroup's BM x BN sums in s_sum (rows of BN + 4, complete for its K range): added over the
// tile's splits by the workgroup that arrives last, then scaled, rounded and stored.
template <int BN, int BM, int NT, class RowScale>
__device__ __forceinline__ void few_finish(const I8FewParams& p, const FewTile& t, int* s_sum, int* s_last,
                                           RowScale row_scale) {
  constexpr int kPitch = BN + 4;
  constexpr int kChunks = BM * BN / 4;   // pieces of 4 columns
  const int tid = threadIdx.x;
  auto piece = [&](int c) { return reinterpret_cast<v4i*>(&s_sum[(c / (BN / 4)) * kPitch + 4 * (c % (BN / 4))]); };
  if (p.splits > 1) {
    // partials leave and return by device-scope accesses (no cache holds another XCD's bytes)
    const __amdgpu_buffer_rsrc_t rs_ws =
        make_rsrc(p.ws + (int64_t)t.id * p.splits * (BM * BN), (int64_t)p.splits * BM * BN * 4);
    for (int c = tid; c < kChunks; c += NT)
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, *piece(c)), rs_ws, (t.split * kChunks + c) * 16, 0,
                                             kCpolSc1);
    __builtin_amdgcn_s_waitcnt(0);   // this thread's partials have arrived
    __syncthreads();
    if (tid == 0) {
      const unsigned prev = __hip_atomic_fetch_add(p.counters + t.id, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      *s_last = prev == (unsigned)(p.splits - 1);
      if (*s_last) __hip_atomic_store(p.counters + t.id, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (!*s_last) return;
  }
  const float* sb = p.sb + (int64_t)t.g * p.n;
  constexpr int kMine = (kChunks + NT - 1) / NT;   // pieces of this thread
  v4i sum[kMine];
#pragma unroll
  for (int u = 0; u < kMine; ++u)
    if (tid + NT * u < kChunks) sum[u] = *piece(tid + NT * u);
  if (p.splits > 1) {
    // the other splits' partials, eight loads together: one by one each costs a trip to memory
    constexpr int kTogether = kMine >= 8 ? 1 : 8 / kMine;
    const __amdgpu_buffer_rsrc_t rs_ws =
        make_rsrc(p.ws + (int64_t)t.id * p.splits * (BM * BN), (int64_t)p.splits * BM * BN * 4);
    for (int o0 = 0; o0 < p.splits; o0 += kTogether) {
      v4i v[kTogether][kMine];
#pragma unroll
      for (int o = 0; o < kTogether; ++o)
#pragma unroll
        for (int u = 0; u < kMine; ++u) {
          const int c = tid + NT * u;
          const uint32_t out = o0 + o < p.splits && o0 + o != t.split && c < kChunks ? 0u : 0xFFFFFFF0u;   // zeros
          v[o][u] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(
                                                rs_ws, (uint32_t)(((o0 + o) * kChunks + c) * 16) | out, 0, kCpolSc1));
        }
#pragma unroll
      for (int o = 0; o < kTogether; ++o)
#pragma unroll
        for (int u = 0; u < kMine; ++u) sum[u] += v[o][u];
    }
  }
#pragma unroll
  for (int u = 0; u < kMine; ++u) {
    const int c = tid + NT * u;
    const int row = t.m0 + c / (BN / 4), col = t.n0 + 4 * (c % (BN / 4));
    const int count = p.n - col;
    if (c >= kChunks || row >= t.m_valid || count <= 0) continue;
    const float sr = row_scale(row);
    float sc[4], v[4];   // (all four loads before the first is used: past the edge the last column's)
#pragma unroll
    for (int r = 0; r < 4; ++r) sc[r] = sb[r < count ? col + r : p.n - 1];
    bool odd = false;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      odd |= !is_normal(sr * sc[r]);
      v[r] = (float)sum[u][r] * (sr * sc[r]);
    }
    if (__ballot(odd) != 0) {   // wave-uniform; the same value for products of scales that are normal
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = scaled_sum(sum[u][r], sr, sc[r]);
    }
    store_out4(p.d, p.out_dtype, ((int64_t)t.g * p.m + row) * p.n + col, v, count);
  }
}

template <int R, int U, int W, class X>
__global__ __launch_bounds__(64 * W) void gemm_int8_direct_kernel(I8FewParams p) {
  constexpr int NT = 64 * W;
  constexpr int BN = 16 * R, BM = 16;
  constexpr int kPitch = BN + 4;
  constexpr int kHold = 2;   // 8-element pieces of a row per thread: k <= 16 NT
  __shared__ __attribute__((aligned(16))) int s_sum[BM * kPitch];
  __shared__ uint32_t s_max[kFewFusedRows * W];
  __shared__ int s_last;
  extern __shared__ __attribute__((aligned(16))) uint8_t s_codes[];   // (m, k) codes
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g4 = lane >> 4;
  const FewTile t = few_tile<BN, BM>(p);
  if (t.m0 >= t.m_valid) return;   // uniform, and so for every split of the tile

  const __amdgpu_buffer_rsrc_t rs_b = make_rsrc(p.b + (int64_t)t.n0 * p.k, (int64_t)(p.n - t.n0) * p.k);
  const int line = 16 * g4 + 64 * (l16 >> 3);
  const uint32_t row_off = (uint32_t)(l16 & 7) * (uint32_t)p.k + (uint32_t)line;
  // the workgroup's `count` chunks from c0 on, a line of each for every wave
  const int c0 = t.split * p.chunks;
  const int count = c0 + p.chunks < p.all_chunks ? p.chunks : p.all_chunks - c0;
  auto byte_of = [&](int i) { return (c0 + i) * (128 * W) + 128 * wave; };

  struct Set { v4i b[U][R][2]; };
  // U lines; pieces past K and past the workgroup's range take an out-of-range offset and read zeros
  auto load = [&](Set& v, int i) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = byte_of(i + u);
      const uint32_t out = i + u < count && at + line < p.k ? 0u : 0xFFFFFFF0u;
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          v.b[u][r][h] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(
                                                     rs_b, (row_off + (uint32_t)(16 * r + 8 * h) * (uint32_t)p.k) | out,
                                                     at, kNontemporal));
    }
  };
  v4i acc[R];
#pragma unroll
  for (int i = 0; i < R; ++i) acc[i] = v4i{0, 0, 0, 0};
  auto multiply = [&](const Set& v, int i) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v4i act[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = byte_of(i + u) + 64 * h + 16 * g4;
        act[h] = l16 < p.m && i + u < count && at < p.k ? *reinterpret_cast<const v4i*>(s_codes + l16 * p.k + at)
                                                        : v4i{0, 0, 0, 0};
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        v4i w[2];
        exchange_halves(v.b[u][r], w);
#pragma unroll
        for (int h = 0; h < 2; ++h) acc[r] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[h], act[h], acc[r], 0, 0, 0);
      }
    }
  };

  // every workgroup quantizes the few rows for itself while its first weights are on the way
  const X* x = reinterpret_cast<const X*>(p.a);
  Raw8<X> held[kFewFusedRows][kHold];
#pragma unroll
  for (int r = 0; r < kFewFusedRows; ++r)
#pragma unroll
    for (int h = 0; h < kHold; ++h)
      if (r < p.m && 8 * (tid + NT * h) < p.k) held[r][h] = load8(x + (int64_t)r * p.k + 8 * (tid + NT * h));
  Set even, odd;
  load(even, 0);
  for (int i = tid; i < BM * kPitch; i += NT) s_sum[i] = 0;
#pragma unroll
  for (int r = 0; r < kFewFusedRows; ++r) {
    if (r >= p.m) break;   // uniform
    uint32_t amax = 0;
#pragma unroll
    for (int h = 0; h < kHold; ++h) {
      if (8 * (tid + NT * h) < p.k) {
        float v[8];
        widen8(held[r][h], v);
#pragma unroll
        for (int c = 0; c < 8; ++c) amax = umax(amax, abs_bits(v[c]));
      }
    }
    amax = wave_max_u32(amax);
    if (lane == 0) s_max[r * W + wave] = amax;
  }
  __syncthreads();
  float scale[kFewFusedRows];
#pragma unroll
  for (int r = 0; r < kFewFusedRows; ++r) {
    if (r >= p.m) break;   // uniform
    uint32_t amax = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) amax = umax(amax, s_max[r * W + w]);
    scale[r] = int8_scale(amax);
#pragma unroll
    for (int h = 0; h < kHold; ++h) {
      if (8 * (tid + NT * h) < p.k) {
        float v[8];
        widen8(held[r][h], v);
        *reinterpret_cast<u32x2_t*>(s_codes + r * p.k + 8 * (tid + NT * h)) =
            u32x2_t{pack4_int8(v, scale[r]), pack4_int8(v + 4, scale[r])};
      }
    }
  }
  __syncthreads();
  for (int i = 0; i < count; i += 2 * U) {
    load(odd, i + U);
    multiply(even, i);
    if (i + U >= count) break;   // uniform
    load(even, i + 2 * U);
    multiply(odd, i + U);
  }

  // the waves' partials: integer atomics, whose order does not matter
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (l16 < p.m) atomicAdd(&s_sum[l16 * kPitch + 16 * i + 4 * g4 + r], acc[i][r]);
  __syncthreads();
  few_finish<BN, BM, NT>(p, t, s_sum, &s_last, [&](int row) {
    float sr = scale[0];
#pragma unroll
    for (int r = 1; r < kFewFusedRows; ++r) sr = row == r ? scale[r] : sr;
    return sr;
  });
}

// NS x KS = 8 waves on 16 R NS weight rows and 16 J activation rows: wave (ns, kh) multiplies line kh of each
// chunk of KS lines with its R fragment rows.
//
// Each strip starts its K range elsewhere: rows a power of two apart meet in the same channels otherwise
// (16 x 7168 x 16384: 28.3 us, 23.5 so; other lengths are the same either way).
//
// Activations: through registers into one of two LDS buffers, one barrier a chunk, D - 1 chunks ahead.  They
// come from L2, but a CU's loads return in order, behind the weights' trips to memory: with R NS small the
// kernel waits for them (64 x 24576 x 7168: strips of 32 rows 51 us, 96 rows 38.7).
constexpr int kStWaves = 8;

template <int NS, int R, int J, int D, int W = kStWaves>
__global__ __launch_bounds__(64 * W) void gemm_int8_staged_kernel(I8FewParams p) {
  constexpr int KS = W / NS, NT = 64 * W;
  constexpr int BN = 16 * R * NS, BM = 16 * J;
  constexpr int kChunk = 128 * KS;
  constexpr int kPitch = kChunk + 16;   // 16 rows of one 16-byte column fall in different banks
  constexpr int kRowPieces = kChunk / 16;
  constexpr int kPieces = (BM * kRowPieces + NT - 1) / NT;   // 16-byte pieces per thread and chunk
  constexpr int kBuf = BM * kPitch;
  constexpr int kSumPitch = BN + 4;
  constexpr int kLds = 2 * kBuf > BM * kSumPitch * 4 ? 2 * kBuf : BM * kSumPitch * 4;
  constexpr int kPolicy = J <= 2 ? kNontemporal : 0;
  __shared__ __attribute__((aligned(16))) uint8_t smem[kLds];
  __shared__ int s_last;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ns = wave % NS, kh = wave / NS;
  const int l16 = lane & 15, g4 = lane >> 4;
  const FewTile t = few_tile<BN, BM>(p);
  if (t.m0 >= t.m_valid) return;   // uniform, and so for every split of the tile

  const __amdgpu_buffer_rsrc_t rs_b = make_rsrc(p.b + ((int64_t)t.g * p.n + t.n0) * p.k, (int64_t)(p.n - t.n0) * p.k);
  const __amdgpu_buffer_rsrc_t rs_a = make_rsrc(p.a + ((int64_t)t.g * p.m + t.m0) * p.k, (int64_t)(t.m_valid - t.m0) * p.k);
  // the workgroup's `count` chunks from c0 on, the strip's own one first
  const int c0 = t.split * p.chunks;
  const int count = c0 + p.chunks < p.all_chunks ? p.chunks : p.all_chunks - c0;
  const int first = (t.n0 / BN) % count;

  struct Set { u32x4 act[kPieces]; v4i b[R][2]; };
  const int line = 128 * kh + 16 * g4 + 64 * (l16 >> 3);
  const uint32_t row_off = (uint32_t)(16 * R * ns + (l16 & 7)) * (uint32_t)p.k + (uint32_t)line;
  auto load = [&](Set& v, int i) {   // the i-th chunk; past the last, and past K, zeros
    const int at = (c0 + (i + first < count ? i + first : i + first - count)) * kChunk;
    const uint32_t out_b = i < count && at + line < p.k ? 0u : 0xFFFFFFF0u;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int u = 0; u < 2; ++u)
        v.b[r][u] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(
                                                rs_b, (row_off + (uint32_t)(16 * r + 8 * u) * (uint32_t)p.k) | out_b, at,
                                                kPolicy));
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int piece = tid + NT * u, row = piece / kRowPieces, col = 16 * (piece % kRowPieces);
      const uint32_t out = i < count && at + col < p.k && row < BM ? 0u : 0xFFFFFFF0u;
      v.act[u] = __builtin_amdgcn_raw_buffer_load_b128(rs_a, ((uint32_t)row * (uint32_t)p.k + (uint32_t)col) | out, at, 0);
    }
  };
  auto store_act = [&](const Set& v, int parity) {
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int piece = tid + NT * u, row = piece / kRowPieces, col = 16 * (piece % kRowPieces);
      if (BM * kRowPieces >= NT || row < BM)
        *reinterpret_cast<u32x4*>(smem + parity * kBuf + row * kPitch + col) = v.act[u];
    }
  };
  v4i acc[R][J];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int j = 0; j < J; ++j) acc[r][j] = v4i{0, 0, 0, 0};
  auto multiply = [&](const Set& v, int parity) {
    const uint8_t* base = smem + parity * kBuf + l16 * kPitch + 128 * kh + 16 * g4;
    v4i w[R][2];
#pragma unroll
    for (int r = 0; r < R; ++r) exchange_halves(v.b[r], w[r]);
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const v4i fa = *reinterpret_cast<const v4i*>(base + 16 * j * kPitch + 64 * u);
#pragma unroll
        for (int r = 0; r < R; ++r) acc[r][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[r][u], fa, acc[r][j], 0, 0, 0);
      }
  };

  Set set[D];
#pragma unroll
  for (int d = 0; d < D - 1; ++d) load(set[d], d);
  constexpr int kUnroll = D % 2 ? 2 * D : D;   // both the set and the buffer of a step are fixed
  for (int i0 = 0; i0 < count; i0 += kUnroll) {
#pragma unroll
    for (int d = 0; d < kUnroll; ++d) {
      if (i0 + d >= count) break;   // uniform
      store_act(set[d % D], d & 1);
      load(set[(d + D - 1) % D], i0 + d + D - 1);
      __syncthreads();   // this chunk is in its buffer; every wave is done with the one before
      multiply(set[d % D], d & 1);
    }
  }

  __syncthreads();   // the buffers become the sums
  int* s_sum = reinterpret_cast<int*>(smem);
#pragma unroll
  for (int h = 0; h < KS; ++h) {
    if (kh == h) {
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int r = 0; r < R; ++r) {
          v4i* at = reinterpret_cast<v4i*>(&s_sum[(16 * j + l16) * kSumPitch + 16 * (R * ns + r) + 4 * g4]);
          *at = h == 0 ? acc[r][j] : *at + acc[r][j];
        }
    }
    __syncthreads();
  }
  few_finish<BN, BM, NT>(p, t, s_sum, &s_last, [&](int row) { return p.sa[(int64_t)t.g * p.m + row]; });
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
using I8Square = I8Cfg<256, 256, 128, 64, 1>;
using I8Small = I8Cfg<128, 128, 64, 32, 2>;
enum I8Tile : int { kSquare = 0, kSmall, kTiles };

struct FewPlan {
  int ns, r, j, waves, unit;   // unit: K bytes of a chunk, one or more lines for each wave
  int bn, bm;
  int strips, mtiles, splits;
  int all_chunks, chunks;   // of K, and of one split
  int64_t tiles;
  size_t ws_bytes;
};

// DG_PLAN: a measurement override of the plan (read at every call, like DG_DEBUG), comma-separated:
// "tile=256x256" or "tile=128x128", or "strip=32", 64, 96 or 128 (weight rows of a strip; forms and sizes that
// may run on the few-row kernel), and "splits=S" where the call may split K.  Anything else is ignored; the
// workspace queries see the same plan.
struct I8Override { int bn = 0, bm = 0, strip = 0, splits = 0; };
static I8Override plan_override() {
  I8Override o;
  const char* e = std::getenv("DG_PLAN");
  for (const char* q = e; q != nullptr && *q;) {
    if (std::sscanf(q, "tile=%dx%d", &o.bn, &o.bm) == 2 || std::sscanf(q, "strip=%d", &o.strip) == 1 ||
        std::sscanf(q, "splits=%d", &o.splits) == 1) {}
    q = std::strchr(q, ',');
    if (q != nullptr) ++q;
  }
  if (o.splits < 0) o.splits = 0;
  if (o.splits > kMaxSplits) o.splits = kMaxSplits;
  return o;
}

// The tiles and the split of K into at most `want` parts, none empty.
static void few_grid(FewPlan* f, int64_t m, int64_t n, int64_t k, int64_t groups, int64_t want) {
  f->bn = 16 * f->r * f->ns;
  f->bm = 16 * f->j;
  f->strips = (int)((n + f->bn - 1) / f->bn);
  f->mtiles = (int)((m + f->bm - 1) / f->bm);
  f->tiles = (int64_t)f->strips * f->mtiles * groups;
  f->all_chunks = (int)((k + f->unit - 1) / f->unit);
  f->chunks = (int)((f->all_chunks + want - 1) / want);
  f->splits = (f->all_chunks + f->chunks - 1) / f->chunks;
  f->ws_bytes = f->splits > 1 ? kCounterBytes + (size_t)f->tiles * f->splits * f->bn * f->bm * 4 : 0;
}

// The kernel that quantizes its rows itself.  What the choices measured: waves a workgroup (they share K):
// 1 x 24576 x 1536 takes 9.7 us with 4, 12.2 with 8, 17.1 with 16; 1 x 4096 x 7168 8.5 with 8, 9.3 with 16;
// the row has to fit the threads' registers, 1024 elements a wave.  32 weight rows a workgroup where that still
// gives ~3/4 of a workgroup per CU: 1 x 24576 x 7168 30.6 us, 36.2 with 16; 1 x 4096 x 7168 10.6 and 8.5.  K is not
// split over workgroups: each would quantize the row again (1 x 2112 x 7168 7.8 us whole, 10.8 in two).
static FewPlan direct_plan(int64_t m, int64_t n, int64_t k, int num_cus) {
  FewPlan f{};
  f.ns = 1;
  f.j = 1;
  f.r = n >= (int64_t)24 * num_cus ? 2 : 1;
  f.waves = k <= 4096 ? 4 : k <= 8192 ? 8 : 16;
  f.unit = 128 * f.waves;
  few_grid(&f, m, n, k, 1, 1);
  return f;
}

// Joining K splits: three trips to memory in turn, and a tile's partials through one workgroup at 70 B/ns.
static double few_split_time(const FewPlan& f) {
  return f.splits > 1 ? 1.5 + 0.2 * f.splits + f.splits * (double)(f.bn * f.bm * 4) / 70e3 : 0.0;
}

// Time estimate (microseconds, MI355X): a fixed part, and per K byte what the fullest CU's workgroups load and
// multiply, fitted to 16, 32 and 64 rows by 4096 x 7168 ... 24576 x 7168 over every tile and split below.
static double few_time(const FewPlan& f, int layout, int64_t n, int64_t k, int64_t groups, int num_cus) {
  const double c = (double)((f.tiles * f.splits + num_cus - 1) / num_cus);
  const double wide = f.j == 8 ? 1.1 : 1.0;   // (fitted to 128 rows: more sums and pieces in each thread's registers)
  const double per_byte = wide * (f.bn * (0.0322 + 0.000183 * f.bm) + 0.0098 * f.bm);
  const double loads = c * 1e-3 * f.chunks * f.unit * per_byte, memory = (double)groups * n * k / 5.9e6;
  const double shared = layout == kDense ? 0.17 * (double)n * k / 5.6e6 : 0.0;   // what of memory nothing hides
  return 4.8 + shared + (loads > memory ? loads : memory) + few_split_time(f);
}

// Strips of 32 to 128 weight rows: wide ones read the activations less often, narrow ones need less of a K
// split to fill the chip (its join costs 2-4 us).  64 rows, fastest split: 24576 x 7168 51.1 us with 32, 45
// with 64, 38.7 with 96, 40.7 with 128; 4096 x 7168 14.2, 13.5, 16.4, 17.6; 7168 x 2048 8.3, 10.2, 12.5, 12.6.
// D: 3 pays where a wave keeps one fragment row and a workgroup has the chunks (16 x 4096 x 7168 10.8 -> 10.2 us;
// 64 x 7168 x 2048, four chunks, 8.3 -> 9.1).
static FewPlan staged_plan(int layout, int64_t m, int64_t n, int64_t k, int64_t groups, int num_cus, bool allow_split,
                           const I8Override& o) {
  static constexpr struct { int ns, r; } kStrips[] = {{2, 1}, {4, 1}, {2, 3}, {4, 2}};
  FewPlan best{};
  double best_us = 0.0;
  for (const auto& strip : kStrips) {
    FewPlan f{};
    f.j = m <= 16 ? 1 : m <= 32 ? 2 : m <= 64 ? 4 : 8;
    if (f.j == 8 && strip.r == 3) continue;   // (not built: 128 rows of its chunks fill the LDS)
    f.ns = strip.ns; f.r = strip.r;
    if (o.strip != 0 && o.strip != 16 * f.r * f.ns) continue;
    // up to 16 rows and long K: one strip of two fragment rows, K over all eight waves (16 x 7168 x 16384
    // 25.3 -> 23.1 us; 16 x 4096 x 7168 10.2 -> 10.5)
    if (f.j == 1 && f.ns * f.r == 2 && k > 8192) f.ns = 1, f.r = 2;
    f.waves = f.j == 8 && f.ns == 2 ? kStWaves / 2 : kStWaves;   // (two workgroups' buffers fit a CU)
    f.unit = 128 * (f.waves / f.ns);
    bool forced = false;
    if (o.splits != 0 && allow_split) {
      few_grid(&f, m, n, k, groups, o.splits);
      forced = f.tiles <= kMaxCounterTiles;
    }
    for (int want = 1; want <= (forced ? 1 : kMaxSplits); ++want) {
      if (!forced) few_grid(&f, m, n, k, groups, want);
      if (want > 1 && (!allow_split || f.tiles > kMaxCounterTiles || f.chunks < 2)) break;
      const double us = few_time(f, layout, n, k, groups, num_cus);
      if (best_us == 0.0 || us <= best_us) best = f, best_us = us;   // (of equals, bound by memory, the widest)
    }
  }
  return best;
}

template <int J>
static const void* staged_fn_of(const FewPlan& f) {
  const bool deep = f.chunks >= 7;
  void (*fn)(I8FewParams);
  if (f.ns == 4)
    fn = f.r == 2 ? gemm_int8_staged_kernel<4, 2, J, 2> : deep ? gemm_int8_staged_kernel<4, 1, J, J < 8 ? 3 : 2>
                                                              : gemm_int8_staged_kernel<4, 1, J, 2>;
  else if constexpr (J == 8)
    fn = gemm_int8_staged_kernel<2, 1, 8, 2, kStWaves / 2>;
  else
    fn = f.ns == 1 ? gemm_int8_staged_kernel<1, 2, 1, 2> : f.r == 3 ? gemm_int8_staged_kernel<2, 3, J, 2>
         : deep ? gemm_int8_staged_kernel<2, 1, J, 3> : gemm_int8_staged_kernel<2, 1, J, 2>;
  return reinterpret_cast<const void*>(fn);
}
static const void* staged_fn(const FewPlan& f) {
  return f.j == 1 ? staged_fn_of<1>(f) : f.j == 2 ? staged_fn_of<2>(f) : f.j == 4 ? staged_fn_of<4>(f) : staged_fn_of<8>(f);
}

template <class X>
static const void* direct_fn_of(const FewPlan& f) {
  void (*fn)(I8FewParams);
  if (f.r == 1)
    fn = f.waves == 4 ? gemm_int8_direct_kernel<1, 4, 4, X> : f.waves == 8 ? gemm_int8_direct_kernel<1, 4, 8, X>
                                                                           : gemm_int8_direct_kernel<1, 4, 16, X>;
  else
    fn = f.waves == 4 ? gemm_int8_direct_kernel<2, 2, 4, X> : f.waves == 8 ? gemm_int8_direct_kernel<2, 2, 8, X>
                                                                           : gemm_int8_direct_kernel<2, 2, 16, X>;
  return reinterpret_cast<const void*>(fn);
}
static const void* direct_fn(const FewPlan& f, int dtype) {
  return dtype == kF32 ? direct_fn_of<float>(f) : dtype == kBf16 ? direct_fn_of<Bf16>(f) : direct_fn_of<_Float16>(f);
}

static int64_t few_blocks(const FewPlan& f, int64_t groups) {
  return groups * ((((int64_t)f.strips * f.splits + 7) & ~(int64_t)7) * f.mtiles);
}

// Every (tile, split) pair is a workgroup.  dg_set_num_cus keeps a call to fewer CUs than the device has by
// launching no more of them at once than those hold, one launch after the other: the pairs do not wait for each
// other, whichever of them arrives last joins a tile's splits.  (A loop over pairs in the kernel would do it in
// one launch, but takes 10 to 40 registers more of the uncapped call, and a wave per SIMD with them.)
static int64_t few_workgroups(const FewPlan& f, const void* fn, size_t lds, int64_t groups, int num_cus) {
  const int64_t blocks = few_blocks(f, groups);
  if (num_cus >= device_cu_count()) return blocks;
  int occ = 0;
  if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&occ, fn, 64 * f.waves, lds) != hipSuccess || occ < 1) {
    (void)hipGetLastError();
    occ = 1;
  }
  int64_t most = (int64_t)num_cus * occ;
  if (most > 8) most = most / 8 * 8;   // (few_tile's runs of 8 stay on their XCDs)
  return blocks < most ? blocks : most;
}

static int launch_few(const FewPlan& f, const void* fn, I8FewParams p, size_t lds, int64_t groups, int64_t workgroups,
                      void* counters, void* partials, hipStream_t stream) {
  p.strips = f.strips; p.mtiles = f.mtiles; p.splits = f.splits;
  p.all_chunks = f.all_chunks; p.chunks = f.chunks;
  p.counters = static_cast<unsigned*>(counters);
  p.ws = static_cast<int*>(partials);
  const int64_t blocks = few_blocks(f, groups);
  if (blocks * 64 * f.waves > 0xffffffffLL) return set_error(kUnsupported, "int8 gemm: too many output tiles");
  for (int64_t at = 0; at < blocks; at += workgroups) {
    p.block0 = (int)at;
    void* args[] = {&p};
    const hipError_t e = hipLaunchKernel(fn, dim3((unsigned)(blocks - at < workgroups ? blocks - at : workgroups)),
                                         dim3(64 * f.waves), args, lds, stream);
    if (e != hipSuccess) return set_error(kHip, "int8 gemm launch: %s", hipGetErrorString(e));
  }
  return kOk;
}

// Time estimates (microseconds, MI355X, 256 CUs).  A workgroup's K block takes longer the more of them run (they
// share caches and power); a tile costs a fixed part as well (first loads, stores); a K split sends its partials
// out and back.  Fitted, with few_time's fixed part, to timings of every choice on 154 shapes of 72 to 1024
// rows, 512 to 24576 columns and K from 512 to 16384: the plan takes 1.0% longer than the fastest choice on
// average, 19% at worst (777 x 2112 x 7168: 34.7 us in three parts, 29.1 in four).  The grouped forms use the same
// constants without a fit of their own.
struct TileModel { int bn, bm, occ; double fixed, alone, busy; };
constexpr TileModel kTileModel[kTiles] = {
    {I8Square::BN, I8Square::BM, I8Square::OCC, 7.0, 0.9, 1.6},
    {I8Small::BN, I8Small::BM, I8Small::OCC, 3.75, 0.59, 1.11}};

static double split_time(int splits, double partial_bytes) { return 0.3 + 0.7 * splits + 0.146e-6 * partial_bytes; }

struct TilePlan {
  int tile;
  int tiles_m, tiles_n, splits, kb_per_split;
  int64_t items;
  size_t ws_bytes;
  double us;
};

static TilePlan tile_choice(int tile, int splits, int layout, int64_t m, int64_t n, int64_t k, int64_t groups,
                            int num_cus) {
  const TileModel& c = kTileModel[tile];
  const int kb_total = (int)((k + kI8Block - 1) / kI8Block);
  TilePlan t{};
  t.tile = tile;
  t.tiles_m = (int)((m + c.bm - 1) / c.bm);
  t.tiles_n = (int)((n + c.bn - 1) / c.bn);
  t.kb_per_split = (kb_total + splits - 1) / splits;
  t.splits = (kb_total + t.kb_per_split - 1) / t.kb_per_split;   // no empty split
  double tiles = (double)t.tiles_m * t.tiles_n;
  // masked: the counts are on the device; any of 0 .. m rows alike use (m-blocks + 1) / 2 blocks on average
  if (layout == kMasked) tiles = (double)groups * 0.5 * (t.tiles_m + 1) * t.tiles_n;
  // A tile that spans two experts runs twice, one pass after the other in its workgroup.  Counted as another tile it
  // costs too much where the tiles fill one round: 4096 x 4096 x 7168, four experts of whole tiles, takes 98 us on
  // 256x256 tiles and 123 on the 128x128 ones that are chosen (every edge inside a tile: 126 and 127).
  if (layout == kContiguous && c.bm > kGroup) {
    const int64_t edges = groups - 1 < t.tiles_m ? groups - 1 : t.tiles_m;
    tiles += (double)edges * t.tiles_n;
  }
  t.items = (int64_t)t.tiles_m * t.tiles_n * t.splits * (layout == kMasked ? groups : 1);
  const double items = tiles * t.splits, slots = (double)c.occ * num_cus;
  const double full = (double)(int64_t)(items / slots), rest = items - full * slots;
  t.us = full * (c.fixed + t.kb_per_split * c.busy);
  if (rest > 0) t.us += c.fixed + t.kb_per_split * (c.alone + (c.busy - c.alone) * rest / slots);
  // the weights come from memory at 5.6 TB/s at best, and at 17 GB/s for each workgroup
  const double rate = items * 0.017e6 < 5.6e6 ? items * 0.017e6 : 5.6e6;
  const double weights = c.fixed + (double)n * k * (layout == kDense ? 1 : groups) / rate;
  if (t.us < weights) t.us = weights;
  if (layout == kDense) t.us += 0.58 * (double)n * k / 5.6e6;   // what the products do not hide of it
  if (t.splits > 1) {
    const double partials = items * (double)(c.bm * c.bn) * 4;
    t.us += split_time(t.splits, partials);
    t.ws_bytes = kCounterBytes + (size_t)partials;
  }
  return t;
}

// The fastest of the tiles and, for the normal form with a workspace, of the K splits that keep at least 4
// K blocks and give each CU about one workgroup (256 x 4096 x 7168 on 128x128 tiles: split in four 22.6 us,
// in eight, two workgroups a CU, 29.6), or two with at most three splits (64 x 24576 x 7168: 56.4 us whole,
// 45.5 in two).
static TilePlan tile_plan(int layout, int64_t m, int64_t n, int64_t k, int64_t groups, int num_cus, bool allow_split,
                          const I8Override& o) {
  TilePlan best{};
  const bool may_split = layout == kDense && allow_split;
  for (int tile = 0; tile < kTiles; ++tile) {
    if (o.bn != 0 && (o.bn != kTileModel[tile].bn || o.bm != kTileModel[tile].bm)) continue;
    if (o.splits != 0 && may_split) {
      const TilePlan t = tile_choice(tile, o.splits, layout, m, n, k, groups, num_cus);
      if (t.items / t.splits <= kMaxCounterTiles) {
        if (best.items == 0 || t.us < best.us) best = t;
        continue;
      }
    }
    for (int splits = 1; splits <= kMaxSplits; ++splits) {
      const TilePlan t = tile_choice(tile, splits, layout, m, n, k, groups, num_cus);
      if (splits > 1) {
        const bool crowded = t.items > (int64_t)(splits <= 3 ? kTileModel[tile].occ : 1) * num_cus;
        if (!may_split || t.kb_per_split < 4 || crowded || t.items / t.splits > kMaxCounterTiles) break;
        if (t.splits != splits) continue;   // the same as a smaller request
      }
      if (best.items == 0 || t.us < best.us) best = t;
    }
  }
  return best;
}

template <int LAYOUT>
static const void* tile_fn_of(int tile) {
  void (*fn)(I8Params) = tile == kSquare ? gemm_int8_kernel<I8Square, LAYOUT> : gemm_int8_kernel<I8Small, LAYOUT>;
  return reinterpret_cast<const void*>(fn);
}
static const void* tile_fn(int layout, int tile) {
  return layout == kMasked ? tile_fn_of<kMasked>(tile) : layout == kContiguous ? tile_fn_of<kContiguous>(tile)
                                                                              : tile_fn_of<kDense>(tile);
}

// The most rows that may run on the few-row kernel (more never measured faster).
constexpr int64_t kFewRowsMost = 1024;

struct I8Plan {
  bool few;
  FewPlan f;
  TilePlan t;
  size_t ws_bytes() const { return few ? f.ws_bytes : t.ws_bytes; }
};

static I8Plan int8_plan(int layout, int64_t m, int64_t n, int64_t k, int64_t groups, int num_cus, bool allow_split) {
  I8Override o = plan_override();
  bool known = false;
  for (const TileModel& t : kTileModel) known |= o.bn == t.bn && o.bm == t.bm;
  if (!known) o.bn = o.bm = 0;
  const bool may_few = layout != kContiguous && m <= kFewRowsMost;
  const bool strip = o.strip == 32 || o.strip == 64 || (o.strip == 96 && m <= 64) || o.strip == 128;
  if (!strip || !may_few || o.bn != 0) o.strip = 0;
  I8Plan p{};
  if (may_few) p.f = staged_plan(layout, m, n, k, groups, num_cus, allow_split, o);
  p.t = tile_plan(layout, m, n, k, groups, num_cus, allow_split, o);
  p.few = may_few && o.bn == 0 && (o.strip != 0 || few_time(p.f, layout, n, k, groups, num_cus) < p.t.us);
  return p;
}

// "BNxBM/Wwaves/splitS", the few-row kernel's after "strip".
static void plan_name(const I8Plan& p, char* buf, size_t len) {
  const TileModel& t = kTileModel[p.t.tile];
  if (p.few) snprintf(buf, len, "strip%dx%d/%dwaves/split%d", p.f.bn, p.f.bm, p.f.waves, p.f.splits);
  else snprintf(buf, len, "%dx%d/%dwaves/split%d", t.bn, t.bm, I8Square::kWaves, p.t.splits);
}

void gemm_int8_config_name(int layout, int64_t m, int64_t n, int64_t k, int64_t groups, int num_cus, char* buf,
                           size_t len) {
  plan_name(int8_plan(layout, m, n, k, layout == kDense ? 1 : groups, num_cus, layout != kContiguous), buf, len);
}

// DG_DEBUG: one line per launch with the plan.
static void log_plan(int layout, const char* name, int64_t m, int64_t n, int64_t k, int64_t groups, int64_t workgroups,
                     size_t need, size_t ws_bytes) {
  static const char* const kNames[] = {"normal", "contiguous", "masked"};
  std::fprintf(stderr, "[dg] int8 gemm %s m=%lld n=%lld k=%lld groups=%lld: %s workgroups=%lld workspace=%zu/%zu bytes\n",
               kNames[layout], (long long)m, (long long)n, (long long)k, (long long)groups, name, (long long)workgroups,
               need, ws_bytes);
}

int launch_quant_int8(const void* x, int dtype, int64_t rows, int64_t k, int8_t* q, float* s, hipStream_t stream);
int launch_check_contiguous(const int32_t* m_indices, int64_t m, int64_t groups, hipStream_t stream);

// One group may be the normal form or a masked buffer, whose plans differ: what either of them takes (only the
// few-row kernel splits the masked one, so more rows need no second plan).
size_t int8_workspace_size(int64_t m, int64_t n, int64_t k, int64_t groups, int num_cus) {
  size_t need = 0;
  if (groups == 1) need = int8_plan(kDense, m, n, k, 1, num_cus, true).ws_bytes();
  if (groups > 1 || m <= kFewRowsMost) {
    const size_t masked = int8_plan(kMasked, m, n, k, groups, num_cus, true).ws_bytes();
    if (masked > need) need = masked;
  }
  return need;
}

// `counters` and `partials`: the K split's workspace, or null for none; ws_bytes: what the caller gave, for the log.
static int launch_planned(int layout, const int8_t* a, const float* sa, const int8_t* b, const float* sb, void* d,
                          int out_dtype, const int32_t* m_indices, const int32_t* masked_m, int64_t groups, int64_t m,
                          int64_t n, int64_t k, const I8Plan& plan, void* counters, void* partials, size_t ws_bytes,
                          hipStream_t stream, int num_cus) {
  const int64_t slots = (int64_t)num_cus * kTileModel[plan.t.tile].occ;
  const void* fn = plan.few ? staged_fn(plan.f) : tile_fn(layout, plan.t.tile);
  const int64_t workgroups = plan.few               ? few_workgroups(plan.f, fn, 0, groups, num_cus)
                             : plan.t.items < slots ? plan.t.items
                                                    : slots;
  if (debug_enabled()) {
    char name[64];
    plan_name(plan, name, sizeof(name));
    log_plan(layout, name, m, n, k, groups, workgroups, plan.ws_bytes(), ws_bytes);
    if (layout == kContiguous) {   // (the kernel itself carries no check)
      const int r = launch_check_contiguous(m_indices, m, groups, stream);
      if (r != kOk) return r;
    }
  }
  if (plan.few) {
    I8FewParams p{};
    p.a = a; p.sa = sa; p.b = b; p.sb = sb; p.d = d; p.masked_m = masked_m;
    p.m = (int)m; p.n = (int)n; p.k = (int)k; p.out_dtype = out_dtype;
    return launch_few(plan.f, fn, p, 0, groups, workgroups, counters, partials, stream);
  }
  const TilePlan& t = plan.t;
  I8Params p{};
  p.a = a; p.sa = sa; p.b = b; p.sb = sb; p.d = d;
  p.m_indices = m_indices; p.masked_m = masked_m;
  p.m = (int)m; p.n = (int)n; p.k = (int)k;
  p.groups = (int)groups;
  p.kb_total = (int)((k + kI8Block - 1) / kI8Block);
  p.tiles_m = t.tiles_m; p.tiles_n = t.tiles_n;
  p.splits = t.splits; p.kb_per_split = t.kb_per_split;
  p.out_dtype = out_dtype;
  p.counters = static_cast<unsigned*>(counters);
  p.ws = static_cast<int*>(partials);
  if (t.items > 0x7fffffffLL) return set_error(kUnsupported, "int8 gemm: too many output tiles");
  void* args[] = {&p};
  const hipError_t e = hipLaunchKernel(fn, dim3((unsigned)workgroups), dim3(I8Square::kThreads), args, 0, stream);
  return e == hipSuccess ? kOk : set_error(kHip, "int8 gemm launch: %s", hipGetErrorString(e));
}

int launch_gemm_int8(int layout, const int8_t* a, const float* sa, const int8_t* b, const float* sb, void* d,
                     int out_dtype, const int32_t* m_indices, const int32_t* masked_m, int64_t groups, int64_t m,
                     int64_t n, int64_t k, void* ws, size_t ws_bytes, hipStream_t stream, int num_cus) {
  I8Plan plan = int8_plan(layout, m, n, k, groups, num_cus, ws != nullptr);
  if (ws_bytes < plan.ws_bytes()) plan = int8_plan(layout, m, n, k, groups, num_cus, false);
  return launch_planned(layout, a, sa, b, sb, d, out_dtype, m_indices, masked_m, groups, m, n, k, plan, ws,
                        static_cast<uint8_t*>(ws) + kCounterBytes, ws_bytes, stream, num_cus);
}

// In-call quantization.  Up to kFewFusedRows rows of at most kFewFusedK elements are quantized by the
// product's own workgroups; more rows by a launch of the quantizer into the workspace: the counter prefix,
// the codes, the scales (256-byte pieces), then the K split's partials.
static size_t align256(size_t v) { return (v + 255) / 256 * 256; }
static bool few_fused(int64_t m, int64_t k) { return m <= kFewFusedRows && k <= kFewFusedK; }

size_t int8_act_quant_workspace_size(int64_t m, int64_t n, int64_t k, int num_cus) {
  if (few_fused(m, k)) return 0;
  const size_t split = int8_plan(kDense, m, n, k, 1, num_cus, true).ws_bytes();
  return kCounterBytes + align256((size_t)(m * k)) + align256((size_t)m * 4) + (split > 0 ? split - kCounterBytes : 0);
}

int launch_gemm_int8_act_quant(const void* x, int dtype, const int8_t* b, const float* sb, void* d, int out_dtype,
                               int64_t m, int64_t n, int64_t k, void* ws, size_t ws_bytes, hipStream_t stream,
                               int num_cus) {
  // (ws_bytes: checked by the caller against int8_act_quant_workspace_size)
  if (few_fused(m, k)) {
    const FewPlan f = direct_plan(m, n, k, num_cus);
    const void* fn = direct_fn(f, dtype);
    const size_t lds = (size_t)(m * k);
    const int64_t workgroups = few_workgroups(f, fn, lds, 1, num_cus);
    if (debug_enabled()) {
      char name[64];
      snprintf(name, sizeof(name), "direct%dx%d/%dwaves/split1", f.bn, f.bm, f.waves);
      log_plan(kDense, name, m, n, k, 1, workgroups, 0, ws_bytes);
    }
    I8FewParams p{};
    p.a = static_cast<const int8_t*>(x); p.b = b; p.sb = sb; p.d = d;
    p.m = (int)m; p.n = (int)n; p.k = (int)k; p.out_dtype = out_dtype;
    return launch_few(f, fn, p, lds, 1, workgroups, nullptr, nullptr, stream);
  }
  uint8_t* w = static_cast<uint8_t*>(ws);
  uint8_t* codes = w + kCounterBytes;
  uint8_t* scales = codes + align256((size_t)(m * k));
  uint8_t* partials = scales + align256((size_t)m * 4);
  int8_t* q = reinterpret_cast<int8_t*>(codes);
  float* s = reinterpret_cast<float*>(scales);
  const int r = launch_quant_int8(x, dtype, m, k, q, s, stream);
  if (r != kOk) return r;
  return launch_planned(kDense, q, s, b, sb, d, out_dtype, nullptr, nullptr, 1, m, n, k,
                        int8_plan(kDense, m, n, k, 1, num_cus, true), w, partials, ws_bytes, stream, num_cus);
}

}  // namespace dg
