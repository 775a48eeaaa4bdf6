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
// Bound by the matrix cores: 16384 x 7168 x 16384 runs at 2.70e15 operations/s (1424 us), 4096 x 4096 x 7168
// at 2.45e15 (98 us, one round of 256 tiles: its first loads and its stores are not hidden).  The rate
// depends on the operands' bits (zeros 3.2e15, random codes 2.7e15): power holds the clock, not the
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
    auto scaled = [&](int i, int j, float* v) {
      const float sr = s_scale[C::BN + wm0 + 16 * j + e16];
      const v4f sc = *reinterpret_cast<const v4f*>(&s_scale[wn0 + 16 * i + 4 * e4]);
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = (float)acc[i][j][r] * (sr * sc[r]);
    };
    // Through LDS: each wave turns 16 output rows of its tile (fp32: of half its columns at a time) into
    // row pieces of 16 bytes (a fragment's own stores would touch 16 rows of 32 or 64 bytes each).
    auto store_rows = [&](auto size_c) {
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
            float v[4];
            scaled(part * (kFN / kParts) + i0, j, v);
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
    if (p.out_dtype == kF32) store_rows(IC<4>{});
    else store_rows(IC<2>{});
  }
}

// ---------------------------------------------------------------------------
// Few rows: the weights are streamed once from memory, and that is what bounds the kernel.  Two kernels, both
// of them on tiles of 16 weight rows per wave and step, multiplied straight from the registers that memory
// filled: a lane reads 16 bytes of one row, so an instruction covers 16 rows x 64 bytes of K.  The waves of
// a workgroup (and S workgroups of one tile) split K; rows past the edges take out-of-range addresses and
// cost no traffic.  The waves' int32 partials are added in LDS with integer atomics, whose order does not
// matter; the S partials of a tile go through the workspace to the workgroup that arrives last.
//  * direct: one or two unquantized rows, which every workgroup quantizes for itself while its first weights
//    are on the way (1 x 4096 x 7168: 9.0 us, 3.3 TB/s of weights; 1 x 24576 x 1536: 10.3 us, 3.7 TB/s).
//  * staged: the activations pass through LDS (64 x 4096 x 7168: 13.1 us; 64 x 7168 x 16384: 36.6 us,
//    3.2 TB/s of weights).
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
  int steps, steps_per_wave;
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
  t.g = blockIdx.x / per_group;
  const int rest = blockIdx.x - t.g * per_group;
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
  const __amdgpu_buffer_rsrc_t rs_ws =
      make_rsrc(p.ws + (int64_t)t.id * p.splits * (BM * BN), p.splits > 1 ? (int64_t)p.splits * BM * BN * 4 : 0);
  for (int c = tid; c < kChunks; c += NT) {
    const int row = t.m0 + c / (BN / 4), col = t.n0 + 4 * (c % (BN / 4));
    const int count = p.n - col;
    if (row >= t.m_valid || count <= 0) continue;
    v4i sum = *piece(c);
    for (int o = 0; o < p.splits; ++o)
      if (o != t.split)
        sum += __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rs_ws, (o * kChunks + c) * 16, 0, kCpolSc1));
    const float sr = row_scale(row);
    float v[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = (float)sum[r] * (sr * (r < count ? sb[col + r] : 0.f));
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
  const uint32_t row_off = (uint32_t)l16 * (uint32_t)p.k + 16u * g4;
  const int s0 = (t.split * W + wave) * p.steps_per_wave;
  const int s1 = s0 + p.steps_per_wave < p.steps ? s0 + p.steps_per_wave : p.steps;

  struct Set { v4i b[U][R]; };
  // U steps of 64 K bytes; chunks past K and steps past s1 take an out-of-range offset and read zeros
  auto load = [&](Set& v, int s) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k0 = 64 * (s + u);
      const uint32_t out = s + u < s1 && k0 + 16 * g4 < p.k ? 0u : 0xFFFFFFF0u;
#pragma unroll
      for (int i = 0; i < R; ++i)
        v.b[u][i] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(
                                                rs_b, (row_off + (uint32_t)(16 * i) * (uint32_t)p.k) | out, k0, 0));
    }
  };
  v4i acc[R];
#pragma unroll
  for (int i = 0; i < R; ++i) acc[i] = v4i{0, 0, 0, 0};
  auto multiply = [&](const Set& v, int s) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = 64 * (s + u) + 16 * g4;
      const v4i act = l16 < p.m && s + u < s1 && at < p.k ? *reinterpret_cast<const v4i*>(s_codes + l16 * p.k + at)
                                                          : v4i{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < R; ++i) acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(v.b[u][i], act, acc[i], 0, 0, 0);
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
  load(even, s0);
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
  for (int s = s0; s < s1; s += 2 * U) {
    load(odd, s + U);
    multiply(even, s);
    if (s + U >= s1) break;
    load(even, s + 2 * U);
    multiply(odd, s + U);
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

// The activations pass through LDS.  Read by every wave straight from memory they cost as many
// vector-memory requests as the weights (16 rows x 64 bytes an instruction), and that request rate, not the
// bytes, then bounds the kernel (64 x 7168 x 16384: 45 us so, 36.6 here).  Here 2 times 16 R weight rows
// each belong to 4 waves that share their K chunk of 512 bytes (256 on 128-row tiles), and the workgroup
// brings the chunk's 16 J activation rows in once, a whole line per 8 lanes, through registers into one of
// two LDS buffers: one barrier per chunk, the next chunk's weights and activations in flight across it.
constexpr int kStNS = 2, kStKS = 4;

template <int R, int J, int CHUNK>
__global__ __launch_bounds__(64 * kStNS * kStKS) void gemm_int8_staged_kernel(I8FewParams p) {
  constexpr int NS = kStNS, KS = kStKS, NT = 64 * NS * KS;
  constexpr int BN = 16 * R * NS, BM = 16 * J;
  constexpr int kPitch = CHUNK + 16;   // 16 rows of one 16-byte column fall in different banks
  constexpr int U = CHUNK / 64 / KS;              // steps of 64 K bytes per wave and chunk
  constexpr int kPieces = BM * CHUNK / 16 / NT;   // 16-byte pieces per thread and chunk
  constexpr int kBuf = BM * kPitch;
  constexpr int kSumPitch = BN + 4;
  static_assert(kPieces * NT * 16 == BM * CHUNK && U * KS * 64 == CHUNK, "a chunk splits evenly");
  constexpr int kLds = 2 * kBuf > BM * kSumPitch * 4 ? 2 * kBuf : BM * kSumPitch * 4;
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
  // steps_per_wave counts chunks here: the workgroup's chunks [c0, c1)
  const int c0 = t.split * p.steps_per_wave;
  const int c1 = c0 + p.steps_per_wave < p.steps ? c0 + p.steps_per_wave : p.steps;

  // this thread's activation pieces: row piece / 32, 16-byte column piece % 32 of the chunk
  u32x4 act[kPieces];
  auto load_act = [&](int c) {
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int piece = tid + NT * u, row = piece / (CHUNK / 16), col = 16 * (piece % (CHUNK / 16));
      const uint32_t out = c < c1 && c * CHUNK + col < p.k ? 0u : 0xFFFFFFF0u;   // past K: zeros
      act[u] = __builtin_amdgcn_raw_buffer_load_b128(rs_a, ((uint32_t)row * (uint32_t)p.k + (uint32_t)col) | out,
                                                     c * CHUNK, 0);
    }
  };
  auto store_act = [&](int c) {
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int piece = tid + NT * u, row = piece / (CHUNK / 16), col = 16 * (piece % (CHUNK / 16));
      *reinterpret_cast<u32x4*>(smem + (c & 1) * kBuf + row * kPitch + col) = act[u];
    }
  };
  struct Set { v4i b[U][R]; };
  const uint32_t row_off = (uint32_t)(16 * R * ns + l16) * (uint32_t)p.k + 16u * g4;
  auto load_b = [&](Set& v, int c) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k0 = c * CHUNK + 64 * (kh * U + u);
      const uint32_t out = c < c1 && k0 + 16 * g4 < p.k ? 0u : 0xFFFFFFF0u;
#pragma unroll
      for (int i = 0; i < R; ++i)
        v.b[u][i] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(
                                                rs_b, (row_off + (uint32_t)(16 * i) * (uint32_t)p.k) | out, k0, 0));
    }
  };
  v4i acc[R][J];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < J; ++j) acc[i][j] = v4i{0, 0, 0, 0};
  auto multiply = [&](const Set& v, int c) {
    const uint8_t* base = smem + (c & 1) * kBuf + l16 * kPitch + 64 * kh * U + 16 * g4;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v4i fa[J];
#pragma unroll
      for (int j = 0; j < J; ++j) fa[j] = *reinterpret_cast<const v4i*>(base + 16 * j * kPitch + 64 * u);
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < J; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(v.b[u][i], fa[j], acc[i][j], 0, 0, 0);
    }
  };

  // one chunk of weights and activations ahead (two or three ahead measured the same or slower);
  // chunks past c1 read nothing
  Set even, odd;
  load_act(c0);
  load_b(even, c0);
  for (int c = c0; c < c1; c += 2) {
    store_act(c);
    load_act(c + 1);
    load_b(odd, c + 1);
    __syncthreads();   // chunk c is in its buffer; every wave is done with chunk c - 1's
    multiply(even, c);
    if (c + 1 >= c1) break;   // uniform
    store_act(c + 1);
    load_act(c + 2);
    load_b(even, c + 2);
    __syncthreads();
    multiply(odd, c + 1);
  }

  __syncthreads();   // the buffers become the sums
  int* s_sum = reinterpret_cast<int*>(smem);
#pragma unroll
  for (int h = 0; h < KS; ++h) {
    if (kh == h) {
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < R; ++i) {
          v4i* at = reinterpret_cast<v4i*>(&s_sum[(16 * j + l16) * kSumPitch + 16 * (R * ns + i) + 4 * g4]);
          *at = h == 0 ? acc[i][j] : *at + acc[i][j];
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
  bool direct;
  int r, j, waves, unit;   // unit: K bytes of a step (direct) or chunk (staged)
  int bn, bm;
  int strips, mtiles, splits, steps, steps_per_wave;
  int64_t tiles;
  size_t ws_bytes;
};

// Few-row plan.  `direct`: the kernel that quantizes its rows itself.  What the choices measured:
//  * direct, waves a workgroup (they share K): 1 x 24576 x 1536 takes 10.3 us with 4, 13.9 with 8, 16.3
//    with 16; 1 x 4096 x 7168 9.0 with 8, 9.9 with 16; K past 8192 needs 16 to hold the row.
//  * direct, 32 weight rows a workgroup where that still gives ~3/4 of a workgroup per CU: 1 x 7168 x 2048
//    5.2 us against 5.7 with 16.
//  * staged, 128-row tiles: chunks of 256 (two workgroups' buffers fit a CU): 128 x 24576 x 1536 23.0 us,
//    two 64-row tiles 26.4; 32 weight rows a wave once K is long enough to pay for splitting it:
//    128 x 7168 x 16384 45.7 us against 52.9 with 16.
static FewPlan few_plan(bool direct, int64_t m, int64_t n, int64_t k, int64_t groups, int num_cus, bool allow_split) {
  FewPlan f{};
  f.direct = direct;
  if (direct) {
    f.j = 1;
    f.r = n >= (int64_t)24 * num_cus ? 2 : 1;
    f.waves = k <= 4096 ? 4 : k <= 8192 ? 8 : 16;
    f.unit = 64;
  } else {
    f.j = m <= 16 ? 1 : m <= 32 ? 2 : m <= 64 ? 4 : 8;
    f.r = f.j == 8 && k >= 8192 && n >= (int64_t)24 * num_cus ? 2 : 1;
    f.waves = kStNS * kStKS;
    f.unit = f.j == 8 ? 256 : 512;
  }
  f.bn = 16 * f.r * (direct ? 1 : kStNS);
  f.bm = 16 * f.j;
  f.strips = (int)((n + f.bn - 1) / f.bn);
  f.mtiles = (int)((m + f.bm - 1) / f.bm);
  f.tiles = (int64_t)f.strips * f.mtiles * groups;
  const int sharing = direct ? f.waves : 1;   // units of K go to waves (direct) or to workgroups (staged)
  f.steps = (int)((k + f.unit - 1) / f.unit);
  // split K until there is about one workgroup per CU, each keeping a few units (64 x 4096 x 7168:
  // unsplit 128 workgroups 20 us, split in two 13.1, in four 15.5)
  int64_t want = (2 * (int64_t)num_cus / f.tiles + 1) / 2;
  const int64_t most = f.steps / (direct ? 4 * sharing : 2);
  if (want > most) want = most;
  if (want > kMaxSplits) want = kMaxSplits;
  if (!allow_split || want < 1 || f.tiles > kMaxCounterTiles) want = 1;
  f.steps_per_wave = (int)((f.steps + want * sharing - 1) / (want * sharing));
  f.splits = (int)((f.steps + (int64_t)f.steps_per_wave * sharing - 1) / ((int64_t)f.steps_per_wave * sharing));   // none empty
  f.ws_bytes = f.splits > 1 ? kCounterBytes + (size_t)f.tiles * f.splits * f.bn * f.bm * 4 : 0;
  return f;
}

static const void* staged_fn(const FewPlan& f) {
  void (*fn)(I8FewParams) = f.j == 1   ? gemm_int8_staged_kernel<1, 1, 512>
                            : f.j == 2 ? gemm_int8_staged_kernel<1, 2, 512>
                            : f.j == 4 ? gemm_int8_staged_kernel<1, 4, 512>
                            : f.r == 1 ? gemm_int8_staged_kernel<1, 8, 256>
                                       : gemm_int8_staged_kernel<2, 8, 256>;
  return reinterpret_cast<const void*>(fn);
}

template <class X>
static const void* direct_fn_of(const FewPlan& f) {
  void (*fn)(I8FewParams);
  if (f.r == 1)
    fn = f.waves == 4 ? gemm_int8_direct_kernel<1, 8, 4, X> : f.waves == 8 ? gemm_int8_direct_kernel<1, 8, 8, X>
                                                                           : gemm_int8_direct_kernel<1, 8, 16, X>;
  else
    fn = f.waves == 4 ? gemm_int8_direct_kernel<2, 4, 4, X> : f.waves == 8 ? gemm_int8_direct_kernel<2, 4, 8, X>
                                                                           : gemm_int8_direct_kernel<2, 4, 16, X>;
  return reinterpret_cast<const void*>(fn);
}
static const void* direct_fn(const FewPlan& f, int dtype) {
  return dtype == kF32 ? direct_fn_of<float>(f) : dtype == kBf16 ? direct_fn_of<Bf16>(f) : direct_fn_of<_Float16>(f);
}

static int launch_few(const FewPlan& f, const void* fn, I8FewParams p, size_t lds, int64_t groups, void* counters,
                      void* partials, hipStream_t stream) {
  p.strips = f.strips; p.mtiles = f.mtiles; p.splits = f.splits;
  p.steps = f.steps; p.steps_per_wave = f.steps_per_wave;
  p.counters = static_cast<unsigned*>(counters);
  p.ws = static_cast<int*>(partials);
  const int64_t blocks = groups * ((((int64_t)f.strips * f.splits + 7) & ~(int64_t)7) * f.mtiles);
  if (blocks * 64 * f.waves > 0xffffffffLL) return set_error(kUnsupported, "int8 gemm: too many output tiles");
  void* args[] = {&p};
  const hipError_t e = hipLaunchKernel(fn, dim3((unsigned)blocks), dim3(64 * f.waves), args, lds, stream);
  return e == hipSuccess ? kOk : set_error(kHip, "int8 gemm launch: %s", hipGetErrorString(e));
}

// Time estimates (microseconds, MI355X, 256 CUs), fitted to timings of every choice on shapes of 1 to 4096
// rows.  A workgroup's K block takes longer the more of them run (they share caches and power); a
// tile costs a fixed part as well (first loads, stores); a K split sends its partials out and back.
struct TileModel { int bn, bm, occ; double fixed, alone, busy; };
constexpr TileModel kTileModel[kTiles] = {
    {I8Square::BN, I8Square::BM, I8Square::OCC, 7.0, 0.9, 1.6},
    {I8Small::BN, I8Small::BM, I8Small::OCC, 3.5, 0.5, 1.15}};

static double split_time(int splits, double partial_bytes) { return 3.0 + 0.5 * splits + 0.22e-6 * partial_bytes; }

// Few-row tiles: the time of a chunk (512 bytes of K, 256 on 128-row tiles) with one workgroup a CU, and
// per workgroup of the fullest CU.
static double few_time(const FewPlan& f, int num_cus) {
  const double c = (double)((f.tiles * f.splits + num_cus - 1) / num_cus);
  const double one = f.j == 8 ? 0.8 * f.r : 0.95, more = f.j == 8 ? 0.7 * f.r : f.j == 4 ? 1.0 : 0.87;
  const double t = 3.5 + f.steps_per_wave * (c * more > one ? c * more : one);
  return t + (f.splits > 1 ? split_time(f.splits, (double)f.tiles * f.splits * f.bn * f.bm * 4) : 0.0);
}

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
  if (layout == kContiguous && c.bm > kGroup) {   // a tile that spans two experts runs twice
    const int64_t edges = groups - 1 < t.tiles_m ? groups - 1 : t.tiles_m;
    tiles += (double)edges * t.tiles_n;
  }
  t.items = (int64_t)t.tiles_m * t.tiles_n * t.splits * (layout == kMasked ? groups : 1);
  const double items = tiles * t.splits, slots = (double)c.occ * num_cus;
  const double full = (double)(int64_t)(items / slots), rest = items - full * slots;
  t.us = full * (c.fixed + t.kb_per_split * c.busy);
  if (rest > 0) t.us += c.fixed + t.kb_per_split * (c.alone + (c.busy - c.alone) * rest / slots);
  // the weights come from memory at 5 TB/s at best, and at 17 GB/s for each workgroup
  const double rate = items * 0.017e6 < 5.0e6 ? items * 0.017e6 : 5.0e6;
  const double weights = c.fixed + (double)n * k * (layout == kDense ? 1 : groups) / rate;
  if (t.us < weights) t.us = weights;
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
static TilePlan tile_plan(int layout, int64_t m, int64_t n, int64_t k, int64_t groups, int num_cus, bool allow_split) {
  TilePlan best{};
  for (int tile = 0; tile < kTiles; ++tile) {
    for (int splits = 1; splits <= kMaxSplits; ++splits) {
      const TilePlan t = tile_choice(tile, splits, layout, m, n, k, groups, num_cus);
      if (splits > 1) {
        const bool crowded = splits <= 3 ? t.items > (int64_t)kTileModel[tile].occ * num_cus
                                         : 8 * t.items > 9 * (int64_t)num_cus;
        if (layout != kDense || !allow_split || t.kb_per_split < 4 || crowded || t.items / t.splits > kMaxCounterTiles)
          break;
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
  I8Plan p{};
  p.few = layout != kContiguous && m <= kFewRowsMost;
  if (p.few) p.f = few_plan(false, m, n, k, groups, num_cus, allow_split);
  p.t = tile_plan(layout, m, n, k, groups, num_cus, allow_split);
  p.few = p.few && few_time(p.f, num_cus) < p.t.us;
  return p;
}

int launch_quant_int8(const void* x, int dtype, int64_t rows, int64_t k, int8_t* q, float* s, hipStream_t stream);

size_t int8_workspace_size(int64_t m, int64_t n, int64_t k, int64_t groups, int num_cus) {
  return int8_plan(groups > 1 ? kMasked : kDense, m, n, k, groups, num_cus, true).ws_bytes();
}

// `counters` and `partials`: the K split's workspace, or null for none.
static int launch_planned(int layout, const int8_t* a, const float* sa, const int8_t* b, const float* sb, void* d,
                          int out_dtype, const int32_t* m_indices, const int32_t* masked_m, int64_t groups, int64_t m,
                          int64_t n, int64_t k, const I8Plan& plan, void* counters, void* partials, hipStream_t stream,
                          int num_cus) {
  if (plan.few) {
    I8FewParams p{};
    p.a = a; p.sa = sa; p.b = b; p.sb = sb; p.d = d; p.masked_m = masked_m;
    p.m = (int)m; p.n = (int)n; p.k = (int)k; p.out_dtype = out_dtype;
    return launch_few(plan.f, staged_fn(plan.f), p, 0, groups, counters, partials, stream);
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
  const int64_t slots = (int64_t)num_cus * kTileModel[t.tile].occ;
  void* args[] = {&p};
  const hipError_t e = hipLaunchKernel(tile_fn(layout, t.tile), dim3((unsigned)(t.items < slots ? t.items : slots)),
                                       dim3(I8Square::kThreads), args, 0, stream);
  return e == hipSuccess ? kOk : set_error(kHip, "int8 gemm launch: %s", hipGetErrorString(e));
}

int launch_gemm_int8(int layout, const int8_t* a, const float* sa, const int8_t* b, const float* sb, void* d,
                     int out_dtype, const int32_t* m_indices, const int32_t* masked_m, int64_t groups, int64_t m,
                     int64_t n, int64_t k, void* ws, size_t ws_bytes, hipStream_t stream, int num_cus) {
  I8Plan plan = int8_plan(layout, m, n, k, groups, num_cus, ws != nullptr);
  if (ws_bytes < plan.ws_bytes()) plan = int8_plan(layout, m, n, k, groups, num_cus, false);
  return launch_planned(layout, a, sa, b, sb, d, out_dtype, m_indices, masked_m, groups, m, n, k, plan, ws,
                        static_cast<uint8_t*>(ws) + kCounterBytes, stream, num_cus);
}

// In-call quantization.  Up to kFewFusedRows rows of at most kFewFusedK elements are quantized by the
// product's own workgroups; more rows by a launch of the quantizer into the workspace: the counter prefix,
// the codes, the scales (256-byte pieces), then the K split's partials.
static size_t align256(size_t v) { return (v + 255) / 256 * 256; }
static bool few_fused(int64_t m, int64_t k) { return m <= kFewFusedRows && k <= kFewFusedK; }

size_t int8_act_quant_workspace_size(int64_t m, int64_t n, int64_t k, int num_cus) {
  if (few_fused(m, k)) {
    const size_t split = few_plan(true, m, n, k, 1, num_cus, true).ws_bytes;
    return split > 0 ? split : kCounterBytes;
  }
  const size_t split = int8_workspace_size(m, n, k, 1, num_cus);
  return kCounterBytes + align256((size_t)(m * k)) + align256((size_t)m * 4) + (split > 0 ? split - kCounterBytes : 0);
}

int launch_gemm_int8_act_quant(const void* x, int dtype, const int8_t* b, const float* sb, void* d, int out_dtype,
                               int64_t m, int64_t n, int64_t k, void* ws, size_t ws_bytes, hipStream_t stream,
                               int num_cus) {
  (void)ws_bytes;   // checked by the caller against int8_act_quant_workspace_size
  if (few_fused(m, k)) {
    const FewPlan f = few_plan(true, m, n, k, 1, num_cus, true);
    I8FewParams p{};
    p.a = static_cast<const int8_t*>(x); p.b = b; p.sb = sb; p.d = d;
    p.m = (int)m; p.n = (int)n; p.k = (int)k; p.out_dtype = out_dtype;
    return launch_few(f, direct_fn(f, dtype), p, (size_t)(m * k), 1, ws, static_cast<uint8_t*>(ws) + kCounterBytes, stream);
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
                        int8_plan(kDense, m, n, k, 1, num_cus, true), w, partials, stream, num_cus);
}

}  // namespace dg
