// The gated FP8 GEMM for few rows: weights streamed from memory into registers.
//
// With few rows a product is the reading of its weights.  A tile is 128 columns of h (128 gate and 128 up rows of the
// weights) and 16 or 64 rows: each of the 8 waves holds 16 columns, one gate and one up fragment, which it loads
// itself, D K blocks ahead, straight into the registers that the matrix instruction reads - no LDS, no barrier and no other
// wave between memory and the product.  Up to 16 rows each wave loads the activations likewise (they are in the caches);
// above, they go through registers into a two-slot ring of LDS (16-byte chunk c of row r in slot c ^ f(r), as in the
// large tiles), with one barrier a K block that waits for LDS only (not __syncthreads, which waits for every load in
// flight).  A loop body has no branch: loads past the last K block take an offset out of range, which reads zeros and no
// memory.
//   in flight per CU: 8 waves x 4 KB x D of weights, against one stage of 32 KB of the ring of the large tiles.
// EXACT, for quantized outputs: the codes are widened to bf16, whose products the matrix instruction adds to 2^-22 of them,
// where the FP8 instruction cuts them at 2^-13 of their largest.  A bf16 output's rounding hides that; a quantized one
// has a few codes in each 10^4 so near to a border that they come out on its other side, a step of 6 to 12%, and
// among few values no others make up for it (1 x 2048 x 7168, SiLU: 13.2 us for 11.8; 64 rows: 21.5 for 19.5).  In the contiguous
// layout a tile is half a block of 128 rows (256 x 512 x 7168 67 us, 52 by the FP8 instruction on the 256x128 tile).
// K is split over workgroups where there are few tiles: fp32 partials of the rows in use go to the workspace.  Their sums,
// in the order of the splits, end the rows: taken by a second launch, or, of few bytes, by the last workgroup of a tile to
// arrive (the hand-off of the plain forms).  A CU takes some 30 bytes a nanosecond from memory, so the last workgroup alone
// is the slower the more there is to add, while a launch costs 3 us whatever it does.
// Bound by what a CU takes from memory, and for one token by the latencies of one pass: 1 x 2048 x 7168, 14 splits, 11.8 us
// (29 MB; 5.9 us at the rate of a copy); 777 x 1057 x 1552 in 117 tiles of 64 rows on 256 CUs 18 us; 64 x 2048
// x 7168 in 8 splits 19.5 us.  Tiles of 128 and 256 rows were no faster than the large tiles.
#include <type_traits>

#include "gemm_common.hpp"
#include "gemm_gated.hpp"

namespace dg {

template <int V>
using IC = std::integral_constant<int, V>;

template <int J_, int D_>
struct CfgStream {
  static constexpr int BN = 256, BM = 16 * J_, kThreads = 512, kWaves = 8;
  static constexpr int J = J_, D = D_;
  static constexpr bool kDirect = J_ == 1;                      // activations without LDS
  static constexpr int kActLoads = J_ >= 4 ? J_ / 4 : 1;        // 16-byte pieces a thread stages per K block
  static constexpr int kStages = D_ - 1;                        // K blocks of activations in registers
  static constexpr int kScaleOffset = BM * kGroup;
  static constexpr int kSlot = kScaleOffset + kThreads * 4;     // activation bytes and scales of one K block
  static constexpr int kEpilogue = (BM < 64 ? BM : 64) * kGatedPitch * 4;
  static constexpr int kRing = kDirect ? 0 : 2 * kSlot;
  static constexpr int kLds = kRing > kEpilogue ? kRing : kEpilogue;
  static_assert(kDirect || (D_ == 3 && J_ % 4 == 0), "registers are named by K block modulo 3 and 2 in steps of six");
};

// First float of a split tile's partials: tiles numbered by (group, row block, strip of columns), whether they have rows or not.
__device__ __forceinline__ int64_t partial_at(const GemmParams& p, int bm, int g, int mb, int nbt, int split) {
  return ((((int64_t)g * p.tiles_m + mb) * p.tiles_n + nbt) * p.splits + split) * bm * (2 * kGroup);
}

// Every wave's LDS operations are done, and every wave is here: __syncthreads with fences of LDS alone, so that loads from
// memory into registers fly on over it.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

template <class C, int LAYOUT, bool EXACT>
__global__ __launch_bounds__(C::kThreads) void gemm_gated_few_kernel(GemmParams p) {
  constexpr int J = C::J, D = C::D, NT = C::kThreads;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[C::kLds];
  __shared__ int s_prefix[LAYOUT == kMasked ? 1025 : 1];
  __shared__ int s_scan[LAYOUT == kMasked ? 256 : 1];
  __shared__ int s_flag;
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g4 = lane >> 4;

  int total_items;
  if constexpr (LAYOUT == kMasked) {
    masked_item_prefix(p.masked_m, p.num_groups, p.m, C::BM, p.tiles_n, s_prefix, s_scan);
    total_items = s_prefix[p.num_groups] * p.splits;
  } else {
    total_items = p.tiles_m * p.tiles_n * p.splits;
  }
  const int grid = gridDim.x;
  int wg = blockIdx.x;   // XCD-aware order, as in the large tiles
  if ((grid & 7) == 0) wg = (blockIdx.x & 7) * (grid >> 3) + (blockIdx.x >> 3);

  for (int item = wg; item < total_items; item += grid) {
    TileCoord t;
    t.m_lo = 0;
    t.split = item % p.splits;
    int rest = item / p.splits;
    if constexpr (LAYOUT == kMasked) {
      t.g = masked_group_of(s_prefix, p.num_groups, rest);
      rest -= s_prefix[t.g];
      const int mv = p.masked_m[t.g];
      t.m_valid = mv < 0 ? 0 : (mv > p.m ? p.m : mv);
    } else {
      t.g = 0;
      t.m_valid = p.m;
    }
    // row blocks of one strip of weights side by side: they share it in their XCD's L2
    const int mblocks = LAYOUT == kMasked ? (t.m_valid + C::BM - 1) / C::BM : p.tiles_m;
    t.mb = rest % mblocks;
    t.nbt = rest / mblocks;
    const int m0 = t.mb * C::BM, n0 = t.nbt * kGroup;
    if constexpr (LAYOUT == kContiguous) {   // a tile lies in one block of 128 rows, so in one expert's rows
      static_assert(kGroup % C::BM == 0, "a block is whole tiles");
      t.g = p.m_indices[m0];
      if (t.g < 0 || t.g >= p.num_groups) continue;   // (uniform)
    }
    const int rows = t.m_valid - m0;   // rows of this tile (more than BM: all)
    const int kb0 = t.split * p.kb_per_split;
    const int kb1 = kb0 + p.kb_per_split < p.kb_total ? kb0 + p.kb_per_split : p.kb_total;
    const int nk = kb1 - kb0;

    const uint8_t* b_g = p.b + (int64_t)t.g * p.b_gstride + (int64_t)n0 * p.k;
    const int64_t b_bytes = (int64_t)(p.n - n0) * p.k;   // the rows of this half that exist; the rest reads zeros
    const __amdgpu_buffer_rsrc_t rs_g = make_rsrc(b_g, b_bytes);
    const __amdgpu_buffer_rsrc_t rs_u = make_rsrc(b_g + (int64_t)p.n * p.k, b_bytes);
    const __amdgpu_buffer_rsrc_t rs_a = make_rsrc(
        p.a + (LAYOUT == kMasked ? (int64_t)t.g * p.a_gstride : 0) + (int64_t)m0 * p.k, (int64_t)rows * p.k);
    const __amdgpu_buffer_rsrc_t rs_sa =
        make_rsrc(p.sa + (LAYOUT == kMasked ? (int64_t)t.g * p.sa_gstride : 0), (int64_t)p.kb_total * p.ld_sa * 4);
    const float* sb_g = p.sb + (int64_t)t.g * p.sb_gstride + (int64_t)t.nbt * p.kb_total + kb0;
    const float* sb_u = sb_g + (int64_t)p.nb128 * p.kb_total;

    // A lane's 32 bytes of a K block, of weights and activations alike, as in the large tiles: the matrix instruction adds
    // the same products together, whatever the tile (16 bytes of each half, 64 of a row in one piece, were no faster).
    // Loads past the last K block, or past k, take an out-of-range offset.
    auto offset = [&](int tk, int half, uint32_t row_off) {
      return tk < nk && (kb0 + tk) * kGroup + 16 * half + 32 * g4 < p.k ? row_off + 16u * half + 32u * g4 : kOut;
    };
    auto load16 = [&](__amdgpu_buffer_rsrc_t rs, int tk, int half, uint32_t row_off) {
      return __builtin_amdgcn_raw_buffer_load_b128(rs, offset(tk, half, row_off), offset_block(kb0 + tk, tk < nk) * kGroup, 0);
    };
    auto load_scale = [&](int tk, int row) {   // of row m0 + row (0 past the rows in use)
      return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                                           rs_sa, tk < nk && row < rows ? (uint32_t)(m0 + row) * 4u : kOut,
                                           offset_block(kb0 + tk, tk < nk) * (int)p.ld_sa * 4, 0));
    };
    const uint32_t w_off = (uint32_t)(16 * wave + l16) * (uint32_t)p.k;
    v8i w[D][2];   // [K block][gate, up]
    auto load_w = [&](int tk, v8i* r) {
      r[0] = make_v8i(load16(rs_g, tk, 0, w_off), load16(rs_g, tk, 1, w_off));
      r[1] = make_v8i(load16(rs_u, tk, 0, w_off), load16(rs_u, tk, 1, w_off));
    };
    // Block scales of 64 K blocks at a time, one a lane, read by lane number.
    float vg = 0.0f, vu = 0.0f;
    auto load_blocks = [&](int tk) {
      const int i = tk + lane < nk ? tk + lane : nk - 1;
      vg = sb_g[i];
      vu = sb_u[i];
    };
    auto block_scale = [&](float v, int tk) {   // 0 past the last K block, whose operands are zeros
      const float s = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), tk & 63));
      return tk < nk ? s : 0.0f;
    };

    v4f acc[2][J];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < J; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    using Weights = std::conditional_t<EXACT, Wide, v8i>;
    auto weights = [&](const v8i& r) {
      if constexpr (EXACT) return widen_codes(r);
      else return r;
    };
    auto multiply = [&](const Weights* r, const v8i& act_codes, float sa, float sbg, float sbu, int j) {
      v4f pg, pu;
      if constexpr (EXACT) {
        const Wide act = widen_codes(act_codes);
        pg = exact_product(r[0], act);
        pu = exact_product(r[1], act);
      } else {
        pg = pu = v4f{0.f, 0.f, 0.f, 0.f};
        pg = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(r[0], act_codes, pg, 0, 0, 0, 127, 0, 127);
        pu = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(r[1], act_codes, pu, 0, 0, 0, 127, 0, 127);
      }
      const float sg = sa * sbg, su = sa * sbu;   // fl32(sa * sb)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[0][j][i] = __builtin_fmaf(pg[i], sg, acc[0][j][i]);
        acc[1][j][i] = __builtin_fmaf(pu[i], su, acc[1][j][i]);
      }
    };

    load_blocks(0);
    if constexpr (C::kDirect) {
      const uint32_t a_off = (uint32_t)l16 * (uint32_t)p.k;   // (rows that are not there: past the resource, zeros)
      v8i av[D];
      float sv[D];
      auto load = [&](int tk, int slot) {
        load_w(tk, w[slot]);
        av[slot] = make_v8i(load16(rs_a, tk, 0, a_off), load16(rs_a, tk, 1, a_off));
        sv[slot] = load_scale(tk, l16);
      };
#pragma unroll
      for (int i = 0; i < D; ++i) load(i, i);
      for (int t0 = 0; t0 < nk; t0 += D) {
        if (t0 > 0 && (t0 & 63) == 0) load_blocks(t0);
#pragma unroll
        for (int u = 0; u < D; ++u) {   // (K blocks past the last are zeros with scales 0)
          const Weights both[2] = {weights(w[u][0]), weights(w[u][1])};
          multiply(both, av[u], sv[u], block_scale(vg, t0 + u), block_scale(vu, t0 + u), 0);
          load(t0 + u + D, u);
        }
      }
    } else {
      // activations: 16-byte piece tid + NT * i is chunk piece % 8 of row piece / 8; scales: thread tid has row tid's
      u32x4 ar[C::kStages][C::kActLoads];
      float sr[C::kStages];
      auto load_a = [&](int tk, int stage) {
#pragma unroll
        for (int i = 0; i < C::kActLoads; ++i) {
          const int piece = tid + NT * i, row = piece >> 3, c = piece & 7;
          const bool there = tk < nk && (kb0 + tk) * kGroup + 16 * c < p.k;
          ar[stage][i] = __builtin_amdgcn_raw_buffer_load_b128(rs_a, there ? (uint32_t)row * (uint32_t)p.k + 16u * c : kOut,
                                                               offset_block(kb0 + tk, tk < nk) * kGroup, 0);
        }
        sr[stage] = load_scale(tk, tid);
      };
      auto put_a = [&](int slot, int stage) {
        uint8_t* base = lds + slot * C::kSlot;
#pragma unroll
        for (int i = 0; i < C::kActLoads; ++i) {
          const int piece = tid + NT * i;
          *reinterpret_cast<u32x4*>(base + lds_off(piece >> 3, piece & 7)) = ar[stage][i];
        }
        *reinterpret_cast<float*>(base + C::kScaleOffset + 4 * tid) = sr[stage];
      };
      const int lane_off = lds_off(l16, 2 * g4);   // the second half's chunk differs in bit 0: address ^ 16
      auto compute = [&](int slot, const v8i* r, float sbg, float sbu) {
        const uint8_t* base = lds + slot * C::kSlot;
        auto read = [&](int j) {
          const int off = 16 * j * kGroup + lane_off;
          return make_v8i(*reinterpret_cast<const u32x4*>(base + off), *reinterpret_cast<const u32x4*>(base + (off ^ 16)));
        };
        const Weights both[2] = {weights(r[0]), weights(r[1])};
        // four fragments read at a time
#pragma unroll
        for (int j0 = 0; j0 < J; j0 += 4) {
          v8i act[4];
          float sa[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            act[i] = read(j0 + i);
            sa[i] = *reinterpret_cast<const float*>(base + C::kScaleOffset + 4 * (16 * (j0 + i) + l16));
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) multiply(both, act[i], sa[i], sbg, sbu, j0 + i);
        }
      };
      // K block tk: the barrier makes its activations visible and frees the other slot, where the next block's go; the loads
      // of the blocks after go out as soon as the registers that they fill are free.  (A K block past the last
      // is zeros with scales 0.)
      auto step = [&](int tk, int u) {
        lds_barrier();
        put_a((u + 1) & 1, (u + 1) & 1);
        load_a(tk + 3, (u + 1) & 1);
        compute(u & 1, w[u % 3], block_scale(vg, tk), block_scale(vu, tk));
        load_w(tk + 3, w[u % 3]);
      };
      __syncthreads();   // the previous tile's readers of the LDS are done
      load_a(0, 0);
      load_w(0, w[0]);
      load_a(1, 1);
      load_w(1, w[1]);
      put_a(0, 0);
      load_a(2, 0);
      load_w(2, w[2]);
      for (int t0 = 0; t0 < nk; t0 += 6) {
#pragma unroll
        for (int u = 0; u < 6; ++u) {
          if (u > 0 && t0 + u >= nk) break;
          if (t0 + u > 0 && ((t0 + u) & 63) == 0) load_blocks(t0 + u);
          step(t0 + u, u);
        }
      }
    }

    float* chunk = reinterpret_cast<float*>(lds);
    auto row_of = [&](int, int r) { return m0 + r; };
    if (p.splits > 1) {   // (row, 256) partials of the rows in use
      const int64_t at = partial_at(p, C::BM, t.g, t.mb, t.nbt, 0);
      constexpr int kSplitBytes = C::BM * 2 * kGroup * 4;
      const __amdgpu_buffer_rsrc_t rs_ws = make_rsrc(p.ws + at, (int64_t)p.splits * kSplitBytes);
      // (agent-scope stores and loads where the tile's last workgroup reads them: they pass the XCD's non-coherent L2)
      auto put = [&](auto policy) {
#pragma unroll
        for (int j = 0; j < J; ++j)
          if (16 * j + l16 < rows)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              __builtin_amdgcn_raw_buffer_store_b128(
                  __builtin_bit_cast(u32x4, acc[i][j]), rs_ws,
                  t.split * kSplitBytes + ((16 * j + l16) * 2 * kGroup + i * kGroup + 16 * wave + 4 * g4) * 4, 0,
                  decltype(policy)::value);
      };
      if constexpr (!C::kDirect) {
        put(IC<0>{});
        continue;
      } else {
        if (p.counters == nullptr) {
          put(IC<0>{});
          continue;
        }
        put(IC<kCpolSc1>{});
        __builtin_amdgcn_s_waitcnt(0);   // every partial store of this thread has completed
        __syncthreads();
        unsigned* counter = p.counters + at / (p.splits * (kSplitBytes / 4));
        if (tid == 0) {
          const unsigned prev = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          s_flag = prev == (unsigned)(p.splits - 1) ? 1 : 0;
        }
        __syncthreads();
        if (!s_flag) continue;
        if (tid == 0)   // leave the counter zeroed for the next call
          __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        gated_epilogue<NT, LAYOUT, false>(
            p, t, n0, 1, C::BM, chunk,
            [&](int) {   // a wave a row, 16 bytes a lane
#pragma unroll 1
              for (int r = wave; r < C::BM && r < rows; r += C::kWaves) {
                const int src = (r * 2 * kGroup + 4 * lane) * 4;
                v4f sum = {0.f, 0.f, 0.f, 0.f};
                for (int s0 = 0; s0 < p.splits; s0 += 16) {   // up to 16 splits' loads in flight
                  v4f v[16];
#pragma unroll
                  for (int u = 0; u < 16; ++u)
                    v[u] = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(
                                                       rs_ws, s0 + u < p.splits ? (s0 + u) * kSplitBytes + src : (int)kOut, 0, kCpolSc1));
#pragma unroll
                  for (int u = 0; u < 16; ++u) sum = s0 + u == 0 ? v[u] : sum + v[u];   // (absent splits read zeros)
                }
                *reinterpret_cast<v4f*>(chunk + r * kGatedPitch + 4 * lane) = sum;
              }
            },
            row_of);
        continue;
      }
    }
    gated_epilogue<NT, LAYOUT, false>(
        p, t, n0, 1, C::BM, chunk,
        [&](int) {
          float* dst = chunk + l16 * kGatedPitch + 16 * wave + 4 * g4;
#pragma unroll
          for (int j = 0; j < J; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) *reinterpret_cast<v4f*>(dst + 16 * j * kGatedPitch + i * kGroup) = acc[i][j];
        },
        row_of);
  }
}

// The sums of the splits' partials, in their order, and the end of the rows: 16 lanes a row and 128 columns of h.
template <int LAYOUT>
__global__ __launch_bounds__(256) void gemm_gated_join_kernel(GemmParams p, int bm) {
  const int lane16 = threadIdx.x & 15;
  const int row = blockIdx.y * 16 + (threadIdx.x >> 4), g = blockIdx.z;
  int m_valid = p.m;
  if constexpr (LAYOUT == kMasked) {
    const int mv = p.masked_m[g];
    m_valid = mv < 0 ? 0 : (mv > p.m ? p.m : mv);
  }
  if (row >= m_valid) return;   // (uniform over the 16 lanes)
  const int nbt = blockIdx.x, mb = row / bm;
  const float* part = p.ws + partial_at(p, bm, g, mb, nbt, 0) + (row - mb * bm) * 2 * kGroup + 8 * lane16;
  const int64_t step = (int64_t)bm * 2 * kGroup;
  v4f sum[4];
  for (int s0 = 0; s0 < p.splits; s0 += 4) {   // the loads of four splits in flight
    v4f v[4][4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float* src = part + (s0 + u < p.splits ? s0 + u : s0) * step;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[u][i] = *reinterpret_cast<const v4f*>(src + (i >> 1) * kGroup + (i & 1) * 4);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[i] = s0 + u == 0 ? v[u][i] : s0 + u < p.splits ? sum[i] + v[u][i] : sum[i];
  }
  float gv[8], uv[8];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    gv[c] = sum[0][c];
    gv[4 + c] = sum[1][c];
    uv[c] = sum[2][c];
    uv[4 + c] = sum[3][c];
  }
  float* scales = p.s + (LAYOUT == kMasked ? (int64_t)g * p.s_gstride : 0) + (int64_t)nbt * p.ld_s;
  gated_piece(p, (LAYOUT == kMasked ? (int64_t)g * p.m : 0) + row, scales + row, nbt * kGroup + 8 * lane16, lane16, gv, uv);
}

int launch_gated_join(int layout, GemmParams p, int bm, hipStream_t stream) {
  void (*fn)(GemmParams, int) = layout == kMasked ? gemm_gated_join_kernel<kMasked> : gemm_gated_join_kernel<kDense>;
  void* args[] = {&p, &bm};
  const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(fn),
                                       dim3((unsigned)p.tiles_n, (unsigned)((p.m + 15) / 16), (unsigned)p.num_groups), dim3(256),
                                       args, 0, stream);
  return e == hipSuccess ? kOk : set_error(kHip, "gated gemm join launch: %s", hipGetErrorString(e));
}

template <class C, bool EXACT>
static const void* few_fn(int layout) {
  if constexpr (EXACT && !C::kDirect)
    if (layout == kContiguous) {
      void (*fn)(GemmParams) = gemm_gated_few_kernel<C, kContiguous, EXACT>;
      return reinterpret_cast<const void*>(fn);
    }
  void (*fn)(GemmParams) = layout == kMasked ? gemm_gated_few_kernel<C, kMasked, EXACT> : gemm_gated_few_kernel<C, kDense, EXACT>;
  return reinterpret_cast<const void*>(fn);
}

// The kernel for tiles of 16 or 64 rows.
using CfgStream16 = CfgStream<1, 4>;
using CfgStream64 = CfgStream<4, 3>;

const void* gated_few_kernel(int layout, int bm, bool quantized) {
  if (quantized) return bm == 16 ? few_fn<CfgStream16, true>(layout) : few_fn<CfgStream64, true>(layout);
  return bm == 16 ? few_fn<CfgStream16, false>(layout) : few_fn<CfgStream64, false>(layout);
}

int gated_few_lds(int bm) { return bm == 16 ? CfgStream16::kLds : CfgStream64::kLds; }

}  // namespace dg
