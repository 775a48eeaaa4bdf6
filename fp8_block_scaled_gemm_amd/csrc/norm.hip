// What lies between two blocks of a transformer, one pass over its rows (the arithmetic is fp32 throughout):
//   z = v * x * rsqrt(mean(x^2) + eps)        the norm after the first block (or z = x without one)
//   s = r + scale * gate * z                  its gate and residual scale, and the residual stream
//   y = w * s * rsqrt(mean(s^2) + eps)        the norm before the second block
// with y in x's type, or quantized for an FP8 or int8 product as the library's quantizers would quantize it.
// And the backward pass: from dy, ds (the gradient that s gets from later blocks), x and s as it was stored,
//   du = ds + rho * (dy w - s rho^2 mean(dy w s)),  rho = rsqrt(mean(s^2) + eps)       -> dr = du
//   dz = scale * gate * du,  dgate = scale * sum(z du),  dw = sum(dy s rho)
//   dx = sigma * (dz v - x sigma^2 mean(dz v x)),  sigma = rsqrt(mean(x^2) + eps),  dv = sum(dz x sigma)
// Bound by memory: a row is read once into registers, its sums of squares are reduced there, so that every input passes
// once and every output once (4096 x 7168 bf16 over an fp32 stream, to FP8: 66 us, 332 MB at 5.0 TB/s, what a copy
// reaches; 8191 x 2048 bf16: 27 us).  One row alone is the latency of two loads and a reduction, 3.3 us.  To int8, with one
// reduction more: 4096 x 7168 68 us, a row 0.5 us more; short rows feel it (65536 x 128 40 us, to FP8 30).
#include "rows.hpp"

namespace dg {

enum NormOut : int { kNormSame = 0, kNormFp8 = 1, kNormInt8 = 2 };

struct NormParams {
  const void* x;              // null: s = r
  const void* residual;
  const float* weight;        // null: ones
  const float* post_weight;   // null: ones
  const void* gate;           // null: none
  void* sum;                  // null: not stored
  void* y;                    // y, or its codes
  float* scales;
  int64_t ld_s;
  int64_t rows, rows_per_gate;
  int hidden, post_norm;
  float scale, eps;
};

// Sums of N values over the LT lanes of a row, the same on each of them: within waves, then over the waves in order.
// Two calls in a row need different `red` arrays (no barrier keeps the first one's readers from the second's writers).
template <int LT, int N>
__device__ __forceinline__ void row_sums(float* v, float (*red)[N], int tid) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (LT > 64) {
    if ((tid & 63) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) red[tid >> 6][i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = red[0][i];
#pragma unroll
      for (int w = 1; w < LT / 64; ++w) s += red[w][i];
      v[i] = s;
    }
  }
}

// 1 / sqrt(mean + eps), both operations IEEE (one per row and lane: they cost nothing beside the row's memory traffic)
__device__ __forceinline__ float inv_rms(float sum_sq, int hidden, float eps) {
  return 1.0f / sqrtf(sum_sq / (float)hidden + eps);
}

constexpr int kNormThreads = 256;   // threads of a workgroup whose rows take one wave each

template <int LT>
constexpr int norm_threads() { return LT > kNormThreads ? LT : kNormThreads; }
template <int LT>
constexpr int norm_rows() { return LT >= kNormThreads ? 1 : kNormThreads / LT; }

// LT lanes a row, V pieces of 8 elements a lane: at most two, so that enough rows are in flight on a CU.
template <class T, class TR, int OUT, int LT, int V>
__global__ __launch_bounds__(norm_threads<LT>()) void residual_norm_kernel(NormParams p) {
  constexpr int kWaves = LT / 64;
  __shared__ float red_x[kWaves][1], red_s[kWaves][1];
  __shared__ uint32_t red_max[kWaves];
  const int tid = threadIdx.x % LT;
  const int64_t row = (blockIdx.x + (int64_t)gridDim.x * blockIdx.y) * norm_rows<LT>() +
                      __builtin_amdgcn_readfirstlane(threadIdx.x / LT);
  if (row >= p.rows) return;   // uniform over the row's waves, which share no barrier with another row's
  const int64_t base = row * p.hidden;
  const T* x = static_cast<const T*>(p.x);
  const TR* r = static_cast<const TR*>(p.residual);
  bool ok[V];
  int at[V];
  Raw8<TR> rr[V];
  Raw8<T> rx[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    at[i] = 8 * (tid + LT * i);
    ok[i] = at[i] < p.hidden;
    if (ok[i]) rr[i] = load8(r + base + at[i]);
    if (ok[i] && x != nullptr) rx[i] = load8(x + base + at[i]);
  }
  float s[V][8];
  if (x != nullptr) {
    float sigma = 1.0f;
    if (p.post_norm) {
      float sq[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (ok[i]) {
          float v[8];
          widen8(rx[i], v);
#pragma unroll
          for (int c = 0; c < 8; ++c) sq[0] = __builtin_fmaf(v[c], v[c], sq[0]);
        }
      row_sums<LT, 1>(sq, red_x, tid);
      sigma = inv_rms(sq[0], p.hidden, p.eps);
    }
    const T* gate = p.gate != nullptr ? static_cast<const T*>(p.gate) + (row / p.rows_per_gate) * p.hidden : nullptr;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (ok[i]) {
        float v[8], z[8];
        widen8(rr[i], v);
        widen8(rx[i], z);
        if (p.post_norm) {
#pragma unroll
          for (int c = 0; c < 8; ++c) z[c] *= sigma;
          if (p.post_weight != nullptr) {
            float w[8];
            widen8(load8(p.post_weight + at[i]), w);
#pragma unroll
            for (int c = 0; c < 8; ++c) z[c] *= w[c];
          }
        }
        if (gate != nullptr) {
          float g[8];
          widen8(load8(gate + at[i]), g);
#pragma unroll
          for (int c = 0; c < 8; ++c) z[c] *= g[c];
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) s[i][c] = __builtin_fmaf(p.scale, z[c], v[c]);
        if (p.sum != nullptr) store8(static_cast<TR*>(p.sum) + base + at[i], narrow8<TR>(s[i]));
      }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (ok[i]) widen8(rr[i], s[i]);
  }
  float sq[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (ok[i])
#pragma unroll
      for (int c = 0; c < 8; ++c) sq[0] = __builtin_fmaf(s[i][c], s[i][c], sq[0]);
  row_sums<LT, 1>(sq, red_s, tid);
  const float rho = inv_rms(sq[0], p.hidden, p.eps);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (ok[i]) {
      float w[8];
      if (p.weight != nullptr) widen8(load8(p.weight + at[i]), w);
#pragma unroll
      for (int c = 0; c < 8; ++c) s[i][c] = p.weight != nullptr ? s[i][c] * rho * w[c] : s[i][c] * rho;
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c) s[i][c] = 0.0f;
    }
  }
  if constexpr (OUT == kNormSame) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (ok[i]) store8(static_cast<T*>(p.y) + base + at[i], narrow8<T>(s[i]));
  } else if constexpr (OUT == kNormFp8) {
    uint8_t* q = static_cast<uint8_t*>(p.y) + base;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      // a group of 128 is the pieces of 16 neighbouring lanes; a partial last one holds zeros past the row
      const GroupScale scale = group16_scale(s[i]);
      if (ok[i]) {
        *reinterpret_cast<u32x2_t*>(q + at[i]) = pack8_e4m3(s[i], scale);
        if ((tid & 15) == 0) p.scales[(int64_t)(at[i] / kGroup) * p.ld_s + row] = scale.d.s;
      }
    }
  } else {
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int c = 0; c < 8; ++c) amax = umax(amax, abs_bits(s[i][c]));
    amax = wave_max_u32(amax);
    if constexpr (LT > 64) {
      if ((tid & 63) == 0) red_max[tid >> 6] = amax;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kWaves; ++w) amax = umax(amax, red_max[w]);
    }
    const float scale = int8_scale(amax);
    uint8_t* q = static_cast<uint8_t*>(p.y) + base;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (ok[i]) *reinterpret_cast<u32x2_t*>(q + at[i]) = u32x2_t{pack4_int8(s[i], scale), pack4_int8(s[i] + 4, scale)};
    if (tid == 0) p.scales[row] = scale;
  }
}

struct NormGradParams {
  const void* dy;
  const void* dsum;           // null: zeros
  const void* x;              // null: s = r
  const void* sum;
  const float* weight;
  const float* post_weight;
  const void* gate;
  void* dx;
  void* dresidual;
  float* dweight;             // null: not wanted
  void* dgate;
  float* dpost;
  float* part;                // partials: dweight, dpost, and two of dgate, (parts, hidden) each
  int64_t rows, rows_per_gate;
  int64_t rows_per_part;
  int parts;
  int gates_shared;           // gates that share a workgroup of the sums
  int hidden, post_norm;
  float scale, eps;
};

// What a norm's backward pass has to do beside the second norm's.
enum NormGradKind : int { kNormAlone = 0, kNormWithX = 1, kNormGateRows = 2 };   // no x; x; x and a gate for every row

// A workgroup takes p.rows_per_part consecutive rows, its row groups (of LT lanes) every norm_rows-th of them, and holds
// the columns' sums in registers.  They end in `part` (one row a workgroup), added by norm_grad_sum_kernel in the order
// of the workgroups: no atomics, the same bits from run to run.  A gate's rows ("segment") may end inside the
// workgroup's range: a segment that lies in it whole is written at once; a piece of one that does not goes to
// slot 0 where the range begins inside the segment, or with it, and to slot 1 where the segment begins later.
// One sum of a piece serves two gradients: with a = sum(scale du x sigma) over its rows, dgate is v a and dv gets gate a
// (held in LDS from piece to piece).  Absent weights, gates and norms are ones and scales of 1 rather than branches (those
// took 190 registers where 110 do).
// Bound by memory: 8191 x 2048 bf16 with a gate 40 us (220 MB at 5.5 TB/s), 16064 x 1536 fp16 over an fp32 stream with 64
// gates 97 us (4.6 TB/s), and 6 us for the sums of the partials.
template <class T, class TR, int KIND, int LT, int V>
__global__ __launch_bounds__(norm_threads<LT>(), V == 1 ? 3 : 2) void residual_norm_grad_kernel(NormGradParams p) {
  constexpr bool HASX = KIND != kNormAlone, GATES = KIND == kNormGateRows;
  constexpr int kWaves = LT / 64, kRows = norm_rows<LT>();
  __shared__ float red_a[kWaves][3], red_b[kWaves][1];
  __shared__ float cols[kRows > 1 ? kRows : 1][kRows > 1 ? 8 * LT * V : 1];
  constexpr bool kPieces = KIND == kNormWithX;   // dv is gathered piece by piece
  __shared__ v4f s_dv[kPieces ? kRows : 1][kPieces ? 2 * V : 1][kPieces ? LT : 1];
  // (a row group is whole waves: with its number in a scalar register the loop over its rows has no lane leave it alone)
  const int tid = threadIdx.x % LT, group = __builtin_amdgcn_readfirstlane(threadIdx.x / LT);
  const int64_t first = (int64_t)blockIdx.x * p.rows_per_part;
  const int64_t end = first + p.rows_per_part < p.rows ? first + p.rows_per_part : p.rows;
  const bool gate_sums = !GATES && p.dgate != nullptr;
  constexpr int VX = HASX ? V : 1;
  float dw[V][8], sum[VX][8];
  int at[V];
  bool ok[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    at[i] = 8 * (tid + LT * i);
    ok[i] = at[i] < p.hidden;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      dw[i][c] = 0.0f;
      if constexpr (HASX) sum[i][c] = 0.0f;
    }
    if constexpr (kPieces) s_dv[group][2 * i][tid] = s_dv[group][2 * i + 1][tid] = v4f{0.f, 0.f, 0.f, 0.f};
  }
  struct Row {
    Raw8<TR> u[V], ds[V];
    Raw8<T> dy[V], x[VX], g[GATES ? V : 1];
  };
  Row cur;
  // (an absent piece loads the row's first one: the loads stand in no branch)
  auto load_row = [&](int64_t row) {   // all but x
    const int64_t base = row * p.hidden;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int64_t from = base + (ok[i] ? at[i] : 0);
      cur.u[i] = load8(static_cast<const TR*>(p.sum) + from);
      cur.dy[i] = load8(static_cast<const T*>(p.dy) + from);
      if (p.dsum != nullptr) cur.ds[i] = load8(static_cast<const TR*>(p.dsum) + from);
      if constexpr (GATES) cur.g[i] = load8(static_cast<const T*>(p.gate) + from);
    }
  };
  auto load_x = [&](int64_t row) {
    if constexpr (HASX)
#pragma unroll
      for (int i = 0; i < V; ++i) cur.x[i] = load8(static_cast<const T*>(p.x) + row * p.hidden + (ok[i] ? at[i] : 0));
  };
  const bool normed = p.post_norm;
  auto columns = [&](const auto* src, int i, float* to) {   // of a weight or gate, ones where there is none
    if (src != nullptr && ok[i]) {
      widen8(load8(src + at[i]), to);
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c) to[c] = 1.0f;
    }
  };
  // weight, and post_weight times the piece's gate (a gate for every row: post_weight), held where the registers suffice, and
  // loaded piece by piece for rows of more than 8192
  constexpr bool kHold = V <= 2;
  const T* gate = nullptr;   // of the piece
  auto gated_weight = [&](int i, float* to) {
    columns(p.post_weight, i, to);
    if constexpr (KIND == kNormWithX) {
      float g[8];
      columns(gate, i, g);
#pragma unroll
      for (int c = 0; c < 8; ++c) to[c] *= g[c];
    }
  };
  float held_w[kHold ? V : 1][8], held_v[kHold ? VX : 1][8];
  auto hold = [&](float (*to)[8], auto&& get) {
    if constexpr (kHold)
#pragma unroll
      for (int i = 0; i < V; ++i) get(i, to[i]);
  };
  auto held = [&](const float (*from)[8], int i, float* to, auto&& get) {
    if constexpr (kHold) {
#pragma unroll
      for (int c = 0; c < 8; ++c) to[c] = from[i][c];
    } else {
      get(i, to);
    }
  };
  auto weight = [&](int i, float* to) { columns(p.weight, i, to); };
  hold(held_w, weight);
  if constexpr (GATES) hold(held_v, gated_weight);
  // a column sum of the whole workgroup (its row groups added in order), written by the first row group
  auto flush = [&](auto&& get, auto&& put) {
    if constexpr (kRows > 1) {
      __syncthreads();   // the previous flush's readers are done
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float t[8];
        get(i, t);
#pragma unroll
        for (int c = 0; c < 8; ++c) cols[group][at[i] + c] = t[c];
      }
      __syncthreads();
    }
    if (group == 0) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (ok[i]) {
          float t[8];
          get(i, t);
          if constexpr (kRows > 1) {
#pragma unroll
            for (int c = 0; c < 8; ++c)
#pragma unroll
              for (int g = 1; g < kRows; ++g) t[c] += cols[g][at[i] + c];
          }
          put(at[i], t);
        }
    }
  };
  const int64_t plane = (int64_t)p.parts * p.hidden;
  for (int64_t piece = first; piece < end;) {
    // the rows up to the segment's end (every row without sums of gates); uniform over the workgroup
    int64_t piece_end = end, segment = 0;
    if constexpr (KIND == kNormWithX) {
      if (p.gate != nullptr) {
        segment = piece / p.rows_per_gate;
        const int64_t e = (segment + 1) * p.rows_per_gate;
        piece_end = e < end ? e : end;
        gate = static_cast<const T*>(p.gate) + segment * p.hidden;
      }
      hold(held_v, gated_weight);
    }
    // rows of the piece in steps of kRows: every row group runs its own (they share barriers only in flush).  The next
    // row's loads go out as soon as the registers that they fill are free.
    if (piece + group < piece_end) {
      load_row(piece + group);
      load_x(piece + group);
    }
    for (int64_t row = piece + group; row < piece_end; row += kRows) {
      const int64_t base = row * p.hidden;
      float sums[3] = {0.0f, 0.0f, 0.0f};   // s^2, dy w s, x^2
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (ok[i]) {
          float u[8], dy[8], w[8];
          widen8(cur.u[i], u);
          widen8(cur.dy[i], dy);
          held(held_w, i, w, weight);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            sums[0] = __builtin_fmaf(u[c], u[c], sums[0]);
            sums[1] = __builtin_fmaf(dy[c] * w[c], u[c], sums[1]);
          }
          if constexpr (HASX) {
            float x[8];
            widen8(cur.x[i], x);
#pragma unroll
            for (int c = 0; c < 8; ++c) sums[2] = __builtin_fmaf(x[c], x[c], sums[2]);
          }
        }
      if constexpr (LT > 64) __syncthreads();   // the previous row's readers of red_a are done
      row_sums<LT, 3>(sums, red_a, tid);
      const float rho = inv_rms(sums[0], p.hidden, p.eps);
      const float back = rho * rho * sums[1] / (float)p.hidden;
      const float sigma = normed ? inv_rms(sums[2], p.hidden, p.eps) : 1.0f;
      float dz[VX][8];   // the gradient of z, times v
      float inner[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (ok[i]) {
          float u[8], dy[8], du[8], w[8];
          widen8(cur.u[i], u);
          widen8(cur.dy[i], dy);
          held(held_w, i, w, weight);
          if (p.dsum != nullptr) {
            widen8(cur.ds[i], du);
          } else {
#pragma unroll
            for (int c = 0; c < 8; ++c) du[c] = 0.0f;
          }
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            du[c] += rho * (dy[c] * w[c] - u[c] * back);
            dw[i][c] = __builtin_fmaf(dy[c], u[c] * rho, dw[i][c]);
          }
          store8(static_cast<TR*>(p.dresidual) + base + at[i], narrow8<TR>(du));
          if constexpr (HASX) {
            float x[8], v[8], g[8], dg[8];
            widen8(cur.x[i], x);
            held(held_v, i, v, gated_weight);
            if constexpr (GATES) widen8(cur.g[i], g);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const float n = x[c] * sigma;
              float dz0 = p.scale * du[c];
              if constexpr (GATES) {
                dg[c] = dz0 * (n * v[c]);
                dz0 *= g[c];
              }
              sum[i][c] = __builtin_fmaf(dz0, n, sum[i][c]);
              dz[i][c] = dz0 * v[c];
              inner[0] = __builtin_fmaf(dz[i][c], x[c], inner[0]);
            }
            if constexpr (GATES)
              if (p.dgate != nullptr) store8(static_cast<T*>(p.dgate) + base + at[i], narrow8<T>(dg));
          }
        }
      if (row + kRows < piece_end) load_row(row + kRows);
      if constexpr (HASX) {
        if (normed) row_sums<LT, 1>(inner, red_b, tid);   // (red_b's readers of the previous row are past the barrier above)
        const float along = sigma * sigma * inner[0] / (float)p.hidden;
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (ok[i]) {
            float x[8], dx[8];
            widen8(cur.x[i], x);
#pragma unroll
            for (int c = 0; c < 8; ++c) dx[c] = sigma * (dz[i][c] - (normed ? x[c] * along : 0.0f));
            store8(static_cast<T*>(p.dx) + base + at[i], narrow8<T>(dx));
          }
        if (row + kRows < piece_end) load_x(row + kRows);
      }
    }
    if constexpr (kPieces) {
      if (gate_sums) {
        const int64_t seg_first = segment * p.rows_per_gate;
        const bool whole = seg_first >= first && seg_first + p.rows_per_gate <= end;
        float* slot = p.part + (seg_first > first ? 3 : 2) * plane + (int64_t)blockIdx.x * p.hidden;
        flush(
            [&](int i, float* t) {
              columns(p.post_weight, i, t);
#pragma unroll
              for (int c = 0; c < 8; ++c) t[c] *= sum[i][c];
            },
            [&](int c0, const float* t) {
              if (whole) {
                store8(static_cast<T*>(p.dgate) + segment * p.hidden + c0, narrow8<T>(t));
              } else {
                store8(slot + c0, narrow8<float>(t));
              }
            });
      }
      if (p.dpost != nullptr) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float g[8];
          columns(gate, i, g);
#pragma unroll
          for (int c = 0; c < 8; ++c) s_dv[group][2 * i + (c >> 2)][tid][c & 3] += g[c] * sum[i][c];
        }
      }
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int c = 0; c < 8; ++c) sum[i][c] = 0.0f;
    }
    piece = piece_end;
  }
  float* mine = p.part + (int64_t)blockIdx.x * p.hidden;
  if (p.dweight != nullptr)
    flush(
        [&](int i, float* t) {
#pragma unroll
          for (int c = 0; c < 8; ++c) t[c] = dw[i][c];
        },
        [&](int c0, const float* t) { store8(mine + c0, narrow8<float>(t)); });
  if constexpr (HASX)
    if (p.dpost != nullptr)
      flush(
          [&](int i, float* t) {
#pragma unroll
            for (int c = 0; c < 8; ++c)
              if constexpr (kPieces)
                t[c] = s_dv[group][2 * i + (c >> 2)][tid][c & 3];
              else
                t[c] = sum[i][c];
          },
          [&](int c0, const float* t) { store8(mine + plane + c0, narrow8<float>(t)); });
}

// Column sums of the partials: 64 columns a workgroup (16 lanes of 4), 64 of the partials side by side, eight loads of each
// in flight, all added in a fixed order.  blockIdx.y = 0: dweight, 1: dpost, the rest the gates whose rows lie in more than
// one workgroup's: 2 + i is gate i, or the p.gates_shared gates from p.gates_shared i on, where gates have at least a
// workgroup's rows; where they have fewer, the 64 borders from 64 i on between workgroups j and j + 1, each with the last
// piece of j and the first of j + 1.
constexpr int kSumAlong = 64;

template <class T>
__global__ __launch_bounds__(16 * kSumAlong) void norm_grad_sum_kernel(NormGradParams p) {
  __shared__ v4f s_sum[kSumAlong][16];
  const int lane = threadIdx.x & 15, along = threadIdx.x >> 4;
  const int col = blockIdx.x * 64 + 4 * lane;
  const bool there = col < p.hidden;
  const int64_t plane = (int64_t)p.parts * p.hidden;
  auto at = [&](int which, int part) { return *reinterpret_cast<const v4f*>(p.part + which * plane + (int64_t)part * p.hidden + col); };
  auto put_gate = [&](int64_t gate, v4f v) {
    T* out = static_cast<T*>(p.dgate) + gate * p.hidden + col;
#pragma unroll
    for (int c = 0; c < 4; ++c) out[c] = narrow<T>(v[c]);
  };
  int which = blockIdx.y, begin = 0, end = p.parts;
  int head = -1;   // the workgroup in which the gate's rows begin, where that piece is in slot 1
  int beside = kSumAlong, place = along;   // partials side by side of this sum, and which of them this thread takes
  int64_t gate_sum = -1;
  if (blockIdx.y < 2) {
    if (blockIdx.y == 0 ? p.dweight == nullptr : p.dpost == nullptr) return;
  } else if (p.rows_per_gate < p.rows_per_part) {
    const int j = (blockIdx.y - 2) * kSumAlong + along;
    if (j + 1 >= p.parts || !there) return;
    const int64_t border = (int64_t)(j + 1) * p.rows_per_part, gate = border / p.rows_per_gate;
    if (gate * p.rows_per_gate != border) put_gate(gate, at(3, j) + at(2, j + 1));
    return;
  } else {
    beside = kSumAlong / p.gates_shared;
    place = along % beside;
    gate_sum = (int64_t)(blockIdx.y - 2) * p.gates_shared + along / beside;
    const int64_t first = gate_sum * p.rows_per_gate;
    begin = end = 0;
    if (first < p.rows) {
      begin = (int)(first / p.rows_per_part);
      end = (int)((first + p.rows_per_gate - 1) / p.rows_per_part) + 1;
      if (end - begin == 1) end = begin;   // written already
      if (first > (int64_t)begin * p.rows_per_part) head = begin;
    }
    which = 2;
  }
  v4f sum = {0.f, 0.f, 0.f, 0.f};
  if (there)
    for (int i0 = begin + place; i0 < end; i0 += 8 * beside) {
      v4f v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int i = i0 + u * beside < end ? i0 + u * beside : i0;
        v[u] = at(i == head ? 3 : which, i);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (i0 + u * beside < end) sum += v[u];
    }
  s_sum[along][lane] = sum;
  __syncthreads();
  if (beside < kSumAlong) {
    if (place != 0 || !there || begin == end) return;
    for (int i = 1; i < beside; ++i) sum += s_sum[along + i][lane];
    put_gate(gate_sum, sum);
    return;
  }
  if (along < 8) {
#pragma unroll
    for (int i = 8; i < kSumAlong; i += 8) sum += s_sum[along + i][lane];
    s_sum[along][lane] = sum;   // (no other thread reads these eight before the barrier)
  }
  __syncthreads();
  if (along != 0 || !there || begin == end) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) sum += s_sum[i][lane];
  if (blockIdx.y == 0) *reinterpret_cast<v4f*>(p.dweight + col) = sum;
  else if (blockIdx.y == 1) *reinterpret_cast<v4f*>(p.dpost + col) = sum;
  else put_gate(gate_sum, sum);
}

// ---- host ------------------------------------------------------------------------------------------
constexpr int kNormMaxHidden = 16384;

template <class T, class TR, int OUT>
static const void* norm_fn(int lt, int v) {
  void (*fn)(NormParams) = lt == 64    ? (v == 1 ? residual_norm_kernel<T, TR, OUT, 64, 1> : residual_norm_kernel<T, TR, OUT, 64, 2>)
                           : lt == 256 ? (v == 1 ? residual_norm_kernel<T, TR, OUT, 256, 1>
                                                 : residual_norm_kernel<T, TR, OUT, 256, 2>)
                           : lt == 512 ? residual_norm_kernel<T, TR, OUT, 512, 2>
                                       : residual_norm_kernel<T, TR, OUT, 1024, 2>;
  return reinterpret_cast<const void*>(fn);
}

template <class T, class TR>
static const void* norm_fn_of(int out, int lt, int v) {
  return out == kNormSame ? norm_fn<T, TR, kNormSame>(lt, v)
         : out == kNormFp8 ? norm_fn<T, TR, kNormFp8>(lt, v) : norm_fn<T, TR, kNormInt8>(lt, v);
}

template <class T, class TR, int KIND>
static const void* norm_grad_fn_of(int lt, int v) {
  void (*fn)(NormGradParams) =
      lt == 64 ? (v == 1 ? residual_norm_grad_kernel<T, TR, KIND, 64, 1> : residual_norm_grad_kernel<T, TR, KIND, 64, 2>)
      : lt == 256 ? (v == 1 ? residual_norm_grad_kernel<T, TR, KIND, 256, 1> : residual_norm_grad_kernel<T, TR, KIND, 256, 2>)
                  : (v == 2 ? residual_norm_grad_kernel<T, TR, KIND, 512, 2> : residual_norm_grad_kernel<T, TR, KIND, 512, 4>);
  return reinterpret_cast<const void*>(fn);
}

template <class T, class TR>
static const void* norm_grad_fn(int kind, int lt, int v) {
  return kind == kNormAlone   ? norm_grad_fn_of<T, TR, kNormAlone>(lt, v)
         : kind == kNormWithX ? norm_grad_fn_of<T, TR, kNormWithX>(lt, v) : norm_grad_fn_of<T, TR, kNormGateRows>(lt, v);
}

// Lanes a row and pieces a lane.
static void norm_shape(int64_t hidden, int* lt, int* v) {
  *lt = hidden <= 1024 ? 64 : hidden <= 4096 ? 256 : hidden <= 8192 ? 512 : 1024;
  *v = (int)((hidden + 8 * *lt - 1) / (8 * *lt));
  if (*lt > 256) *v = 2;
}

static int check_norm_size(int64_t rows, int64_t hidden) {
  if (hidden > kNormMaxHidden)
    return set_error(kUnsupported, "residual_norm: hidden = %lld, rows of at most %d are held in registers",
                     (long long)hidden, kNormMaxHidden);
  if (rows > 0x7fffffffLL) return set_error(kUnsupported, "residual_norm: 2^31 rows");
  return kOk;
}

int launch_residual_norm(int out, const void* x, const void* residual, int dtype, int residual_dtype, const float* weight,
                         const void* gate, int64_t gate_rows, bool post_norm, const float* post_weight, float scale,
                         float eps, int64_t rows, int64_t hidden, void* sum, void* y, float* scales, int64_t ld_s,
                         hipStream_t stream) {
  const int c = check_norm_size(rows, hidden);
  if (c != kOk) return c;
  NormParams p{};
  p.x = x;
  p.residual = residual;
  p.weight = weight;
  p.post_weight = post_weight;
  p.gate = gate;
  p.sum = sum;
  p.y = y;
  p.scales = scales;
  p.ld_s = ld_s;
  p.rows = rows;
  p.rows_per_gate = gate_rows > 0 ? rows / gate_rows : 1;
  p.hidden = (int)hidden;
  p.post_norm = post_norm;
  p.scale = scale;
  p.eps = eps;
  int lt, v;
  norm_shape(hidden, &lt, &v);
  const bool wide = residual_dtype == kF32;
  const void* fn = dtype == kF32 ? norm_fn_of<float, float>(out, lt, v)
                   : dtype == kBf16 ? (wide ? norm_fn_of<Bf16, float>(out, lt, v) : norm_fn_of<Bf16, Bf16>(out, lt, v))
                                    : (wide ? norm_fn_of<_Float16, float>(out, lt, v) : norm_fn_of<_Float16, _Float16>(out, lt, v));
  const int threads = lt > kNormThreads ? lt : kNormThreads, per_wg = lt >= kNormThreads ? 1 : kNormThreads / lt;
  void* args[] = {&p};
  const int64_t blocks = (rows + per_wg - 1) / per_wg, gx = blocks < kGridRow ? blocks : kGridRow;
  const hipError_t e = hipLaunchKernel(fn, dim3((unsigned)gx, (unsigned)((blocks + gx - 1) / gx)), dim3(threads), args, 0, stream);
  return e == hipSuccess ? kOk : set_error(kHip, "residual_norm launch: %s", hipGetErrorString(e));
}

// The backward pass: at most 512 lanes a row, whose registers hold the columns' sums too.
static void norm_grad_shape(int64_t hidden, int* lt, int* v) {
  norm_shape(hidden, lt, v);
  if (*lt == 1024) {
    *lt = 512;
    *v = 4;
  }
}

// Its workgroups and the rows of each: as many as the CUs hold at once (three of 256 threads, two with twice the columns,
// one of 512; 8191 x 2048 42.9 us with the sums, 47.9 with 1024 workgroups).
// A lane adds at most 256 rows of a column one after the other (more only past 2^24 rows of up to 1024, 2^22 of longer
// ones, where the partials of the second step would be the longer chain): the error of a sum is below 2^-24 times its two
// chains, rows and partials, of its terms' magnitudes.
static void norm_grad_parts(int64_t rows, int64_t hidden, int64_t* per_part, int* parts) {
  int lt, v;
  norm_grad_shape(hidden, &lt, &v);
  const int64_t most = v == 1 ? 768 : lt <= 256 ? 512 : 256;
  const int64_t groups = lt >= kNormThreads ? 1 : kNormThreads / lt;
  int64_t chain = 256;
  while (kSumAlong * groups * chain * chain < rows) chain *= 2;
  *per_part = (rows + most - 1) / most;
  if (*per_part > groups * chain) *per_part = groups * chain;
  *parts = rows == 0 ? 0 : (int)((rows + *per_part - 1) / *per_part);
}

size_t residual_norm_grad_workspace_size(int64_t rows, int64_t hidden) {
  int64_t per_part;
  int parts;
  norm_grad_parts(rows, hidden, &per_part, &parts);
  return (size_t)parts * hidden * 4 * sizeof(float);
}

int launch_fill_zero_bf16(uint16_t* d, int64_t count, hipStream_t stream);

int launch_residual_norm_grad(const void* dy, const void* dsum, const void* x, const void* sum, int dtype,
                              int residual_dtype, const float* weight, const void* gate, int64_t gate_rows, bool post_norm,
                              const float* post_weight, float scale, float eps, int64_t rows, int64_t hidden, void* dx,
                              void* dresidual, float* dweight, void* dgate, float* dpost, void* ws, hipStream_t stream) {
  const int c = check_norm_size(rows, hidden);
  if (c != kOk) return c;
  if (rows == 0) {   // sums over no rows
    int r = kOk;
    if (dweight != nullptr) r = launch_fill_zero_bf16(reinterpret_cast<uint16_t*>(dweight), 2 * hidden, stream);
    if (r == kOk && dpost != nullptr) r = launch_fill_zero_bf16(reinterpret_cast<uint16_t*>(dpost), 2 * hidden, stream);
    if (r == kOk && dgate != nullptr)
      r = launch_fill_zero_bf16(static_cast<uint16_t*>(dgate), gate_rows * hidden * (dtype == kF32 ? 2 : 1), stream);
    return r;
  }
  NormGradParams p{};
  p.dy = dy;
  p.dsum = dsum;
  p.x = x;
  p.sum = sum;
  p.weight = weight;
  p.post_weight = post_weight;
  p.gate = gate;
  p.dx = dx;
  p.dresidual = dresidual;
  p.dweight = dweight;
  p.dgate = dgate;
  p.dpost = dpost;
  p.part = static_cast<float*>(ws);
  p.rows = rows;
  p.rows_per_gate = gate_rows > 0 ? rows / gate_rows : 1;
  p.hidden = (int)hidden;
  p.post_norm = post_norm;
  p.scale = scale;
  p.eps = eps;
  norm_grad_parts(rows, hidden, &p.rows_per_part, &p.parts);
  int lt, v;
  norm_grad_shape(hidden, &lt, &v);
  const bool wide = residual_dtype == kF32;
  const int kind = x == nullptr ? kNormAlone : gate != nullptr && p.rows_per_gate == 1 ? kNormGateRows : kNormWithX;
  const void* fn = dtype == kF32 ? norm_grad_fn<float, float>(kind, lt, v)
                   : dtype == kBf16 ? (wide ? norm_grad_fn<Bf16, float>(kind, lt, v) : norm_grad_fn<Bf16, Bf16>(kind, lt, v))
                                    : (wide ? norm_grad_fn<_Float16, float>(kind, lt, v) : norm_grad_fn<_Float16, _Float16>(kind, lt, v));
  void* args[] = {&p};
  hipError_t e = hipLaunchKernel(fn, dim3((unsigned)p.parts), dim3(lt > kNormThreads ? lt : kNormThreads), args, 0, stream);
  if (e != hipSuccess) return set_error(kHip, "residual_norm_grad launch: %s", hipGetErrorString(e));
  int64_t gates = 0;   // rows of the sums' grid for gates
  p.gates_shared = 1;
  if (dgate != nullptr && p.rows_per_gate > 1 && p.parts > 1) {
    if (p.rows_per_gate < p.rows_per_part) {
      gates = (p.parts - 1 + kSumAlong - 1) / kSumAlong;
    } else {
      // as many threads to a gate as leave each at most two of its partials (64 gates of 251 rows: 103 -> 99.5 us with the sums)
      const int64_t pieces = p.rows_per_gate / p.rows_per_part + 2;
      while (p.gates_shared < 16 && 2 * (kSumAlong / (2 * p.gates_shared)) >= pieces) p.gates_shared *= 2;
      gates = (gate_rows + p.gates_shared - 1) / p.gates_shared;
    }
  }
  if (dweight == nullptr && dpost == nullptr && gates == 0) return kOk;
  void (*sum_fn)(NormGradParams) = dtype == kF32 ? norm_grad_sum_kernel<float>
                                   : dtype == kBf16 ? norm_grad_sum_kernel<Bf16> : norm_grad_sum_kernel<_Float16>;
  e = hipLaunchKernel(reinterpret_cast<const void*>(sum_fn),
                      dim3((unsigned)((hidden + 63) / 64), (unsigned)(2 + gates)), dim3(16 * kSumAlong), args, 0, stream);
  return e == hipSuccess ? kOk : set_error(kHip, "residual_norm_grad sums launch: %s", hipGetErrorString(e));
}

}  // namespace dg
