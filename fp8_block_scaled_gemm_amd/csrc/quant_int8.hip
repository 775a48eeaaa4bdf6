// Per-row 8-bit integer quantizer for gfx950: activations (one scale per token) and weights (one
// scale per output channel).  For each row
//   amax = max |x|,  s = amax / 127 (1 for amax = 0),  q = rne(x / s)  in [-127, 127],
// both divisions IEEE fp32, so codes and scales are bit-exact with any correct implementation.  A row
// that holds a NaN or an infinity gets a NaN or infinite scale, which the product carries on.
#include "rows.hpp"

namespace dg {

constexpr int kQ8Threads = 256;

// One workgroup per row: the row is read once for its maximum and again (from the caches) for its codes.
template <class T>
__global__ __launch_bounds__(kQ8Threads) void quant_int8_kernel(const T* __restrict__ x, int k, uint8_t* __restrict__ q,
                                                                float* __restrict__ s_out) {
  __shared__ uint32_t s_max[kQ8Threads / 64];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const T* src = x + row * k;
  uint8_t* dst = q + row * k;
  uint32_t amax = 0;
  for (int i = 16 * tid; i < k; i += 16 * kQ8Threads) {
    float v[16];
    widen8(load8(src + i), v);
    widen8(load8(src + i + 8), v + 8);
#pragma unroll
    for (int u = 0; u < 16; ++u) amax = umax(amax, abs_bits(v[u]));
  }
  amax = wave_max_u32(amax);
  if ((tid & 63) == 0) s_max[tid >> 6] = amax;
  __syncthreads();
  amax = umax(umax(s_max[0], s_max[1]), umax(s_max[2], s_max[3]));
  const float s = int8_scale(amax);
  for (int i = 16 * tid; i < k; i += 16 * kQ8Threads) {
    float v[16];
    widen8(load8(src + i), v);
    widen8(load8(src + i + 8), v + 8);
    *reinterpret_cast<u32x4_t*>(dst + i) =
        u32x4_t{pack4_int8(v, s), pack4_int8(v + 4, s), pack4_int8(v + 8, s), pack4_int8(v + 12, s)};
  }
  if (tid == 0) s_out[row] = s;
}

int launch_quant_int8(const void* x, int dtype, int64_t rows, int64_t k, int8_t* q, float* s, hipStream_t stream) {
  if (rows * kQ8Threads > 0xffffffffLL || k > 0x7fffffffLL)
    return set_error(kUnsupported, "quantize_int8_per_token: shape too large for the launch grid");
  uint8_t* codes = reinterpret_cast<uint8_t*>(q);
  const dim3 grid((unsigned)rows), block(kQ8Threads);
  switch (dtype) {
    case kF32:
      hipLaunchKernelGGL(quant_int8_kernel<float>, grid, block, 0, stream, static_cast<const float*>(x), (int)k, codes, s);
      break;
    case kBf16:
      hipLaunchKernelGGL(quant_int8_kernel<Bf16>, grid, block, 0, stream, static_cast<const Bf16*>(x), (int)k, codes, s);
      break;
    default:
      hipLaunchKernelGGL(quant_int8_kernel<_Float16>, grid, block, 0, stream, static_cast<const _Float16*>(x), (int)k,
                         codes, s);
  }
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? kOk : set_error(kHip, "quantize_int8_per_token launch: %s", hipGetErrorString(e));
}

}  // namespace dg
