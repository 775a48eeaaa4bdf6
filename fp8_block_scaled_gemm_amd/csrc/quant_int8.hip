// Per-row 8-bit integer quantizer for gfx950: activations (one scale per token) and weights (one
// scale per output channel).  For each row
//   amax = max |x|,  s = amax / 127 (1 for amax = 0),  q = rne(x / s)  in [-127, 127],
// both divisions IEEE fp32, so codes and scales are bit-exact with any correct implementation.  A row
// that holds a NaN or an infinity gets a NaN or infinite scale, which the product carries on.
#include "rows.hpp"

namespace dg {

// One workgroup of NT threads per row.  Each thread holds HOLD pieces of 8 elements in registers, so that a
// row of up to 8 * NT * HOLD elements is read once; the rest of a longer row is read again (from the
// caches) for its codes.  Bound by memory: 32768 x 7168 bf16 135 us, 5.2 TB/s; 16384 x 16384 bf16 150 us, 5.4;
// 65536 x 2048 fp32 113 us, 5.9 TB/s (nontemporal loads of rows past the last-level cache: 2% of that, either way).
template <class T, int NT, int HOLD>
__global__ __launch_bounds__(NT) void quant_int8_kernel(const T* __restrict__ x, int k, uint8_t* __restrict__ q,
                                                        float* __restrict__ s_out) {
  constexpr int W = NT / 64;
  __shared__ uint32_t s_max[W];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const T* src = x + row * k;
  uint8_t* dst = q + row * k;
  Raw8<T> held[HOLD];
#pragma unroll
  for (int h = 0; h < HOLD; ++h)
    if (8 * (tid + NT * h) < k) held[h] = load8(src + 8 * (tid + NT * h));
  uint32_t amax = 0;
  auto largest = [&](const Raw8<T>& r) {
    float v[8];
    widen8(r, v);
#pragma unroll
    for (int c = 0; c < 8; ++c) amax = umax(amax, abs_bits(v[c]));
  };
#pragma unroll
  for (int h = 0; h < HOLD; ++h)
    if (8 * (tid + NT * h) < k) largest(held[h]);
  // (unsigned: past the last piece of a row of almost 2^31 elements the index must not wrap)
  const uint32_t len = (uint32_t)k;
  for (uint32_t i = 8 * (tid + NT * HOLD); i < len; i += 8 * NT) largest(load8(src + i));
  amax = wave_max_u32(amax);
  if constexpr (W > 1) {
    if ((tid & 63) == 0) s_max[tid >> 6] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W; ++w) amax = umax(amax, s_max[w]);
  }
  const float s = int8_scale(amax);
  auto encode = [&](const Raw8<T>& r, uint32_t i) {
    float v[8];
    widen8(r, v);
    *reinterpret_cast<u32x2_t*>(dst + i) = u32x2_t{pack4_int8(v, s), pack4_int8(v + 4, s)};
  };
#pragma unroll
  for (int h = 0; h < HOLD; ++h)
    if (8 * (tid + NT * h) < k) encode(held[h], 8 * (tid + NT * h));
  for (uint32_t i = 8 * (tid + NT * HOLD); i < len; i += 8 * NT) encode(load8(src + i), i);
  if (tid == 0) s_out[row] = s;
}

template <class T>
static const void* quant_int8_fn(int nt) {
  void (*fn)(const T*, int, uint8_t*, float*) = nt == 64    ? quant_int8_kernel<T, 64, 2>
                                                : nt == 256 ? quant_int8_kernel<T, 256, 2>
                                                            : quant_int8_kernel<T, 512, 4>;
  return reinterpret_cast<const void*>(fn);
}

int launch_quant_int8(const void* x, int dtype, int64_t rows, int64_t k, int8_t* q, float* s, hipStream_t stream) {
  // threads for one to four pieces each (bf16, 16384 x 16384: 512 threads 12% faster than 256 and 28% faster than 1024
  // that read the row twice; 65536 x 1024: 64 threads 31% faster than 256)
  const int nt = k <= 1024 ? 64 : k <= 4096 ? 256 : 512;
  if (rows > 0xffffffffLL / nt || k > 0x7fffffffLL)
    return set_error(kUnsupported, "quantize_int8_per_token: shape too large for the launch grid");
  const void* fn = dtype == kF32 ? quant_int8_fn<float>(nt) : dtype == kBf16 ? quant_int8_fn<Bf16>(nt)
                                                                            : quant_int8_fn<_Float16>(nt);
  int ki = (int)k;
  uint8_t* codes = reinterpret_cast<uint8_t*>(q);
  void* args[] = {&x, &ki, &codes, &s};
  const hipError_t e = hipLaunchKernel(fn, dim3((unsigned)rows), dim3(nt), args, 0, stream);
  return e == hipSuccess ? kOk : set_error(kHip, "quantize_int8_per_token launch: %s", hipGetErrorString(e));
}

}  // namespace dg
