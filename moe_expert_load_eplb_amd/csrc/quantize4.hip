// Weights to 4-bit floating point with a power of two for each 32.
//
// A scale is a power of two, so x / 2^e is exact and a value has one right
// answer.  With a the largest magnitude, e is the least with a <= 7 * 2^e: what
// lies between 6 and 7 rounds to 6, off by at most the half step that values
// between 4 and 6 are off by.
//
// Bound by memory: 9 experts of 2048 x 4096 in 32 bits: 59 us, 5.8 TB/s.  Four lanes to
// a block, 16 or 32 bytes of each, so that a wave reads whole lines.
#include "experts_device.h"
#include "layer_internal.h"

namespace eplb {

namespace {

constexpr int kThreads = 256;

// Four lanes to a block of 32, eight elements each.
template <int DTYPE>
__global__ __launch_bounds__(kThreads) void quantize4_kernel(const void* w, int64_t groups, uint32_t* q,
                                                            uint8_t* scale) {
  const int64_t part = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t parts = groups * 4;
  const int64_t from = part < parts ? part : parts - 1;        // every lane takes part in its block's maximum
  float v[8];
  if (DTYPE == kF32) {
    const f32x4* p = static_cast<const f32x4*>(w) + from * 2;
    const f32x4 lo = p[0], hi = p[1];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = lo[j], v[4 + j] = hi[j];
  } else {
    const uint4 h = static_cast<const uint4*>(w)[from];
    const uint32_t word[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const u16 x = (u16)(word[j >> 1] >> (j & 1) * 16);
      v[j] = DTYPE == kBf16 ? bf16_to_float(x) : f16_to_float(x);
    }
  }
  uint32_t top = 0;                        // as integers magnitudes keep their order, infinities and NaN last
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  top = max(top, (uint32_t)__shfl_xor((int)top, 1));
  top = max(top, (uint32_t)__shfl_xor((int)top, 2));
  const int exponent = (int)(top >> 23);
  const bool fine = exponent < 255;
  // 1.75 * 2^(e + 2) = 7 * 2^e
  const int s = fine ? max((top & 0x7FFFFFu) <= 0x600000u ? exponent - 2 : exponent - 1, 27) : 255;
  const float factor = fine ? __uint_as_float((uint32_t)(254 - s) << 23) : 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = fine ? v[j] * factor : 0.0f;
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], 1.0f, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], 1.0f, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], 1.0f, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], 1.0f, 3);
  if (part < parts) {
    q[part] = c;
    if ((part & 3) == 0) scale[part >> 2] = (uint8_t)s;
  }
}

}  // namespace

hipError_t launch_quantize_weights4(const void* w, int32_t dtype, int64_t groups, uint8_t* q, uint8_t* scale,
                                    hipStream_t stream) {
  const dim3 grid((unsigned)ceil_div(groups * 4, kThreads));
  uint32_t* out = reinterpret_cast<uint32_t*>(q);
  if (dtype == kF32) quantize4_kernel<kF32><<<grid, kThreads, 0, stream>>>(w, groups, out, scale);
  else if (dtype == kBf16) quantize4_kernel<kBf16><<<grid, kThreads, 0, stream>>>(w, groups, out, scale);
  else quantize4_kernel<kF16><<<grid, kThreads, 0, stream>>>(w, groups, out, scale);
  return hipGetLastError();
}

}  // namespace eplb
