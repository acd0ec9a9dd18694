// qk_norm_rope.cu -- per-head RMS norm of q and k and the position rotation in
// one pass:  y = x * rsqrt(mean(x^2) + eps) * w per head, then each channel
// pair (a, b) becomes (a cos - b sin, b cos + a sin) with the angle
// position * inv_freq.  fp32 throughout, one rounding to bf16 at the end; the
// angle is a 64-bit product reduced to a fraction of a turn, so that far
// positions keep it (131072 * 1 rad in fp32 would be off by 4e-3 rad).
#include "q4.h"

namespace flux {

namespace {

__device__ __forceinline__ float bf16_bits_to_f32(uint16_t x) {
  return __uint_as_float(static_cast<uint32_t>(x) << 16);
}
__device__ __forceinline__ uint16_t f32_to_bf16_bits(float x) {
  return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

// One warp per (token, head); a lane holds D / 64 channel pairs.
template <int D>
__global__ void __launch_bounds__(256) norm_rope_kernel(const NormRopeLaunch a) {
  constexpr int NP = D / 64;
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int H = a.Hq + a.Hkv;
  if (row >= static_cast<long long>(a.N) * H) return;
  const long long n = row / H;
  int h = static_cast<int>(row % H);
  const bool is_q = h < a.Hq;
  if (!is_q) h -= a.Hq;
  const uint16_t* src = is_q ? a.q + n * a.q_stride + h * D : a.k + n * a.k_stride + h * D;
  uint16_t* dst = is_q ? a.q_out + n * a.q_out_stride + h * D : a.k_out + n * a.k_out_stride + h * D;
  const uint16_t* w = is_q ? a.q_weight : a.k_weight;
  const int half = a.rot / 2;
  int c0[NP], c1[NP];
  float x0[NP], x1[NP], sum = 0.f;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int p = lane + 32 * i;
    if (p < half && !a.interleaved) {
      c0[i] = p;
      c1[i] = p + half;
    } else {               // neighbouring pairs; the channels behind rot are paired any way
      c0[i] = 2 * p;
      c1[i] = 2 * p + 1;
    }
    x0[i] = bf16_bits_to_f32(src[c0[i]]);
    x1[i] = bf16_bits_to_f32(src[c1[i]]);
    sum += x0[i] * x0[i] + x1[i] * x1[i];
  }
  float r = 1.f;
  if (w) {
    for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
    r = rsqrtf(sum * (1.f / D) + a.eps);
  }
  __syncwarp();            // in place: every read of the row comes before a write to it
  const int pos = a.positions[n];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int p = lane + 32 * i;
    float y0 = x0[i] * r, y1 = x1[i] * r;
    if (w) {
      y0 *= bf16_bits_to_f32(w[c0[i]]);
      y1 *= bf16_bits_to_f32(w[c1[i]]);
    }
    if (p < half) {
      double t = static_cast<double>(pos) * (static_cast<double>(a.inv_freq[p]) * 0.15915494309189535);
      t -= rint(t);
      float s, c;
      sincospif(2.f * static_cast<float>(t), &s, &c);
      const float z0 = y0 * c - y1 * s;
      y1 = y1 * c + y0 * s;
      y0 = z0;
    }
    dst[c0[i]] = f32_to_bf16_bits(y0);
    dst[c1[i]] = f32_to_bf16_bits(y1);
  }
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeLaunch& p, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  const long long rows = static_cast<long long>(p.N) * (p.Hq + p.Hkv);
  const unsigned grid = static_cast<unsigned>((rows + 7) / 8);
  if (p.d == 64) norm_rope_kernel<64><<<grid, 256, 0, stream>>>(p);
  else norm_rope_kernel<128><<<grid, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace flux
