// qk_norm_rope.cu -- per-head RMS norm of q and k and the position rotation in
// one pass:  y = x * rsqrt(mean(x^2) + eps) * w per head, then each channel
// pair (a, b) becomes (a cos - b sin, b cos + a sin) with the angle
// position * inv_freq.  fp32 throughout, one rounding to bf16 at the end; the
// angle is a 64-bit product reduced to a fraction of a turn, so that far
// positions keep it (131072 * 1 rad in fp32 would be off by 4e-3 rad).
//
// Bound: HBM, every row read and written once.  D / 16 lanes hold a head, each
// two 16-byte chunks of which one is the other's partner in the rotation, so
// the rotation and the in-place form need no exchange between lanes; a warp
// takes 512 / D heads at a time.  The cosines and sines of a token are computed
// once per warp (a pair or two per lane, passed on in shared memory) and stay
// in registers while the warp walks the token's heads.
#include "q4.h"

namespace flux {

namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16lo_to_f32(w[i]);
    x[2 * i + 1] = bf16hi_to_f32(w[i]);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// One warp: token n, heads [h0, h1) of q and k taken as one list of Hq + Hkv.
template <int D, bool INTER>
__global__ void __launch_bounds__(32 * kWarps) norm_rope_kernel(const NormRopeLaunch a, int heads_per_warp,
                                                                int parts) {
  constexpr int LANES = D / 16;             // per head
  constexpr int PER = 32 / LANES;           // heads at a time
  __shared__ float2 table[kWarps][D / 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_launch_dependents();
  griddep_wait();
  const long long unit = static_cast<long long>(blockIdx.x) * kWarps + warp;
  const int n = static_cast<int>(unit / parts);
  if (n >= a.N) return;
  const int H = a.Hq + a.Hkv, half = a.rot / 2;
  const int h0 = static_cast<int>(unit % parts) * heads_per_warp, h1 = min(h0 + heads_per_warp, H);

  // cos, sin of the token's pairs
  const double pos = static_cast<double>(a.positions[n]);
  for (int p = lane; p < half; p += 32) {
    double t = pos * (static_cast<double>(a.inv_freq[p]) * 0.15915494309189535);
    t -= rint(t);
    float s, c;
    sincospif(2.f * static_cast<float>(t), &s, &c);
    table[warp][p] = make_float2(c, s);
  }
  __syncwarp();

  // The lane's chunks: c0 and its partner c1 (channels c0 + i and c1 + i are a
  // pair), or two neighbours that hold whole pairs (interleaved) or pass.
  const int l = lane % LANES, sub = lane / LANES;
  const bool turned = l < half / 8;
  const int c0 = turned && !INTER ? 8 * l : INTER ? 16 * l : a.rot + 16 * (l - half / 8);
  const int c1 = turned && !INTER ? 8 * l + half : c0 + 8;
  float2 cs[8];                             // of pair i; passing channels turn by nothing
#pragma unroll
  for (int i = 0; i < 8; ++i) cs[i] = turned ? table[warp][8 * l + i] : make_float2(1.f, 0.f);

  const bool norm = a.q_weight != nullptr;
  uint4 wq[2] = {}, wk[2] = {};
  if (norm) {
    wq[0] = *reinterpret_cast<const uint4*>(a.q_weight + c0);
    wq[1] = *reinterpret_cast<const uint4*>(a.q_weight + c1);
    wk[0] = *reinterpret_cast<const uint4*>(a.k_weight + c0);
    wk[1] = *reinterpret_cast<const uint4*>(a.k_weight + c1);
  }
  const uint16_t* qrow = a.q + n * a.q_stride;
  const uint16_t* krow = a.k + n * a.k_stride;
  uint16_t* qdst = a.q_out + n * a.q_out_stride;
  uint16_t* kdst = a.k_out + n * a.k_out_stride;
#pragma unroll 4
  for (int hb = h0; hb < h1; hb += PER) {
    const int h = hb + sub;
    const bool there = h < h1, is_q = h < a.Hq;
    const uint16_t* src = is_q ? qrow + h * D : krow + (h - a.Hq) * D;
    uint4 v0 = {0, 0, 0, 0}, v1 = {0, 0, 0, 0};
    if (there) {
      v0 = *reinterpret_cast<const uint4*>(src + c0);
      v1 = *reinterpret_cast<const uint4*>(src + c1);
    }
    float x0[8], x1[8];
    unpack8(v0, x0);
    unpack8(v1, x1);
    if (norm) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(x0[i], x0[i], fmaf(x1[i], x1[i], sum));
#pragma unroll
      for (int s = LANES / 2; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
      const float r = rsqrtf(sum * (1.f / D) + a.eps);
      float w0[8], w1[8];
      unpack8(is_q ? wq[0] : wk[0], w0);
      unpack8(is_q ? wq[1] : wk[1], w1);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x0[i] = x0[i] * r * w0[i];
        x1[i] = x1[i] * r * w1[i];
      }
    }
    // a non-finite passing channel stays as it is: its partner is turned by (1, 0) too
    if (turned) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (INTER) {
          float& p = i < 4 ? x0[2 * i] : x1[2 * i - 8];
          float& q = i < 4 ? x0[2 * i + 1] : x1[2 * i - 7];
          const float z = p * cs[i].x - q * cs[i].y;
          q = q * cs[i].x + p * cs[i].y;
          p = z;
        } else {
          const float z = x0[i] * cs[i].x - x1[i] * cs[i].y;
          x1[i] = x1[i] * cs[i].x + x0[i] * cs[i].y;
          x0[i] = z;
        }
      }
    }
    if (there) {
      uint16_t* dst = is_q ? qdst + h * D : kdst + (h - a.Hq) * D;
      *reinterpret_cast<uint4*>(dst + c0) = pack8(x0);
      *reinterpret_cast<uint4*>(dst + c1) = pack8(x1);
    }
  }
}

template <int D, bool INTER>
cudaError_t launch_t(const NormRopeLaunch& p, int num_sms, cudaStream_t stream) {
  constexpr int PER = 512 / D;
  const int H = p.Hq + p.Hkv;
  // All heads of a token by one warp, unless that leaves the SMs short of warps
  // (a decode step): then as many as a warp takes at a time.
  const bool few = static_cast<long long>(p.N) < 16LL * num_sms;
  const int per = few ? PER : H, parts = (H + per - 1) / per;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((static_cast<long long>(p.N) * parts + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_rope_kernel<D, INTER>, p, per, parts);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeLaunch& p, int num_sms, cudaStream_t stream) {
  if (p.d == 64)
    return p.interleaved ? launch_t<64, true>(p, num_sms, stream) : launch_t<64, false>(p, num_sms, stream);
  return p.interleaved ? launch_t<128, true>(p, num_sms, stream) : launch_t<128, false>(p, num_sms, stream);
}

}  // namespace flux
