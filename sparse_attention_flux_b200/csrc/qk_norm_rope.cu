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
// takes 512 / D heads at a time, the loads of four such groups at once.  The
// cosines and sines of a token are computed once per warp (a pair or two per
// lane, passed on in shared memory) while its first rows are on their way, and
// multiplied into the weights, which leaves three operations a channel.  32768
// tokens, 32 + 8 heads, d 128: 118 us, 5.7 TB/s of 671 MB (weights and sines
// applied one after the other, no early loads: 136 us; 4 CTAs per SM without
// the register limit 124, 6 with it 121-123; the limit of 5 spills 12 registers
// of the half-split form).
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

// One warp: token n, groups [t0, t1) of PER heads, those of q before those of k.
template <int D, bool INTER>
__global__ void __launch_bounds__(32 * kWarps, 5) norm_rope_kernel(const NormRopeLaunch a, int groups_per_warp,
                                                                int parts) {
  constexpr int LANES = D / 16;             // per head
  constexpr int PER = 32 / LANES;           // heads at a time
  constexpr int U = 4;                      // groups in flight
  __shared__ float2 table[kWarps][D / 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_launch_dependents();
  griddep_wait();
  const long long unit = static_cast<long long>(blockIdx.x) * kWarps + warp;
  const int n = static_cast<int>(unit / parts);
  if (n >= a.N) return;
  const int half = a.rot / 2, gq = (a.Hq + PER - 1) / PER, gk = (a.Hkv + PER - 1) / PER;
  const int t0 = static_cast<int>(unit % parts) * groups_per_warp, t1 = min(t0 + groups_per_warp, gq + gk);

  // The lane's chunks: c0 and its partner c1 (channels c0 + i and c1 + i are a
  // pair), or two neighbours that hold whole pairs (interleaved) or pass.
  const int l = lane % LANES, sub = lane / LANES;
  const bool turned = l < half / 8;
  const int c0 = turned && !INTER ? 8 * l : INTER ? 16 * l : a.rot + 16 * (l - half / 8);
  const int c1 = turned && !INTER ? 8 * l + half : c0 + 8;

  uint4 v0[U], v1[U];
  auto load = [&](const uint16_t* row, int H, int g, int ge) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = (g + u) * PER + sub;
      if (g + u < ge && h < H) {
        v0[u] = __ldcs(reinterpret_cast<const uint4*>(row + h * D + c0));
        v1[u] = __ldcs(reinterpret_cast<const uint4*>(row + h * D + c1));
      } else {
        v0[u] = v1[u] = make_uint4(0, 0, 0, 0);
      }
    }
  };
  const uint16_t* qrow = a.q + n * a.q_stride;
  const uint16_t* krow = a.k + n * a.k_stride;
  // The first rows are on their way while the sines are computed.
  if (t0 < gq) load(qrow, a.Hq, t0, min(t1, gq));
  else load(krow, a.Hkv, t0 - gq, t1 - gq);

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

  auto heads = [&](const uint16_t* row, uint16_t* dst, const uint16_t* weight, int H, int g0, int ge, bool loaded) {
    // Pair (x0, x1) -> r (x0 a0 - x1 b0), r (x1 a1 + x0 b1) with the weights in the coefficients.
    float a0[8], a1[8], b0[8], b1[8];
    if (weight) {
      unpack8(*reinterpret_cast<const uint4*>(weight + c0), a0);
      unpack8(*reinterpret_cast<const uint4*>(weight + c1), a1);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) a0[i] = a1[i] = 1.f;
    }
    if (turned) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 cs = table[warp][8 * l + i];
        if (INTER) {           // pair i: channels 2 i, 2 i + 1 of the 16
          float& wa = i < 4 ? a0[2 * i] : a1[2 * i - 8];
          float& wb = i < 4 ? a0[2 * i + 1] : a1[2 * i - 7];
          (i < 4 ? b0[2 * i] : b1[2 * i - 8]) = wb * cs.y;
          (i < 4 ? b0[2 * i + 1] : b1[2 * i - 7]) = wa * cs.y;
          wa *= cs.x;
          wb *= cs.x;
        } else {
          b0[i] = a1[i] * cs.y;
          b1[i] = a0[i] * cs.y;
          a0[i] *= cs.x;
          a1[i] *= cs.x;
        }
      }
    }
    for (int g = g0; g < ge; g += U) {
      if (!loaded) load(row, H, g, ge);
      loaded = false;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (g + u >= ge) break;
        float x0[8], x1[8];
        unpack8(v0[u], x0);
        unpack8(v1[u], x1);
        float r = 1.f;
        if (weight) {
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) sum = fmaf(x0[i], x0[i], fmaf(x1[i], x1[i], sum));
#pragma unroll
          for (int s = LANES / 2; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
          r = rsqrtf(sum * (1.f / D) + a.eps);
        }
        float y0[8], y1[8];
        if (turned) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (INTER) {
              const float p0 = i % 2 ? x0[i ^ 1] : -x0[i ^ 1], p1 = i % 2 ? x1[i ^ 1] : -x1[i ^ 1];
              y0[i] = r * fmaf(p0, b0[i], x0[i] * a0[i]);
              y1[i] = r * fmaf(p1, b1[i], x1[i] * a1[i]);
            } else {
              y0[i] = r * fmaf(-x1[i], b0[i], x0[i] * a0[i]);
              y1[i] = r * fmaf(x0[i], b1[i], x1[i] * a1[i]);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            y0[i] = r * (x0[i] * a0[i]);
            y1[i] = r * (x1[i] * a1[i]);
          }
        }
        const int h = (g + u) * PER + sub;
        if (h < H) {
          *reinterpret_cast<uint4*>(dst + h * D + c0) = pack8(y0);
          *reinterpret_cast<uint4*>(dst + h * D + c1) = pack8(y1);
        }
      }
    }
  };
  if (t0 < gq) heads(qrow, a.q_out + n * a.q_out_stride, a.q_weight, a.Hq, t0, min(t1, gq), true);
  if (t1 > gq)
    heads(krow, a.k_out + n * a.k_out_stride, a.k_weight, a.Hkv, max(t0, gq) - gq, t1 - gq, t0 >= gq);
}

template <int D, bool INTER>
cudaError_t launch_t(const NormRopeLaunch& p, int num_sms, cudaStream_t stream) {
  constexpr int PER = 512 / D;
  const int groups = (p.Hq + PER - 1) / PER + (p.Hkv + PER - 1) / PER;
  // All heads of a token by one warp, unless that leaves the SMs short of warps
  // (a decode step): then a group each.
  const bool few = static_cast<long long>(p.N) < 16LL * num_sms;
  const int per = few ? 1 : groups, parts = few ? groups : 1;
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
