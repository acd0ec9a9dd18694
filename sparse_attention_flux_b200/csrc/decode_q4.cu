// decode_q4.cu -- decode attention over the paged 4-bit KV cache (layout in
// q4.h): one query token per sequence, the routing bit, the SA mask and the
// output of decode.cu.
//
// One CTA per (kv head, sequence); its warps take 16-token records in turn.  A
// warp's lane owns D / 32 channels, scores are warp sums, and each query head of
// the group keeps the running maximum and sum of its softmax.  The warps'
// partials are merged in shared memory at the end.
#include "q4.h"

namespace flux {

namespace {

constexpr int kWarps = 8;
constexpr int kMaxG = 8;

template <int D>
__global__ void __launch_bounds__(32 * kWarps) decode_q4_kernel(const DecodeQ4Launch a) {
  using L = Q4Layout<D>;
  constexpr int C = D / 32;
  __shared__ float sm_m[kWarps][kMaxG], sm_l[kWarps][kMaxG], sm_o[kWarps][kMaxG][D];
  const int g = blockIdx.x, b = blockIdx.y;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int G = a.Hq / a.Hkv;
  const bool fa = a.layer_mode == nullptr || a.layer_mode[a.layer] != 0;
  const size_t row0 = static_cast<size_t>(b) * a.Hq + g * G;
  int s = a.seqlens[b];
  if (s < 0 || s > static_cast<long long>(a.max_pages) * a.page_size) {
    if (g == 0 && threadIdx.x == 0) raise_error(a.st.err, DEV_ERR_SEQLEN);
    s = 0;
  }
  const int nb = s > 0 ? (s - 1) / a.block + 1 : 0;
  const int n_sink = fa ? s : static_cast<int>(min(static_cast<long long>(a.sink_blocks) * a.block,
                                                   static_cast<long long>(s)));
  const int win = fa ? 0 : max(0, nb - a.window_blocks) * a.block;
  float q[kMaxG][C], o[kMaxG][C], m[kMaxG], l[kMaxG];
  for (int h = 0; h < kMaxG; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
    for (int c = 0; c < C; ++c) {
      o[h][c] = 0.f;
      q[h][c] = h < G ? __uint_as_float(static_cast<uint32_t>(a.q[(row0 + h) * D + lane * C + c]) << 16)
                      : 0.f;
    }
  }
  const float sl2 = a.scale * 1.4426950408889634f;
  const int recs = a.page_size / kQ4Rec;
  for (int rr = warp; rr < (s + kQ4Rec - 1) / kQ4Rec; rr += kWarps) {
    const int u0 = rr * kQ4Rec;
    if (u0 >= n_sink && u0 + kQ4Rec <= win) continue;
    const int page = a.page_table[static_cast<size_t>(b) * a.max_pages + u0 / a.page_size];
    if (page < 0 || page >= a.num_pages) {
      if (lane == 0) raise_error(a.st.err, DEV_ERR_PAGE);
      continue;
    }
    const uint8_t* rec = a.pool + ((static_cast<size_t>(page) * a.Hkv + g) * recs +
                                   u0 % a.page_size / kQ4Rec) * L::BYTES;
    for (int r = 0; r < kQ4Rec; ++r) {
      const int u = u0 + r;
      if (u >= s || !(u < n_sink || u >= win)) continue;
      float k[C], v[C];
      for (int c = 0; c < C; ++c) {
        const int ch = lane * C + c, w = ch / 32, t = ch % 32 / 8, e = ch % 8;
        uint32_t word = *reinterpret_cast<const uint32_t*>(rec + r * (D / 2) + t * (D / 8) + 4 * w);
        word = __funnelshift_r(word, word, 3);
        const int nk = static_cast<int>((word >> (16 * (e & 1) + 4 * (e >> 1))) & 15) - 8;
        const int gv = ch / (D / 8), j = ch % (D / 8) / 4, i = ch % 4;
        const uint32_t half = *reinterpret_cast<const uint16_t*>(
            rec + L::VC + (r / 8) * 4 * D + (4 * gv + r % 8 / 2) * (D / 8) + 4 * j + 2 * (r & 1));
        const int nv = static_cast<int>((half >> (4 * i)) & 15) - 8;
        k[c] = nk * __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(
                        rec + L::KS)[r * L::G + w]) << 16);
        v[c] = nv * __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(
                        rec + L::VS)[w * 16 + r]) << 16);
      }
#pragma unroll
      for (int h = 0; h < kMaxG; ++h) {
        if (h >= G) break;
        float x = 0.f;
        for (int c = 0; c < C; ++c) x += q[h][c] * k[c];
        for (int st = 16; st > 0; st >>= 1) x += __shfl_xor_sync(0xffffffffu, x, st);
        x *= sl2;
        const float mn = fmaxf(m[h], x);
        const float mu = mn == -INFINITY ? 0.f : mn;
        const float alpha = exp2f(m[h] - mu), p = exp2f(x - mu);
        m[h] = mn;
        l[h] = l[h] * alpha + p;
        for (int c = 0; c < C; ++c) o[h][c] = o[h][c] * alpha + p * v[c];
      }
    }
  }
  for (int h = 0; h < kMaxG; ++h) {
    if (lane == 0) {
      sm_m[warp][h] = m[h];
      sm_l[warp][h] = l[h];
    }
    for (int c = 0; c < C; ++c) sm_o[warp][h][lane * C + c] = o[h][c];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < G * D; i += 32 * kWarps) {
    const int h = i / D, c = i % D;
    float M = -INFINITY, ls = 0.f, O = 0.f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w][h]);
    const float mu = M == -INFINITY ? 0.f : M;
    for (int w = 0; w < kWarps; ++w) {
      const float wt = exp2f(sm_m[w][h] - mu);
      ls += wt * sm_l[w][h];
      O += wt * sm_o[w][h][c];
    }
    const float out = ls != 0.f ? O / ls : 0.f;
    a.o[(row0 + h) * D + c] = __bfloat16_as_ushort(__float2bfloat16_rn(out));
    if (c == 0 && a.lse)
      a.lse[row0 + h] = ls != 0.f ? (M + log2f(ls)) * 0.69314718055994531f : -INFINITY;
  }
}

}  // namespace

size_t decode_q4_workspace_bytes(int d, int num_sms) {
  (void)d;
  (void)num_sms;
  return 0;
}

cudaError_t launch_decode_q4(const DecodeQ4Launch& p, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  const dim3 grid(p.Hkv, p.B);
  if (p.d == 64) decode_q4_kernel<64><<<grid, 32 * kWarps, 0, stream>>>(p);
  else decode_q4_kernel<128><<<grid, 32 * kWarps, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace flux
