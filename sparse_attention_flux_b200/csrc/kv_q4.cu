// kv_q4.cu -- rows into and out of the paged 4-bit KV cache (layout in q4.h).
//
// Write: per group of 32 channels a = max|x|, scale = a / 7 cut to 5
// significant bits, code = 8 + round-half-even(x / scale).  The cut makes
// x / scale at most 7 * (1 + 1/16) = 7.44, so the code stays within 1..15, and
// the largest element always gets 15 or 1: quantising a stored group again
// returns the same bits.  x has 8 significant bits and a rounding border
// (n + 1/2) scale at most 9, so x / scale is either a border exactly (fp32
// division returns it and rint goes to even) or further from it than fp32's
// rounding: the codes are those of exact arithmetic.
// Read: (code - 8) * scale, exactly a bf16 number.
#include "q4.h"

namespace flux {

namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ uint8_t* record_of(const KvQ4Launch& a, int64_t slot, int h, int bytes) {
  const int64_t page = slot / a.page_size;
  const int at = static_cast<int>(slot - page * a.page_size);
  const int recs = a.page_size / kQ4Rec;
  return a.pool + ((page * a.Hkv + h) * recs + at / kQ4Rec) * bytes;
}

// One warp per (token, kv head): lanes 0 .. D/8 - 1 hold 8 channels of K each,
// the next D/8 lanes 8 channels of V.
template <int D>
__global__ void __launch_bounds__(32 * kWarps) kv_write_q4_kernel(const KvQ4Launch a) {
  using L = Q4Layout<D>;
  constexpr int LANES = D / 8;
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (row >= static_cast<long long>(a.N) * a.Hkv) return;
  const long long n = row / a.Hkv;
  const int h = static_cast<int>(row % a.Hkv);
  const int64_t slot = a.slots[n];
  if (slot < 0) return;
  if (slot >= static_cast<int64_t>(a.num_pages) * a.page_size) {
    if (lane == 0) raise_error(a.err, DEV_ERR_PAGE);
    return;
  }
  const bool is_k = lane < LANES, active = lane < 2 * LANES;
  const int ch = lane % LANES;                   // 8-channel chunk
  uint4 x = {0, 0, 0, 0};
  if (active) {
    const uint16_t* src = is_k ? a.k + n * a.k_stride : a.v + n * a.v_stride;
    x = reinterpret_cast<const uint4*>(src + h * D)[ch];
  }
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  float f[8];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16lo_to_f32(w[i]);
    f[2 * i + 1] = bf16hi_to_f32(w[i]);
    top = max(top, max((w[i] << 16) & 0x7fffffffu, w[i] & 0x7fff0000u));
  }
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  uint32_t sbits = __float_as_uint(__uint_as_float(top) / 7.f) & 0xfff80000u;
  if (top < kQ4LowBits) sbits = 0;
  const bool plain = top >= kQ4LowBits && top <= kQ4HighBits;
  if (top > kQ4HighBits) sbits = 0x7fc00000u;
  const float s = __uint_as_float(sbits);
  uint32_t code[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) code[e] = plain ? 8 + __float2int_rn(f[e] / s) : 8;
  if (!active) return;
  uint8_t* rec = record_of(a, slot, h, L::BYTES);
  const int r = static_cast<int>(slot % kQ4Rec);
  if (is_k) {
    uint32_t word = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) word |= code[e] << (16 * (e & 1) + 4 * (e >> 1));
    const int g = ch / 4, t = ch % 4;
    *reinterpret_cast<uint32_t*>(rec + r * (D / 2) + t * (D / 8) + 4 * g) =
        __funnelshift_l(word, word, 3);
    if (t == 0) reinterpret_cast<uint16_t*>(rec + L::KS)[r * L::G + g] = sbits >> 16;
  } else {
    const int t = (r % 8) / 2;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int c = 8 * ch + 4 * q;              // 4 channels of one half-word
      const int g = c / (D / 8), j = c % (D / 8) / 4;
      const uint32_t half = code[4 * q] | code[4 * q + 1] << 4 | code[4 * q + 2] << 8 |
                            code[4 * q + 3] << 12;
      *reinterpret_cast<uint16_t*>(rec + L::VC + (r / 8) * 4 * D + (4 * g + t) * (D / 8) + 4 * j +
                                   2 * (r & 1)) = static_cast<uint16_t>(half);
    }
    if (ch % 4 == 0) reinterpret_cast<uint16_t*>(rec + L::VS)[(ch / 4) * 16 + r] = sbits >> 16;
  }
}

template <int D>
__global__ void __launch_bounds__(32 * kWarps) kv_read_q4_kernel(const KvQ4Launch a) {
  using L = Q4Layout<D>;
  constexpr int LANES = D / 8;
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (row >= static_cast<long long>(a.N) * a.Hkv) return;
  const long long n = row / a.Hkv;
  const int h = static_cast<int>(row % a.Hkv);
  const int64_t slot = a.slots[n];
  if (slot < 0) return;
  if (slot >= static_cast<int64_t>(a.num_pages) * a.page_size) {
    if (lane == 0) raise_error(a.err, DEV_ERR_PAGE);
    return;
  }
  if (lane >= 2 * LANES) return;
  const bool is_k = lane < LANES;
  const int ch = lane % LANES;
  const uint8_t* rec = record_of(a, slot, h, L::BYTES);
  const int r = static_cast<int>(slot % kQ4Rec);
  int code[8];
  uint16_t sb;
  if (is_k) {
    const int g = ch / 4, t = ch % 4;
    uint32_t word = *reinterpret_cast<const uint32_t*>(rec + r * (D / 2) + t * (D / 8) + 4 * g);
    word = __funnelshift_r(word, word, 3);
#pragma unroll
    for (int e = 0; e < 8; ++e) code[e] = (word >> (16 * (e & 1) + 4 * (e >> 1))) & 15;
    sb = reinterpret_cast<const uint16_t*>(rec + L::KS)[r * L::G + g];
  } else {
    const int t = (r % 8) / 2;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int c = 8 * ch + 4 * q;
      const int g = c / (D / 8), j = c % (D / 8) / 4;
      const uint32_t half = *reinterpret_cast<const uint16_t*>(
          rec + L::VC + (r / 8) * 4 * D + (4 * g + t) * (D / 8) + 4 * j + 2 * (r & 1));
#pragma unroll
      for (int i = 0; i < 4; ++i) code[4 * q + i] = (half >> (4 * i)) & 15;
    }
    sb = reinterpret_cast<const uint16_t*>(rec + L::VS)[(ch / 4) * 16 + r];
  }
  const float s = __uint_as_float(static_cast<uint32_t>(sb) << 16);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = pack_bf16x2((code[2 * i] - 8) * s, (code[2 * i + 1] - 8) * s);
  uint16_t* dst = (is_k ? a.k_out : a.v_out) + row * D;
  reinterpret_cast<uint4*>(dst)[ch] = make_uint4(w[0], w[1], w[2], w[3]);
}

unsigned grid_of(const KvQ4Launch& p) {
  return static_cast<unsigned>((static_cast<long long>(p.N) * p.Hkv + kWarps - 1) / kWarps);
}

}  // namespace

cudaError_t launch_kv_write_q4(const KvQ4Launch& p, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  if (p.d == 64) kv_write_q4_kernel<64><<<grid_of(p), 32 * kWarps, 0, stream>>>(p);
  else kv_write_q4_kernel<128><<<grid_of(p), 32 * kWarps, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_kv_read_q4(const KvQ4Launch& p, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  if (p.d == 64) kv_read_q4_kernel<64><<<grid_of(p), 32 * kWarps, 0, stream>>>(p);
  else kv_read_q4_kernel<128><<<grid_of(p), 32 * kWarps, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace flux
