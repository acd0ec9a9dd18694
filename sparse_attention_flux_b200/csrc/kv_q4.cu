// kv_q4.cu -- rows into and out of the paged 4-bit KV cache (layout in q4.h).
//
// Write: per group of 32 channels a = max|x|, scale = a / 7 cut to 5
// significant bits, code = 8 + round-half-even(x / scale).  The cut makes
// x / scale at most 7 * (1 + 1/16) = 7.44, so the code stays within 1..15, and
// the largest element always gets 15 or 1: quantising a stored group again
// returns the same bits.  x has 8 significant bits and a rounding border
// (n + 1/2) scale at most 9, so x / scale is either a border exactly or 2^-18 of
// itself away from it: an fp32 quotient that is exact where the quotient is a
// float, and within 2^-22 elsewhere, gives the codes of exact arithmetic.
// Read: (code - 8) * scale, exactly a bf16 number.
//
// Bound: HBM.  A token's bytes are scattered over its record (its V codes are
// 2-byte pieces), so one token at a time writes eight times the bytes in
// partial sectors.  Calls of some length therefore work by windows of 16 tokens
// of the call, one warp per window and kv head: 16 tokens in a row that fill a
// record (found from the slots alone, wherever they start) go through shared
// memory as a whole record by the warp in whose window they start; the tokens
// that are in no such run (the ends of a prompt's part of a page, requests of
// one token) go one at a time.  Short calls take a warp per token and kv head.
// 65536 tokens, 8 kv heads, d 128, written and read back: 122 us, 5.6 TB/s of
// 687 MB (a warp per token 369 us; 4 CTAs per SM writing, 100 registers, 131; one
// quotient at a time 124; V rows read back by 16-byte instead of 32-byte stores 138).
#include "q4.h"

namespace flux {

namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ uint8_t* record_of(const KvQ4Launch& a, int64_t slot, int h, int bytes) {
  const int64_t page = slot / a.page_size;
  const int at = static_cast<int>(slot - page * a.page_size);
  const int recs = a.page_size / kQ4Rec;
  return a.pool + ((page * a.Hkv + h) * recs + at / kQ4Rec) * bytes;
}
// Does the slot name a place?  A negative one says to skip the token.
__device__ __forceinline__ bool valid_slot(const KvQ4Launch& a, int64_t slot, bool report) {
  if (slot < 0) return false;
  if (slot < static_cast<int64_t>(a.num_pages) * a.page_size) return true;
  if (report) raise_error(a.err, DEV_ERR_PAGE);
  return false;
}

// 8 consecutive channels of the lane, quantised; the group of 32 is the lane's
// aligned quartet.  bits[e] = kCodeBits + code (mod 2^32).
constexpr uint32_t kCodeBits = 0x4b400000u;      // 1.5 * 2^23: adding it to a float rounds to whole numbers
__device__ __forceinline__ unsigned long long pack2(float lo, float hi) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
struct Quant {
  uint32_t bits[8];
  uint32_t scale;          // bf16 bits
  bool plain;              // else every code is 8
};
__device__ __forceinline__ Quant quantise8(const uint4& x) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  // |x| as bit patterns, which order like the values with infinities and NaN on top
  uint32_t top2 = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                           __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
  top2 = __vmaxu2(top2, __shfl_xor_sync(0xffffffffu, top2, 1));
  top2 = __vmaxu2(top2, __shfl_xor_sync(0xffffffffu, top2, 2));
  const uint32_t top = max(top2 << 16, top2 & 0xffff0000u);
  // top / 7 by a product with a little more than 1 / 7 (by 2^-20 of it): top has 8
  // significant bits, so top / 7 is a 5-bit number exactly, which the product
  // passes by less than the cut takes off, or at least 2^-9 of itself below the next.
  uint32_t sbits = __float_as_uint(__uint_as_float(top) * 0x1.24925cp-3f) & 0xfff80000u;
  Quant out;
  out.plain = top >= kQ4LowBits && top <= kQ4HighBits;
  if (top < kQ4LowBits) sbits = 0;
  if (top > kQ4HighBits) sbits = 0x7fc00000u;
  out.scale = sbits >> 16;
  const float s = __uint_as_float(sbits);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  // f / s by a product and one residual step (Markstein), two at a time: where
  // f / s is a float, the residual is exact and so is the result, whatever the last
  // bits of r; else it is off by a rounding or two, and no border is that near.
  const unsigned long long r2 = pack2(r, r), s2 = pack2(-s, -s);
  const unsigned long long m2 = pack2(12582920.f, 12582920.f);      // 1.5 * 2^23 + 8
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const unsigned long long f = pack2(bf16lo_to_f32(w[i]), bf16hi_to_f32(w[i]));
    unsigned long long q, t;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(q) : "l"(f), "l"(r2));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(t) : "l"(q), "l"(s2), "l"(f));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(q) : "l"(t), "l"(r2), "l"(q));
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(q) : "l"(q), "l"(m2));
    asm("mov.b64 {%0, %1}, %2;" : "=r"(out.bits[2 * i]), "=r"(out.bits[2 * i + 1]) : "l"(q));
  }
  return out;
}
// The K word of 8 channels, and the two V half-words of a token (16 bits each).
// A sum of bits[e] << place is the sum of the codes' plus a constant (mod 2^32).
__device__ __forceinline__ uint32_t k_word(const Quant& x) {
  uint32_t word = 0u - kCodeBits * 0x11111111u;
#pragma unroll
  for (int e = 0; e < 8; ++e) word += x.bits[e] << (16 * (e & 1) + 4 * (e >> 1));
  word = x.plain ? word : 0x88888888u;
  return __funnelshift_l(word, word, 3);
}
__device__ __forceinline__ uint32_t v_half(const Quant& x, int q) {
  uint32_t half = 0u - kCodeBits * 0x1111u;
#pragma unroll
  for (int i = 0; i < 4; ++i) half += x.bits[4 * q + i] << (4 * i);
  return x.plain ? half : 0x8888u;
}
// Byte of channels 8 ch + 4 q .. + 3 of token r (its 16-bit half) in the record.
template <int D>
__device__ __forceinline__ int v_byte(int r, int ch, int q) {
  const int c = 8 * ch + 4 * q, g = c / (D / 8), j = c % (D / 8) / 4;
  return Q4Layout<D>::VC + (r / 8) * 4 * D + (4 * g + r % 8 / 2) * (D / 8) + 4 * j + 2 * (r & 1);
}

// One token of one kv head by one warp: lanes 0 .. D/8 - 1 hold 8 channels of K
// each, the next D/8 lanes of V.
template <int D>
__device__ __forceinline__ void write_token(const KvQ4Launch& a, int n, int h, int64_t slot, int lane) {
  using L = Q4Layout<D>;
  constexpr int LANES = D / 8;
  const bool is_k = lane < LANES, active = lane < 2 * LANES;
  const int ch = lane % LANES;
  uint4 x = {0, 0, 0, 0};
  if (active) {
    const uint16_t* src = is_k ? a.k + n * a.k_stride : a.v + n * a.v_stride;
    x = reinterpret_cast<const uint4*>(src + h * D)[ch];
  }
  const Quant z = quantise8(x);
  if (!active) return;
  uint8_t* rec = record_of(a, slot, h, L::BYTES);
  const int r = static_cast<int>(slot % kQ4Rec);
  if (is_k) {
    const int g = ch / 4, t = ch % 4;
    *reinterpret_cast<uint32_t*>(rec + r * (D / 2) + t * (D / 8) + 4 * g) = k_word(z);
    if (t == 0) reinterpret_cast<uint16_t*>(rec + L::KS)[r * L::G + g] = static_cast<uint16_t>(z.scale);
  } else {
#pragma unroll
    for (int q = 0; q < 2; ++q)
      *reinterpret_cast<uint16_t*>(rec + v_byte<D>(r, ch, q)) = static_cast<uint16_t>(v_half(z, q));
    if (ch % 4 == 0) reinterpret_cast<uint16_t*>(rec + L::VS)[(ch / 4) * 16 + r] = static_cast<uint16_t>(z.scale);
  }
}

template <int D>
__device__ __forceinline__ void read_token(const KvQ4Launch& a, int n, int h, int64_t slot, int lane) {
  using L = Q4Layout<D>;
  constexpr int LANES = D / 8;
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
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint32_t half = *reinterpret_cast<const uint16_t*>(rec + v_byte<D>(r, ch, q));
#pragma unroll
      for (int i = 0; i < 4; ++i) code[4 * q + i] = (half >> (4 * i)) & 15;
    }
    sb = reinterpret_cast<const uint16_t*>(rec + L::VS)[(ch / 4) * 16 + r];
  }
  const float s = __uint_as_float(static_cast<uint32_t>(sb) << 16);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2((code[2 * i] - 8) * s, (code[2 * i + 1] - 8) * s);
  uint16_t* dst = (is_k ? a.k_out : a.v_out) + (static_cast<long long>(n) * a.Hkv + h) * D;
  reinterpret_cast<uint4*>(dst)[ch] = make_uint4(w[0], w[1], w[2], w[3]);
}

// 16 tokens n .. n + 15 that fill the record of `slot` (its first token's).
template <int D>
__device__ __forceinline__ void write_record(const KvQ4Launch& a, int n, int h, int64_t slot, int lane,
                                             uint8_t* buf) {
  using L = Q4Layout<D>;
  constexpr int CH = D / 8, PER = 32 / CH;       // 8-channel chunks per row, rows at a time
  const int ch = lane % CH, sub = lane / CH;
  uint4 xk[16 / PER], xv[16 / PER];
#pragma unroll
  for (int i = 0; i < 16 / PER; ++i)
    xk[i] = __ldcs(reinterpret_cast<const uint4*>(a.k + (n + i * PER + sub) * a.k_stride + h * D) + ch);
#pragma unroll
  for (int i = 0; i < 16 / PER; ++i)
    xv[i] = __ldcs(reinterpret_cast<const uint4*>(a.v + (n + i * PER + sub) * a.v_stride + h * D) + ch);
#pragma unroll
  for (int i = 0; i < 16 / PER; ++i) {
    const int r = i * PER + sub;
    Quant z = quantise8(xk[i]);
    *reinterpret_cast<uint32_t*>(buf + r * (D / 2) + (ch % 4) * (D / 8) + 4 * (ch / 4)) = k_word(z);
    if (ch % 4 == 0)
      reinterpret_cast<uint16_t*>(buf + L::KS)[r * L::G + ch / 4] = static_cast<uint16_t>(z.scale);
    z = quantise8(xv[i]);
#pragma unroll
    for (int q = 0; q < 2; ++q)
      *reinterpret_cast<uint16_t*>(buf + v_byte<D>(r, ch, q)) = static_cast<uint16_t>(v_half(z, q));
    if (ch % 4 == 0)
      reinterpret_cast<uint16_t*>(buf + L::VS)[(ch / 4) * 16 + r] = static_cast<uint16_t>(z.scale);
  }
  __syncwarp();
  uint4* rec = reinterpret_cast<uint4*>(record_of(a, slot, h, L::BYTES));
  for (int i = lane; i < L::BYTES / 16; i += 32) rec[i] = reinterpret_cast<const uint4*>(buf)[i];
  __syncwarp();
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
// 4-bit fields in mantissa bits 3..6 of both halves -> (code - 8): 16 + u less 24, exact.
__device__ __forceinline__ uint32_t codes_of(uint32_t x) {
  uint32_t r;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"((x & 0x00780078u) | 0x41804180u), "r"(0xc1c0c1c0u));
  return r;
}

__device__ __forceinline__ void store_sector(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// The record of `slot` to rows n .. n + 15.  Lane 4 g + t reads what it reads in
// the decode kernel: K of tokens g and g + 8, V of tokens 2 t and 2 t + 1 (+ 8).
template <int D>
__device__ __forceinline__ void read_record(const KvQ4Launch& a, int n, int h, int64_t slot, int lane) {
  using L = Q4Layout<D>;
  constexpr int GR = L::G;
  const int g = lane >> 2, t = lane & 3;
  const uint8_t* rec = record_of(a, slot, h, L::BYTES);
  uint32_t kw[2][GR], vw[2][GR], ks[2][GR / 2], vs[2];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const uint8_t* kp = rec + m * 4 * D + lane * (D / 8);
    const uint8_t* vp = kp + L::VC;
    const uint8_t* sp = rec + L::KS + (g + 8 * m) * (2 * GR);
    if constexpr (D == 128) {
      const uint4 x = *reinterpret_cast<const uint4*>(kp), y = *reinterpret_cast<const uint4*>(vp);
      kw[m][0] = x.x, kw[m][1] = x.y, kw[m][2] = x.z, kw[m][3] = x.w;
      vw[m][0] = y.x, vw[m][1] = y.y, vw[m][2] = y.z, vw[m][3] = y.w;
      const uint2 s = *reinterpret_cast<const uint2*>(sp);
      ks[m][0] = s.x, ks[m][1] = s.y;
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(kp), y = *reinterpret_cast<const uint2*>(vp);
      kw[m][0] = x.x, kw[m][1] = x.y;
      vw[m][0] = y.x, vw[m][1] = y.y;
      ks[m][0] = *reinterpret_cast<const uint32_t*>(sp);
    }
    vs[m] = *reinterpret_cast<const uint32_t*>(rec + L::VS + (g * (D / 8) / 32) * 32 + 16 * m + 4 * t);
  }
  const long long row = static_cast<long long>(a.Hkv) * D;      // elements from token to token
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    uint16_t* dst = a.k_out + (n + g + 8 * m) * row + h * D;
#pragma unroll
    for (int i = 0; i < GR; ++i) {
      const uint32_t w = kw[m][i];
      const uint32_t s = __byte_perm(ks[m][i / 2], 0, i % 2 ? 0x3232 : 0x1010);
      *reinterpret_cast<uint4*>(dst + 32 * i + 8 * t) =
          make_uint4(mul_bf16x2(codes_of(w), s), mul_bf16x2(codes_of(w >> 4), s),
                     mul_bf16x2(codes_of(w >> 8), s), mul_bf16x2(codes_of(__funnelshift_r(w, w, 12)), s));
    }
    // V: tokens 2 t (low halves) and 2 t + 1, channels g D/8 + 4 j + i
    uint32_t lo[2 * GR], hi[2 * GR];
#pragma unroll
    for (int j = 0; j < GR; ++j) {
      const uint32_t w = vw[m][j];
      const uint32_t x0 = mul_bf16x2(codes_of(w << 3), vs[m]), x1 = mul_bf16x2(codes_of(w >> 1), vs[m]);
      const uint32_t x2 = mul_bf16x2(codes_of(w >> 5), vs[m]), x3 = mul_bf16x2(codes_of(w >> 9), vs[m]);
      lo[2 * j] = __byte_perm(x0, x1, 0x5410);
      lo[2 * j + 1] = __byte_perm(x2, x3, 0x5410);
      hi[2 * j] = __byte_perm(x0, x1, 0x7632);
      hi[2 * j + 1] = __byte_perm(x2, x3, 0x7632);
    }
    uint16_t* d0 = a.v_out + (n + 2 * t + 8 * m) * row + h * D + g * (D / 8);
    uint16_t* d1 = d0 + row;
    bool stored = false;
    if constexpr (D == 128) {
      if ((reinterpret_cast<uintptr_t>(a.v_out) & 31) == 0) {      // whole 32-byte sectors
        store_sector(d0, lo);
        store_sector(d1, hi);
        stored = true;
      }
    }
    if (!stored) {
#pragma unroll
      for (int j = 0; j < GR / 2; ++j) {
        reinterpret_cast<uint4*>(d0)[j] = make_uint4(lo[4 * j], lo[4 * j + 1], lo[4 * j + 2], lo[4 * j + 3]);
        reinterpret_cast<uint4*>(d1)[j] = make_uint4(hi[4 * j], hi[4 * j + 1], hi[4 * j + 2], hi[4 * j + 3]);
      }
    }
  }
}

// The runs around a window of 16 tokens at n0: lane i looks at token n0 - 15 + i.
// record: the token of the window at which a full record's run starts, or -1;
// alone: bit i = token n0 + i is in no such run of this or the window before.
struct Window {
  int record;
  uint32_t alone;
};
__device__ __forceinline__ Window window_of(const KvQ4Launch& a, int n0, int lane) {
  // slots of tokens n0 - 15 .. n0 + 30, two per lane
  const int na = n0 - 15 + lane, nb = na + 32;
  const int64_t sa = na >= 0 && na < a.N ? a.slots[na] : -1;
  const int64_t sb = lane < 14 && nb < a.N ? a.slots[nb] : -1;
  // follows: token i + 1 stands in the slot behind token i's
  const int64_t na1 = __shfl_down_sync(0xffffffffu, sa, 1), b0 = __shfl_sync(0xffffffffu, sb, 0);
  const int64_t nb1 = __shfl_down_sync(0xffffffffu, sb, 1);
  const int64_t next_a = lane < 31 ? na1 : b0;
  const int64_t limit = static_cast<int64_t>(a.num_pages) * a.page_size;
  const bool in = sa >= 0 && sa < limit;
  const uint32_t fa = __ballot_sync(0xffffffffu, sa >= 0 && next_a == sa + 1);
  const uint32_t fb = __ballot_sync(0xffffffffu, lane < 13 && sb >= 0 && nb1 == sb + 1);
  const uint64_t follows = static_cast<uint64_t>(fb) << 32 | fa;
  // starts: the token opens a record and the 15 behind it follow
  const uint32_t starts = __ballot_sync(
      0xffffffffu, lane < 31 && in && sa % kQ4Rec == 0 && (follows >> lane & 0x7fffu) == 0x7fffu);
  uint64_t covered = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) covered |= static_cast<uint64_t>(starts) << i;
  Window w;
  w.record = (starts >> 15) ? n0 + __ffs(starts >> 15) - 1 : -1;
  w.alone = ~static_cast<uint32_t>(covered >> 15) & 0xffffu;
  const int left = a.N - n0;
  if (left < 16) w.alone &= (1u << left) - 1u;
  return w;
}

template <int D, bool WRITE>
__global__ void __launch_bounds__(32 * kWarps, WRITE ? 6 : 1) kv_q4_window_kernel(const KvQ4Launch a) {
  __shared__ __align__(16) uint8_t buf[WRITE ? kWarps : 1][WRITE ? Q4Layout<D>::BYTES : 16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_launch_dependents();
  griddep_wait();
  const long long unit = static_cast<long long>(blockIdx.x) * kWarps + warp;
  const int n0 = static_cast<int>(unit / a.Hkv) * 16, h = static_cast<int>(unit % a.Hkv);
  if (n0 >= a.N) return;
  const Window w = window_of(a, n0, lane);
  if (w.record >= 0) {
    const int64_t slot = a.slots[w.record];
    if constexpr (WRITE) write_record<D>(a, w.record, h, slot, lane, buf[warp]);
    else read_record<D>(a, w.record, h, slot, lane);
  }
  for (uint32_t m = w.alone; m; m &= m - 1) {
    const int n = n0 + __ffs(m) - 1;
    const int64_t slot = a.slots[n];
    if (!valid_slot(a, slot, lane == 0)) continue;
    if constexpr (WRITE) write_token<D>(a, n, h, slot, lane);
    else read_token<D>(a, n, h, slot, lane);
  }
}

template <int D, bool WRITE>
__global__ void __launch_bounds__(32 * kWarps) kv_q4_token_kernel(const KvQ4Launch a) {
  const int lane = threadIdx.x & 31;
  griddep_launch_dependents();
  griddep_wait();
  const long long unit = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (unit >= static_cast<long long>(a.N) * a.Hkv) return;
  const int n = static_cast<int>(unit / a.Hkv), h = static_cast<int>(unit % a.Hkv);
  const int64_t slot = a.slots[n];
  if (!valid_slot(a, slot, lane == 0)) return;
  if constexpr (WRITE) write_token<D>(a, n, h, slot, lane);
  else read_token<D>(a, n, h, slot, lane);
}

template <int D, bool WRITE>
cudaError_t launch_t(const KvQ4Launch& p, int num_sms, cudaStream_t stream) {
  // Windows, once there are enough of them to give every SM a few warps; below
  // that a warp per token, whose latency is one token's.
  const long long windows = (static_cast<long long>(p.N) + 15) / 16 * p.Hkv;
  const bool by_window = windows >= 2LL * num_sms;
  const long long units = by_window ? windows : static_cast<long long>(p.N) * p.Hkv;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((units + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return by_window ? cudaLaunchKernelEx(&cfg, kv_q4_window_kernel<D, WRITE>, p)
                   : cudaLaunchKernelEx(&cfg, kv_q4_token_kernel<D, WRITE>, p);
}

}  // namespace

cudaError_t launch_kv_write_q4(const KvQ4Launch& p, int num_sms, cudaStream_t stream) {
  return p.d == 64 ? launch_t<64, true>(p, num_sms, stream) : launch_t<128, true>(p, num_sms, stream);
}

cudaError_t launch_kv_read_q4(const KvQ4Launch& p, int num_sms, cudaStream_t stream) {
  return p.d == 64 ? launch_t<64, false>(p, num_sms, stream) : launch_t<128, false>(p, num_sms, stream);
}

}  // namespace flux
