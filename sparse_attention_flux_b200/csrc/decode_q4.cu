// decode_q4.cu -- decode attention over the paged 4-bit KV cache (layout in
// q4.h): one query token per sequence, the routing bit, the SA mask and the
// output of decode.cu.
//
// Bound: the cache bytes (18 d per 16 tokens and kv head); the work per byte
// is the unpacking, so the kernel is built to keep HBM busy with as few issued
// instructions per record as possible.
//
// Work split.  The live records of all (sequence, kv head) rows, in pairs, are
// laid end to end and cut into equal ranges, one per CTA (one wave), so a ragged
// batch loads every SM alike.  A row counts kRowCost empty slots more than its
// pairs for what it costs beside them; without any, the CTA that got a batch's
// short requests, 45 rows of one or two pairs, took 90 us of a call whose others
// ended after 25.  Where the rows are alike and few, each is cut by itself instead.
// A CTA walks its range row by row; within a row its warps take pairs in turn and
// merge at the row's end in shared memory.  A row that crosses a range border (at
// most the first and the last of a CTA) leaves a partial in the workspace; the CTA
// that delivers a row's last partial (a ticket) merges them in range order, so the
// result does not depend on timing.
//
// Stream.  Records are taken in pairs.  Each warp keeps a ring of two pairs in
// shared memory, filled by bulk copies (one, when the page holds both records):
// when the warp has taken a pair's operands into registers it refills the stage
// itself, so a full barrier per stage is all the synchronisation there is.  The
// places of a warp's next 16 pairs are looked up at once, a lane each record.
//
// Arithmetic per record, one warp, warp MMAs (m16n8k16, bf16, fp32 sums).  A
// 4-bit field u = code + 8 that stands alone in the low byte of a bf16 number is
// u times a power of two (exponent 0 or 1: the subnormals and the first normals
// lie on one line), so an AND makes an operand, and one shift serves two pairs.
//   S = K q^T: the 16 tokens are the rows, the group's query heads (up to 8)
//     the columns.  The query is scaled by a power of two per head (exact) to
//     meet the operands' 2^-133; the products of one 32-channel group are
//     multiplied by the token's scale in fp32, and the 8 sum(q) that u adds per
//     group comes off by an MMA of the scales with it (three bf16 pieces, 24
//     bits).
//   O^T += V^T P^T: the lane's channels are the rows; u s - 8 s is one packed
//     fma with s brought up by 2^108, and exactly the stored value times 2^-25.
//     The softmax sum keeps the weights P in fp32; the MMA takes them as two bf16
//     pieces, 16 bits, so that the output's one rounding is the error left.  (One
//     piece, 8 bits, made a batch's outputs 1.4 times as far off: 0.00234 against
//     0.00166 in the mean.  The second costs 1-2 % of short calls, 4 % of long ones
//     with up to 4 heads a group, where it rides in the operand's idle columns, and
//     9 % with more.)  movmatrix turns them.
// Unpacking by shift and AND-OR into 16 + u instead, seven or eight operations
// for four pairs where these take six and five: 249 us against 224 (16 x 65536
// tokens, 8 kv heads, d 128; both with P in one piece).
// The softmax runs against a reference that only grows when a score passes it
// by 8 (in log2 units): p <= 2^8, and the common record needs no rescaling and
// one vote.
#include "q4.h"

namespace flux {

namespace {

// Two shapes, 16 warps of 128 registers per SM each: 2 CTAs of 8 warps, or 1 of 16.
// With no more rows than SMs the second: half the range borders and parts to merge
// (an SA layer of 16 sequences, 8 kv heads: 18.3 us against 20.6; 65536 tokens FA:
// 224-242 against 232-250; one sequence of 131072 tokens, 1 kv head: 21.1 against 32.4;
// but 31.3 against 30.1 where the 16 are ragged up to 32768, and 14.5 against 13.0 where
// 24 are up to 9000, 4 kv heads, d 64).  With more rows the first: a row's merge holds
// up 8 warps, and the SM's other CTA goes on meanwhile (60 sequences up to 3000 tokens,
// 8 kv heads: 23.7 us against 34.3; 64 sequences SA: 50 against 59); nor do 16 warps help
// rows of a few pairs (100 tokens: 7.1 against 6.0).
template <int W>
struct Shape {
  static constexpr int kThreads = 32 * W;
  static constexpr int kCtasPerSm = 16 / W;
  // What a row costs beside its pairs, in pairs.  A ragged batch of 16 up to 32768
  // tokens, 8 kv heads: 38.1, 30.5, 30.1, 30.1, 30.6 us with 8, 14, 16, 20, 28 at 8
  // warps; 32.3, 31.3, 32.0, 35.2 with 32, 48, 64, 96 at 16.  One of 24 up to 9000, 4 kv
  // heads, d 64: 14.8, 14.5, 14.5 with 32, 48, 64 at 16.
  static constexpr int kRowCost = W == 16 ? 48 : 16;
};
constexpr int kMaxParts = 320;              // of a row, so of CTAs: the merge buffer begins with their weights
constexpr int kComb = kMaxParts * 8 * 4;    // (a full die pair has 160 SMs)
constexpr int kDepth = 2;                   // ring stages of a warp, a pair of records each
constexpr uint32_t kNoRecord = 0xffffffffu;
constexpr int kMergeCost = 24;              // of a row in parts (3 us), in pairs of a range
constexpr float kGrow = 8.f;                // log2 growth of a score that is tolerated
constexpr float kLowest = -3.0e38f;         // reference of a row without tokens: finite, so that
                                            // no difference of two references is NaN

// Raw accumulator order: float4 (tile m, lane 4 g + t) = channels g D/8 + 2 m
// and + 1 of heads 2 t and 2 t + 1, as the MMA leaves them.
template <int D, int W>
struct Q4Smem {
  static constexpr int NT = D / 16;                       // channel tiles
  static constexpr int RING = W * kDepth * 2 * Q4Layout<D>::BYTES;
  static constexpr int PART4 = NT * 32;                   // float4 per partial
  static constexpr int ACC = W * PART4 * 16;
  static constexpr int ML = RING + ACC;                   // m, l [warp][8]
  static constexpr int FIN = ML + 2 * W * 8 * 4;     // 1 / l of the final merge
  static constexpr int BAR = FIN + 8 * 4;
  static constexpr int MISC = BAR + W * kDepth * 8;          // start row, totals, ticket
  static constexpr int WHERE = MISC + 64;                 // where each warp is
  static constexpr int BYTES = WHERE + W * 32;
};

// The live records of one sequence: [0, head) and [tail, end) of its records;
// the tokens inside them are live below n_sink and from win on.  They are taken
// two at a time: pair j is the live records 2 j and 2 j + 1 (the last may be
// one).  Pairs below plain1 and from plain2 to plain3 have live tokens only.
struct Live {
  int s, n_sink, win, head, tail, count, pairs;
  int plain1, plain2, plain3;
};

__device__ __forceinline__ Live live_of(const DecodeQ4Launch& a, int b, bool fa) {
  Live v;
  int s = a.seqlens[b];
  if (s < 0 || s > static_cast<long long>(a.max_pages) * a.page_size) s = 0;
  const int recs = s > 0 ? (s - 1) / kQ4Rec + 1 : 0;
  v.s = s;
  v.n_sink = s;
  v.win = 0;
  v.head = recs;
  v.tail = recs;
  v.plain2 = v.plain3 = 0;
  if (!fa && s > 0) {
    const int nb = (s - 1) / a.block + 1;
    const int win = max(0, nb - a.window_blocks) * a.block;
    const int sink = static_cast<int>(min(static_cast<long long>(a.sink_blocks) * a.block,
                                          static_cast<long long>(s)));
    if (win > sink) {
      v.n_sink = sink;
      v.win = win;
      v.head = sink > 0 ? (sink - 1) / kQ4Rec + 1 : 0;
      v.tail = max(win / kQ4Rec, v.head);
      const int first = v.tail * kQ4Rec < win ? v.head + 1 : v.head;   // first record behind the border
      v.plain2 = (first + 1) / 2;
      v.plain3 = (v.head + s / kQ4Rec - v.tail) / 2;
    }
  }
  v.plain1 = v.n_sink / (2 * kQ4Rec);
  v.count = v.head + recs - v.tail;
  v.pairs = (v.count + 1) / 2;
  return v;
}

// How the rows are laid end to end: each row's pairs and some empty slots.
// even == 0: a row has `cost` empty slots; else every row has `even` slots.
struct Plan {
  uint32_t even, cost;
};
__device__ __forceinline__ uint32_t slots_of(const Plan& p, uint32_t pairs) {
  return pairs == 0 ? 0u : p.even ? p.even : pairs + p.cost;
}

// Row (b, g), its pairs and its slots; rows without records are skipped.
struct Row {
  int b, g;
  uint32_t pairs, slots;
};

__device__ __forceinline__ void next_row(const DecodeQ4Launch& a, bool fa, const Plan& p, Row& w) {
  if (++w.g == a.Hkv) {
    w.g = 0;
    do {
      ++w.b;
      if (w.b >= a.B) {    // behind the last row: never reached while records remain
        w.pairs = w.slots = 0xffffffffu;
        return;
      }
      w.pairs = live_of(a, w.b, fa).pairs;
      w.slots = slots_of(p, w.pairs);
    } while (w.slots == 0);
  }
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t x, uint32_t y, uint32_t z) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(y), "r"(z));
  return r;
}

__device__ __forceinline__ void mma_add(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

// d = a b.
__device__ __forceinline__ void mma_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Two fp32 numbers in one operation.
__device__ __forceinline__ unsigned long long bits_of(float2 x) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x.x), "f"(x.y));
  return r;
}
__device__ __forceinline__ float2 pair_of(unsigned long long x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits_of(x)), "l"(bits_of(y)), "l"(bits_of(z)));
  return pair_of(r);
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits_of(x)), "l"(bits_of(y)));
  return pair_of(r);
}

// The weights of 8 tokens and the group's heads as the second operand of a value MMA,
// in two bf16 pieces, p = high + low to 2^-16 of p.
//   Paired (up to 4 heads): the query stands in the 8 columns twice, and column h + 4
//     takes the low piece of head h; its accumulators join those of h where the
//     warps merge.  minus is -1 in the lanes of those columns, else 0.
//   Else the low pieces take an MMA of their own, and minus is -1.
template <bool PAIRED>
struct Weights {
  uint32_t high, low;
  __device__ __forceinline__ Weights(float2 p, float minus) {
    high = pack_bf16x2(p.x, p.y);
    const float2 rest = fma2(make_float2(minus, minus), make_float2(bf16lo_to_f32(high), bf16hi_to_f32(high)), p);
    if constexpr (PAIRED) {
      high = movmatrix_trans(pack_bf16x2(rest.x, rest.y));
    } else {
      low = movmatrix_trans(pack_bf16x2(rest.x, rest.y));
      high = movmatrix_trans(high);
    }
  }
};
template <bool PAIRED>
__device__ __forceinline__ void add_values(float (&d)[4], const uint32_t (&a)[4], const Weights<PAIRED>& b0,
                                           const Weights<PAIRED>& b1) {
  mma_add(d, a, b0.high, b1.high);
  if constexpr (!PAIRED) mma_add(d, a, b0.low, b1.low);
}

// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}

// Two 4-bit fields, one of each 16-bit half.  A field alone at bits 0..3 (even I)
// or 4..7 (odd I) is a bf16 number whose exponent is zero or one, and linear in u
// through both: u 2^-133, or u 2^-129.
template <int I>
__device__ __forceinline__ uint32_t fields(uint32_t y) {    // y: the word, or for I > 1 the word >> 8
  return y & (I % 2 ? 0x00f000f0u : 0x000f000fu);
}
// The values are brought up by S = scale 2^108 (odd fields: 2^104), so that the
// operand (u - 8) scale 2^-25 is exact for every stored scale below 2^20; larger
// ones, and NaN, take another way.
constexpr uint32_t kUpEven = 0x75807580u, kUpOdd = 0x73807380u;    // 2^108, 2^104
constexpr uint32_t kDown8 = 0xb480b480u;                            // -8 2^-25 = -2^-22
constexpr uint32_t kLarge = 0x36803680u;        // carries a half >= 2^20 into its upper bit
constexpr float kValueUnit = 33554432.f;        // 2^25

template <int D>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[D / 32]) {
  if constexpr (D == 128) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x;
    w[1] = v.y;
  }
}
// The G bf16 scales of a token as fp32.
template <int D>
__device__ __forceinline__ void load_scales(const uint8_t* p, float (&s)[D / 32]) {
  if constexpr (D == 128) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    s[0] = bf16lo_to_f32(v.x);
    s[1] = bf16hi_to_f32(v.x);
    s[2] = bf16lo_to_f32(v.y);
    s[3] = bf16hi_to_f32(v.y);
  } else {
    const uint32_t v = *reinterpret_cast<const uint32_t*>(p);
    s[0] = bf16lo_to_f32(v);
    s[1] = bf16hi_to_f32(v);
  }
}

__device__ __forceinline__ long long div_of(long long x, long long y) {
  return (static_cast<unsigned long long>(x) | static_cast<unsigned long long>(y)) >> 32
             ? x / y
             : static_cast<long long>(static_cast<uint32_t>(x) / static_cast<uint32_t>(y));
}
// R slots cut into N ranges of q or q + 1: the first slot of range c, and the range of a slot.
struct Cuts {
  long long q;
  int N, rem;
};
__device__ __forceinline__ Cuts cuts_of(long long R, int N) {
  Cuts c;
  c.N = N;
  c.q = div_of(R, N);
  c.rem = static_cast<int>(R - c.q * N);
  return c;
}
__device__ __forceinline__ long long range_of(const Cuts& c, int i) { return c.q * i + min(i, c.rem); }
__device__ __forceinline__ int cta_of(const Cuts& c, long long x) {
  const long long wide = (c.q + 1) * c.rem;
  return static_cast<int>(x < wide ? div_of(x, c.q + 1) : c.rem + div_of(x - wide, c.q));
}

template <int D, int W, bool PAIRED>
__global__ void __launch_bounds__(Shape<W>::kThreads, Shape<W>::kCtasPerSm)
    decode_q4_kernel(const DecodeQ4Launch a) {
  using L = Q4Layout<D>;
  using S = Q4Smem<D, W>;
  constexpr int kThreads = Shape<W>::kThreads, kRowCost = Shape<W>::kRowCost;
  constexpr int NT = S::NT, GR = L::G;
  extern __shared__ __align__(128) uint8_t smem[];
  float4* sm_acc = reinterpret_cast<float4*>(smem + S::RING);
  float* sm_m = reinterpret_cast<float*>(smem + S::ML);
  float* sm_l = sm_m + W * 8;
  float* sm_fl = reinterpret_cast<float*>(smem + S::FIN);       // [8] 1 / sum of the merged row
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::BAR);
  long long* sm_total = reinterpret_cast<long long*>(smem + S::MISC);        // [0] R, [1] R0 in sequence *sm_start
  int* sm_start = reinterpret_cast<int*>(smem + S::MISC + 16);               // b of the start
  int* sm_ticket = sm_start + 1;
  int* sm_ranges = sm_start + 2;                                             // N
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid < W * kDepth) mbar_init(full + tid, 1);
  fence_barrier_init();
  griddep_launch_dependents();
  griddep_wait();

  const bool fa = a.layer_mode == nullptr || a.layer_mode[a.layer] != 0;
  const int G = a.Hq / a.Hkv;

  // ---- slots of all rows, and where this CTA's range starts -------------
  // Thread t owns `per` consecutive sequences; one block scan of their slots and
  // (upper bits) of how many have any, and the longest row.
  const int per = a.B <= kThreads ? 1 : (a.B + kThreads - 1) / kThreads;
  const int bt0 = tid * per, bt1 = min(bt0 + per, a.B);
  constexpr int kCountBit = 46;           // 2^16 rows of 2^27 pairs stay below it
  long long mine = 0;
  uint32_t longest = 0;
  for (int b = bt0; b < bt1; ++b) {
    const uint32_t pairs = live_of(a, b, fa).pairs;
    if (pairs) mine += (1LL << kCountBit) + static_cast<long long>(pairs + kRowCost) * a.Hkv;
    longest = max(longest, pairs);
  }
  long long incl = mine;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, incl, s);
    if (lane >= s) incl += x;
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  long long* wsum = reinterpret_cast<long long*>(sm_acc);        // [W], and the longest
  uint32_t* wmax = reinterpret_cast<uint32_t*>(wsum + W);
  if (lane == 31) {
    wsum[warp] = incl;
    wmax[warp] = longest;
  }
  __syncthreads();
  long long before = incl - mine, all = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    const long long x = wsum[w];
    if (w < warp) before += x;
    all += x;
    longest = max(longest, wmax[w]);
  }
  constexpr long long kSlotMask = (1LL << kCountBit) - 1;
  const int grid = gridDim.x, cta = blockIdx.x;
  const long long rows = (all >> kCountBit) * a.Hkv;
  Plan plan = {0u, kRowCost};
  Cuts cuts = {};
  long long R = all & kSlotMask, at0 = before & kSlotMask, n0 = mine & kSlotMask;
  int N = static_cast<int>(min(static_cast<long long>(grid), (R + W - 1) / W));
  if (rows > 0 && rows <= grid) {
    // Every row by itself, in k equal parts or, up to three pairs a warp, whole; if
    // that is no longer than an equal share of everything, with what the merges cost
    // (an SA layer, a batch of equal lengths, few requests).
    const uint32_t k = static_cast<uint32_t>(grid) / static_cast<uint32_t>(rows);
    const uint32_t part = longest <= 3 * W ? longest : max((longest + k - 1) / k, static_cast<uint32_t>(W));
    const uint32_t parts = (longest + part - 1) / part;
    const int cost = static_cast<int>(part) + (parts > 1 ? kMergeCost : 0) - 3 * kMergeCost / 2;
    if (static_cast<long long>(cost) * grid <= max(R, static_cast<long long>(W) * grid)) {
      plan.even = part * parts;
      R = rows * plan.even;
      N = static_cast<int>(rows * parts);
      at0 = (before >> kCountBit) * a.Hkv * plan.even;
      n0 = (mine >> kCountBit) * a.Hkv * plan.even;
      cuts.q = part;
    }
  }
  const bool works = cta < N, empties = (all >> kCountBit) != a.B;
  if (N > 0 && !plan.even) cuts = cuts_of(R, N);
  cuts.N = N;
  const long long R0 = works ? range_of(cuts, cta) : 0, R1 = works ? range_of(cuts, cta + 1) : 0;
  if (works && R0 >= at0 && R0 < at0 + n0) {                     // one thread
    long long at = at0;
    int b = bt0;
    for (;; ++b) {
      const long long n = static_cast<long long>(slots_of(plan, live_of(a, b, fa).pairs)) * a.Hkv;
      if (R0 < at + n) break;
      at += n;
    }
    *sm_start = b;
    sm_total[0] = R;
    *sm_ranges = N;
    sm_total[1] = R0 - at;
  }
  __syncthreads();

  const int g = lane >> 2, t = lane & 3;

  const float sl2 = a.scale * 1.4426950408889634f;
  const float minus = PAIRED && t < 2 ? 0.f : -1.f;       // of the weights' low pieces
  // The position in the range: row w, of which `done` slots are behind us, at
  // slot `pos` of the CTA's `len`.
  Row w = {};
  uint32_t done = 0, pos = 0;
  const uint32_t len = static_cast<uint32_t>(R1 - R0);
  if (works) {
    w.b = *sm_start;
    w.pairs = live_of(a, w.b, fa).pairs;
    w.slots = slots_of(plan, w.pairs);
    const long long off = sm_total[1];
    w.g = static_cast<int>(div_of(off, w.slots));
    done = static_cast<uint32_t>(off - static_cast<long long>(w.g) * w.slots);
  }
  // ---- the warp's stream of slots ---------------------------------------------
  // Slot n of the warp is number warp + W n of the CTA's range and goes
  // to stage n mod kDepth of the warp's ring.
  uint8_t* ring = smem + warp * kDepth * 2 * L::BYTES;
  uint64_t* bars = full + warp * kDepth;
  const uint32_t total = (len + W - 1 - warp) / W;
  // Row, done and pos stand in shared memory too: the loop over pairs, which is
  // short of registers, wants them only at every 16th.
  volatile uint32_t* where = reinterpret_cast<uint32_t*>(smem + S::WHERE) + warp * 8;
  auto keep = [&]() {
    __syncwarp();              // nobody recalls the old place any more
    if (lane == 0) {
      where[0] = w.b, where[1] = w.g, where[2] = w.slots;
      where[3] = done, where[4] = pos, where[5] = w.pairs;
    }
    __syncwarp();
  };
  auto recall = [&]() {
    w.b = where[0], w.g = where[1], w.slots = where[2];
    done = where[3], pos = where[4], w.pairs = where[5];
  };
  keep();
  uint32_t taken = 0;          // slots consumed
  uint32_t src = kNoRecord;    // lane's record of the current 16 pairs (index into the pool), or none
  uint32_t joined = 0;         // bit 2 i: the records of the i-th of them stand side by side
  uint32_t missing = 0;        // two bits per pair in flight, the oldest lowest: no such record
  bool ok = true;
  auto fill = [&](uint32_t n, int place) {
    if ((n & 15u) == 0) {      // places of pairs n .. n + 15
      src = kNoRecord;
      const uint32_t nl = n + (lane >> 1);
      if (nl < total) {
        uint32_t x = where[3] + (warp + W * nl - where[4]);   // counted from the row's start
        Row t;
        t.b = where[0], t.g = where[1], t.slots = where[2];
        while (x >= t.slots) {
          x -= t.slots;
          next_row(a, fa, plan, t);
        }
        const int k = 2 * static_cast<int>(x) + (lane & 1);
        const Live v = live_of(a, t.b, fa);
        if (k < v.count) {
          const int rec = k < v.head ? k : v.tail + (k - v.head);
          const int recs = a.page_size / kQ4Rec, lp = rec / recs;
          const int page = a.page_table[static_cast<size_t>(t.b) * a.max_pages + lp];
          if (page >= 0 && page < a.num_pages)
            src = (static_cast<uint32_t>(page) * a.Hkv + t.g) * recs + (rec - lp * recs);
          else
            raise_error(a.st.err, DEV_ERR_PAGE);
        }
      }
      __syncwarp();
      const uint32_t other = __shfl_xor_sync(0xffffffffu, src, 1);
      joined = __ballot_sync(0xffffffffu, src != kNoRecord && other == src + 1 && other != kNoRecord);
    }
    const uint32_t stage = n & (kDepth - 1), i = (2 * n) & 31u;
    const uint32_t i0 = __shfl_sync(0xffffffffu, src, i);
    uint8_t* dst = ring + stage * 2 * L::BYTES;
    if (joined >> i & 1u) {
      if (elect_one()) {
        mbar_arrive_expect_tx(bars + stage, 2 * L::BYTES);
        bulk_load(dst, a.pool + static_cast<size_t>(i0) * L::BYTES, 2 * L::BYTES, bars + stage);
      }
    } else {
      const uint32_t i1 = __shfl_sync(0xffffffffu, src, i + 1);
      const uint32_t none = (i0 == kNoRecord ? 1u : 0u) | (i1 == kNoRecord ? 2u : 0u);
      missing |= none << (2 * place);
      if (lane == 0) {
        if (none == 3) mbar_arrive(bars + stage);
        else mbar_arrive_expect_tx(bars + stage, none ? L::BYTES : 2 * L::BYTES);
        if (!(none & 1u)) bulk_load(dst, a.pool + static_cast<size_t>(i0) * L::BYTES, L::BYTES, bars + stage);
        if (!(none & 2u))
          bulk_load(dst + L::BYTES, a.pool + static_cast<size_t>(i1) * L::BYTES, L::BYTES, bars + stage);
      }
    }
  };
  for (uint32_t n = 0; n < kDepth && n < total; ++n) fill(n, n);

  // Sequences with no live token: zero output, lse -inf.
  for (int b = empties ? cta : a.B; b < a.B; b += gridDim.x) {
    if (live_of(a, b, fa).pairs != 0) continue;
    if (tid == 0) {
      const int s = a.seqlens[b];
      if (s < 0 || s > static_cast<long long>(a.max_pages) * a.page_size)
        raise_error(a.st.err, DEV_ERR_SEQLEN);
    }
    uint32_t* o = reinterpret_cast<uint32_t*>(a.o + static_cast<size_t>(b) * a.Hq * D);
    for (int i = tid; i < a.Hq * (D / 2); i += kThreads) o[i] = 0;
    if (a.lse)
      for (int i = tid; i < a.Hq; i += kThreads) a.lse[static_cast<size_t>(b) * a.Hq + i] = -INFINITY;
  }

  while (pos < len) {
    float o[NT][4];
    float2 l = {0.f, 0.f};
    float m0 = kLowest, m1 = kLowest;          // softmax references (log2 units) of heads 2 t, 2 t + 1
    const uint32_t stop = min(w.slots, done + (len - pos));        // of the row, in this range
    const uint32_t first_head = static_cast<uint32_t>(w.b) * a.Hq + w.g * G;

    // Query operands: lane 4 g + t holds head g (paired: g mod 4), channels 32 i + 8 t + e.  And
    // -8 times the head's group sums, cut into three bf16 numbers, as the
    // second operand of an MMA whose first is the tokens' scales: row 2 t + e
    // of that product is (at d 128) piece t / 2 of group 2 (t % 2) + e, rows 8
    // and up the last piece; at d 64 piece t of group e.
    uint32_t qf[GR][4], bq0 = 0, bq1 = 0;
    float sc0, sc1;            // log2 units per unit of a score, of heads 2 t and 2 t + 1
    {
      float c[GR];
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < GR; ++i) {
        uint4 v = {0, 0, 0, 0};
        const int head = PAIRED ? g & 3 : g;
        if (head < G)
          v = *reinterpret_cast<const uint4*>(a.q + static_cast<size_t>(first_head + head) * D + 32 * i + 8 * t);
        qf[i][0] = v.x;
        qf[i][1] = v.y;
        qf[i][2] = v.z;
        qf[i][3] = v.w;
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, max(qf[i][e] << 16 & 0x7fffffffu, qf[i][e] & 0x7fff0000u));
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // The head times 2^k, its largest channel then next to 2^126; the odd pairs
      // 2^4 less.  Scores come out times 2^(k - 133).
      const int k = min(126, max(6, 126 + 127 - static_cast<int>(top >> 23)));
      const float up = __uint_as_float((127 + k) << 23), less = __uint_as_float((127 + k - 4) << 23);
      const float down = __uint_as_float(max(1, 127 + k - 130) << 23);
#pragma unroll
      for (int i = 0; i < GR; ++i) {
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float lo = bf16lo_to_f32(qf[i][e]), hi = bf16hi_to_f32(qf[i][e]);
          sum += lo * down + hi * down;
          qf[i][e] = e & 1 ? pack_bf16x2(lo * less, hi * less) : pack_bf16x2(lo * up, hi * up);
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        c[i] = -sum;
      }
      const float back = sl2 * __uint_as_float((127 + 133 - k) << 23);
      sc0 = __shfl_sync(0xffffffffu, back, 8 * t);
      sc1 = __shfl_sync(0xffffffffu, back, 8 * t + 4);
      float e0 = c[0], e1 = c[1];
      if constexpr (D == 128) {
        if (t & 1) {
          e0 = c[2];
          e1 = c[3];
        }
      }
      const uint32_t hi = pack_bf16x2(e0, e1);
      e0 -= bf16lo_to_f32(hi);
      e1 -= bf16hi_to_f32(hi);
      const uint32_t mid = pack_bf16x2(e0, e1);
      e0 -= bf16lo_to_f32(mid);
      e1 -= bf16hi_to_f32(mid);
      const uint32_t lo = pack_bf16x2(e0, e1);
      if constexpr (D == 128) {
        bq0 = t < 2 ? hi : mid;
        bq1 = t < 2 ? lo : 0u;
      } else {
        bq0 = t == 0 ? hi : t == 1 ? mid : t == 2 ? lo : 0u;
      }
    }

    // The next row's query, for when it is its turn.
    if (pos + (stop - done) < len && lane < G * D / 64 && first_head + 2 * G <= static_cast<uint32_t>(a.B) * a.Hq)
      asm volatile("prefetch.global.L1 [%0];" ::"l"(a.q + static_cast<size_t>(first_head + G) * D + lane * 64));

#pragma unroll
    for (int m = 0; m < NT; ++m) o[m][0] = o[m][1] = o[m][2] = o[m][3] = 0.f;
    float th0 = kLowest, th1 = kLowest;        // a score (before the scale) above it moves the reference

    // The warp takes every W-th slot of the CTA's range.
    const uint32_t skip = (warp - pos) % W;
    int plain1, plain2, plain3;
    {
      const Live v = live_of(a, w.b, fa);
      plain1 = v.plain1;
      plain2 = v.plain2;
      plain3 = v.plain3;
    }
    const int j_end = static_cast<int>(stop);
    for (int j = static_cast<int>(done + skip); j < j_end && ok; j += W, ++taken) {
      const uint32_t stage = taken & (kDepth - 1), parity = (taken / kDepth) & 1u;
      const uint32_t none = missing & 3u;
      missing >>= 2;
      if (none == 3u) {        // an empty slot, or no valid page: nothing was copied
        if (taken + kDepth < total) fill(taken + kDepth, kDepth - 1);
        continue;
      }
      if (!__all_sync(0xffffffffu, mbar_try_wait(bars + stage, parity))) {
        ok = __all_sync(0xffffffffu, mbar_drain(bars + stage, parity, a.st.spin_ns));
        if (!ok) {             // gave up: the copies in flight land before anything else
          raise_error(a.st.err, DEV_ERR_TIMEOUT);
          for (uint32_t n = taken; n < total && n < taken + kDepth; ++n)
            mbar_drain(bars + (n & (kDepth - 1)), (n / kDepth) & 1u);
          break;
        }
      }
      const uint8_t* rec = ring + stage * 2 * L::BYTES;

      uint32_t v0[2][GR], v1[2][GR], sv0[2], sv1[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint8_t* p = rec + r * L::BYTES;
        load_words<D>(p + L::VC + lane * (D / 8), v0[r]);
        load_words<D>(p + L::VC + 4 * D + lane * (D / 8), v1[r]);
        const uint8_t* vs = p + L::VS + (g * (D / 8) / 32) * 32 + 4 * t;
        sv0[r] = *reinterpret_cast<const uint32_t*>(vs);
        sv1[r] = *reinterpret_cast<const uint32_t*>(vs + 16);
      }
      float x[2][4];           // scores: tokens g, g + 8, heads 2 t, 2 t + 1
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint8_t* p = rec + r * L::BYTES;
        uint32_t k0[GR], k1[GR];
        float s0[GR], s1[GR];
        load_words<D>(p + lane * (D / 8), k0);
        load_words<D>(p + 4 * D + lane * (D / 8), k1);
        load_scales<D>(p + L::KS + g * (2 * GR), s0);
        load_scales<D>(p + L::KS + (g + 8) * (2 * GR), s1);
        {
          const uint32_t w0 = *reinterpret_cast<const uint32_t*>(p + L::KS + g * (2 * GR) + (t & (GR / 2 - 1)) * 4);
          const uint32_t w1 =
              *reinterpret_cast<const uint32_t*>(p + L::KS + (g + 8) * (2 * GR) + (t & (GR / 2 - 1)) * 4);
          const uint32_t af[4] = {w0, w1, w0, w1};
          mma_zero(x[r], af, bq0, bq1);
        }
#pragma unroll
        for (int i = 0; i < GR; ++i) {
          float acc[4];
          const uint32_t y0 = __funnelshift_r(k0[i], k0[i], 3), y1 = __funnelshift_r(k1[i], k1[i], 3);
          {
            const uint32_t af[4] = {fields<0>(y0), fields<0>(y1), fields<1>(y0), fields<1>(y1)};
            mma_zero(acc, af, qf[i][0], qf[i][1]);
          }
          {
            const uint32_t z0 = y0 >> 8, z1 = y1 >> 8;
            const uint32_t af[4] = {fields<2>(z0), fields<2>(z1), fields<3>(z0), fields<3>(z1)};
            mma_add(acc, af, qf[i][2], qf[i][3]);
          }
          x[r][0] = fmaf(s0[i], acc[0], x[r][0]);
          x[r][1] = fmaf(s0[i], acc[1], x[r][1]);
          x[r][2] = fmaf(s1[i], acc[2], x[r][2]);
          x[r][3] = fmaf(s1[i], acc[3], x[r][3]);
        }
      }
      __syncwarp();
      if (taken + kDepth < total) fill(taken + kDepth, kDepth - 1);
      // A pair at the end of the sequence or of the sink or window, or with a
      // missing page: tokens that are not live score -inf, and their values
      // count as zero whatever bytes stand there.
      if (none != 0 || !(j < plain1 || (j >= plain2 && j < plain3))) {
        const Live v = live_of(a, w.b, fa);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int k = 2 * j + r;
          const int u0 = (k < v.head ? k : v.tail + (k - v.head)) * kQ4Rec;
          const bool there = !(none >> r & 1u);
          auto live = [&](int u) { return there && u < v.s && (u < v.n_sink || u >= v.win); };
          if (!live(u0 + g)) x[r][0] = x[r][1] = -INFINITY;
          if (!live(u0 + g + 8)) x[r][2] = x[r][3] = -INFINITY;
          if (!live(u0 + 2 * t)) sv0[r] &= 0xffff0000u;
          if (!live(u0 + 2 * t + 1)) sv0[r] &= 0x0000ffffu;
          if (!live(u0 + 2 * t + 8)) sv1[r] &= 0xffff0000u;
          if (!live(u0 + 2 * t + 9)) sv1[r] &= 0x0000ffffu;
        }
      }
      const uint32_t carried = (sv0[0] + kLarge) | (sv1[0] + kLarge) | (sv0[1] + kLarge) | (sv1[1] + kLarge);
      bool large = (carried & 0x80008000u) != 0;
      const float t0 = fmaxf(fmaxf(x[0][0], x[0][2]), fmaxf(x[1][0], x[1][2]));
      const float t1 = fmaxf(fmaxf(x[0][1], x[0][3]), fmaxf(x[1][1], x[1][3]));
      if (__any_sync(0xffffffffu, t0 > th0 || t1 > th1 || large)) {
        large = __any_sync(0xffffffffu, large);
        float n0 = t0, n1 = t1;
#pragma unroll
        for (int s = 4; s < 32; s <<= 1) {
          n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, s));
          n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, s));
        }
        n0 = fmaxf(m0, n0 * sc0);
        n1 = fmaxf(m1, n1 * sc1);
        const float f0 = ex2(m0 - n0), f1 = ex2(m1 - n1);
        m0 = n0;
        m1 = n1;
        th0 = (n0 + kGrow) / sc0;
        th1 = (n1 + kGrow) / sc1;
        l.x *= f0;
        l.y *= f1;
#pragma unroll
        for (int m = 0; m < NT; ++m) {
          o[m][0] *= f0;
          o[m][1] *= f1;
          o[m][2] *= f0;
          o[m][3] *= f1;
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float2 p0 = {ex2(fmaf(x[r][0], sc0, -m0)), ex2(fmaf(x[r][1], sc1, -m1))};
        const float2 p1 = {ex2(fmaf(x[r][2], sc0, -m0)), ex2(fmaf(x[r][3], sc1, -m1))};
        l = add2(l, add2(p0, p1));
        if (!large) {
          const Weights<PAIRED> b0(p0, minus), b1(p1, minus);
          const uint32_t e0 = mul_bf16x2(sv0[r], kUpEven), e1 = mul_bf16x2(sv1[r], kUpEven);
          const uint32_t o0 = mul_bf16x2(sv0[r], kUpOdd), o1 = mul_bf16x2(sv1[r], kUpOdd);
          const uint32_t n0 = mul_bf16x2(sv0[r], kDown8), n1 = mul_bf16x2(sv1[r], kDown8);
#pragma unroll
          for (int i = 0; i < GR; ++i) {
            const uint32_t y0 = v0[r][i], y1 = v1[r][i], z0 = y0 >> 8, z1 = y1 >> 8;
            {
              const uint32_t af[4] = {fma_bf16x2(fields<0>(y0), e0, n0), fma_bf16x2(fields<1>(y0), o0, n0),
                                      fma_bf16x2(fields<0>(y1), e1, n1), fma_bf16x2(fields<1>(y1), o1, n1)};
              add_values(o[2 * i], af, b0, b1);
            }
            {
              const uint32_t af[4] = {fma_bf16x2(fields<2>(z0), e0, n0), fma_bf16x2(fields<3>(z0), o0, n0),
                                      fma_bf16x2(fields<2>(z1), e1, n1), fma_bf16x2(fields<3>(z1), o1, n1)};
              add_values(o[2 * i + 1], af, b0, b1);
            }
          }
        } else {
          // Large values: 16 + u from the mantissa, (16 + u) scale - 24 scale the
          // value itself, and 2^-25 on the other operand.
          const float f = 1.f / kValueUnit;
          const Weights<PAIRED> b0(make_float2(p0.x * f, p0.y * f), minus), b1(make_float2(p1.x * f, p1.y * f), minus);
          const uint32_t n0 = mul_bf16x2(sv0[r], 0xc1c0c1c0u), n1 = mul_bf16x2(sv1[r], 0xc1c0c1c0u);   // -24
          auto value = [](uint32_t x, uint32_t scale, uint32_t n) {
            return fma_bf16x2((x & 0x00780078u) | 0x41804180u, scale, n);
          };
#pragma unroll
          for (int i = 0; i < GR; ++i) {
            const uint32_t y0 = v0[r][i], y1 = v1[r][i];
            {
              const uint32_t af[4] = {value(y0 << 3, sv0[r], n0), value(y0 >> 1, sv0[r], n0),
                                      value(y1 << 3, sv1[r], n1), value(y1 >> 1, sv1[r], n1)};
              add_values(o[2 * i], af, b0, b1);
            }
            {
              const uint32_t af[4] = {value(y0 >> 5, sv0[r], n0), value(y0 >> 9, sv0[r], n0),
                                      value(y1 >> 5, sv1[r], n1), value(y1 >> 9, sv1[r], n1)};
              add_values(o[2 * i + 1], af, b0, b1);
            }
          }
        }
      }
    }
    recall();
    const uint32_t pairs = w.pairs, until = min(w.slots, done + (len - pos));
    const uint32_t head0 = static_cast<uint32_t>(w.b) * a.Hq + w.g * G;
    const bool begins = done == 0, ends = until >= pairs;
    if (done >= pairs) {       // the range began in the row's empty slots
      pos += until - done;
      done = 0;
      if (pos < len) next_row(a, fa, plan, w);
      keep();
      continue;
    }
    // ---- merge the warps --------------------------------------------------
#pragma unroll
    for (int s = 4; s < 32; s <<= 1) {
      l.x += __shfl_xor_sync(0xffffffffu, l.x, s);
      l.y += __shfl_xor_sync(0xffffffffu, l.y, s);
    }
#pragma unroll
    for (int m = 0; m < NT; ++m)
      sm_acc[warp * S::PART4 + m * 32 + lane] = make_float4(o[m][0], o[m][1], o[m][2], o[m][3]);
    if (g == 0) {
      sm_m[warp * 8 + 2 * t] = m0;
      sm_m[warp * 8 + 2 * t + 1] = m1;
      sm_l[warp * 8 + 2 * t] = l.x;
      sm_l[warp * 8 + 2 * t + 1] = l.y;
    }
    const bool fine = named_bar_and(1, kThreads, ok);
    const bool whole = begins && ends;
    const int slot = 2 * cta + (begins ? 1 : 0);
    float4* part = reinterpret_cast<float4*>(a.part);            // [2 gridDim][PART4], then m, l [..][8]
    float* part_m = a.part + static_cast<size_t>(2) * gridDim.x * S::PART4 * 4;
    float* part_l = part_m + 2 * gridDim.x * 8;
    for (int i = tid; i < S::PART4; i += kThreads) {
      const int h = 2 * (PAIRED ? i & 1 : i & 3), gi = (i & 31) >> 2, m = i >> 5;
      float M0 = kLowest, M1 = kLowest;
#pragma unroll
      for (int v = 0; v < W; ++v) {
        M0 = fmaxf(M0, sm_m[v * 8 + h]);
        M1 = fmaxf(M1, sm_m[v * 8 + h + 1]);
      }
      float ls0 = 0.f, ls1 = 0.f;
      float4 r = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int v = 0; v < W; ++v) {
        const float w0 = ex2(sm_m[v * 8 + h] - M0), w1 = ex2(sm_m[v * 8 + h + 1] - M1);
        const float4 c = sm_acc[v * S::PART4 + i];
        ls0 = fmaf(w0, sm_l[v * 8 + h], ls0);
        ls1 = fmaf(w1, sm_l[v * 8 + h + 1], ls1);
        r.x = fmaf(w0, c.x, r.x);
        r.y = fmaf(w1, c.y, r.y);
        r.z = fmaf(w0, c.z, r.z);
        r.w = fmaf(w1, c.w, r.w);
      }
      if constexpr (PAIRED) {                  // high and low pieces
        r.x += __shfl_xor_sync(0xffffffffu, r.x, 2);
        r.y += __shfl_xor_sync(0xffffffffu, r.y, 2);
        r.z += __shfl_xor_sync(0xffffffffu, r.z, 2);
        r.w += __shfl_xor_sync(0xffffffffu, r.w, 2);
        if (i & 2) continue;
      }
      if (h >= G) continue;
      if (!fine) {                             // a wait ran out: the row's output is zero
        ls0 = ls1 = whole ? 0.f : -1.f;
        r = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      if (whole) {
        const float i0 = ls0 != 0.f ? kValueUnit / ls0 : 0.f, i1 = ls1 != 0.f ? kValueUnit / ls1 : 0.f;
        uint16_t* out = a.o + static_cast<size_t>(head0 + h) * D + gi * (D / 8) + 2 * m;
        *reinterpret_cast<uint32_t*>(out) = pack_bf16x2(r.x * i0, r.z * i0);
        if (h + 1 < G) *reinterpret_cast<uint32_t*>(out + D) = pack_bf16x2(r.y * i1, r.w * i1);
        if (a.lse && m == 0 && gi == 0) {
          a.lse[head0 + h] = ls0 != 0.f ? (M0 + log2f(ls0)) * 0.69314718055994531f : -INFINITY;
          if (h + 1 < G) a.lse[head0 + h + 1] = ls1 != 0.f ? (M1 + log2f(ls1)) * 0.69314718055994531f : -INFINITY;
        }
      } else {
        __stcg(part + static_cast<size_t>(slot) * S::PART4 + i, r);
        if (m == 0 && gi == 0) {
          __stcg(part_m + slot * 8 + h, M0);
          __stcg(part_m + slot * 8 + h + 1, M1);
          __stcg(part_l + slot * 8 + h, ls0);
          __stcg(part_l + slot * 8 + h + 1, ls1);
        }
      }
    }
    if (!whole) {
      // ---- merge the CTAs of a row: the one that comes last ----------------
      const Cuts c = cuts_of(sm_total[0], *sm_ranges);
      const long long row0 = range_of(c, cta) + pos - done;
      const int first = cta_of(c, row0), last = cta_of(c, row0 + pairs - 1);
      named_bar_sync(1, kThreads);
      if (tid == 0) {
        // The barrier orders the CTA's stores before the ticket, which releases them
        // and acquires those of the CTAs before; the next barrier passes that on.
        int* ticket = a.tickets + static_cast<size_t>(w.b) * a.Hkv + w.g;
        int n;
        asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(n) : "l"(ticket) : "memory");
        *sm_ticket = n;
        if (n == last - first) *ticket = 0;
      }
      named_bar_sync(1, kThreads);
      if (*sm_ticket == last - first) {
        // slot of part c: the first CTA's row begins there, the others' before
        const int f0 = 2 * first + 1;
        float* wt = reinterpret_cast<float*>(sm_acc);              // [part][8] weights
        const int np = last - first + 1;
        // The parts are shared out to NG groups of threads, a float4 per thread.  The
        // first ones are loaded while the weights are worked out.
        constexpr int NG = kThreads / S::PART4, kAhead = 8;
        static_assert(NG >= 1 && kThreads % S::PART4 == 0 && kComb + NG * S::PART4 * 16 <= S::ACC, "merge layout");
        const int i = tid % S::PART4, group = tid / S::PART4;
        const int h = 2 * (i & 3), gi = (i & 31) >> 2, m = i >> 5;
        const bool act = h < G;
        auto part_of = [&](int c) {
          return part + static_cast<size_t>(c == 0 ? f0 : 2 * (first + c)) * S::PART4 + i;
        };
        float4 ahead[kAhead];
#pragma unroll
        for (int c = 0; c < kAhead; ++c)
          ahead[c] = act && c * NG + group < np ? __ldcg(part_of(c * NG + group)) : make_float4(0.f, 0.f, 0.f, 0.f);
        // Warp v: the weights of head v's parts, and the row's sum.
        if (warp < G) {
          float M = kLowest, ls = 0.f;
          bool lost = false;
          for (int c = lane; c < np; c += 32) {
            const int at = (c == 0 ? f0 : 2 * (first + c)) * 8 + warp;
            const float pm = __ldcg(part_m + at), pl = __ldcg(part_l + at);
            lost |= pl < 0.f;
            const float M1 = fmaxf(M, pm);
            ls = fmaf(pl, ex2(pm - M1), ls * ex2(M - M1));
            M = M1;
            wt[c * 8 + warp] = pm;
          }
          const float mine = M;
#pragma unroll
          for (int s = 1; s < 32; s <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, s));
          ls *= ex2(mine - M);
          for (int c = lane; c < np; c += 32) wt[c * 8 + warp] = ex2(wt[c * 8 + warp] - M);
#pragma unroll
          for (int s = 1; s < 32; s <<= 1) ls += __shfl_xor_sync(0xffffffffu, ls, s);
          if (__any_sync(0xffffffffu, lost)) ls = 0.f;
          if (lane == 0) {
            sm_fl[warp] = ls != 0.f ? kValueUnit / ls : 0.f;
            if (a.lse) a.lse[head0 + warp] = ls != 0.f ? (M + log2f(ls)) * 0.69314718055994531f : -INFINITY;
          }
        }
        named_bar_sync(1, kThreads);
        float4 r = {0.f, 0.f, 0.f, 0.f};
        if (act) {
          auto add = [&](int c, const float4& v) {
            const float w0 = wt[c * 8 + h], w1 = h + 1 < G ? wt[c * 8 + h + 1] : 0.f;
            r.x = fmaf(w0, v.x, r.x);
            r.y = fmaf(w1, v.y, r.y);
            r.z = fmaf(w0, v.z, r.z);
            r.w = fmaf(w1, v.w, r.w);
          };
#pragma unroll
          for (int c = 0; c < kAhead; ++c)
            if (c * NG + group < np) add(c * NG + group, ahead[c]);
#pragma unroll 8
          for (int c = kAhead * NG + group; c < np; c += NG) add(c, __ldcg(part_of(c)));
        }
        if (NG > 1) {
          float4* comb = sm_acc + kComb / 16;
          comb[tid] = r;
          named_bar_sync(1, kThreads);
          if (group == 0) {
#pragma unroll
            for (int k = 1; k < NG; ++k) {
              const float4 v = comb[k * S::PART4 + i];
              r = make_float4(r.x + v.x, r.y + v.y, r.z + v.z, r.w + v.w);
            }
          }
        }
        if (act && group == 0) {
          const float i0 = sm_fl[h], i1 = h + 1 < G ? sm_fl[h + 1] : 0.f;
          uint16_t* out = a.o + static_cast<size_t>(head0 + h) * D + gi * (D / 8) + 2 * m;
          *reinterpret_cast<uint32_t*>(out) = pack_bf16x2(r.x * i0, r.z * i0);
          if (h + 1 < G) *reinterpret_cast<uint32_t*>(out + D) = pack_bf16x2(r.y * i1, r.w * i1);
        }
      }
    }
    pos += until - done;
    done = 0;
    if (pos < len) {
      next_row(a, fa, plan, w);
      keep();
      named_bar_sync(1, kThreads);      // the merge buffer is free again
    }
  }
}

template <int W>
int ctas_of(int num_sms) {
  return min(Shape<W>::kCtasPerSm * num_sms, kMaxParts);
}

template <int D, int W, bool PAIRED>
cudaError_t launch_t(const DecodeQ4Launch& p, int num_sms, cudaStream_t stream) {
  constexpr int smem = Q4Smem<D, W>::BYTES;
  static_assert(smem * Shape<W>::kCtasPerSm <= 226 << 10, "shared memory");
  cudaError_t e =
      cudaFuncSetAttribute(decode_q4_kernel<D, W, PAIRED>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas_of<W>(num_sms));
  cfg.blockDim = dim3(Shape<W>::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_q4_kernel<D, W, PAIRED>, p);
}

template <int D>
cudaError_t launch_d(const DecodeQ4Launch& p, int num_sms, cudaStream_t stream) {
  // At most one row per SM; of some length, and if they are few, of a length that is
  // cut into many parts either way (8 rows of 1200 tokens: 9.6 us by 8 warps, 11.3 by
  // 16; 64 rows of 300: 9.1 and 8.0).  The lengths are on the device: the bound that the
  // host has is the table's capacity.  A table wider than its requests need takes the
  // second shape for short ones too: up to 16 rows, 5.7-6.1 us become 6.8-7.2 at 100
  // tokens, 8.9-10.6 become 11.1-11.4 at 1200, and from 4000 (one row: 9000) tokens on,
  // or with 64 rows from 300 on, there is no difference.
  const long long rows = static_cast<long long>(p.B) * p.Hkv;
  const long long longest = static_cast<long long>(p.max_pages) * p.page_size;
  const bool wide = rows <= num_sms && longest > (rows >= 32 ? 256 : 8192);
  if (p.Hq / p.Hkv <= 4)
    return wide ? launch_t<D, 16, true>(p, num_sms, stream) : launch_t<D, 8, true>(p, num_sms, stream);
  return wide ? launch_t<D, 16, false>(p, num_sms, stream) : launch_t<D, 8, false>(p, num_sms, stream);
}

}  // namespace

// Two partials per CTA, of either shape: float4 accumulators, m and l of 8 heads.
size_t decode_q4_workspace_bytes(int d, int num_sms) {
  const size_t parts = static_cast<size_t>(2) * ctas_of<8>(num_sms);
  return parts * (static_cast<size_t>(d) / 16 * 32 * 16 + 2 * 8 * 4);
}

cudaError_t launch_decode_q4(const DecodeQ4Launch& p, int num_sms, cudaStream_t stream) {
  return p.d == 64 ? launch_d<64>(p, num_sms, stream) : launch_d<128>(p, num_sms, stream);
}

}  // namespace flux
