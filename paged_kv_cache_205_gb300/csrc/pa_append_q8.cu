// pa_append_q8.cu -- KV append with Llama-3-scaled RoPE into the 8-bit cache
// (pa_q8.cuh has the format).
//
// Both entry points run the page allocation kernel of the bf16 appends, then
// a store kernel launched with programmatic dependent launch:
//   append_store_q8_kernel   one CTA per sequence: rotates q and k, quantises
//                            k and v to the page's scale; where the new token
//                            needs a larger scale than the page has, the
//                            page's earlier tokens are brought to it.
//   prefill_store_q8_kernel  one CTA per page that the call's rows touch (its
//                            values stay in registers between the maximum that
//                            sets the scale and the rounding), and one per 8
//                            or 16 rows of q.
// Both are bound by memory (large) or latency (small): a row costs 2 KiB of k
// and v read, 1 KiB of bytes written, 4 KiB of q read and 4 KiB written.
#include <algorithm>
#include <cuda_fp16.h>

#include "pa_append_shared.cuh"
#include "pa_q8.cuh"

namespace pa {
namespace {

// What the rotations need, worked out on the host and passed by value: cos and
// sin of 2 pi i / 64, and the pairs' frequencies as fp32 head and rest.
constexpr int kAngles = 64;
struct AngleTable {
  float2 e[kAngles];
  float2 f[kD / 2];
  double2 exact[kAngles];   // (cos, sin) again
};

AngleTable angle_table(const RopeFreqs &freqs) {
  AngleTable t;
  for (int i = 0; i < kAngles; ++i) {
    const double a = i * (6.283185307179586476925 / kAngles);
    t.exact[i] = make_double2(std::cos(a), std::sin(a));
    t.e[i] = make_float2(static_cast<float>(t.exact[i].x), static_cast<float>(t.exact[i].y));
  }
  for (int d = 0; d < kD / 2; ++d) {
    t.f[d].x = static_cast<float>(freqs.f[d]);
    t.f[d].y = static_cast<float>(freqs.f[d] - t.f[d].x);
  }
  return t;
}

struct Q8Out {
  uint16_t *q_out;   // where rotated q goes (may be q itself)
  float *scales;
  AngleTable table;
};

// The angle pos * f less at * 2 pi / 64, as fp32 head and rest, |.| <= pi / 64.
struct BaseAngle {
  float r, rest;
  int at;
};

// Formed and reduced in fp64; the multiple of 2 pi / 64 is taken off in two fused
// multiply-adds, head first (W. J. Cody, W. Waite, "Software Manual for the
// Elementary Functions", 1980).
__device__ __forceinline__ BaseAngle base_angle(int pos, double f) {
  constexpr double kStepHi = 6.283185307179586232 / kAngles;
  constexpr double kStepLo = 2.4492935982947064e-16 / kAngles;
  constexpr double kInteger = 6755399441055744.0;   // 1.5 * 2^52: adding it rounds to an integer
  const double a = static_cast<double>(pos) * f;
  const double t = fma(a, 0.15915494309189533577 * kAngles, kInteger);
  const double k = t - kInteger;
  const double r = fma(-k, kStepLo, fma(-k, kStepHi, a));
  BaseAngle b;
  b.r = static_cast<float>(r);
  b.rest = static_cast<float>(r - static_cast<double>(b.r));
  b.at = __double2loint(t) & (kAngles - 1);
  return b;
}

// (cos, sin) of the angle of `step` (< 32) positions after b's, within 2^-23.
// Everything in fp32, so that fp64, at a sixteenth of a warp a cycle and SM, works
// out one row's angles of a CTA and not all rows': step * f and the sum with the
// base keep their rounding errors, the multiple k <= 327 of 2 pi / 64 is taken
// off with an 8-bit head (k times it is exact) and a rest, the table holds the
// grid point, and the addition theorem adds what is left, |r| <= pi / 64 + 2^-20,
// whose sine and 1 - cosine are short Taylor sums (r^7 / 5040 < 2^-42).
__device__ __forceinline__ float2 angle_cos_sin(const BaseAngle &b, int step, float2 f,
                                                const float2 *table) {
  constexpr float kStepHead = 0.09814453125f;                            // 2 pi / 64 to 8 bits
  constexpr float kStepRest = static_cast<float>(0.098174770424681038701 - 0.09814453125);
  const float t = static_cast<float>(step);
  const float p = t * f.x, pe = fmaf(t, f.x, -p);
  const float s = b.r + p, v = s - b.r;
  const float se = (b.r - (s - v)) + (p - v);                            // s + se = b.r + p
  const float k = rintf(s * 10.185916357881302f);
  const float low = se + fmaf(t, f.y, b.rest + pe);
  const float r = fmaf(-k, kStepHead, s) + fmaf(-k, kStepRest, low);
  const float2 e = table[(b.at + static_cast<int>(k)) & (kAngles - 1)];
  const float r2 = r * r;
  const float cm1 = r2 * fmaf(r2, 1.f / 24, -0.5f);                      // cos r - 1
  const float sn = fmaf(r * r2, fmaf(r2, 1.f / 120, -1.f / 6), r);       // sin r
  return make_float2(e.x + fmaf(e.x, cm1, -e.y * sn), e.y + fmaf(e.y, cm1, e.x * sn));
}

// A key's byte rounds twice, to bf16 and to e4m3, and an error of the fp32 rotation
// changes it only where the value lies next to a bf16 border beside an e4m3
// border: mantissa bits 0x78000 and 0x88000 (of 20; bytes below e4m3's normal range
// have theirs elsewhere, and steps that weigh nothing).  near_border is below 2 kNear
// within kNear ulps of one.  The fp32 error is mostly below 2^-24 (|a| + |b|), which
// is 4 ulps where the products cancel to a quarter; the few words of a prompt's keys
// that near a border (one in 16,000) are rotated again in fp64, 2% of the call's
// time, and 8 x 2048 tokens' bytes then differ from the definition's in 2 of 17
// million, both where the products cancel to 2^-6 and less (7 without).
constexpr uint32_t kNear = 4;
__device__ __forceinline__ uint32_t near_border(float x) {
  return (__float_as_uint(x) + (0x88000u + kNear)) & 0xeffffu;   // (both borders at 0)
}

// x to fp32 so that a later rounding to fewer bits comes out as x's own.
__device__ __forceinline__ float round_to_odd(double x) {
  const float f = __double2float_rz(x);
  return static_cast<double>(f) == x ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

// The bytes of a pair of key elements (a, b) rotated by the angle pos * f in fp64,
// the first in the low byte.
__device__ __forceinline__ uint32_t exact_key_pair(float a, float b, int pos, double f, float inv,
                                                const double2 *table) {
  constexpr double kStepHi = 6.283185307179586232 / kAngles;
  constexpr double kStepLo = 2.4492935982947064e-16 / kAngles;
  const double angle = static_cast<double>(pos) * f;
  const double k = rint(angle * (0.15915494309189533577 * kAngles));
  const double r = fma(-k, kStepLo, fma(-k, kStepHi, angle)), r2 = r * r;
  const double2 e = table[static_cast<int>(static_cast<long long>(k) & (kAngles - 1))];
  // Taylor sums for |r| <= pi / 64: r^9 / 9! < 2^-57, r^10 / 10! < 2^-65
  const double cm1 = r2 * fma(r2, fma(r2, fma(r2, 1. / 40320, -1. / 720), 1. / 24), -0.5);
  const double sn = fma(r * r2, fma(r2, fma(r2, -1. / 5040, 1. / 120), -1. / 6), r);
  const double c = e.x + fma(e.x, cm1, -e.y * sn), s = e.y + fma(e.y, cm1, e.x * sn);
  const double da = a, db = b;
  const float2 t = bf16x2_to_float2(
      float2_to_bf16x2(round_to_odd(fma(da, c, -db * s)), round_to_odd(fma(db, c, da * s))));
  return e4m3x2(t.x * inv, t.y * inv);
}

// Pairs d and d + 1 (d even) of the key at k, rotated so, into its bytes at row.
__device__ __forceinline__ void exact_key_word(const uint16_t *k, unsigned char *row, int d, int pos,
                                               float inv, const RopeFreqs &freqs,
                                               const double2 *table) {
#pragma unroll 1
  for (int i = d; i < d + 2; ++i) {
    const uint32_t x =
        exact_key_pair(__uint_as_float(static_cast<uint32_t>(k[i]) << 16),
                       __uint_as_float(static_cast<uint32_t>(k[i + kD / 2]) << 16), pos, freqs.f[i], inv, table);
    row[i] = static_cast<unsigned char>(x);
    row[i + kD / 2] = static_cast<unsigned char>(x >> 8);
  }
}

// The pairs (lo, hi) of one bf16 word each, rotated by (x, y) and (z, w).
__device__ __forceinline__ void rotate2(uint32_t *lo, uint32_t *hi, float4 cs) {
  const float2 a = bf16x2_to_float2(*lo), b = bf16x2_to_float2(*hi);
  *lo = float2_to_bf16x2(fmaf(a.x, cs.x, -b.x * cs.y), fmaf(a.y, cs.z, -b.y * cs.w));
  *hi = float2_to_bf16x2(fmaf(b.x, cs.x, a.x * cs.y), fmaf(b.y, cs.z, a.y * cs.w));
}

// The same for keys; bit `bit` of *borders: one of the four nears a border.
__device__ __forceinline__ void rotate2_key(uint32_t *lo, uint32_t *hi, float4 cs, int bit,
                                            uint32_t *borders) {
  const float2 a = bf16x2_to_float2(*lo), b = bf16x2_to_float2(*hi);
  const float l0 = fmaf(a.x, cs.x, -b.x * cs.y), l1 = fmaf(a.y, cs.z, -b.y * cs.w);
  const float h0 = fmaf(b.x, cs.x, a.x * cs.y), h1 = fmaf(b.y, cs.z, a.y * cs.w);
  if (min(min(near_border(l0), near_border(l1)), min(near_border(h0), near_border(h1))) < 2 * kNear)
    *borders |= 1u << bit;
  *lo = float2_to_bf16x2(l0, l1);
  *hi = float2_to_bf16x2(h0, h1);
}

// (lo, hi) of 4 consecutive pairs of one head row: bf16 words of dims
// 4j..4j+3 and 32+4j..32+4j+3.
struct HeadPart {
  uint2 lo, hi;
};

__device__ __forceinline__ HeadPart load_part(const uint16_t *row, int j) {
  HeadPart h;
  h.lo = *reinterpret_cast<const uint2 *>(row + 4 * j);
  h.hi = *reinterpret_cast<const uint2 *>(row + kD / 2 + 4 * j);
  return h;
}

constexpr int kStoreQ8Threads = (2 * kHkv + kHq) * 8;   // 8 threads per head row: k, v, q

template <int BT>
__global__ void __launch_bounds__(kStoreQ8Threads) append_store_q8_kernel(AppendParams p, Q8Out o) {
  constexpr size_t kHalfPage = static_cast<size_t>(BT) * kQ8TokBytes;
  __shared__ float2 cs[kD / 2];
  pdl_launch_dependents();   // the next kernel may start its own set-up
  const int s = blockIdx.x;
  const int tid = threadIdx.x;
  const int pos = p.context_lens[s];
  if (pos < 0 || pos >= p.max_blocks * BT) {   // reported by the allocation kernel
    pdl_wait_primary();
    return;
  }
  const int head = tid >> 3;   // 0..7 k, 8..15 v, 16..47 q
  const int j = tid & 7;
  const bool is_k = head < kHkv, is_v = head >= kHkv && head < 2 * kHkv;
  HeadPart x;
  x.lo = x.hi = make_uint2(0, 0);
  if (is_k) {
    x = load_part(p.k_new + (static_cast<size_t>(s) * kHkv + head) * kD, j);
  } else if (is_v) {
    // (v: dims 8j..8j+7)
    const uint4 w = *reinterpret_cast<const uint4 *>(
        p.v_new + (static_cast<size_t>(s) * kHkv + head - kHkv) * kD + 8 * j);
    x.lo = make_uint2(w.x, w.y);
    x.hi = make_uint2(w.z, w.w);
  } else if (p.q) {
    x = load_part(p.q + (static_cast<size_t>(s) * kHq + head - 2 * kHkv) * kD, j);
  }
  if (tid < kD / 2)
    cs[tid] = angle_cos_sin(base_angle(pos, p.freqs.f[tid]), 0, make_float2(0.f, 0.f), o.table.e);
  // the largest magnitude of the head's 64 values, before the rotation
  uint32_t top = q8_top(x.hi.y, q8_top(x.hi.x, q8_top(x.lo.y, q8_top(x.lo.x, 0u))));
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
  __syncthreads();
  if (!is_v) rotate4(x.lo, x.hi, cs, j, &x.lo, &x.hi);
  if (!is_k && !is_v) {
    if (p.q) {
      uint16_t *row = o.q_out + (static_cast<size_t>(s) * kHq + head - 2 * kHkv) * kD;
      *reinterpret_cast<uint2 *>(row + 4 * j) = x.lo;
      *reinterpret_cast<uint2 *>(row + kD / 2 + 4 * j) = x.hi;
    }
    pdl_wait_primary();   // this grid ends after the allocation kernel
    return;
  }

  // the entry of a page that starts now is written by the allocation kernel;
  // an existing page's entry was written before that kernel started
  const int slot = pos % BT;
  if (slot == 0) pdl_wait_primary();
  const int blk = p.block_table[table_row(s, p.n_layers, p.layer, p.max_blocks) + pos / BT];
  if (blk < 0 || blk >= p.num_blocks) {
    // a new page that was refused or popped invalid is reported by the
    // allocation kernel; an invalid existing entry is reported here
    if (tid == 0 && slot != 0) report(p.err, PA_DEV_BAD_BLOCK);
    pdl_wait_primary();
    return;
  }
  const int kv = is_k ? 0 : 1, h = is_k ? head : head - kHkv;
  unsigned char *half = p.kv + (static_cast<size_t>(blk) * 2 + kv) * kHalfPage + h * kQ8HeadBytes;
  float *scale = o.scales + (static_cast<size_t>(blk) * 2 + kv) * kHkv + h;
  int e = q8_exponent(top, is_k ? kMantK : kMantV);
  if (slot != 0) {
    const int held = q8_scale_exponent(*scale);
    // (the head's 8 threads read the scale before one of them writes it)
    __syncwarp(0xffu << (threadIdx.x & 24));
    if (held < kMinExp) {
      if (j == 0) report(p.err, PA_DEV_BAD_SCALE);
      pdl_wait_primary();
      return;
    }
    if (e > held) {
      const float ratio = pow2(max(held - e, -126));
      for (int t = 0; t < slot; ++t) {
        uint2 *w = reinterpret_cast<uint2 *>(half + t * kQ8TokBytes + 8 * j);
        const uint2 v = *w;
        *w = make_uint2(e4m3x4_rescale(v.x, ratio), e4m3x4_rescale(v.y, ratio));
      }
    } else {
      e = held;
    }
  }
  if (j == 0) *scale = pow2(e);
  const float inv = pow2(-e);
  unsigned char *row = half + slot * kQ8TokBytes;
  const uint32_t lo = bf16x4_to_e4m3x4(x.lo.x, x.lo.y, inv);
  const uint32_t hi = bf16x4_to_e4m3x4(x.hi.x, x.hi.y, inv);
  if (is_k) {
    *reinterpret_cast<uint32_t *>(row + 4 * j) = lo;
    *reinterpret_cast<uint32_t *>(row + kD / 2 + 4 * j) = hi;
  } else {
    *reinterpret_cast<uint2 *>(row + 8 * j) = make_uint2(lo, hi);
  }
  pdl_wait_primary();   // this grid ends after the allocation kernel
}

// ------------------------------------------------------------------ prefill
// (cos, sin) of a row's 32 pairs: thread c of a head row takes pairs 8c..8c+7,
// two at a time; pairs 8c + 2w and 8c + 2w + 1 lie at [4w + c], so that the four
// threads of a row read 64 consecutive bytes.
struct __align__(16) RowAngles {
  float4 a[kD / 4];
  __device__ __forceinline__ void set(int d, float2 cs) {
    const int c = d >> 3, w = (d >> 1) & 3;
    reinterpret_cast<float2 *>(&a[4 * w + c])[d & 1] = cs;
  }
};

// 16 bytes (8 bf16) of one half of a head row, rotated against the other half.
__device__ __forceinline__ void rotate8(uint4 *lo, uint4 *hi, const RowAngles &r, int c) {
  rotate2(&lo->x, &hi->x, r.a[c]);
  rotate2(&lo->y, &hi->y, r.a[4 + c]);
  rotate2(&lo->z, &hi->z, r.a[8 + c]);
  rotate2(&lo->w, &hi->w, r.a[12 + c]);
}

// The same for keys: bits bit .. bit + 3.
__device__ __forceinline__ void rotate8_key(uint4 *lo, uint4 *hi, const RowAngles &r, int c, int bit,
                                            uint32_t *borders) {
  rotate2_key(&lo->x, &hi->x, r.a[c], bit, borders);
  rotate2_key(&lo->y, &hi->y, r.a[4 + c], bit + 1, borders);
  rotate2_key(&lo->z, &hi->z, r.a[8 + c], bit + 2, borders);
  rotate2_key(&lo->w, &hi->w, r.a[12 + c], bit + 3, borders);
}

__device__ __forceinline__ uint32_t q8_top4(uint4 w, uint32_t top) {
  return q8_top(w.w, q8_top(w.z, q8_top(w.y, q8_top(w.x, top))));
}

// The largest magnitudes (bf16 patterns, infinities and NaN among them) of the
// even and the odd elements of w, and of `top`.
__device__ __forceinline__ uint32_t any_top4(uint4 w, uint32_t top) {
  constexpr uint32_t kMag = 0x7fff7fffu;
  return __vmaxu2(top, __vmaxu2(__vmaxu2(w.x & kMag, w.y & kMag), __vmaxu2(w.z & kMag, w.w & kMag)));
}

// Eight bf16 times `inv` to eight e4m3; plain: none of them is infinite.
__device__ __forceinline__ uint2 quantise8(uint4 w, float inv, bool plain) {
  if (plain) {
    uint2 r;
    float2 a = bf16x2_to_float2(w.x), b = bf16x2_to_float2(w.y);
    r.x = e4m3x2_plain(a.x * inv, a.y * inv) | (e4m3x2_plain(b.x * inv, b.y * inv) << 16);
    a = bf16x2_to_float2(w.z);
    b = bf16x2_to_float2(w.w);
    r.y = e4m3x2_plain(a.x * inv, a.y * inv) | (e4m3x2_plain(b.x * inv, b.y * inv) << 16);
    return r;
  }
  return make_uint2(bf16x4_to_e4m3x4(w.x, w.y, inv), bf16x4_to_e4m3x4(w.z, w.w, inv));
}

// A page CTA takes the rows of one call that fall into one page.  Sequence s owns
// CTAs cu_tokens[s] / BT + 2 s and up: n rows touch at most n / BT + 2 pages, so
// the ranges do not meet, and total_tokens / BT + 2 num_seqs CTAs hold them all.
// The other CTAs take kQRows packed rows of q each: one per SM (`lead`) before the
// page CTAs, which meanwhile wait for the pages that the allocation kernel hands
// out, and the rest after them.  CTAs of 64 registers, four (256 threads) an SM.
// Bound by memory and by each CTA's chain of load, angle, maximum, table entry and
// store: 8 x 2048 tokens 33.6 us, 184 MB at 5.5 TB/s (no q CTA first 34.7, 304
// first 33.2; q in the page CTAs, every row's angles in fp64 36.5; a CTA per window
// of rows with every warp on k, v and q in turn 53), 31 tokens 6.5 to 7.4 us.
template <int BT>
struct StoreGeom {
  static constexpr int kThreads = BT == 32 ? 512 : 256;
  static constexpr int kPassRows = kThreads / 32;    // rows of k and v a pass takes: 4 threads per kv head
  static constexpr int kPasses = BT / kPassRows;     // 1, 2, 2
  static constexpr int kQRows = kThreads / 32;
  static constexpr int kQParts = 4;                  // 16-byte parts (and their partners) a thread holds
  static constexpr int kRows = BT > kQRows ? BT : kQRows;
  static_assert(kPassRows * kPasses == BT && kThreads * kQParts == kQRows * kHq * 4, "");
};

// The number of s in [lo, hi) with start(s) <= x, plus lo, for start that does not
// decrease: every thread of the CTA probes, so that each round divides the range
// by their number.
template <int kThreads, class Start>
__device__ __forceinline__ int first_after(int lo, int hi, int x, Start start) {
  while (hi - lo > kThreads) {
    const int step = (hi - lo + kThreads - 1) / kThreads;
    const long long s = lo + static_cast<long long>(threadIdx.x) * step;
    const int c = __syncthreads_count(s < hi && start(static_cast<int>(s)) <= x);
    if (c == 0) return lo;
    lo += (c - 1) * step;
    hi = min(hi, lo + step);
  }
  const int s = lo + threadIdx.x;
  return lo + __syncthreads_count(s < hi && start(s) <= x);
}

// The packed rows [r0, r0 + kQRows) of q, rotated.
template <int BT>
__device__ __forceinline__ void rotate_q_rows(const PrefillAppendParams &p, const Q8Out &o, int r0,
                                              RowAngles *cs, int *row_pos, int *row_run,
                                              BaseAngle (*base)[kD / 2], const float2 *table_f,
                                              const float2 *table_e) {
  using G = StoreGeom<BT>;
  const int tid = threadIdx.x, c = tid & 3;
  uint4 lo[G::kQParts], hi[G::kQParts];
  auto at = [&](int i) -> size_t {   // part i of the thread: row, head, part c
    const int item = tid + i * G::kThreads;
    return (static_cast<size_t>(r0 + (item >> 7)) * kHq + ((item >> 2) & 31)) * kD + 8 * c;
  };
  auto row_of = [&](int i) { return (tid + i * G::kThreads) >> 7; };
#pragma unroll
  for (int i = 0; i < G::kQParts; ++i) {
    lo[i] = hi[i] = make_uint4(0, 0, 0, 0);
    if (r0 + row_of(i) < p.total_tokens) {
      lo[i] = *reinterpret_cast<const uint4 *>(p.q + at(i));
      hi[i] = *reinterpret_cast<const uint4 *>(p.q + at(i) + kD / 2);
    }
  }
  if (tid < G::kQRows) row_pos[tid] = -1;   // rows of refused chunks stay as they are
  int s0 = 0, s1 = p.num_seqs;
  if (s1 > G::kThreads) {   // the sequences that may have rows here
    auto start = [&](int s) { return p.cu_tokens[s]; };
    s0 = max(first_after<G::kThreads>(0, s1, r0, start) - 1, 0);
    s1 = first_after<G::kThreads>(s0, s1, r0 + G::kQRows - 1, start);
  }
  __syncthreads();
  for (int s = s0 + tid; s < s1; s += G::kThreads) {
    const int a = p.cu_tokens[s], b = p.cu_tokens[s + 1];
    if (a >= r0 + G::kQRows || b <= r0) continue;
    int ctx, n;
    if (!chunk_fits<BT>(p, s, &ctx, &n)) continue;
    const int run = max(a, r0);
    for (int r = run; r < min(b, r0 + G::kQRows); ++r) {
      row_pos[r - r0] = ctx + (r - a);
      row_run[r - r0] = run - r0;
    }
  }
  __syncthreads();
  for (int x = tid; x < G::kQRows * (kD / 2); x += G::kThreads) {
    const int t = x / (kD / 2), d = x % (kD / 2);
    if (row_pos[t] >= 0 && row_run[t] == t) base[t][d] = base_angle(row_pos[t], p.freqs.f[d]);
  }
  __syncthreads();
  for (int x = tid; x < G::kQRows * (kD / 2); x += G::kThreads) {
    const int t = x / (kD / 2), d = x % (kD / 2);
    if (row_pos[t] < 0) continue;
    cs[t].set(d, angle_cos_sin(base[row_run[t]][d], t - row_run[t], table_f[d], table_e));
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < G::kQParts; ++i) {
    if (row_pos[row_of(i)] < 0) continue;
    rotate8(&lo[i], &hi[i], cs[row_of(i)], c);
    *reinterpret_cast<uint4 *>(o.q_out + at(i)) = lo[i];
    *reinterpret_cast<uint4 *>(o.q_out + at(i) + kD / 2) = hi[i];
  }
}

template <int BT>
__global__ void __launch_bounds__(StoreGeom<BT>::kThreads, 1024 / StoreGeom<BT>::kThreads)
prefill_store_q8_kernel(PrefillAppendParams p, Q8Out o, int lead, int page_ctas) {
  using G = StoreGeom<BT>;
  constexpr size_t kHalfPage = static_cast<size_t>(BT) * kQ8TokBytes;
  __shared__ RowAngles cs[G::kRows];
  __shared__ float2 table_e[kAngles], table_f[kD / 2];
  __shared__ BaseAngle base[G::kQRows][kD / 2];
  __shared__ int row_pos[G::kQRows], row_run[G::kQRows];
  __shared__ int owner_s, ctx_s, n_s, row0_s;   // the sequence, its context, rows and first row
  __shared__ uint32_t top_s[2][kHkv];
  __shared__ int e_s[2][kHkv], held_s[2][kHkv];   // held: exponent of the page's scale so far
  __shared__ int blk_s;
  pdl_launch_dependents();   // the next kernel may start its own set-up
  const int tid = threadIdx.x;
  if (tid < kAngles) table_e[tid] = o.table.e[tid];
  else if (tid < kAngles + kD / 2) table_f[tid - kAngles] = o.table.f[tid - kAngles];
  const int page_cta = static_cast<int>(blockIdx.x) - lead;
  if (page_cta < 0 || page_cta >= page_ctas) {
    rotate_q_rows<BT>(p, o, (page_cta < 0 ? blockIdx.x : blockIdx.x - page_ctas) * G::kQRows, cs, row_pos, row_run, base,
                      table_f, table_e);
    pdl_wait_primary();   // this grid ends after the allocation kernel
    return;
  }
  if (tid == 0) owner_s = -1;
  if (tid < 2 * kHkv) top_s[tid >> 3][tid & 7] = 0u;
  __syncthreads();
  int s0 = 0, s1 = p.num_seqs;
  if (s1 > G::kThreads) {
    s1 = first_after<G::kThreads>(0, s1, page_cta, [&](int s) { return p.cu_tokens[s] / BT + 2 * s; });
    s0 = max(s1 - 1, 0);
  }
  int mine = -1, my_ctx = 0, my_n = 0;
  for (int s = s0 + tid; s < s1; s += G::kThreads) {
    int ctx, n;
    // (a refused chunk is reported by the allocation kernel)
    if (!chunk_fits<BT>(p, s, &ctx, &n) || n == 0) continue;
    const long long j = static_cast<long long>(page_cta) - (p.cu_tokens[s] / BT + 2ll * s);
    if (j < 0 || j > (ctx + n - 1) / BT - ctx / BT) continue;
    mine = s;
    my_ctx = ctx;
    my_n = n;
  }
  // (more than one claim only where cu_tokens decreases somewhere)
  if (mine >= 0) atomicMax(&owner_s, mine);
  __syncthreads();
  const int seq = owner_s;
  if (seq < 0) {
    pdl_wait_primary();   // this grid ends after the allocation kernel
    return;
  }
  if (mine == seq) {
    ctx_s = my_ctx;
    n_s = my_n;
    row0_s = p.cu_tokens[seq];
  }
  __syncthreads();
  const int ctx = ctx_s;
  const int page_at = ctx / BT + page_cta - (row0_s / BT + 2 * seq);
  const int pos0 = max(ctx, page_at * BT);
  const int len = min(ctx + n_s, page_at * BT + BT) - pos0;
  const size_t first = static_cast<size_t>(row0_s) + (pos0 - ctx);   // packed row of pos0
  const int c = tid & 3;
  if (tid < kD / 2) base[0][tid] = base_angle(pos0, p.freqs.f[tid]);
  const int krow = tid >> 5, khead = (tid >> 2) & 7;
  uint4 klo[G::kPasses], khi[G::kPasses], v0[G::kPasses], v1[G::kPasses];
#pragma unroll
  for (int i = 0; i < G::kPasses; ++i) {
    const int t = krow + i * G::kPassRows;
    klo[i] = khi[i] = v0[i] = v1[i] = make_uint4(0, 0, 0, 0);
    if (t < len) {
      const size_t row = ((first + t) * kHkv + khead) * kD;
      klo[i] = *reinterpret_cast<const uint4 *>(p.k_new + row + 8 * c);
      khi[i] = *reinterpret_cast<const uint4 *>(p.k_new + row + kD / 2 + 8 * c);
      v0[i] = *reinterpret_cast<const uint4 *>(p.v_new + row + 16 * c);
      v1[i] = *reinterpret_cast<const uint4 *>(p.v_new + row + 16 * c + 8);
    }
  }
  // ---- the largest magnitudes of each head's keys (before the rotation) and values
  uint32_t top_k = 0, top_v = 0;
#pragma unroll
  for (int i = 0; i < G::kPasses; ++i) {
    top_k = any_top4(khi[i], any_top4(klo[i], top_k));
    top_v = any_top4(v1[i], any_top4(v0[i], top_v));
  }
  top_k = max(top_k & 0xffffu, top_k >> 16);
  top_v = max(top_v & 0xffffu, top_v >> 16);
  // rare: infinities and NaN do not count (nor stay plain the keys that a
  // rotation might make infinite, from 2^126)
  const bool plain_k = top_k < 0x7e80u, plain_v = top_v < 0x7f80u;
  if (!plain_k || !plain_v) {
    top_k = top_v = 0;
#pragma unroll
    for (int i = 0; i < G::kPasses; ++i) {
      top_k = q8_top4(khi[i], q8_top4(klo[i], top_k));
      top_v = q8_top4(v1[i], q8_top4(v0[i], top_v));
    }
  }
  top_k = max(top_k, __shfl_xor_sync(0xffffffffu, top_k, 1));
  top_k = max(top_k, __shfl_xor_sync(0xffffffffu, top_k, 2));
  top_v = max(top_v, __shfl_xor_sync(0xffffffffu, top_v, 1));
  top_v = max(top_v, __shfl_xor_sync(0xffffffffu, top_v, 2));
  if (c == 0) {
    atomicMax(&top_s[0][khead], top_k);
    atomicMax(&top_s[1][khead], top_v);
  }
  __syncthreads();
  // ---- the page and its scales
  const int slot0 = pos0 % BT;
  if (tid < 2 * kHkv) {
    const bool opened = slot0 == 0;   // this call opens the page
    if (opened) pdl_wait_primary();   // its entry comes from the allocation kernel
    const int blk = p.block_table[table_row(seq, p.n_layers, p.layer, p.max_blocks) + page_at];
    const bool ok = blk >= 0 && blk < p.num_blocks;
    const int kv = tid >> 3, h = tid & 7;
    int e = q8_exponent(top_s[kv][h], kv ? kMantV : kMantK), held = e;
    if (ok) {
      float *scale = o.scales + (static_cast<size_t>(blk) * 2 + kv) * kHkv + h;
      if (!opened) {
        held = q8_scale_exponent(*scale);
        if (held < kMinExp) report(p.err, PA_DEV_BAD_SCALE);
        e = max(e, held);
      }
      if (held >= kMinExp) *scale = pow2(e);
    } else if (!opened && tid == 0) {
      // a page of this chunk that was refused or popped invalid is reported
      // by the allocation kernel; an invalid page from before is reported here
      report(p.err, PA_DEV_BAD_BLOCK);
    }
    e_s[kv][h] = e;
    held_s[kv][h] = held;
    if (tid == 0) blk_s = ok ? blk : -1;
  }
  for (int x = tid; x < len * (kD / 2); x += G::kThreads) {   // (meanwhile)
    const int t = x / (kD / 2), d = x % (kD / 2);
    cs[t].set(d, angle_cos_sin(base[0][d], t, table_f[d], table_e));
  }
  __syncthreads();
  uint32_t borders = 0;   // bit 4 i + w: word w of row i's parts
#pragma unroll
  for (int i = 0; i < G::kPasses; ++i) {
    const int t = krow + i * G::kPassRows;
    if (t < len) rotate8_key(&klo[i], &khi[i], cs[t], c, 4 * i, &borders);
  }
  if (blk_s >= 0) {
    unsigned char *page = p.kv + static_cast<size_t>(blk_s) * 2 * kHalfPage;
    // ---- tokens that the page holds already are brought to its new scale
    for (int x = tid; x < slot0 * 64; x += G::kThreads) {   // 16-byte parts: 32 of K, 32 of V a token
      const int t = x >> 6, kv = (x >> 5) & 1, part = x & 31, h = part >> 2;
      const int held = held_s[kv][h], e = e_s[kv][h];
      if (held < kMinExp || held == e) continue;
      const float ratio = pow2(max(held - e, -126));
      uint4 *w = reinterpret_cast<uint4 *>(page + kv * kHalfPage + t * kQ8TokBytes + 16 * part);
      uint4 u = *w;
      u.x = e4m3x4_rescale(u.x, ratio);
      u.y = e4m3x4_rescale(u.y, ratio);
      u.z = e4m3x4_rescale(u.z, ratio);
      u.w = e4m3x4_rescale(u.w, ratio);
      *w = u;
    }
    const float inv_k = pow2(-e_s[0][khead]), inv_v = pow2(-e_s[1][khead]);
#pragma unroll
    for (int i = 0; i < G::kPasses; ++i) {
      const int t = krow + i * G::kPassRows;
      if (t >= len) continue;
      unsigned char *row = page + (slot0 + t) * kQ8TokBytes + khead * kQ8HeadBytes;
      if (held_s[0][khead] >= kMinExp) {
        *reinterpret_cast<uint2 *>(row + 8 * c) = quantise8(klo[i], inv_k, plain_k);
        *reinterpret_cast<uint2 *>(row + kD / 2 + 8 * c) = quantise8(khi[i], inv_k, plain_k);
      }
      if (held_s[1][khead] >= kMinExp) {
        const uint2 a = quantise8(v0[i], inv_v, plain_v), b = quantise8(v1[i], inv_v, plain_v);
        *reinterpret_cast<uint4 *>(row + kHalfPage + 16 * c) = make_uint4(a.x, a.y, b.x, b.y);
      }
    }
    if (!plain_k || held_s[0][khead] < kMinExp) borders = 0;
#pragma unroll 1
    for (; borders; borders &= borders - 1) {
      const int i = (__ffs(borders) - 1) >> 2, d = 8 * c + 2 * ((__ffs(borders) - 1) & 3);
      const int t = krow + i * G::kPassRows;
      exact_key_word(p.k_new + ((first + t) * kHkv + khead) * kD,
                     page + (slot0 + t) * kQ8TokBytes + khead * kQ8HeadBytes, d, pos0 + t, inv_k, p.freqs,
                     o.table.exact);
    }
  }
  pdl_wait_primary();   // this grid ends after the allocation kernel
}

}  // namespace
}  // namespace pa

using namespace pa;

namespace {

template <int BT>
int kv_append_q8_impl(const uint16_t *k_new, const uint16_t *v_new, const uint16_t *q_or_null,
                      uint16_t *q_out, uint8_t *kv_cache, float *kv_scales, int num_blocks,
                      int32_t *block_table, int n_layers, int max_blocks_per_seq,
                      const int32_t *context_lens, int num_seqs, int layer, int32_t *free_list,
                      int32_t *free_count, int32_t *err, void *stream) {
  if (num_seqs < 0 || num_blocks <= 0 || n_layers <= 0 || max_blocks_per_seq <= 0)
    return PA_ERR_ARG;
  if (static_cast<long long>(max_blocks_per_seq) * BT > INT_MAX) return PA_ERR_ARG;
  if (layer < 0 || layer >= n_layers) return PA_ERR_LAYER;
  if (num_seqs == 0) return PA_OK;
  if (!k_new || !v_new || !kv_cache || !kv_scales || !block_table || !context_lens || !free_list ||
      !free_count || !err || (q_or_null && !q_out))
    return PA_ERR_NULL;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(kv_cache) || !aligned16(kv_scales) ||
      (q_or_null && (!aligned16(q_or_null) || !aligned16(q_out))))
    return PA_ERR_ALIGN;
  DeviceInfo di;
  const int rc = current_device(&di);
  if (rc != PA_OK) return rc;

  static const RopeFreqs freqs = llama3_freqs();
  AppendParams prm;
  prm.freqs = freqs;
  prm.k_new = k_new;
  prm.v_new = v_new;
  prm.q = const_cast<uint16_t *>(q_or_null);   // read only: rotated rows go to q_out
  prm.kv = kv_cache;
  prm.block_table = block_table;
  prm.context_lens = context_lens;
  prm.free_list = free_list;
  prm.free_count = free_count;
  prm.err = err;
  prm.num_blocks = num_blocks;
  prm.n_layers = n_layers;
  prm.max_blocks = max_blocks_per_seq;
  prm.num_seqs = num_seqs;
  prm.layer = layer;
  static const AngleTable table = angle_table(freqs);
  const Q8Out o{q_out, kv_scales, table};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (launch_pdl(append_alloc_kernel<BT>, dim3(1), dim3(kScanCta), 0, st, prm) != cudaSuccess)
    return PA_ERR_CUDA;
  if (launch_pdl(append_store_q8_kernel<BT>, dim3(num_seqs), dim3(kStoreQ8Threads), 0, st, prm,
                 o) != cudaSuccess)
    return PA_ERR_CUDA;
  return PA_OK;
}

template <int BT>
int prefill_append_q8_impl(const uint16_t *k_new, const uint16_t *v_new, const uint16_t *q_or_null,
                           uint16_t *q_out, int total_tokens, const int32_t *cu_tokens,
                           uint8_t *kv_cache, float *kv_scales, int num_blocks,
                           int32_t *block_table, int n_layers, int max_blocks_per_seq,
                           const int32_t *context_lens, int num_seqs, int layer,
                           int32_t *free_list, int32_t *free_count, int32_t *err, void *stream) {
  if (num_seqs < 0 || total_tokens < 0 || num_blocks <= 0 || n_layers <= 0 ||
      max_blocks_per_seq <= 0)
    return PA_ERR_ARG;
  if (static_cast<long long>(max_blocks_per_seq) * BT > INT_MAX) return PA_ERR_ARG;
  if (layer < 0 || layer >= n_layers) return PA_ERR_LAYER;
  if (num_seqs > (1 << 29)) return PA_ERR_ARG;   // the grid: total_tokens / BT + 2 num_seqs + total_tokens / 8
  if (num_seqs == 0 || total_tokens == 0) return PA_OK;
  if (!k_new || !v_new || !cu_tokens || !kv_cache || !kv_scales || !block_table ||
      !context_lens || !free_list || !free_count || !err || (q_or_null && !q_out))
    return PA_ERR_NULL;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(kv_cache) || !aligned16(kv_scales) ||
      (q_or_null && (!aligned16(q_or_null) || !aligned16(q_out))))
    return PA_ERR_ALIGN;
  DeviceInfo di;
  const int rc = current_device(&di);
  if (rc != PA_OK) return rc;
  static const RopeFreqs freqs = llama3_freqs();
  PrefillAppendParams prm;
  prm.freqs = freqs;
  prm.k_new = k_new;
  prm.v_new = v_new;
  prm.q = const_cast<uint16_t *>(q_or_null);   // read only: rotated rows go to q_out
  prm.kv = kv_cache;
  prm.block_table = block_table;
  prm.cu_tokens = cu_tokens;
  prm.context_lens = context_lens;
  prm.free_list = free_list;
  prm.free_count = free_count;
  prm.err = err;
  prm.total_tokens = total_tokens;
  prm.num_blocks = num_blocks;
  prm.n_layers = n_layers;
  prm.max_blocks = max_blocks_per_seq;
  prm.num_seqs = num_seqs;
  prm.layer = layer;
  static const AngleTable table = angle_table(freqs);
  const Q8Out o{q_out, kv_scales, table};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (launch_pdl(prefill_alloc_kernel<BT>, dim3(1), dim3(kScanCta), 0, st, prm) != cudaSuccess)
    return PA_ERR_CUDA;
  using G = StoreGeom<BT>;
  const int page_ctas = total_tokens / BT + 2 * num_seqs;
  const int q_ctas = q_or_null ? (total_tokens + G::kQRows - 1) / G::kQRows : 0;
  if (launch_pdl(prefill_store_q8_kernel<BT>, dim3(page_ctas + q_ctas), dim3(G::kThreads), 0, st, prm,
                 o, std::min(q_ctas, di.sm_count), page_ctas) != cudaSuccess)
    return PA_ERR_CUDA;
  return PA_OK;
}

}  // namespace

extern "C" int pa_kv_append_rope_q8(const uint16_t *k_new, const uint16_t *v_new,
                                    const uint16_t *q_or_null, uint16_t *q_out, uint8_t *kv_cache,
                                    float *kv_scales, int num_blocks, int block_tokens,
                                    int32_t *block_table, int n_layers, int max_blocks_per_seq,
                                    const int32_t *context_lens, int num_seqs, int layer,
                                    int32_t *free_list, int32_t *free_count, int32_t *err,
                                    void *stream) {
  auto *impl = block_tokens == 8    ? kv_append_q8_impl<8>
               : block_tokens == 16 ? kv_append_q8_impl<16>
               : block_tokens == 32 ? kv_append_q8_impl<32>
                                    : nullptr;
  if (!impl) return PA_ERR_ARG;
  return impl(k_new, v_new, q_or_null, q_out, kv_cache, kv_scales, num_blocks, block_table,
              n_layers, max_blocks_per_seq, context_lens, num_seqs, layer, free_list, free_count,
              err, stream);
}

extern "C" int pa_prefill_append_rope_q8(const uint16_t *k_new, const uint16_t *v_new,
                                         const uint16_t *q_or_null, uint16_t *q_out,
                                         int total_tokens, const int32_t *cu_tokens,
                                         uint8_t *kv_cache, float *kv_scales, int num_blocks,
                                         int block_tokens, int32_t *block_table, int n_layers,
                                         int max_blocks_per_seq, const int32_t *context_lens,
                                         int num_seqs, int layer, int32_t *free_list,
                                         int32_t *free_count, int32_t *err, void *stream) {
  auto *impl = block_tokens == 8    ? prefill_append_q8_impl<8>
               : block_tokens == 16 ? prefill_append_q8_impl<16>
               : block_tokens == 32 ? prefill_append_q8_impl<32>
                                    : nullptr;
  if (!impl) return PA_ERR_ARG;
  return impl(k_new, v_new, q_or_null, q_out, total_tokens, cu_tokens, kv_cache, kv_scales,
              num_blocks, block_table, n_layers, max_blocks_per_seq, context_lens, num_seqs, layer,
              free_list, free_count, err, stream);
}
