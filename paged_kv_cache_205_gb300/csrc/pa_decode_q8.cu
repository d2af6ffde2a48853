// pa_decode_q8.cu -- decode attention over the 8-bit cache (pa_q8.cuh).
//
//   out[h] = sum_t softmax_t(scale * q[h] . (sK K_t)) (sV V_t)
//
// decode_q8_kernel: the 16-token tiles of all sequences are laid end to end
// and cut into one equal run for each CTA (two CTAs an SM).  A producer warp
// streams the run's tiles into a ring of shared-memory stages, one 16 KiB TMA
// copy (16 tokens x 8 kv heads x K, V) and one 64-byte copy of the page's
// scales a tile, and the sequence's q with the first tile of a piece; eight
// consumer warps, one per kv head, follow.  A sequence that lies in one run
// is written by its CTA; the pieces of the others are merged by
// decode_q8_merge_kernel.  Tables of at most kDirectTiles tiles a sequence run
// one CTA a sequence and no merge.
// Measured on the way (us, 4 x 32768 tokens / 256 ragged sequences; floors at
// the copy peak 19.8 / 39.1):
//   46.1 / 92.8  consumer warps load tiles into registers, two ahead: each
//                chunk's first loads wait for its page ids
//   36.1 / 64.1  the producer warp; chunks of 1/4 of a CTA's share from a counter
//   33.2 / 63.2  q with the tiles, page ids a batch ahead, half a share a chunk
//   29.2 / 52.8  one run a CTA: the finer cuts balance SMs of unequal speed
//                better (the last tile at 45.9 instead of 47.3 us), but every
//                piece costs 8.4 KiB of partial written and read again
//   26.9 / 53.5  the plan made, and 4 tiles a CTA prefetched, while the kernels
//                before end (2 rows of 14 to 17 tokens, direct: 5.5 to 3.5)
//   26.3 / 49.9  the reference below the largest score (fewer moves), shared
//                memory addressed as such
// Of the 53.5: 4.4 to the first data, 37 at 7.1 TB/s, 5 between the CTAs' last
// tiles (SMs of unequal speed), 5 to end, launch and run the merge.
// The copies' rows are two heads wide (128 bytes): the TMA unit takes a box row
// by row.
//
// A consumer computes the transposed products, so that the 4 q heads of the
// group fill half of the MMAs' 8 columns (as rows they would fill a quarter of
// 16): S^T = K Q^T (tokens x heads, 4 m16n8k16) and O^T = V^T P^T (dims x
// heads, 4 m16n8k16) a tile.  The inner and output dimensions are permuted to
// what wide shared-memory loads deliver (a sum may be taken in any order):
//   S^T  lane (g, c) (g = lane / 4, c = lane % 4) reads dims 16c..16c+15 of
//        the tokens that rows g and g + 8 stand for (one 16-byte load each);
//        k-step ks takes dims 16c + 4 ks + {0, 1} and {2, 3}.
//   P    S^T's fragments in f16 become P^T's with one movmatrix per 8 tokens.
//   O^T  ldmatrix.trans on byte pairs: a register holds dims 2g, 2g + 1 of a
//        16-dim group for two tokens; one byte permute and two conversions
//        make A's rows g (even dims) and g + 8 (odd dims).
//   Row n of a group of 8 stands for token n / 2 + 4 (n % 2): with two heads'
//   64 bytes in a 128-byte row, swizzled by the token, the loads of both
//   products are then free of bank conflicts.
// The running maximum is a reference set 2^7 below the largest score that moves
// only when a score exceeds it by more than 2^15 (one vote a tile instead of a
// reduction over the tokens and a rescale of O), so P <= 2^15.
// e4m3 becomes f16 exactly; q is scaled by a power of two per head to f16
// (exact for values down to 2^-29 of the head's largest).  P enters the MMA in
// f16: half a step is 2^-12 of a weight (2^-25 absolute below 2^-14, which is
// 2^-32 of the largest weight), an eighth of the output's own bf16 rounding; m
// and l stay fp32.  K's scale
// multiplies the scores; V's multiplies the tile's product when it is added
// to the running output.
#include <climits>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include "pa_decode_tile.cuh"
#include "pa_host.h"
#include "pa_q8.cuh"

namespace pa {
namespace {

constexpr int kWarps = kHkv;               // consumer warps, one per kv head
constexpr int kThreads = (kWarps + 1) * 32;   // + producer warp
constexpr int kScanThreads = kWarps * 32;
constexpr int kCtasPerSm = 2;
constexpr int kStages = 5;
constexpr int kMaxSeqs = 2048;             // the tile prefix is kept in shared memory
constexpr int kMaxGrid = 512;
constexpr int kTile = 16;                  // tokens
constexpr int kDirectTiles = 8;            // longest table served by one CTA a sequence
constexpr int kPrefetchTiles = 4;          // tiles brought into L2 before the wait
constexpr int kTileBytes = 2 * kTile * kQ8TokBytes;   // K and V of 8 heads: 16 KiB
constexpr int kPairBytes = 2 * kQ8HeadBytes;          // one token, two heads: a row of the copies
constexpr float kNoScore = -3e38f;       // the reference before a score is seen
constexpr float kBelow = 7.f;            // log2 units the reference is set below the largest score
constexpr float kMove = 15.f;            // and a score may lie above it
constexpr float kLog2e = 1.4426950408889634f;

constexpr int kSegStart = 1;   // first tile of a sequence's piece in the run
constexpr int kSegEnd = 2;     // last tile of that piece
constexpr int kEndOfWork = 4;  // no more tiles; the stage carries no data

struct StageDesc {
  int seq;
  int flags;
  int slot;      // partial slot of the piece, or -1: the sequence is in one piece
  uint32_t use;  // bit t: token t of the tile is used
};

struct Q8DecodeParams {
  __nv_bfloat16 *out;
  const uint16_t *q;
  const unsigned char *kv;
  const float *scales;
  const int32_t *block_table;
  const int32_t *context_lens;
  // partials: the piece of sequence s in run k is slot k + s
  float2 *ml;          // [slots][32] (m, l), m in the log2 domain
  float *acc;          // [slots][32][64] unnormalised output
  int32_t *err;
  int num_blocks;
  int n_layers;
  int max_blocks;
  int num_seqs;
  int layer;
  int cap_tokens;
  float qscale;        // scale * log2(e)
  int direct;          // one CTA a sequence
  // test hook (pa_decode_set_test_fault): the stage of CTA 0 whose copies are
  // left out (-1: none), and the limit of every wait
  int fault_stage;
  unsigned long long wait_ns;
};

struct __align__(1024) Smem {
  unsigned char kv[kStages][kTileBytes];   // [K|V][head pair][16 tokens][2][64], 128-byte swizzled;
                                           // 8-token pages: two of [K|V][pair][8][2][64]
  unsigned char q[kStages][kHq * kD * 2];  // first tile of a piece: the sequence's q
  float scale[kStages][2][2 * kHkv];       // [page of the tile][K|V][head]
  StageDesc desc[kStages];
  uint64_t full[kStages];
  uint64_t empty[kStages];
  int warp_sum[kWarps];
  int prefix[1];                           // [num_seqs + 1] tiles of sequences 0..s-1
};

// D = A B + D and D = A B, m16n8k16 and m16n8k8, f16 in, fp32 out.
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_16816_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_1688_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, "
      "{%7, %7, %7, %7};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(b), "f"(0.f));
}

// The transpose of an 8 x 8 matrix of f16 held as an MMA fragment.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Packed two-lane fp32 product.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long ra, rb, rd;
  asm("mov.b64 %0, {%1, %2};" : "=l"(ra) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(rb) : "f"(b.x), "f"(b.y));
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(rd) : "l"(ra), "l"(rb));
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(rd));
  return d;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}

__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// A warp's running softmax of one kv head.  Lane (g, c) holds q heads 2c and
// 2c + 1 of the group (lanes c < 2; the others compute columns of zeros):
// dims 16 i + 2 g (o[2 i]) and 16 i + 2 g + 1 (o[2 i + 1]) of both, and the sums over its
// own tokens.
struct State {
  float2 o[8];
  float2 m, l;   // m (log2 domain) is the same in the 8 lanes of a head pair
  __device__ __forceinline__ void reset() {
    m = make_float2(kNoScore, kNoScore);
    l = make_float2(0.f, 0.f);
#pragma unroll
    for (int t = 0; t < 8; ++t) o[t] = make_float2(0.f, 0.f);
  }
};

// q head g of the group in f16, scaled by a power of two to [2^12, 2^13);
// returns the head's score factor: qscale / that power, or NaN for a head that is
// not finite (its scores are NaN, or all -inf: so is its output).  Lane c holds dims
// 16c .. 16c+15 (the order of the K loads): B's columns of S^T.  q_group: the
// group's q in shared memory.
__device__ __forceinline__ float load_q(uint32_t q_group, int g, int c, float qscale,
                                        uint32_t (&qa)[8]) {
  uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
  if (g < kGqa) {
    const uint32_t at = q_group + (g * kD + 16 * c) * 2;
    w0 = lds16(at);
    w1 = lds16(at + 16);
  }
  const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
  top = max(top & 0xffffu, top >> 16);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const int f = min(266 - static_cast<int>(top >> 7), 253);   // exponent field of the factor
  const float up = __int_as_float(f << 23), down = __int_as_float((254 - f) << 23);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 x = bf16x2_to_float2(w[i]);
    qa[i] = f16x2(x.x * up, x.y * up);
  }
  return top < 0x7f80u ? qscale * down : __int_as_float(0x7fc00000);
}

// Folds a tile into the state.  k0 / k1: the head pair's K rows of tokens 0..7
// and 8..15 in shared memory, v0 / v1 its V rows; chunk0: the head's first
// 16-byte chunk of a row (0 or 4).  use: tokens to use (not 0).
template <int BT>
__device__ __forceinline__ void attend(uint32_t k0, uint32_t k1, uint32_t v0, uint32_t v1,
                                       int chunk0, float2 sk, float2 sv, uint32_t use,
                                       const uint32_t (&qa)[8], float2 qs, int lane, State &st) {
  const int g = lane >> 2, c = lane & 3;
  const int kt = (g >> 1) + 4 * (g & 1);   // the token of column g
  const uint32_t koff = kt * kPairBytes + (((chunk0 + c) ^ kt) << 4);
  const uint4 ka = lds16(k0 + koff), kb = lds16(k1 + koff);
  const int vt = ((lane & 7) >> 1) + 4 * (lane & 1);
  const uint32_t voff = vt * kPairBytes + (((chunk0 + (lane >> 3)) ^ vt) << 4);
  uint32_t va[4], vb[4];
  ldsm_x4_trans(v0 + voff, va[0], va[1], va[2], va[3]);
  ldsm_x4_trans(v1 + voff, vb[0], vb[1], vb[2], vb[3]);
  if (use != 0xffffu) {
    // unused tokens may hold anything, NaN included: they meet P = 0.  (V's
    // registers hold tokens c and c + 4 of each group of 8.)
    const uint32_t ma = ((use >> c) & 1u ? 0xffffu : 0u) | ((use >> (c + 4)) & 1u ? 0xffff0000u : 0u);
    const uint32_t mb = ((use >> (c + 8)) & 1u ? 0xffffu : 0u) | ((use >> (c + 12)) & 1u ? 0xffff0000u : 0u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      va[i] &= ma;
      vb[i] &= mb;
    }
  }
  // ---- S^T = K Q^T: s[0], s[1] = heads 2c, 2c + 1 of row g's token, s[2], s[3] of row g + 8's
  float s[4];
  const uint32_t kw0[4] = {ka.x, ka.y, ka.z, ka.w}, kw1[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) {
    const uint32_t a[4] = {e4m3x2_to_f16x2(kw0[ks]), e4m3x2_to_f16x2(kw1[ks]),
                           e4m3x2_to_f16x2(kw0[ks] >> 16), e4m3x2_to_f16x2(kw1[ks] >> 16)};
    if (ks == 0) mma_16816_zero(s, a, qa[0], qa[1]);
    else mma_16816(s, a, qa[2 * ks], qa[2 * ks + 1]);
  }
  // ---- scores against the reference (log2 domain)
  const float2 f0 = make_float2(qs.x * sk.x, qs.y * sk.x);
  const float2 f1 = BT == 8 ? make_float2(qs.x * sk.y, qs.y * sk.y) : f0;
  // (the product is rounded before the reference is taken off: a fused
  // x - m would leave m's rounding error, which for scores of 2^28 and more
  // overflows the exponential)
  float2 x0 = mul2(make_float2(s[0], s[1]), f0), x1 = mul2(make_float2(s[2], s[3]), f1);
  if (use != 0xffffu) {   // (K rows of unused tokens may hold anything too)
    if (!((use >> kt) & 1u)) x0 = make_float2(neg_inf(), neg_inf());
    if (!((use >> (kt + 8)) & 1u)) x1 = make_float2(neg_inf(), neg_inf());
  }
  float over = fmaxf(fmaxf(x0.x, x1.x) - st.m.x, fmaxf(x0.y, x1.y) - st.m.y);
  if (__any_sync(0xffffffffu, over > kMove)) {
    // the reference moves to the largest score so far
    float nx = fmaxf(x0.x, x1.x), ny = fmaxf(x0.y, x1.y);
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
      nx = fmaxf(nx, __shfl_xor_sync(0xffffffffu, nx, d));
      ny = fmaxf(ny, __shfl_xor_sync(0xffffffffu, ny, d));
    }
    nx = fmaxf(nx - kBelow, st.m.x);
    ny = fmaxf(ny - kBelow, st.m.y);
    const float2 al = make_float2(fast_exp2(st.m.x - nx), fast_exp2(st.m.y - ny));
    st.m = make_float2(nx, ny);
    st.l = mul2(st.l, al);
#pragma unroll
    for (int i = 0; i < 8; ++i) st.o[i] = mul2(st.o[i], al);
  }
  const float y0 = x0.x - st.m.x, y1 = x0.y - st.m.y, y2 = x1.x - st.m.x, y3 = x1.y - st.m.y;
  const float p0 = fast_exp2(y0), p1 = fast_exp2(y1), p2 = fast_exp2(y2), p3 = fast_exp2(y3);
  st.l.x += p0 + p2;
  st.l.y += p1 + p3;
  const uint32_t b0 = transpose8x8(f16x2(p0, p1)), b1 = transpose8x8(f16x2(p2, p3));
  // ---- O^T += sV V^T P^T, 16 dims a step
  const float2 sv0 = make_float2(sv.x, sv.x), sv1 = make_float2(sv.y, sv.y);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // bytes (t0 d0, t0 d1, t1 d0, t1 d1) to (t0 d0, t1 d0, t0 d1, t1 d1)
    const uint32_t x = prmt(va[i], 0u, 0x3120), z = prmt(vb[i], 0u, 0x3120);
    const uint32_t a[4] = {e4m3x2_to_f16x2(x), e4m3x2_to_f16x2(x >> 16), e4m3x2_to_f16x2(z),
                           e4m3x2_to_f16x2(z >> 16)};
    float d[4];
    if (BT == 8) {
      // the two pages' products apart: their scales differ
      float d2[4];
      mma_1688_zero(d, a[0], a[1], b0);
      mma_1688_zero(d2, a[2], a[3], b1);
      st.o[2 * i] = fma2(make_float2(d2[0], d2[1]), sv1, st.o[2 * i]);
      st.o[2 * i + 1] = fma2(make_float2(d2[2], d2[3]), sv1, st.o[2 * i + 1]);
    } else {
      mma_16816_zero(d, a, b0, b1);
    }
    st.o[2 * i] = fma2(make_float2(d[0], d[1]), sv0, st.o[2 * i]);
    st.o[2 * i + 1] = fma2(make_float2(d[2], d[3]), sv0, st.o[2 * i + 1]);
  }
}

// Context lengths and page ids are read past L1: they may be read before the
// wait on the kernels before (to know what to prefetch) and again after it.
__device__ __forceinline__ int ctx_now(const Q8DecodeParams &p, int s) {
  return __ldcg(p.context_lens + s);
}
__device__ __forceinline__ int clamp_ctx(const Q8DecodeParams &p, int t) {
  return min(max(t, 0), p.cap_tokens);
}
__device__ __forceinline__ int tiles_in(int ctx) { return (ctx + kTile - 1) / kTile; }

// Sequence holding tile b (b < total): the smallest s with prefix[s+1] > b.
__device__ __forceinline__ int seq_of_tile(const int *prefix, int n, int b) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid + 1] > b) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// A tile as the producer's lane that issues it knows it.
struct TileWork {
  int blk, blk2;   // page ids (blk2: second page of a tile over 8-token pages, -2: there is none)
  int j;           // tile of the sequence
  int n_tok;
  StageDesc d;     // (d.use is set when the tile is issued)
};

// Lane i: tile t + i of the CTA's run [b0, b1).  Its page ids are read here
// and first looked at when the tile is issued.
template <int BT>
__device__ __forceinline__ TileWork tile_work(const Q8DecodeParams &p, const Smem &sm, int t, int b0,
                                              int b1, int lane) {
  TileWork w;
  w.blk = -1;
  w.blk2 = -2;
  w.j = w.n_tok = 0;
  w.d.seq = w.d.flags = 0;
  w.d.slot = -1;
  w.d.use = 0;
  const int b = t + lane;
  if (b < b1) {
    const int s = p.direct ? static_cast<int>(blockIdx.x) : seq_of_tile(sm.prefix, p.num_seqs, b);
    const int B = p.direct ? 0 : sm.prefix[s], E = p.direct ? b1 : sm.prefix[s + 1];
    w.j = b - B;
    const int32_t *row =
        p.block_table + (static_cast<size_t>(s) * p.n_layers + p.layer) * p.max_blocks;
    w.blk = __ldcg(row + (BT == 32 ? w.j >> 1 : BT == 8 ? 2 * w.j : w.j));
    w.n_tok = kTile;
    if (b == E - 1) w.n_tok = clamp_ctx(p, ctx_now(p, s)) - w.j * kTile;
    if (BT == 8 && w.n_tok > 8) w.blk2 = __ldcg(row + 2 * w.j + 1);
    w.d.seq = s;
    w.d.flags = (w.j == 0 || b == b0 ? kSegStart : 0) | (b == E - 1 || b == b1 - 1 ? kSegEnd : 0);
    if (B < b0 || E > b1) w.d.slot = blockIdx.x + s;   // the sequence is cut into several pieces
  }
  return w;
}

// Brings a tile into L2.
template <int BT>
__device__ __forceinline__ void prefetch_tile(const Q8DecodeParams &p, const TileWork &w) {
  constexpr size_t kPage = static_cast<size_t>(BT) * 2 * kQ8TokBytes;
  if (w.blk < 0 || w.blk >= p.num_blocks) return;
  const unsigned char *page = p.kv + static_cast<size_t>(w.blk) * kPage;
  if (BT == 32) {
    page += (w.j & 1) * (kTile * kQ8TokBytes);
    prefetch_bulk_l2(page, kTile * kQ8TokBytes);
    prefetch_bulk_l2(page + kPage / 2, kTile * kQ8TokBytes);
  } else {
    prefetch_bulk_l2(page, kPage);
    if (BT == 8 && w.blk2 >= 0 && w.blk2 < p.num_blocks)
      prefetch_bulk_l2(p.kv + static_cast<size_t>(w.blk2) * kPage, kPage);
  }
  prefetch_l2(p.scales + static_cast<size_t>(w.blk) * 2 * kHkv);
}

// Tile prefix over the sequences into sm.prefix; returns the total.  Every
// thread of the CTA calls it.
__device__ __forceinline__ int tile_prefix(const Q8DecodeParams &p, Smem &sm, int tid, int warp,
                                           int lane) {
  int carry = 0;
  for (int base = 0; base < p.num_seqs; base += kScanThreads) {
    const int i = base + tid;
    int nb = 0;
    if (tid < kScanThreads && i < p.num_seqs) nb = tiles_in(clamp_ctx(p, ctx_now(p, i)));
    int incl = nb;
    if (tid < kScanThreads) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (lane == 31) sm.warp_sum[warp] = incl;
    }
    __syncthreads();
    int before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const int v = sm.warp_sum[w];
      if (w < warp) before += v;
      sum += v;
    }
    if (tid < kScanThreads && i < p.num_seqs) sm.prefix[i + 1] = carry + before + incl;
    carry += sum;
    __syncthreads();
  }
  if (tid == 0) sm.prefix[0] = 0;
  __syncthreads();
  return carry;
}

// The CTA's run of tiles.
__device__ __forceinline__ void run_of(int total, int G, int *b0, int *b1) {
  const int C = max((total + G - 1) / G, 1);
  *b0 = static_cast<int>(min(static_cast<long long>(blockIdx.x) * C, static_cast<long long>(total)));
  *b1 = min(total, *b0 + C);
}

template <int BT>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    decode_q8_kernel(const __grid_constant__ CUtensorMap kv_map, Q8DecodeParams p) {
  extern __shared__ unsigned char smem_raw[];
  // (an offset, so that the compiler still knows it for shared memory)
  Smem &sm = *reinterpret_cast<Smem *>(smem_raw + (-smem_u32(smem_raw) & 1023u));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = gridDim.x;
  if (tid == 0) {
    prefetch_tensormap(&kv_map);
    for (int st = 0; st < kStages; ++st) {
      mbar_init(&sm.full[st], 1);
      mbar_init(&sm.empty[st], kWarps);
    }
    fence_mbar_init();
  }
  int b0 = 0, b1 = 0;
  TileWork w;
  if (p.direct) {
    pdl_wait_primary();        // everything read below may come from the previous kernel
    pdl_launch_dependents();
    const int ctx = ctx_now(p, blockIdx.x);
    if (tid == 0 && (ctx < 0 || ctx > p.cap_tokens)) report(p.err, PA_DEV_CTX_RANGE);
    b1 = tiles_in(clamp_ctx(p, ctx));
    if (b1 == 0) {
      uint4 *o = reinterpret_cast<uint4 *>(p.out + static_cast<size_t>(blockIdx.x) * kHq * kD);
      for (int e = tid; e < kHq * kD * 2 / 16; e += kThreads) o[e] = make_uint4(0, 0, 0, 0);
    }
    if (warp == kWarps) w = tile_work<BT>(p, sm, 0, 0, b1, lane);
    __syncthreads();           // the barriers are initialised
  } else {
    // ---- while the kernels before end: a plan from the lengths and page ids
    // as they read now, which may still change, to bring the run's first tiles
    // into L2.  Nothing else is done with it unless it still holds afterwards.
    int total = tile_prefix(p, sm, tid, warp, lane);
    run_of(total, G, &b0, &b1);
    if (warp == kWarps) {
      w = tile_work<BT>(p, sm, b0, b0, b1, lane);
      if (lane < kPrefetchTiles) prefetch_tile<BT>(p, w);
    }
    pdl_wait_primary();        // everything read below is current
    pdl_launch_dependents();   // the merge kernel may take its place in the queue
    if (warp == kWarps) w = tile_work<BT>(p, sm, b0, b0, b1, lane);
    int changed = 0;
    for (int i = tid; i < p.num_seqs; i += kThreads) {
      const int t = ctx_now(p, i);
      if (blockIdx.x == 0 && (t < 0 || t > p.cap_tokens)) report(p.err, PA_DEV_CTX_RANGE);
      changed |= tiles_in(clamp_ctx(p, t)) != sm.prefix[i + 1] - sm.prefix[i];
    }
    if (__syncthreads_or(changed)) {
      total = tile_prefix(p, sm, tid, warp, lane);
      run_of(total, G, &b0, &b1);
      if (warp == kWarps) w = tile_work<BT>(p, sm, b0, b0, b1, lane);
    }
    // the CTAs' share of zeros for the sequences with an empty context
    for (int s = blockIdx.x; s < p.num_seqs; s += G)
      if (sm.prefix[s] == sm.prefix[s + 1]) {
        uint4 *o = reinterpret_cast<uint4 *>(p.out + static_cast<size_t>(s) * kHq * kD);
        for (int e = tid; e < kHq * kD * 2 / 16; e += kThreads) o[e] = make_uint4(0, 0, 0, 0);
      }
  }

  if (warp == kWarps) {
    // ===================================================== producer warp ==
    // Batches of up to 32 tiles, whatever sequences they belong to: lane i
    // works out tile i and later issues it.  The next batch's page ids are on
    // their way while a batch is issued.
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    uint32_t issued = 0, issued_parity = 0;   // per stage: used / parity of its last phase
    int published = 0;                        // stages published so far
    for (int t = b0; t < b1 && ok; t += 32) {
      const int cnt = min(32, b1 - t);
      const TileWork cur = w;
      if (t + 32 < b1) w = tile_work<BT>(p, sm, t + 32, b0, b1, lane);
      for (int e = 0; e < cnt; ++e) {
        int good = 1;
        if (lane == e) {
          if (!mbar_wait(&sm.empty[stage], phase ^ 1, p.wait_ns)) {
            good = 0;
          } else {
            const bool valid = cur.blk >= 0 && cur.blk < p.num_blocks;
            const bool valid2 = BT == 8 && cur.blk2 >= 0 && cur.blk2 < p.num_blocks;
            if (!valid || (BT == 8 && cur.blk2 != -2 && !valid2)) report(p.err, PA_DEV_BAD_BLOCK);
            StageDesc d = cur.d;
            d.use = ((1u << cur.n_tok) - 1u) &
                    (BT == 8 ? (valid ? 0x00ffu : 0u) | (valid2 ? 0xff00u : 0u) : (valid ? 0xffffu : 0u));
            sm.desc[stage] = d;
            constexpr int kPageCopy = BT == 8 ? kTileBytes / 2 : kTileBytes;
            const int copies = (valid ? 1 : 0) + (valid2 ? 1 : 0);
            const bool first = d.flags & kSegStart;
            mbar_arrive_expect_tx(&sm.full[stage], copies * (kPageCopy + 2 * kHkv * 4) +
                                                       (first ? kHq * kD * 2 : 0));
            // test hook: this stage's copies are left out, so its barrier
            // never completes and every wait on it runs out
            const bool fault = p.fault_stage == published && blockIdx.x == 0;
            if (first && !fault)
              bulk_g2s(sm.q[stage], p.q + static_cast<size_t>(d.seq) * kHq * kD, kHq * kD * 2,
                       &sm.full[stage]);
            if (valid && !fault) {
              tma_load_5d(sm.kv[stage], &kv_map, 0, BT == 32 ? (cur.j & 1) * kTile : 0, 0, 0,
                          cur.blk, &sm.full[stage]);
              bulk_g2s(sm.scale[stage][0], p.scales + static_cast<size_t>(cur.blk) * 2 * kHkv,
                       2 * kHkv * 4, &sm.full[stage]);
            }
            if (valid2 && !fault) {
              tma_load_5d(sm.kv[stage] + kPageCopy, &kv_map, 0, 0, 0, 0, cur.blk2, &sm.full[stage]);
              bulk_g2s(sm.scale[stage][1], p.scales + static_cast<size_t>(cur.blk2) * 2 * kHkv,
                       2 * kHkv * 4, &sm.full[stage]);
            }
          }
        }
        ok = __shfl_sync(0xffffffffu, good, e) != 0;
        if (!ok) break;
        issued |= 1u << stage;
        issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
        ++published;
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (lane == 0) {
      if (ok && mbar_wait(&sm.empty[stage], phase ^ 1, p.wait_ns)) {
        sm.desc[stage].flags = kEndOfWork;
        mbar_arrive(&sm.full[stage]);
        // this arrive is now the stage's last phase; the copy before it on
        // the same stage has landed, or the consumers could not have freed it
        issued |= 1u << stage;
        issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
      } else {
        report(p.err, PA_DEV_TIMEOUT);
      }
      // no copy may still be landing in shared memory when the CTA exits
      for (int st = 0; st < kStages; ++st)
        if ((issued >> st) & 1u)
          if (!mbar_wait(&sm.full[st], (issued_parity >> st) & 1u, p.wait_ns))
            report(p.err, PA_DEV_TIMEOUT);
    }
    __syncwarp();
  } else {
    // ===================================================== consumer warps ==
    const int g = lane >> 2, c = lane & 3;
    constexpr int kRows = BT == 8 ? 8 : kTile;                  // token rows of a head in a stage
    constexpr uint32_t kPairTile = kRows * kPairBytes;          // a head pair's K (or V) there
    constexpr uint32_t kHalf = kHkv / 2 * kPairTile;            // V behind K
    constexpr uint32_t kSecond = BT == 8 ? kTileBytes / 2 : 8 * kPairBytes;   // tokens 8..15
    uint32_t qa[8];
    float2 qs = make_float2(0.f, 0.f);
    State st;
    st.reset();
#pragma unroll
    for (int i = 0; i < 8; ++i) qa[i] = 0u;
    int stage = 0;
    uint32_t phase = 0;
    while (true) {
      if (!mbar_wait(&sm.full[stage], phase, p.wait_ns)) {
        report(p.err, PA_DEV_TIMEOUT);
        break;
      }
      const StageDesc d = sm.desc[stage];
      if (d.flags & kEndOfWork) break;
      if (d.flags & kSegStart) {
        const float mine = load_q(smem_u32(sm.q[stage]) + warp * kGqa * kD * 2, g, c, p.qscale, qa);
        qs.x = __shfl_sync(0xffffffffu, mine, 8 * c);       // heads 2c, 2c + 1
        qs.y = __shfl_sync(0xffffffffu, mine, 8 * c + 4);
        st.reset();
      }
      if (d.use) {
        const uint32_t k0 = smem_u32(sm.kv[stage]) + (warp >> 1) * kPairTile;
        const float(&sc)[2][2 * kHkv] = sm.scale[stage];
        float2 sk, sv;
        sk.x = sc[0][warp];
        sv.x = sc[0][kHkv + warp];
        sk.y = sv.y = 0.f;
        if (BT == 8) {
          // a page that was not loaded left what the stage held before
          if (!(d.use & 0x00ffu)) sk.x = sv.x = 0.f;
          if (d.use & 0xff00u) {
            sk.y = sc[1][warp];
            sv.y = sc[1][kHkv + warp];
          }
        }
        attend<BT>(k0, k0 + kSecond, k0 + kHalf, k0 + kHalf + kSecond, 4 * (warp & 1), sk, sv, d.use,
                   qa, qs, lane, st);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.empty[stage]);
      if (d.flags & kSegEnd) {
        // ---- finish this piece of sequence d.seq
        float2 lt = st.l;
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          lt.x += __shfl_xor_sync(0xffffffffu, lt.x, x);
          lt.y += __shfl_xor_sync(0xffffffffu, lt.y, x);
        }
        if (c < kGqa / 2) {
          const int h = warp * kGqa + 2 * c;   // and h + 1
          if (d.slot < 0) {
            // 0: no page of the context is valid
            const float ix = lt.x == 0.f ? 0.f : 1.f / lt.x, iy = lt.y == 0.f ? 0.f : 1.f / lt.y;
            uint32_t *dst = reinterpret_cast<uint32_t *>(
                p.out + (static_cast<size_t>(d.seq) * kHq + h) * kD) + g;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              dst[8 * i] = float2_to_bf16x2(st.o[2 * i].x * ix, st.o[2 * i + 1].x * ix);
              dst[8 * i + kD / 2] = float2_to_bf16x2(st.o[2 * i].y * iy, st.o[2 * i + 1].y * iy);
            }
          } else {
            const size_t at = static_cast<size_t>(d.slot) * kHq + h;
            float2 *dst = reinterpret_cast<float2 *>(p.acc + at * kD) + g;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              dst[8 * i] = make_float2(st.o[2 * i].x, st.o[2 * i + 1].x);
              dst[8 * i + kD / 2] = make_float2(st.o[2 * i].y, st.o[2 * i + 1].y);
            }
            if (g == 0) {
              p.ml[at] = make_float2(st.m.x, lt.x);
              p.ml[at + 1] = make_float2(st.m.y, lt.y);
            }
          }
        }
      }
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
  }
}

// Combines the partials of every sequence cut into several pieces.  Grid
// (num_seqs, 32 / kHeads): a CTA takes kHeads q heads, kShares warps a head, each half warp
// every (2 kShares)-th partial, 4 dims a lane.  The cut follows from the context
// lengths, which are read before the first kernel has ended (it waited for
// everything before it), so that one round of loads is left after it.
template <int kHeads, int kShares>
__global__ void __launch_bounds__(kHeads * kShares * 32)
    decode_q8_merge_kernel(Q8DecodeParams p, int G) {
  pdl_launch_dependents();   // the next kernel may start its own set-up
  constexpr int kMergeThreads = kHeads * kShares * 32;
  __shared__ int sm_sum[2];
  __shared__ float2 sm_ml[kHeads][kShares];
  __shared__ float4 sm_o[kHeads][kShares][kD / 4];
  const int s = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < 2) sm_sum[tid] = 0;
  __syncthreads();
  int before = 0, all = 0;
  for (int i = tid; i < p.num_seqs; i += kMergeThreads) {
    const int nb = tiles_in(clamp_ctx(p, ctx_now(p, i)));
    all += nb;
    if (i < s) before += nb;
  }
  const int mine = tiles_in(clamp_ctx(p, ctx_now(p, s)));
  if ((tid & ~31) < p.num_seqs) {
    before = __reduce_add_sync(0xffffffffu, before);
    all = __reduce_add_sync(0xffffffffu, all);
    if (lane == 0) {
      atomicAdd(&sm_sum[0], before);
      atomicAdd(&sm_sum[1], all);
    }
  }
  __syncthreads();
  const int B = sm_sum[0], E = B + mine;
  const int C = max((sm_sum[1] + G - 1) / G, 1);
  const int k0 = B / C, np = mine > 0 ? (E - 1) / C - k0 + 1 : 0;   // the runs it lies in
  // (one CTA always waits, so that this grid ends after the first kernel)
  if (np <= 1 && (blockIdx.x != 0 || blockIdx.y != 0)) return;
  pdl_wait_primary();
  if (np <= 1) return;
  const int h = warp % kHeads, share = warp / kHeads, half = lane >> 4, d4 = lane & 15;
  const size_t row = static_cast<size_t>(blockIdx.y) * kHeads + h;
  float m = neg_inf(), l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto fold = [&](float m2, float l2, float4 o2) {
    const float mn = fmaxf(m, m2);
    const float ref = mn == neg_inf() ? 0.f : mn;
    const float so = fast_exp2(m - ref), sn = fast_exp2(m2 - ref);
    l = fmaf(l, so, l2 * sn);
    o = make_float4(fmaf(o.x, so, o2.x * sn), fmaf(o.y, so, o2.y * sn), fmaf(o.z, so, o2.z * sn),
                    fmaf(o.w, so, o2.w * sn));
    m = mn;
  };
  // loads are issued kBatch partials at a time before any of them is folded
  constexpr int kBatch = 6;
  for (int i0 = 2 * share + half; i0 < np; i0 += 2 * kShares * kBatch) {
    float2 mk[kBatch];
    float4 a[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int i = i0 + b * 2 * kShares;
      mk[b] = make_float2(neg_inf(), 0.f);
      a[b] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < np) {
        const size_t at = static_cast<size_t>(k0 + s + i) * kHq + row;
        mk[b] = p.ml[at];
        a[b] = reinterpret_cast<const float4 *>(p.acc + at * kD)[d4];
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) fold(mk[b].x, mk[b].y, a[b]);
  }
  // the two halves of the warp, then the shares
  __syncwarp();
  auto other = [](float x) { return __shfl_xor_sync(0xffffffffu, x, 16); };
  {
    const float m2 = other(m), l2 = other(l);
    const float4 o2 = make_float4(other(o.x), other(o.y), other(o.z), other(o.w));
    fold(m2, l2, o2);
  }
  if (kShares > 1) {
    if (lane == 0) sm_ml[h][share] = make_float2(m, l);
    if (half == 0) sm_o[h][share][d4] = o;
    __syncthreads();
    if (share != 0) return;
#pragma unroll
    for (int w = 1; w < kShares; ++w) fold(sm_ml[h][w].x, sm_ml[h][w].y, sm_o[h][w][d4]);
  }
  if (half == 0) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    reinterpret_cast<uint2 *>(p.out + (static_cast<size_t>(s) * kHq + row) * kD)[d4] =
        make_uint2(float2_to_bf16x2(o.x * inv, o.y * inv), float2_to_bf16x2(o.z * inv, o.w * inv));
  }
}

struct WsLayout {
  size_t acc_off, total;
};

constexpr size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

long long slots_for(int num_seqs, int grid) { return static_cast<long long>(grid) + num_seqs; }

// Tensor map over the pool: dims (two heads' d 128, token bt, head pair 4, K|V
// 2, block), the token dimension before the pairs although its stride is the
// larger one, so that a copy writes each pair's token rows together; box
// (128, 8 or 16, 4, 2, 1), 128-byte swizzle.
int make_q8_tile_map(CUtensorMap *map, const void *kv_cache, int num_blocks, int bt) {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult qr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &qr) != cudaSuccess ||
        qr != cudaDriverEntryPointSuccess)
      return PA_ERR_CUDA;
    fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }
  const cuuint64_t half = static_cast<cuuint64_t>(bt) * kQ8TokBytes;
  const cuuint64_t dims[5] = {kPairBytes, static_cast<cuuint64_t>(bt), kHkv / 2, 2,
                              static_cast<cuuint64_t>(num_blocks)};
  const cuuint64_t strides[4] = {kQ8TokBytes, kPairBytes, half, 2 * half};
  const cuuint32_t box[5] = {kPairBytes, bt == 8 ? 8u : 16u, kHkv / 2, 2, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void *>(kv_cache), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PA_OK : PA_ERR_CUDA;
}

WsLayout ws_layout(long long slots) {
  WsLayout w;
  w.acc_off = align256(sizeof(float2) * kHq * static_cast<size_t>(slots));
  w.total = w.acc_off + align256(sizeof(float) * kHq * kD * static_cast<size_t>(slots));
  return w;
}

long long tiles_of(int max_blocks, int bt) {
  return (static_cast<long long>(max_blocks) * bt + kTile - 1) / kTile;
}

int grid_for(const DeviceInfo &di, int num_seqs, long long tiles) {
  long long g = static_cast<long long>(di.sm_count) * kCtasPerSm;
  g = min(g, static_cast<long long>(num_seqs) * tiles);
  g = min(g, static_cast<long long>(kMaxGrid));
  return static_cast<int>(max(g, 1LL));
}

template <int BT>
int decode_q8_impl(uint16_t *out, const uint16_t *q, const uint8_t *kv_cache,
                   const float *kv_scales, int num_blocks, const int32_t *block_table,
                   int n_layers, int max_blocks_per_seq, const int32_t *context_lens, int num_seqs,
                   int layer, float scale, void *workspace, size_t workspace_bytes, int32_t *err,
                   void *stream) {
  if (num_seqs < 0 || num_seqs > kMaxSeqs || num_blocks <= 0 || n_layers <= 0 ||
      max_blocks_per_seq <= 0)
    return PA_ERR_ARG;
  const long long tiles = tiles_of(max_blocks_per_seq, BT);
  if (static_cast<long long>(max_blocks_per_seq) * BT > INT_MAX ||
      static_cast<long long>(num_seqs) * tiles > INT_MAX)
    return PA_ERR_ARG;
  if (layer < 0 || layer >= n_layers) return PA_ERR_LAYER;
  if (num_seqs == 0) return PA_OK;
  if (!out || !q || !kv_cache || !kv_scales || !block_table || !context_lens || !err)
    return PA_ERR_NULL;
  if (!workspace) return PA_ERR_WORKSPACE;
  if (!aligned16(out) || !aligned16(q) || !aligned16(kv_cache) || !aligned16(kv_scales) ||
      !aligned16(workspace))
    return PA_ERR_ALIGN;
  DeviceInfo di;
  int rc = current_device(&di);
  if (rc != PA_OK) return rc;
  const int G = grid_for(di, num_seqs, tiles);
  const long long slots = slots_for(num_seqs, G);
  const WsLayout w = ws_layout(slots);
  if (w.total > workspace_bytes) return PA_ERR_WORKSPACE;
  // + room to align the base to 1 KiB
  const size_t smem = sizeof(Smem) + sizeof(int) * static_cast<size_t>(num_seqs) + 1024;
  if (cudaFuncSetAttribute(decode_q8_kernel<BT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(sizeof(Smem) + sizeof(int) * kMaxSeqs + 1024)) !=
      cudaSuccess)
    return PA_ERR_CUDA;
  alignas(64) CUtensorMap map;
  rc = make_q8_tile_map(&map, kv_cache, num_blocks, BT);
  if (rc != PA_OK) return rc;

  Q8DecodeParams prm;
  unsigned char *ws = static_cast<unsigned char *>(workspace);
  prm.out = reinterpret_cast<__nv_bfloat16 *>(out);
  prm.q = q;
  prm.kv = kv_cache;
  prm.scales = kv_scales;
  prm.block_table = block_table;
  prm.context_lens = context_lens;
  prm.ml = reinterpret_cast<float2 *>(ws);
  prm.acc = reinterpret_cast<float *>(ws + w.acc_off);
  prm.err = err;
  prm.num_blocks = num_blocks;
  prm.n_layers = n_layers;
  prm.max_blocks = max_blocks_per_seq;
  prm.num_seqs = num_seqs;
  prm.layer = layer;
  prm.cap_tokens = max_blocks_per_seq * BT;
  prm.qscale = scale * kLog2e;
  decode_fault(&prm.fault_stage, &prm.wait_ns);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  prm.direct = tiles <= kDirectTiles ? 1 : 0;
  if (prm.direct)
    return launch_pdl(decode_q8_kernel<BT>, dim3(num_seqs), dim3(kThreads), smem, st, map, prm) ==
                   cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
  if (launch_pdl(decode_q8_kernel<BT>, dim3(G), dim3(kThreads), smem, st, map, prm) != cudaSuccess)
    return PA_ERR_CUDA;
  // few sequences have many partials each
  const cudaError_t e =
      num_seqs >= 64
          ? launch_pdl(decode_q8_merge_kernel<16, 2>, dim3(num_seqs, 2), dim3(1024), 0, st, prm, G)
      : num_seqs >= 8
          ? launch_pdl(decode_q8_merge_kernel<4, 4>, dim3(num_seqs, 8), dim3(512), 0, st, prm, G)
          : launch_pdl(decode_q8_merge_kernel<1, 16>, dim3(num_seqs, 32), dim3(512), 0, st, prm, G);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" size_t pa_decode_workspace_size_q8(int num_seqs, int max_blocks_per_seq,
                                              int block_tokens) {
  if (num_seqs <= 0 || max_blocks_per_seq <= 0 ||
      (block_tokens != 8 && block_tokens != 16 && block_tokens != 32))
    return 0;
  DeviceInfo di;
  if (current_device(&di) != PA_OK) di.sm_count = kMaxGrid;   // generous when no device answers
  const int G = grid_for(di, num_seqs, tiles_of(max_blocks_per_seq, block_tokens));
  return ws_layout(slots_for(num_seqs, G)).total;
}

extern "C" int pa_decode_attention_q8(uint16_t *out, const uint16_t *q, const uint8_t *kv_cache,
                                      const float *kv_scales, int num_blocks, int block_tokens,
                                      const int32_t *block_table, int n_layers,
                                      int max_blocks_per_seq, const int32_t *context_lens,
                                      int num_seqs, int layer, float scale, void *workspace,
                                      size_t workspace_bytes, int32_t *err, void *stream) {
  auto *impl = block_tokens == 8    ? decode_q8_impl<8>
               : block_tokens == 16 ? decode_q8_impl<16>
               : block_tokens == 32 ? decode_q8_impl<32>
                                    : nullptr;
  if (!impl) return PA_ERR_ARG;
  return impl(out, q, kv_cache, kv_scales, num_blocks, block_table, n_layers, max_blocks_per_seq,
              context_lens, num_seqs, layer, scale, workspace, workspace_bytes, err, stream);
}
