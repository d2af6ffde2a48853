// pa_decode_q8.cu -- decode attention over the 8-bit cache (pa_q8.cuh).
//
//   out[h] = sum_t softmax_t(scale * q[h] . (sK K_t)) (sV V_t)
//
// decode_q8_kernel: the 16-token tiles of all sequences are laid end to end
// and cut into chunks; a CTA takes its own index first, then chunks from a
// counter in the workspace.  A CTA is 8 warps, one per kv head; a warp reads
// its head's K and V of a tile straight from global memory into the
// registers that the MMAs take them from, several tiles ahead, so there is no
// shared-memory ring and no barrier in the loop.  That works because the
// sums of a dot product may be taken in any order, so the MMAs' inner and
// output dimensions are permuted to what wide loads deliver:
//   S = Q K^T  lane (g, c) (g = lane / 4, c = lane % 4) loads dims 16c..16c+15
//              of tokens g and g + 8 (two 16-byte loads); k-step ks of the
//              m16n8k16 MMAs takes dims 16c + 4 ks + {0, 1} and {2, 3} where
//              the plain order has 2c + {0, 1} and 8 + 2c + {0, 1}.
//   O = P V    lane (g, c) loads dims 8g..8g+7 of tokens 2c, 2c+1, 2c+8, 2c+9
//              (four 8-byte loads); output column g of MMA nt is dim 8g + nt,
//              so a lane ends with the 16 consecutive dims 16c..16c+15 of its
//              q head.
// e4m3 becomes f16 exactly; q is scaled by a power of two per head to f16
// (exact for values down to 2^-29 of the head's largest).  P <= 1 enters the
// MMA in f16: half a step is 2^-12 of a weight (2^-25 absolute below 2^-14),
// an eighth of the output's own bf16 rounding; m and l stay fp32.  K's scale
// multiplies the scores; V's multiplies the tile's product when it is added
// to the running output, in the FMA that rescales it anyway.
#include <climits>
#include <cuda_fp16.h>

#include "pa_decode_tile.cuh"
#include "pa_host.h"
#include "pa_q8.cuh"

namespace pa {
namespace {

constexpr int kWarps = kHkv;               // one per kv head
constexpr int kThreads = kWarps * 32;
constexpr int kCtasPerSm = 2;
constexpr int kMaxSeqs = 2048;             // tile prefix kept in shared memory
constexpr int kMaxGrid = 512;
constexpr int kChunksPerCta = 4;           // average chunks a CTA takes
constexpr int kTile = 16;                  // tokens
constexpr int kAhead = 2;                  // tiles in flight per warp beside the one worked on
constexpr float kLog2e = 1.4426950408889634f;

struct Q8DecodeParams {
  __nv_bfloat16 *out;
  const uint16_t *q;
  const unsigned char *kv;
  const float *scales;
  const int32_t *block_table;
  const int32_t *context_lens;
  int *chunk_counter;  // zero between calls; reset by the merge kernel
  int2 *meta;          // [num_seqs] (first partial slot, number of partials)
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
  long long n_slots;
};

struct Smem {
  int prefix[kMaxSeqs + 1];   // tiles of sequences 0..s-1
  int warp_sum[kWarps];
  int next;
};

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a2, uint32_t b0,
                                              uint32_t b1) {
  // rows 8..15 of A are zero
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(0u), "r"(a2), "r"(0u), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_f16_1688(float (&d)[4], uint32_t a0, uint32_t b0) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(0u), "r"(b0));
}

// Loads of pool data: once used, not kept in L1.  (volatile: they stay where
// they are written, ahead of the tile that is worked on.)
__device__ __forceinline__ uint4 load16(const unsigned char *p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 load8(const unsigned char *p) {
  uint2 v;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
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

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// One tile of one kv head as loaded.
struct TileRegs {
  uint4 k[2];          // tokens g, g + 8: dims 16c..16c+15
  uint2 v[4];          // tokens 2c, 2c+1, 2c+8, 2c+9: dims 8g..8g+7
  float sk[2], sv[2];  // scales of the tile's first and second 8 tokens
  int n_valid;         // tokens to use: 0..16
  uint32_t use;        // 8-token pages: bit t = token t is used
};

// A warp's running softmax of one kv head: q head g (rows g < 4 are real),
// dims 16c + nt (o[nt].x) and 16c + 8 + nt (o[nt].y).
struct State {
  float2 o[8];
  float m, l;
  __device__ __forceinline__ void reset() {
    m = neg_inf();
    l = 0.f;
#pragma unroll
    for (int t = 0; t < 8; ++t) o[t] = make_float2(0.f, 0.f);
  }
};

// q head g of the group in f16, scaled by a power of two to [2^12, 2^13);
// returns the row's score factor: qscale / that power.
__device__ __forceinline__ float load_q(const uint16_t *q_token, int head0, int g, int c,
                                        float qscale, uint32_t (&qa)[8]) {
  uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
  if (g < kGqa) {
    const uint4 *row = reinterpret_cast<const uint4 *>(q_token + (head0 + g) * kD + 16 * c);
    w0 = row[0];
    w1 = row[1];
  }
  const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = q8_top(w[i], top);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const int f = min(266 - static_cast<int>(top >> 7), 253);   // exponent field of the factor
  const float up = __int_as_float(f << 23), down = __int_as_float((254 - f) << 23);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 x = bf16x2_to_float2(w[i]);
    qa[i] = f16x2(x.x * up, x.y * up);
  }
  return qscale * down;
}

// Folds a tile into the state.  qa[2 ks], qa[2 ks + 1]: the A operand of k-step ks.
template <int BT>
__device__ __forceinline__ void attend(TileRegs &t, const uint32_t (&qa)[8], float qs, int c,
                                       State &st) {
  const bool part = BT == 8 ? t.use != 0xffffu : t.n_valid < kTile;
  bool u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int tok = 2 * c + (i & 1) + 8 * (i >> 1);
    u[i] = BT == 8 ? ((t.use >> tok) & 1u) != 0 : tok < t.n_valid;
  }
  if (part) {
    // unused tokens may hold anything, NaN included: they meet P = 0
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!u[i]) t.v[i] = make_uint2(0, 0);
  }
  // ---- S = Q K^T for tokens 0..7 (s0) and 8..15 (s1)
  float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
  const uint32_t k0[4] = {t.k[0].x, t.k[0].y, t.k[0].z, t.k[0].w};
  const uint32_t k1[4] = {t.k[1].x, t.k[1].y, t.k[1].z, t.k[1].w};
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) {
    mma_f16_16816(s0, qa[2 * ks], qa[2 * ks + 1], e4m3x2_to_f16x2(k0[ks]),
                  e4m3x2_to_f16x2(k0[ks] >> 16));
    mma_f16_16816(s1, qa[2 * ks], qa[2 * ks + 1], e4m3x2_to_f16x2(k1[ks]),
                  e4m3x2_to_f16x2(k1[ks] >> 16));
  }
  // ---- online softmax of row g over tokens 2c, 2c+1, 2c+8, 2c+9
  const float f0 = qs * t.sk[0], f1 = BT == 8 ? qs * t.sk[1] : f0;
  const float x0 = u[0] ? s0[0] * f0 : neg_inf();
  const float x1 = u[1] ? s0[1] * f0 : neg_inf();
  const float x2 = u[2] ? s1[0] * f1 : neg_inf();
  const float x3 = u[3] ? s1[1] * f1 : neg_inf();
  float mx = fmaxf(fmaxf(x0, x1), fmaxf(x2, x3));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
  const float m_new = fmaxf(st.m, mx);
  const float base = m_new == neg_inf() ? 0.f : m_new;   // nothing seen yet
  const float alpha = fast_exp2(st.m - base);
  const float p0 = fast_exp2(x0 - base), p1 = fast_exp2(x1 - base);
  const float p2 = fast_exp2(x2 - base), p3 = fast_exp2(x3 - base);
  st.l = fmaf(st.l, alpha, (p0 + p1) + (p2 + p3));
  st.m = m_new;
  const uint32_t pa = f16x2(p0, p1), pc = f16x2(p2, p3);
  // ---- O = alpha O + sV P V, 8 dims a step
  const float2 al = make_float2(alpha, alpha);
  const float2 sv0 = make_float2(t.sv[0], t.sv[0]), sv1 = make_float2(t.sv[1], t.sv[1]);
#pragma unroll
  for (int w = 0; w < 2; ++w) {   // dims 8g + 4w .. 8g + 4w + 3
    const uint32_t a = w ? t.v[0].y : t.v[0].x, b = w ? t.v[1].y : t.v[1].x;
    const uint32_t d = w ? t.v[2].y : t.v[2].x, e = w ? t.v[3].y : t.v[3].x;
    const uint32_t lo[2] = {prmt(a, b, 0x5140), prmt(a, b, 0x7362)};
    const uint32_t hi[2] = {prmt(d, e, 0x5140), prmt(d, e, 0x7362)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int nt = 4 * w + i;
      const uint32_t b0 = e4m3x2_to_f16x2(lo[i >> 1] >> (16 * (i & 1)));
      const uint32_t b1 = e4m3x2_to_f16x2(hi[i >> 1] >> (16 * (i & 1)));
      float r[4] = {0.f, 0.f, 0.f, 0.f};
      if (BT == 8) {
        // the two pages' products apart: their scales differ
        float r2[4] = {0.f, 0.f, 0.f, 0.f};
        mma_f16_1688(r, pa, b0);
        mma_f16_1688(r2, pc, b1);
        st.o[nt] = fma2(make_float2(r2[0], r2[1]), sv1,
                        fma2(make_float2(r[0], r[1]), sv0, mul2(st.o[nt], al)));
      } else {
        mma_f16_16816(r, pa, pc, b0, b1);
        st.o[nt] = fma2(make_float2(r[0], r[1]), sv0, mul2(st.o[nt], al));
      }
    }
  }
}

__device__ __forceinline__ int clamped_ctx(const Q8DecodeParams &p, int s) {
  return min(max(p.context_lens[s], 0), p.cap_tokens);
}

// Chunk length in tiles: about kChunksPerCta chunks per CTA, at least 8
// tiles (or one CTA's fair share when that is smaller).
__device__ __forceinline__ int chunk_tiles(int total, int g) {
  const int fair = (total + g - 1) / g;
  const int c = (total + kChunksPerCta * g - 1) / (kChunksPerCta * g);
  return max(1, max(min(8, fair), c));
}

// First sequence s with prefix[s+1] > b or prefix[s] >= b (one that reaches
// past tile b, or an empty one starting at b or later).
__device__ __forceinline__ int first_seq_at(const int *prefix, int n, int b) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid + 1] > b || prefix[mid] >= b) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// The warp's tile loads.  Lane i holds the page ids of tile j0 + i of the
// piece (two for 8-token pages) and the scales of its head there.
struct TileIds {
  int blk[2];
  float sk[2], sv[2];
};

template <int BT>
__device__ __forceinline__ TileIds load_ids(const Q8DecodeParams &p, const int32_t *row, int j,
                                            bool have, int n_tok, int head) {
  TileIds t;
#pragma unroll
  for (int i = 0; i < (BT == 8 ? 2 : 1); ++i) {
    t.blk[i] = -1;
    t.sk[i] = t.sv[i] = 0.f;
    if (have && (i == 0 || n_tok > 8)) {
      const int blk = row[BT == 32 ? j >> 1 : BT == 8 ? 2 * j + i : j];
      if (blk >= 0 && blk < p.num_blocks) {
        t.blk[i] = blk;
        const float *s = p.scales + static_cast<size_t>(blk) * 2 * kHkv + head;
        t.sk[i] = s[0];
        t.sv[i] = s[kHkv];
      } else {
        report(p.err, PA_DEV_BAD_BLOCK);
      }
    }
  }
  return t;
}

// Starts the loads of tile j (lane e of the ids holds it).  A page that is
// missing is read as page 0 and not used.
template <int BT>
__device__ __forceinline__ void load_tile(const Q8DecodeParams &p, const TileIds &ids, int e, int j,
                                          int n_tok, int head, int g, int c, TileRegs &t) {
  constexpr size_t kPage = static_cast<size_t>(BT) * 2 * kQ8TokBytes;
  constexpr size_t kHalf = static_cast<size_t>(BT) * kQ8TokBytes;
  const int blk0 = __shfl_sync(0xffffffffu, ids.blk[0], e);
  t.sk[0] = __shfl_sync(0xffffffffu, ids.sk[0], e);
  t.sv[0] = __shfl_sync(0xffffffffu, ids.sv[0], e);
  const unsigned char *p0 = p.kv + static_cast<size_t>(max(blk0, 0)) * kPage + head * kQ8HeadBytes;
  if (BT == 32) p0 += (j & 1) * (kTile * kQ8TokBytes);
  const unsigned char *p1 = p0 + 8 * kQ8TokBytes;   // tokens 8..15
  t.n_valid = blk0 >= 0 ? n_tok : 0;
  t.use = 0;
  if (BT == 8) {
    const int blk1 = __shfl_sync(0xffffffffu, ids.blk[1], e);
    t.sk[1] = __shfl_sync(0xffffffffu, ids.sk[1], e);
    t.sv[1] = __shfl_sync(0xffffffffu, ids.sv[1], e);
    p1 = p.kv + static_cast<size_t>(max(blk1, 0)) * kPage + head * kQ8HeadBytes;
    t.use = ((1u << n_tok) - 1u) & ((blk0 >= 0 ? 0x00ffu : 0u) | (blk1 >= 0 ? 0xff00u : 0u));
  } else {
    t.sk[1] = t.sk[0];
    t.sv[1] = t.sv[0];
  }
  t.k[0] = load16(p0 + g * kQ8TokBytes + 16 * c);
  t.k[1] = load16(p1 + g * kQ8TokBytes + 16 * c);
  const unsigned char *v0 = p0 + kHalf + 2 * c * kQ8TokBytes + 8 * g;
  const unsigned char *v1 = p1 + kHalf + 2 * c * kQ8TokBytes + 8 * g;
  t.v[0] = load8(v0);
  t.v[1] = load8(v0 + kQ8TokBytes);
  t.v[2] = load8(v1);
  t.v[3] = load8(v1 + kQ8TokBytes);
}

template <int BT>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) decode_q8_kernel(Q8DecodeParams p) {
  __shared__ Smem sm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  const int G = gridDim.x;
  pdl_launch_dependents();   // the merge kernel may take its place in the queue
  pdl_wait_primary();        // everything read below may come from the previous kernel

  // ---- tile prefix over the sequences
  int carry = 0;
  for (int base = 0; base < p.num_seqs; base += kThreads) {
    const int i = base + tid;
    int nb = 0;
    if (i < p.num_seqs) {
      const int t = p.context_lens[i];
      if (blockIdx.x == 0 && (t < 0 || t > p.cap_tokens)) report(p.err, PA_DEV_CTX_RANGE);
      nb = (clamped_ctx(p, i) + kTile - 1) / kTile;
    }
    int incl = nb;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) sm.warp_sum[warp] = incl;
    __syncthreads();
    int before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const int v = sm.warp_sum[w];
      if (w < warp) before += v;
      sum += v;
    }
    if (i < p.num_seqs) sm.prefix[i + 1] = carry + before + incl;
    carry += sum;
    __syncthreads();
  }
  if (tid == 0) sm.prefix[0] = 0;
  __syncthreads();
  const int total = carry;
  const int C = chunk_tiles(total, G);
  const int n_chunks = max(1, (total + C - 1) / C);

  int k = blockIdx.x;
  while (k < n_chunks) {
    if (tid == 0) sm.next = G + atomicAdd(p.chunk_counter, 1);
    const int b0 = k * C, b1 = min(total, b0 + C);
    const bool last_chunk = k == n_chunks - 1;
    for (int s = first_seq_at(sm.prefix, p.num_seqs, b0); s < p.num_seqs; ++s) {
      const int B = sm.prefix[s];
      if (B >= b1 && !last_chunk) break;
      const int nb = sm.prefix[s + 1] - B;
      if (nb == 0) {
        // empty context: the chunk holding its start owns it; output zero
        uint4 *o = reinterpret_cast<uint4 *>(p.out + static_cast<size_t>(s) * kHq * kD);
        for (int e = tid; e < kHq * kD * 2 / 16; e += kThreads) o[e] = make_uint4(0, 0, 0, 0);
        if (tid == 0) p.meta[s] = make_int2(0, 0);
        continue;
      }
      if (B >= b1) break;   // last chunk: only empty sequences may follow
      const int tail = clamped_ctx(p, s) - (nb - 1) * kTile;
      const int jb = max(b0, B) - B, je = min(b1, B + nb) - B;
      const int k_first = B / C;
      const int n_parts = (B + nb - 1) / C - k_first + 1;
      const int slot = k + s;
      if (k == k_first && tid == 0) p.meta[s] = make_int2(k_first + s, n_parts);
      const int32_t *row =
          p.block_table + (static_cast<size_t>(s) * p.n_layers + p.layer) * p.max_blocks;
      uint32_t qa[8];
      State st;
      st.reset();
      const float qs = load_q(p.q + static_cast<size_t>(s) * kHq * kD, warp * kGqa, g, c, p.qscale, qa);
      for (int j0 = jb; j0 < je; j0 += 32) {
        const int cnt = min(32, je - j0);
        auto tok = [&](int j) { return j == nb - 1 ? tail : kTile; };
        const TileIds ids = load_ids<BT>(p, row, j0 + lane, lane < cnt, tok(j0 + lane), warp);
        TileRegs t[kAhead + 1];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
          if (i < cnt) load_tile<BT>(p, ids, i, j0 + i, tok(j0 + i), warp, g, c, t[i]);
        for (int e0 = 0; e0 < cnt; e0 += kAhead + 1) {
#pragma unroll
          for (int i = 0; i <= kAhead; ++i) {
            const int e = e0 + i;
            if (e < cnt) {
              const int f = e + kAhead;
              if (f < cnt)
                load_tile<BT>(p, ids, f, j0 + f, tok(j0 + f), warp, g, c, t[(i + kAhead) % (kAhead + 1)]);
              attend<BT>(t[i], qa, qs, c, st);
            }
          }
        }
      }
      // ---- finish this piece of sequence s
      float lt = st.l;
      lt += __shfl_xor_sync(0xffffffffu, lt, 1);
      lt += __shfl_xor_sync(0xffffffffu, lt, 2);
      if (g < kGqa) {
        const int h = warp * kGqa + g;
        if (n_parts == 1) {
          const float inv = lt == 0.f ? 0.f : 1.f / lt;   // 0: no page of the context is valid
          uint32_t w[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            w[i] = float2_to_bf16x2(st.o[2 * i].x * inv, st.o[2 * i + 1].x * inv);
            w[4 + i] = float2_to_bf16x2(st.o[2 * i].y * inv, st.o[2 * i + 1].y * inv);
          }
          uint4 *dst = reinterpret_cast<uint4 *>(p.out + (static_cast<size_t>(s) * kHq + h) * kD + 16 * c);
          dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
          dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
          float4 *dst = reinterpret_cast<float4 *>(p.acc + (static_cast<size_t>(slot) * kHq + h) * kD + 16 * c);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            dst[i] = make_float4(st.o[4 * i].x, st.o[4 * i + 1].x, st.o[4 * i + 2].x, st.o[4 * i + 3].x);
            dst[2 + i] = make_float4(st.o[4 * i].y, st.o[4 * i + 1].y, st.o[4 * i + 2].y, st.o[4 * i + 3].y);
          }
          if (c == 0) p.ml[static_cast<size_t>(slot) * kHq + h] = make_float2(st.m, lt);
        }
      }
    }
    __syncthreads();
    k = sm.next;
    if (k < G) k = n_chunks;   // a counter that was never zeroed
    __syncthreads();
  }
}

// Combines the partials of every sequence cut into several pieces, and
// returns the chunk counter to zero for the next call.  Grid (num_seqs, 32 q
// heads), kShares warps = interleaved shares of the partials, lane = 2 dims.
template <int kShares>
__global__ void __launch_bounds__(kShares * 32) decode_q8_merge_kernel(Q8DecodeParams p) {
  pdl_launch_dependents();   // the next kernel may start its own set-up
  pdl_wait_primary();
  __shared__ float sm_m[kShares], sm_l[kShares];
  __shared__ float2 sm_o[kShares][32];
  const int s = blockIdx.x, h = blockIdx.y;
  const int lane = threadIdx.x & 31, share = threadIdx.x >> 5;
  if (s == 0 && h == 0 && threadIdx.x == 0) *p.chunk_counter = 0;   // the first kernel is done
  const int2 mt = p.meta[s];
  const int np = mt.y;
  if (np <= 1) return;
  // meta left by another call may name slots beyond this workspace
  if (mt.x < 0 || static_cast<long long>(mt.x) + np > p.n_slots) return;
  const size_t slot0 = static_cast<size_t>(mt.x);
  const float2 *acc = reinterpret_cast<const float2 *>(p.acc);
  float m = neg_inf(), l = 0.f;
  float2 o = make_float2(0.f, 0.f);
  // loads are issued kBatch partials at a time before any of them is folded
  constexpr int kBatch = 8;
  for (int k0 = share; k0 < np; k0 += kShares * kBatch) {
    float2 mk[kBatch], a[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int k = k0 + b * kShares;
      mk[b] = make_float2(neg_inf(), 0.f);
      a[b] = make_float2(0.f, 0.f);
      if (k < np) {
        mk[b] = p.ml[(slot0 + k) * kHq + h];
        a[b] = acc[((slot0 + k) * kHq + h) * (kD / 2) + lane];
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (mk[b].x == neg_inf() && mk[b].y == 0.f) continue;
      const float mn = fmaxf(m, mk[b].x);
      const float ref = mn == neg_inf() ? 0.f : mn;
      const float so = fast_exp2(m - ref), sn = fast_exp2(mk[b].x - ref);
      l = fmaf(l, so, mk[b].y * sn);
      o.x = fmaf(o.x, so, a[b].x * sn);
      o.y = fmaf(o.y, so, a[b].y * sn);
      m = mn;
    }
  }
  if (lane == 0) {
    sm_m[share] = m;
    sm_l[share] = l;
  }
  sm_o[share][lane] = o;
  __syncthreads();
  if (share == 0) {
    float M = neg_inf();
#pragma unroll
    for (int w = 0; w < kShares; ++w) M = fmaxf(M, sm_m[w]);
    const float ref = M == neg_inf() ? 0.f : M;
    float L = 0.f;
    float2 t = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kShares; ++w) {
      const float sc = fast_exp2(sm_m[w] - ref);   // empty shares carry m = -inf: weight 0
      L = fmaf(sm_l[w], sc, L);
      t.x = fmaf(sm_o[w][lane].x, sc, t.x);
      t.y = fmaf(sm_o[w][lane].y, sc, t.y);
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    uint32_t *dst = reinterpret_cast<uint32_t *>(p.out + (static_cast<size_t>(s) * kHq + h) * kD);
    dst[lane] = float2_to_bf16x2(t.x * inv, t.y * inv);
  }
}

struct WsLayout {
  size_t meta_off, ml_off, acc_off, total;
};

constexpr size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

long long slots_for(int num_seqs, int grid) {
  return static_cast<long long>(kChunksPerCta) * grid + 2 + num_seqs;
}

WsLayout ws_layout(int num_seqs, long long slots) {
  WsLayout w;
  w.meta_off = 256;   // the chunk counter lies before it
  w.ml_off = w.meta_off + align256(sizeof(int2) * static_cast<size_t>(num_seqs));
  w.acc_off = w.ml_off + align256(sizeof(float2) * kHq * static_cast<size_t>(slots));
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
  const int rc = current_device(&di);
  if (rc != PA_OK) return rc;
  const int G = grid_for(di, num_seqs, tiles);
  const long long slots = slots_for(num_seqs, G);
  const WsLayout w = ws_layout(num_seqs, slots);
  if (w.total > workspace_bytes) return PA_ERR_WORKSPACE;

  Q8DecodeParams prm;
  unsigned char *ws = static_cast<unsigned char *>(workspace);
  prm.out = reinterpret_cast<__nv_bfloat16 *>(out);
  prm.q = q;
  prm.kv = kv_cache;
  prm.scales = kv_scales;
  prm.block_table = block_table;
  prm.context_lens = context_lens;
  prm.chunk_counter = reinterpret_cast<int *>(ws);
  prm.meta = reinterpret_cast<int2 *>(ws + w.meta_off);
  prm.ml = reinterpret_cast<float2 *>(ws + w.ml_off);
  prm.acc = reinterpret_cast<float *>(ws + w.acc_off);
  prm.err = err;
  prm.num_blocks = num_blocks;
  prm.n_layers = n_layers;
  prm.max_blocks = max_blocks_per_seq;
  prm.num_seqs = num_seqs;
  prm.layer = layer;
  prm.cap_tokens = max_blocks_per_seq * BT;
  prm.qscale = scale * kLog2e;
  prm.n_slots = slots;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (launch_pdl(decode_q8_kernel<BT>, dim3(G), dim3(kThreads), 0, st, prm) != cudaSuccess)
    return PA_ERR_CUDA;
  const cudaError_t e =
      num_seqs >= 8
          ? launch_pdl(decode_q8_merge_kernel<4>, dim3(num_seqs, kHq), dim3(4 * 32), 0, st, prm)
          : launch_pdl(decode_q8_merge_kernel<16>, dim3(num_seqs, kHq), dim3(16 * 32), 0, st, prm);
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
  return ws_layout(num_seqs, slots_for(num_seqs, G)).total;
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
