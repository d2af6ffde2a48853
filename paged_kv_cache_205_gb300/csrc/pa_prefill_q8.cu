// pa_prefill_q8.cu -- causal attention of a prompt chunk over its sequence's
// pages in the 8-bit cache (pa_q8.cuh), on the sm_103a tensor cores.
//
// For row i of sequence s (position context_lens[s] + i):
//   out = sum_t softmax_t(scale * q . (sK K_t)) (sV V_t), t = 0 .. position.
// The pipeline is the bf16 prefill kernel's (pa_prefill.cu: persistent CTAs
// over (64-token query tile, kv head) items, two halves of 32 tokens x 4 q
// heads, 128-key chunks, S and O in TMEM, one MMA warp and one softmax
// warpgroup a half) with a converter warpgroup between the copies and the
// MMAs: the TMA brings a chunk's bytes (16 KiB, half of the bf16 cache's) into
// a small ring, and four warps widen them into f16 operand tiles, one
// conversion for two values.  (Widened to bf16 with the scales multiplied in,
// six instructions for two values, 8 x 2048 tokens took 259 us and 32 x 512
// after 4096 860 us.)  The pages' scales come in in two steps.  Within a chunk a
// page's values are multiplied by its scale over the chunk's largest, a power
// of two; what is left is one scale a chunk for K (sK) and one for V (sV), and
// the softmax is
//   y = s * (f sK) + log2 sV - M     (one FMA, as for the bf16 cache)
//   P = 2^y,  O = sum P V16,  l = sum P / sV
// with f the row's score factor and M a reference 2^7 below the row's largest
// s f sK + log2 sV, which moves when a chunk exceeds it by more than 2^15: M
// follows the weights times the values' scale, so that P fits f16 (<= 2^15)
// however far the scales lie apart.  f16 rounds a P by half a step, 2^-12 of it or
// 2^-25 absolute below 2^-14, which is 2^-32 of the row's largest P.  A chunk
// whose V scales lie further than 2^7 apart keeps V's bytes as they are and takes
// log2 sV page by page, so that a heavy key in a page of small scale does not lift
// the reference by the others' scale; rows whose scores may pass 2^22, where the
// FMA's unrounded product and the rounded M differ by whole units, take the same
// way.  (K's scales may lie any distance apart: f16
// takes a factor down to 2^-15 without rounding, and what is lost below weighs
// 2^-33 of the largest key's score.)
// The converter also turns q into f16, a row scaled by a power of two (f undoes
// it), exact for values down to 2^-29 of the row's largest.
//
// What bounds it: the instructions issued (the issue slots are 55% busy, with the
// conversion or, in the bf16 kernel, without it).  So the work is laid out to
// issue little: one thread, the producer's lane 0, works an item out and hands it
// on with q (each softmax and MMA warp for itself: 229 / 765 us), and the
// converter's loop skips the multiplication where a page's factor is 1 and the
// masks in chunks that need none, and stays rolled (unrolled it runs in bursts
// against the softmax warps: 240 / 790 us).  8 x 2048 tokens 218 us, 631 TFLOP/s
// (the bf16 kernel over the same values 186), 32 x 512 after 4096 742 us, 787
// TFLOP/s (629).  Tried and slower: K's bytes as the tensor core's own e4m3 operand
// against q in two e4m3 parts, which halves the converter's work but leaves the
// pages' K scales to the softmax, whose registers they outgrow (267 / 815 us).
#include "pa_prefill_shared.cuh"
#include "pa_q8.cuh"
#include <cuda_fp16.h>

namespace pa {
namespace {

constexpr int kSortQ = 2048;                  // tiles ordered by weight; beyond, by index
constexpr int kRaw = 3;                       // chunks of bytes in flight
constexpr int kWide = 3;                      // widened chunks
constexpr int kConvWarp = 12;                 // first of 4 converter warps
constexpr int kConvThreads = 128;
constexpr int kQThreads = 16 * 32;
// A score factor's floor: a masked score (-inf) times it stays -inf, and a score
// of at most 2^28 times it is as good as 0.
constexpr float kTiny = 1.2e-38f;
constexpr float kLargeFactor = 0.015625f;     // 2^-6
constexpr uint32_t kOnes = 0x3c003c00u;       // two f16 1.0
// V scales below 2^-94 (exponent field 33) leave the rest to V's f16 values, so
// that l = sum P / sV stays in fp32's range (2^15 2^94 for each of 2^18 keys).
constexpr int kLeastV = 33;
// Register budget: 512 threads x 128 at launch; the softmax warpgroups take
// kQRegsSoft, the producer/MMA warpgroup and the converters give up to theirs.
constexpr int kQRegsSoft = 192;
constexpr int kQRegsMma = 72;
constexpr int kQRegsConv = 56;
static_assert(128 * (2 * kQRegsSoft + kQRegsMma + kQRegsConv) <= kQThreads * 128,
              "register split above the launch budget");

// What the producer tells the converter about a chunk.
struct __align__(16) RawChunk {
  int mask;      // pages that were loaded
  int n_live;    // keys of the chunk up to the tile's last
  int pos;       // position of its first key
  int flags;
  float sk;      // the chunk's K scale
  float lv;      // log2 of its V scale
};
// An item as the producer hands it to the MMA and softmax warps, with its q.
struct __align__(16) ItemRec {
  int ctx, row0, t0, g;
  int rows0, rows1;   // query tokens of half 0 / half 1 (<= 0: no work)
  int n_chunks, nc0;  // 128-key chunks: the tile's (0: no more items), half 0's
  __device__ __forceinline__ int nc1() const { return rows1 > 0 ? n_chunks : 0; }
};
constexpr int kFirst = 1;       // the item's first chunk: its q comes with it
constexpr int kTwoHalves = 2;
constexpr int kDiagonal = 4;    // some row of the tile does not see some key
constexpr int kFarApart = 8;    // V's scales spread over more than 2^7
constexpr int kMasked = 32;     // a key past the tile's last, or a page not loaded
constexpr int kEnd = 16;        // no more chunks

struct __align__(1024) QSmem {
  unsigned char q[kQBufs][kHalves][kOperandBytes]; // per half [32 tok][4 heads][64], swizzled
  unsigned char k[kWide][kOperandBytes];           // [128 keys][64] f16
  unsigned char v[kWide][kOperandBytes];
  unsigned char raw[kRaw][2][kChunk * kQ8HeadBytes];   // [128 keys][64] e4m3, K and V
  int tile_prefix[kMaxSeqsP + 1];
  int bin_start[kWeightBins];                      // counting sort of the tiles by weight
  uint16_t order[kSortQ];                          // tiles, heaviest first
  uint8_t tile_bins[kSortQ];                       // each tile's bin
  uint2 raw_mul[kRaw][kChunk / 8];                 // per page: f16x2 factors of K's and V's bytes
  float raw_lv[kRaw][kChunk / 8];                  // per page: log2 of what its V bytes still lack
  RawChunk raw_rec[kRaw];
  ItemRec item[kQBufs];
  float4 scale[kWide];                             // (sK, log2 sV, 1 / sV, 1: V's pages far apart)
  float lv[kWide][kChunk / 8];
  uint8_t q_exp[kQBufs][kHalves][kRows];           // per row: exponent field of its largest |q|
  // per dim: the first position in an item's diagonal chunks whose value is NaN,
  // below the item's number inverted (a later item's record is the smaller one)
  unsigned long long nan_from[kQBufs][kD];
  int nan_item[kQBufs];                            // the last item with such a record
  uint64_t q_full[kQBufs];
  uint64_t q_ready[kQBufs];                        // q is f16
  uint64_t q_empty[kQBufs];
  uint64_t raw_full[kRaw];
  uint64_t raw_empty[kRaw];
  uint64_t kv_full[kWide];
  uint64_t kv_empty[kWide];
  uint64_t s_full[kHalves];
  uint64_t s_free[kHalves];                        // the softmax has read S: the next S may land
  uint64_t p_full[kHalves];
  uint64_t o_full[kHalves];
  uint64_t o_free[kHalves];
  uint64_t staged[kHalves];                        // the half's output rows are in shared memory
  uint64_t mma_done[kHalves];                      // every MMA of the half's warp has completed
  uint32_t tmem_base;
  int pmask[kWide];
  int warp_sum[kQThreads / 32];
};

static_assert(sizeof(QSmem) + 1024 <= 227 * 1024, "shared memory above the per-CTA limit");

// Two f16 2^d (d <= 0; 0 below f16's smallest number).
__device__ __forceinline__ uint32_t pow2_f16x2(int d) {
  const uint32_t h = d >= -14 ? static_cast<uint32_t>(15 + d) << 10 : d >= -24 ? 1u << (24 + d) : 0u;
  return h | (h << 16);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// 8 e4m3 values as f16, and 8 f16 values times m (two f16).
__device__ __forceinline__ uint4 widen8(uint32_t a, uint32_t b) {
  return make_uint4(e4m3x2_to_f16x2(a), e4m3x2_to_f16x2(a >> 16), e4m3x2_to_f16x2(b),
                    e4m3x2_to_f16x2(b >> 16));
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint4 mul8(uint4 a, uint32_t m) {
  return make_uint4(mul2(a.x, m), mul2(a.y, m), mul2(a.z, m), mul2(a.w, m));
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void sts16(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}

// The largest |q| (bf16 pattern) of row r of a half's q tile (128-byte rows,
// 16-byte chunk e at e ^ (r & 7)).
__device__ __forceinline__ uint32_t q_row_top(const unsigned char *row, int r) {
  uint32_t top = 0;
#pragma unroll 2
  for (int e = 0; e < kD / 8; ++e) {
    const uint4 w = *reinterpret_cast<const uint4 *>(row + ((e ^ (r & 7)) << 4));
    top = __vmaxu2(top, __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu),
                                 __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu)));
  }
  return max(top & 0xffffu, top >> 16);
}

// Exponent field of the power of two that brings a row whose largest |q| has
// exponent field e to [2^12, 2^13).
__device__ __forceinline__ int q_scale_field(int e) { return min(266 - e, 253); }

// The row from bf16 to f16 in place, times `up`.
__device__ __forceinline__ void q_row_to_f16(unsigned char *row, int r, float up) {
#pragma unroll 2
  for (int e = 0; e < kD / 8; ++e) {
    uint4 *at = reinterpret_cast<uint4 *>(row + ((e ^ (r & 7)) << 4));
    const uint4 w = *at;
    const float2 a = bf16x2_to_float2(w.x), b = bf16x2_to_float2(w.y);
    const float2 c = bf16x2_to_float2(w.z), d = bf16x2_to_float2(w.w);
    *at = make_uint4(pack_f16(a.x * up, a.y * up), pack_f16(b.x * up, b.y * up),
                     pack_f16(c.x * up, c.y * up), pack_f16(d.x * up, d.y * up));
  }
}

// The top bits of the bytes that are NaN (0x7f or 0xff).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// w with its NaN bytes replaced by zeros; from[d] takes the position of a NaN
// in dim d when it is the item's first.  Rare.
__device__ __forceinline__ uint32_t without_nan(uint32_t w, int dim0, int item, int pos,
                                                unsigned long long *from) {
  for (uint32_t m = nan_bytes(w); m; m &= m - 1) {
    const int byte = (__ffs(m) - 1) >> 3;
    w &= ~(0xffu << (8 * byte));
    atomicMin(from + dim0 + byte,
              (static_cast<unsigned long long>(~static_cast<uint32_t>(item)) << 32) | pos);
  }
  return w;
}

// Whether a dim with record `from` is NaN for the row at qpos of item k.
__device__ __forceinline__ bool sees_nan(unsigned long long from, int k, int qpos) {
  return static_cast<uint32_t>(from >> 32) == ~static_cast<uint32_t>(k) &&
         static_cast<uint32_t>(from) <= static_cast<uint32_t>(qpos);
}

// MMA warp: waits until chunk gc is widened (every MMA warp does, for every
// chunk of the item, before it releases the stage).
__device__ __forceinline__ bool mma_wait_chunk(QSmem &sm, int gc, int lane,
                                               unsigned long long wait_ns) {
  int good = 1;
  if (lane == 0) good = mbar_wait_short(&sm.kv_full[gc % kWide], (gc / kWide) & 1, wait_ns) ? 1 : 0;
  good = __shfl_sync(0xffffffffu, good, 0);
  return good != 0;
}

// S of half h = Q_h K^T for chunk gc into the half's S columns (one thread).
__device__ __forceinline__ void mma_issue_s(QSmem &sm, uint32_t tmem, int qb, int h, int gc,
                                            uint32_t id_s) {
  const uint32_t k_addr = smem_u32(sm.k[gc % kWide]);
  const uint32_t q_addr = smem_u32(sm.q[qb][h]);
#pragma unroll
  for (int ks = 0; ks < kD / 16; ++ks)
    tc::mma_bf16(tmem + h * kChunk, tc::sdesc_sw128(q_addr + 32 * ks, 16, 1024),
                 tc::sdesc_sw128(k_addr + 32 * ks, 16, 1024), id_s, ks > 0);
  tc::mma_commit(&sm.s_full[h]);
}

// O of half h += P_h V for chunk gc in the half's O columns (one thread),
// P read from the half's P columns of tensor memory (16 keys = 8 columns per
// k-step); the item's first chunk starts the sum.
__device__ __forceinline__ void mma_issue_pv(QSmem &sm, uint32_t tmem, int h, int gc, bool first,
                                             uint32_t id_o) {
  const uint32_t v_addr = smem_u32(sm.v[gc % kWide]);
#pragma unroll
  for (int ks = 0; ks < kChunk / 16; ++ks)
    tc::mma_bf16_ts(tmem + kTmemO + h * kD, tmem + kTmemP + h * (kChunk / 2) + 8 * ks,
                    tc::sdesc_sw128(v_addr + 2048 * ks, 16, 1024), id_o,
                    (!first || ks > 0) ? 1u : 0u);
  tc::mma_commit(&sm.o_full[h]);
}

template <int BT>
__global__ void __launch_bounds__(kQThreads, 1) prefill_attention_q8_kernel(
    const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ CUtensorMap q_map,
    const __grid_constant__ CUtensorMap out_map, PrefillParams p,
    const float *__restrict__ scales) {
  extern __shared__ unsigned char smem_raw[];
  // (an offset, so that the compiler still knows it for shared memory)
  QSmem &sm = *reinterpret_cast<QSmem *>(smem_raw + (-smem_u32(smem_raw) & 1023u));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int i = tid; i < kQBufs * kD; i += kQThreads) sm.nan_from[i / kD][i % kD] = ~0ull;
  if (tid < kQBufs) sm.nan_item[tid] = -1;
  if (tid == 0) {
    prefetch_tensormap(&kv_map);
    prefetch_tensormap(&q_map);
    prefetch_tensormap(&out_map);
    for (int b = 0; b < kQBufs; ++b) {
      mbar_init(&sm.q_full[b], 1);
      mbar_init(&sm.q_ready[b], kConvThreads);
      // the MMA warps' commits and each softmax half once its output left
      // the buffer (it stages the half's output tile there)
      mbar_init(&sm.q_empty[b], 2 * kHalves);
    }
    for (int st = 0; st < kRaw; ++st) {
      mbar_init(&sm.raw_full[st], 1);
      mbar_init(&sm.raw_empty[st], kConvThreads);
    }
    for (int st = 0; st < kWide; ++st) {
      mbar_init(&sm.kv_full[st], kConvThreads);
      mbar_init(&sm.kv_empty[st], kHalves);     // one release per MMA warp
    }
    for (int h = 0; h < kHalves; ++h) {
      mbar_init(&sm.s_full[h], 1);
      mbar_init(&sm.s_free[h], kSoftThreads);
      mbar_init(&sm.p_full[h], kSoftThreads);
      mbar_init(&sm.o_full[h], 1);
      mbar_init(&sm.o_free[h], kSoftThreads);
    }
    for (int h = 0; h < kHalves; ++h) {
      mbar_init(&sm.staged[h], kSoftThreads);
      mbar_init(&sm.mma_done[h], 1);
    }
    fence_mbar_init();
  }
  pdl_launch_dependents();
  pdl_wait_primary();   // q and the cache come from the kernels before

  constexpr int kPagesPerChunk = PageGeom<BT>::kPages;
  constexpr unsigned kAllPages = PageGeom<BT>::kAll;
  const int total_tiles = order_tiles<BT, kQThreads, kSortQ>(sm, p, tid, warp, lane);
  const int n_items = total_tiles * kHkv;
  if (static_cast<int>(blockIdx.x) >= n_items) return;
  const bool sorted = total_tiles <= kSortQ;

  if (warp == kMmaWarp) {
    tc::tmem_alloc(&sm.tmem_base, kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sm.tmem_base;
  if (warp >= 8 && warp < kConvWarp) {
    // this warpgroup and the converters' give registers to the softmax warpgroups
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kQRegsMma));
    if (warp == kProducerWarp) {
      // ===================================================== producer warp ==
      bool ok = true;
      int gc = 0, k = 0;
      uint32_t issued = 0, issued_parity = 0;   // per stage: used / parity of its last fill
      // Page ids and scales are read for 32 pages (kBatch chunks) at a time, a
      // lane per page: a batch's ids when the batch before it starts, its scales
      // once that one's first chunk is on its way.
      constexpr int kBatch = 32 / kPagesPerChunk;
      struct Pages {
        int blk;
        float sk, sv;
      };
      auto page_ids = [&](const Item &x, int first) -> int {
        const int32_t *row =
            p.block_table + (static_cast<size_t>(x.s) * p.n_layers + p.layer) * p.max_blocks;
        const int pg = first + lane;
        return static_cast<long long>(pg) * BT < x.n_keys ? row[pg] : -1;
      };
      auto page_scales = [&](int g, Pages &d) {
        d.sk = d.sv = 1.f;
        if (d.blk >= 0 && d.blk < p.num_blocks) {
          const float *s = scales + static_cast<size_t>(d.blk) * 2 * kHkv + g;
          d.sk = s[0];
          d.sv = s[kHkv];
        }
      };
      Pages cur = {-1, 1.f, 1.f}, next = cur;
      int next_g = 0, next_has = 0;   // of `next`: kv head; 0 nothing, 1 ids, 2 scales too
      int q_asked = 0;    // lane 0: items whose Q has been asked for
      // Q buffer kk % 2: the item before last has left it
      auto ask_q = [&](const Item &x, int kk, unsigned long long wait_ns) -> bool {
        const int qb = kk % kQBufs;
        if (kk >= kQBufs && !mbar_wait(&sm.q_empty[qb], (kk / kQBufs - 1) & 1, wait_ns)) return false;
        ItemRec rec;
        rec.ctx = x.ctx;
        rec.row0 = x.row0;
        rec.t0 = x.t0;
        rec.g = x.g;
        rec.rows0 = x.rows0;
        rec.rows1 = x.rows1;
        rec.n_chunks = x.n_chunks;
        rec.nc0 = x.nc0;
        sm.item[qb] = rec;
        mbar_arrive_expect_tx(&sm.q_full[qb], x.halves * kOperandBytes);
        for (int h = 0; h < x.halves; ++h)
          tma_load_3d(sm.q[qb][h], &q_map, 0, x.g * kGqa, x.row0 + x.t0 + h * kQTok, &sm.q_full[qb]);
        q_asked = kk + 1;
        return true;
      };
      ItemRef ref = fetch_item(sm, p, total_tiles, sorted, 0, n_items);
      for (; ok && ref.i >= 0; ++k) {
        const Item it = decode_item(sm, ref);
        if (next_has == 0) {
          next.blk = page_ids(it, 0);
          next_g = it.g;
          next_has = 1;
        }
        int good = 1;
        if (lane == 0 && q_asked <= k) good = ask_q(it, k, p.wait_ns) ? 1 : 0;
        ok = __shfl_sync(0xffffffffu, good, 0) != 0;
        // an item whose Q was not asked for is not waited for below
        if (!ok) break;
        ref = fetch_item(sm, p, total_tiles, sorted, k + 1, n_items);
        for (int j = 0; j < it.n_chunks && ok; ++j, ++gc) {
          const int st = gc % kRaw;
          const uint32_t ph = (gc / kRaw) & 1;
          if (j % kBatch == 0) {
            if (next_has == 1) page_scales(next_g, next);
            cur = next;
            next_has = 0;
            if (j + kBatch < it.n_chunks) {
              next.blk = page_ids(it, (j / kBatch + 1) * 32);
              next_g = it.g;
              next_has = 1;
            } else if (ref.i >= 0) {
              const Item nx = decode_item(sm, ref);
              next.blk = page_ids(nx, 0);
              next_g = nx.g;
              next_has = 1;
            }
          }
          // the next item's Q, once the item before this one has left its buffer
          if (ref.i >= 0 && lane == 0 && q_asked <= k + 1 &&
              (k == 0 || mbar_try_wait_short(&sm.q_empty[(k + 1) % kQBufs], ((k + 1) / kQBufs - 1) & 1)))
            ask_q(decode_item(sm, ref), k + 1, p.wait_ns);
          // lane l: page l mod kPagesPerChunk of the chunk
          const int src = (j % kBatch) * kPagesPerChunk + (lane & (kPagesPerChunk - 1));
          Pages now;
          now.blk = __shfl_sync(0xffffffffu, cur.blk, src);
          const int pg = j * kPagesPerChunk + (lane & (kPagesPerChunk - 1));
          const bool needed = lane < kPagesPerChunk && pg * BT < it.n_keys;
          const bool valid = needed && now.blk >= 0 && now.blk < p.num_blocks;
          const unsigned vm = __ballot_sync(0xffffffffu, valid) & kAllPages;
          const unsigned nm = __ballot_sync(0xffffffffu, needed) & kAllPages;
          good = 1;
          if (lane == 0) {
            if (vm != nm) report(p.err, PA_DEV_BAD_BLOCK);
            if (!mbar_wait(&sm.raw_empty[st], ph ^ 1, p.wait_ns)) good = 0;
          }
          ok = __shfl_sync(0xffffffffu, good, 0) != 0;
          if (!ok) break;
          // The copies go out before the scales are there (the barrier's bytes are
          // announced after that: its phase cannot end before).
          // lane l < 2 kPagesPerChunk: the K rows (l < kPagesPerChunk) or the
          // V rows of page l mod kPagesPerChunk
          const int pl = lane & (kPagesPerChunk - 1), kv = (lane / kPagesPerChunk) & 1;
          // (test hook: CTA 0 leaves this chunk's copies out, so that the
          // waits on it run out)
          const bool fault = p.fault_chunk == gc && blockIdx.x == 0;
          if (!fault && lane < 2 * kPagesPerChunk && ((vm >> pl) & 1u))
            tma_load_5d(sm.raw[st][kv] + pl * BT * kQ8HeadBytes, &kv_map, 0, it.g, 0, kv, now.blk,
                        &sm.raw_full[st]);
          now.sk = __shfl_sync(0xffffffffu, cur.sk, src);
          now.sv = __shfl_sync(0xffffffffu, cur.sv, src);
          // the chunk's scales are its largest page's (exponent fields)
          const int ek = __float_as_int(now.sk) >> 23, ev = __float_as_int(now.sv) >> 23;
          const int top_k = __reduce_max_sync(0xffffffffu, valid ? ek : 1);
          const int ev1 = max(ev, kLeastV);
          const int top_v = __reduce_max_sync(0xffffffffu, valid ? ev1 : kLeastV);
          const bool far = __reduce_min_sync(0xffffffffu, valid ? ev1 : top_v) < top_v - 7;
          if (lane < kPagesPerChunk) {
            sm.raw_mul[st][lane] = make_uint2(pow2_f16x2(valid ? ek - top_k : 0),
                                              pow2_f16x2(!valid ? 0 : ev - (far ? ev1 : top_v)));
            sm.raw_lv[st][lane] = static_cast<float>((valid && far ? ev1 : top_v) - 127);
          }
          __syncwarp();
          if (lane == 0) {
            RawChunk c;
            c.mask = static_cast<int>(vm);
            c.pos = j * kChunk;
            c.n_live = it.n_keys - c.pos;
            c.flags = (j == 0 ? kFirst : 0) | (it.halves == 2 ? kTwoHalves : 0) |
                      (c.pos + kChunk - 1 > it.ctx + it.t0 ? kDiagonal : 0) | (far ? kFarApart : 0) |
                      (vm != kAllPages || c.n_live < kChunk ? kMasked : 0);
            c.sk = __int_as_float(top_k << 23);
            c.lv = static_cast<float>(top_v - 127);
            sm.raw_rec[st] = c;
            mbar_arrive_expect_tx(&sm.raw_full[st], __popc(vm) * 2 * BT * kQ8HeadBytes);
            issued |= 1u << st;
            issued_parity = (issued_parity & ~(1u << st)) | (ph << st);
          }
          __syncwarp();
          if (next_has == 1) {
            page_scales(next_g, next);
            next_has = 2;
          }
        }
      }
      if (lane == 0) {
        const int st = gc % kRaw;
        const uint32_t ph = (gc / kRaw) & 1;
        if (ok && mbar_wait(&sm.raw_empty[st], ph ^ 1, p.wait_ns)) {
          sm.raw_rec[st].flags = kEnd;
          mbar_arrive(&sm.raw_full[st]);
          issued |= 1u << st;
          issued_parity = (issued_parity & ~(1u << st)) | (ph << st);
        } else {
          report(p.err, PA_DEV_TIMEOUT);
        }
        // no copy may still be landing in shared memory when the CTA exits
        for (int kk = max(0, q_asked - kQBufs); kk < q_asked; ++kk)
          if (!mbar_wait(&sm.q_full[kk % kQBufs], (kk / kQBufs) & 1, p.wait_ns)) report(p.err, PA_DEV_TIMEOUT);
        for (int st = 0; st < kRaw; ++st)
          if ((issued >> st) & 1u)
            if (!mbar_wait(&sm.raw_full[st], (issued_parity >> st) & 1u, p.wait_ns))
              report(p.err, PA_DEV_TIMEOUT);
        // no more items
        if (ok) {
          if (k < kQBufs || mbar_wait(&sm.q_empty[k % kQBufs], (k / kQBufs - 1) & 1, p.wait_ns)) {
            sm.item[k % kQBufs].n_chunks = 0;
            mbar_arrive(&sm.q_full[k % kQBufs]);
          } else {
            report(p.err, PA_DEV_TIMEOUT);
          }
        }
      }
      __syncwarp();
    } else if (warp < kMmaWarp + kHalves) {
      // ======================================================== MMA warps ==
      const int h = warp - kMmaWarp;     // the half whose MMAs this warp issues
      const uint32_t id_s = tc::idesc_f16(kRows, kChunk, false);
      const uint32_t id_o = tc::idesc_f16(kRows, kD, true);
      int ok = 1;
      int gc = 0, k = 0;
      int n_p = 0;             // P chunks of this half consumed
      int n_active = 0;        // items in which the half had work
      int n_s = 0;             // S chunks issued
      // Lane 0 waits on the mbarriers and the warp takes its result; the
      // MMAs and commits are issued by one elected lane of the converged
      // warp, which keeps the tensor core fed at its own rate.
      int qb = 0;              // the item's Q buffer
      // S of chunk gcs once the softmax has read the previous S (whole warp)
      auto issue_s = [&](int gcs) -> bool {
        int good = 1;
        if (lane == 0 && n_s > 0 && !mbar_wait_short(&sm.s_free[h], (n_s - 1) & 1, p.wait_ns)) good = 0;
        if (!__shfl_sync(0xffffffffu, good, 0)) return false;
        tc::fence_after_sync();
        if (tc::elect_one()) mma_issue_s(sm, tmem, qb, h, gcs, id_s);
        __syncwarp();
        ++n_s;
        return true;
      };
      for (; ok; ++k) {
        qb = k % kQBufs;
        if (lane == 0) ok = mbar_wait_short(&sm.q_full[qb], (k / kQBufs) & 1, p.wait_ns) ? 1 : 0;
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        __syncwarp();   // (what lane 0 waited for, for every lane)
        const int n_chunks = sm.item[qb].n_chunks;
        if (n_chunks == 0) break;
        const int nch = h == 0 ? sm.item[qb].nc0 : sm.item[qb].nc1();
        if (lane == 0) ok = mbar_wait_short(&sm.q_ready[qb], (k / kQBufs) & 1, p.wait_ns) ? 1 : 0;
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (ok) ok = mma_wait_chunk(sm, gc, lane, p.wait_ns);
        if (ok && nch > 0) ok = issue_s(gc) ? 1 : 0;
        for (int j = 0; j < n_chunks && ok; ++j, ++gc) {
          if (j + 1 < n_chunks &&
              !mma_wait_chunk(sm, gc + 1, lane, p.wait_ns)) {
            ok = 0;
            break;
          }
          if (j < nch) {
            int good = 1;
            if (j + 1 < nch && !issue_s(gc + 1)) good = 0;
            if (lane == 0) {
              // the half's previous item has read its O (the first PV clears it)
              if (good && j == 0 && n_active > 0 &&
                  !mbar_wait_short(&sm.o_free[h], (n_active - 1) & 1, p.wait_ns))
                good = 0;
              // the half's softmax has written P
              if (good && !mbar_wait_short(&sm.p_full[h], n_p & 1, p.wait_ns)) good = 0;
            }
            good = __shfl_sync(0xffffffffu, good, 0);
            if (good) {
              tc::fence_after_sync();
              if (tc::elect_one()) mma_issue_pv(sm, tmem, h, gc, j == 0, id_o);
              __syncwarp();
            }
            ++n_p;
            ok = good;
          }
          if (ok && tc::elect_one()) tc::mma_commit(&sm.kv_empty[gc % kWide]);
          __syncwarp();
        }
        if (ok && tc::elect_one()) tc::mma_commit(&sm.q_empty[qb]);   // every MMA that reads Q is issued
        __syncwarp();
        if (nch > 0) ++n_active;
      }
      if (!ok && lane == 0) report(p.err, PA_DEV_TIMEOUT);
      // the tensor core has finished every MMA this warp issued before the
      // TMEM columns go back (after a time-out too)
      if (tc::elect_one()) tc::mma_commit(&sm.mma_done[h]);
      __syncwarp();
      if (lane == 0 && !mbar_wait(&sm.mma_done[h], 0, p.wait_ns)) report(p.err, PA_DEV_TIMEOUT);
      __syncwarp();
    }
  } else if (warp >= kConvWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kQRegsConv));
    // ================================================== converter warps ==
    // A chunk's bytes as the TMA left them ([128 keys][64] of K and of V) become
    // f16 operand tiles in the swizzled layout that the MMAs read; an item's q
    // becomes f16 first.  V rows past the tile's last key or in a page that was
    // not loaded become zeros: they meet P = 0.
    bool ok = true;
    const int ct = tid - kConvWarp * 32;
    // this thread's 16-byte units of a chunk are u = ct + 128 i: key ct / 4 +
    // 32 i, dims 16 (ct % 4) ..; their two 16-byte places in the wide row
    const int key0 = ct >> 2, part = ct & 3;
    const uint32_t at0 = key0 * kTileRowBytes + (((2 * part) ^ (key0 & 7)) << 4), at1 = at0 ^ 16;
    int items = 0;
    for (int gc = 0;; ++gc) {
      const int rs = gc % kRaw, ws = gc % kWide;
      ok = mbar_wait_short(&sm.raw_full[rs], (gc / kRaw) & 1, p.wait_ns);
      if (!ok) break;
      const RawChunk rec = sm.raw_rec[rs];
      if (rec.flags & kEnd) break;
      const int qb = (items + ((rec.flags & kFirst) ? 0 : 1)) % kQBufs;   // (items counts this one already)
      if (rec.flags & kFirst) {
        // the item's Q is in, so the outputs of the item that had its buffer are out
        ok = mbar_wait_short(&sm.q_full[qb], (items / kQBufs) & 1, p.wait_ns);
        if (!ok) break;
        // thread ct turns row ct of each half into f16, scaled to [2^12, 2^13).
        // The scores of a row that is not finite are NaN, or all -inf: its
        // output is NaN.
        const int halves = (rec.flags & kTwoHalves) ? 2 : 1;
#pragma unroll 1
        for (int h = 0; h < halves; ++h) {
          unsigned char *row = sm.q[qb][h] + ct * kTileRowBytes;
          const int e = static_cast<int>(q_row_top(row, ct) >> 7);
          q_row_to_f16(row, ct, __int_as_float(q_scale_field(e) << 23));
          sm.q_exp[qb][h][ct] = static_cast<uint8_t>(e);
        }
        fence_proxy_async_smem();       // the tensor core reads q through the async proxy
        mbar_arrive(&sm.q_ready[qb]);
        ++items;
      }
      ok = mbar_wait_short(&sm.kv_empty[ws], ((gc / kWide) & 1) ^ 1, p.wait_ns);
      if (!ok) break;
      const uint32_t mul_step = kConvThreads / 4 / BT * 8;
      uint32_t src = smem_u32(sm.raw[rs][0]) + 16 * ct, mul_at = smem_u32(&sm.raw_mul[rs][key0 / BT]);
      uint32_t dst = smem_u32(sm.k[ws]) + at0;
      const uint32_t flip = at1 - at0, to_v = smem_u32(sm.v[ws]) - smem_u32(sm.k[ws]);
      int key = key0;
#pragma unroll 1
      for (int i = 0; i < kChunk * 4 / kConvThreads; ++i) {
        const uint2 mul = lds8(mul_at);
        const uint4 kr = lds16(src);
        uint4 vr = lds16(src + kChunk * kQ8HeadBytes);
        uint4 w0 = widen8(kr.x, kr.y), w1 = widen8(kr.z, kr.w);
        if (mul.x != kOnes) {
          w0 = mul8(w0, mul.x);
          w1 = mul8(w1, mul.x);
        }
        sts16(dst, w0);
        sts16(dst + flip, w1);
        if (rec.flags & (kMasked | kDiagonal)) {
          if (key >= rec.n_live || !((rec.mask >> (key / BT)) & 1)) vr = make_uint4(0, 0, 0, 0);
          // a NaN value would reach the rows before it too (P = 0 times NaN)
          if ((rec.flags & kDiagonal) &&
              (nan_bytes(vr.x) | nan_bytes(vr.y) | nan_bytes(vr.z) | nan_bytes(vr.w)) != 0) {
            unsigned long long *from = sm.nan_from[qb] + 16 * part;
            vr.x = without_nan(vr.x, 0, items - 1, rec.pos + key, from);
            vr.y = without_nan(vr.y, 4, items - 1, rec.pos + key, from);
            vr.z = without_nan(vr.z, 8, items - 1, rec.pos + key, from);
            vr.w = without_nan(vr.w, 12, items - 1, rec.pos + key, from);
            sm.nan_item[qb] = items - 1;
          }
        }
        w0 = widen8(vr.x, vr.y);
        w1 = widen8(vr.z, vr.w);
        if (mul.y != kOnes) {
          w0 = mul8(w0, mul.y);
          w1 = mul8(w1, mul.y);
        }
        sts16(dst + to_v, w0);
        sts16(dst + to_v + flip, w1);
        src += 16 * kConvThreads;
        mul_at += mul_step;
        dst += kConvThreads / 4 * kTileRowBytes;
        key += kConvThreads / 4;
      }
      if (ct < kPagesPerChunk) sm.lv[ws][ct] = sm.raw_lv[rs][ct];
      if (ct == 0) {
        sm.pmask[ws] = rec.mask;
        sm.scale[ws] = make_float4(rec.sk, rec.lv, p_exp2(-rec.lv),
                                   (rec.flags & kFarApart) ? 1.f : 0.f);
      }
      mbar_arrive(&sm.raw_empty[rs]);
      fence_proxy_async_smem();         // the tensor core reads the tiles through the async proxy
      mbar_arrive(&sm.kv_full[ws]);
    }
    if (!ok) report(p.err, PA_DEV_TIMEOUT);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kQRegsSoft));
    // ==================================================== softmax warps ==
    // O accumulates in TMEM.  Each row keeps the reference m its P values are
    // taken against: kBelow (log2 units) below the largest so far when it is
    // set; it moves (and O, l are rescaled) only when a chunk's maximum exceeds
    // it by more than kRescale, so P stays below 2^kRescale and most chunks touch
    // O not at all.
    // S_{j+1} is issued before PV_j, so O (for a rescale) and the P
    // columns are touched only once PV_{j-1}'s commit is there.
    constexpr float kBelow = 7.f, kRescale = 15.f;
    const int h = tid >> 7;                   // half
    const int r = tid & (kRows - 1);          // MMA row = TMEM lane
    const int tok = r >> 2, hh = r & 3;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_addr = lane_addr + h * kChunk, o_addr = lane_addr + kTmemO + h * kD;
    const uint32_t p_addr = lane_addr + kTmemP + h * (kChunk / 2);
    bool ok = true;
    int gc = 0, n_s = 0, n_o = 0;   // S chunks read; PV commits waited for
    int n_staged = 0;               // output tiles staged
    // Thread r == 0: the Q buffer its last output store reads from, released
    // to the producer only after the next item's first P (the store has read
    // it long before), so that the wait for the read is off the warp's path.
    int pend_qb = -1;
    auto release_stored = [&]() {
      if (pend_qb >= 0) {
        bulk_wait_group_read0();
        mbar_arrive(&sm.q_empty[pend_qb]);
        pend_qb = -1;
      }
    };
    for (int k = 0;; ++k) {
      const int qb = k % kQBufs;
      ok = mbar_wait_short(&sm.q_full[qb], (k / kQBufs) & 1, p.wait_ns);
      if (!ok) break;
      const ItemRec it = sm.item[qb];
      if (it.n_chunks == 0) break;
      const int rows = h == 0 ? it.rows0 : it.rows1;
      const int nch = h == 0 ? it.nc0 : it.nc1();
      if (nch == 0) {
        // nothing staged: release the Q buffer (it holds this item's Q: an
        // earlier arrival would count for the item before last)
        if (r == 0) {
          release_stored();
          mbar_arrive(&sm.q_empty[qb]);
        }
        gc += it.n_chunks;
        continue;
      }
      const int first_pos = it.ctx + it.t0 + h * kQTok;   // the half's first query position
      const int last_pos = first_pos + rows - 1;
      const int qpos = min(first_pos + tok, last_pos);
      float m = p_neg_inf(), l = 0.f, factor = 0.f;
      for (int j = 0; j < nch; ++j) {
        const int st = (gc + j) % kWide;
        if (!mbar_wait_short(&sm.s_full[h], n_s & 1, p.wait_ns) ||
            !mbar_wait_short(&sm.kv_full[st], ((gc + j) / kWide) & 1, p.wait_ns)) {
          ok = false;
          break;
        }
        if (j == 0) {   // (q was converted before the item's first chunk was widened)
          const int e = sm.q_exp[qb][h][r];
          factor = e < 255 ? p.qscale * __int_as_float((254 - q_scale_field(e)) << 23)
                           : __int_as_float(0x7fc00000);
        }
        ++n_s;
        tc::fence_after_sync();
        const int pm = sm.pmask[st];
        const int kbase = j * kChunk;
        // every key of the chunk is visible to every row of the half and was loaded
        const bool full = pm == static_cast<int>(kAllPages) && kbase + kChunk - 1 <= first_pos;
        const int lim = qpos - kbase;           // keys c <= lim are at or before the row
        const float4 sc = sm.scale[st];         // sK, log2 sV, 1 / sV, V's pages far apart
        const float fk = fmaxf(factor * sc.x, kTiny);
        bool pv_done = j == 0;                  // PV_{j-1} complete: O stable, P columns read
        auto wait_pv = [&]() -> bool {
          if (pv_done) return true;
          if (!mbar_wait_short(&sm.o_full[h], n_o & 1, p.wait_ns)) return false;
          ++n_o;
          pv_done = true;
          tc::fence_after_sync();
          return true;
        };
        // The reference moves to the chunk's maximum mc where that lies far
        // above it; O and l follow.
        auto move_to = [&](float mc) -> bool {
          const bool move = mc > m + kRescale || (m == p_neg_inf() && mc != p_neg_inf());
          if (__any_sync(0xffffffffu, move) && j > 0) {
            if (!wait_pv()) return false;
            // (the whole warp takes part in the TMEM round trip)
            const float alpha = move ? p_exp2(m - (mc - kBelow)) : 1.f;
#pragma unroll 1
            for (int c0 = 0; c0 < kD; c0 += 32) {
              uint32_t ov[32];
              tc::tmem_ld32(o_addr + c0, ov);
              tc::tmem_ld_wait();
#pragma unroll
              for (int c = 0; c < 32; ++c) ov[c] = __float_as_uint(__uint_as_float(ov[c]) * alpha);
              tc::tmem_st32(o_addr + c0, ov);
            }
            tc::tmem_st_wait();
            l *= alpha;
          }
          if (move) m = mc - kBelow;
          return true;
        };
        // P = 2^(s f sK + log2 sV - m) in f16 pairs (key 2c in the low half of
        // column c) goes into the half's P columns of tensor memory.
        // A fused product keeps m's rounding error: below 2^-2 for scores up to 2^22,
        // which fk bounds (|S| < 2^28), but enough to overflow the exponential above.
        if (!__any_sync(0xffffffffu, sc.w != 0.f || fk > kLargeFactor)) {
          uint32_t v[kChunk];
#pragma unroll
          for (int c0 = 0; c0 < kChunk; c0 += 32)
            tc::tmem_ld32(s_addr + c0, *reinterpret_cast<uint32_t(*)[32]>(&v[c0]));
          tc::tmem_ld_wait();
          tc::fence_before_sync();
          mbar_arrive(&sm.s_free[h]);           // S_{j+1} may land in the S columns
          if (!full) {
            // masked keys: -inf (loaded K rows past the tile or in a missing page may be anything)
            if (pm != static_cast<int>(kAllPages)) {
#pragma unroll
              for (int c = 0; c < kChunk; ++c)
                if (!((pm >> (c / BT)) & 1)) v[c] = 0xff800000u;
            }
            // (the warp's rows are 8 tokens: columns before the first one's need no test)
            const int lim0 = __shfl_sync(0xffffffffu, lim, 0);
#pragma unroll
            for (int c0 = 0; c0 < kChunk; c0 += 16)
              if (c0 + 15 > lim0) {
#pragma unroll
                for (int c = c0; c < c0 + 16; ++c)
                  if (c > lim) v[c] = 0xff800000u;
              }
          }
          // row maximum: 8 chains of three-input maxima over keys q, q+8, ..
          float mx8[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) mx8[q] = p_neg_inf();
#pragma unroll
          for (int c = 0; c < kChunk; c += 16)
#pragma unroll
            for (int q = 0; q < 8; ++q)
              mx8[q] = fmax3(mx8[q], __uint_as_float(v[c + q]), __uint_as_float(v[c + 8 + q]));
          const float mx = fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
                                 fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])));
          if (!move_to(fmaf(mx, fk, sc.y))) {
            ok = false;
            break;
          }
          const float bias = sc.y - ((m == p_neg_inf()) ? 0.f : m);
          const float2 b2 = make_float2(bias, bias), f2 = make_float2(fk, fk);
          float2 ls[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                          make_float2(0.f, 0.f)};
          uint32_t pw[kChunk / 2];
#pragma unroll
          for (int c = 0; c < kChunk; c += 2) {
            const float2 x =
                fma2(make_float2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), f2, b2);
            const float2 e = make_float2(p_exp2(x.x), p_exp2(x.y));
            ls[(c >> 1) & 3] = add2(ls[(c >> 1) & 3], e);
            pw[c >> 1] = pack_f16(e.x, e.y);
          }
          if (!wait_pv()) {
            ok = false;
            break;
          }
          tc::tmem_st32(p_addr, *reinterpret_cast<uint32_t(*)[32]>(&pw[0]));
          tc::tmem_st32(p_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(&pw[32]));
          l = fmaf(((ls[0].x + ls[0].y) + (ls[1].x + ls[1].y)) +
                       ((ls[2].x + ls[2].y) + (ls[3].x + ls[3].y)), sc.z, l);
        } else {
          // pages far apart (log2 sV page by page) or huge scores (each rounded
          // as m is): S read twice, 8 keys at a time (rare, so kept small)
          auto load8 = [&](int c0, float (&x)[8]) {
            uint32_t u[8];
            tc::tmem_ld8(s_addr + c0, u);
            tc::tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 8; ++c)
              x[c] = (c0 + c <= lim && ((pm >> (c0 / BT)) & 1)) ? __uint_as_float(u[c]) : p_neg_inf();
          };
          float mc = p_neg_inf();
#pragma unroll 1
          for (int c0 = 0; c0 < kChunk; c0 += 8) {
            float x[8];
            load8(c0, x);
            float mx = x[0];
#pragma unroll
            for (int c = 1; c < 8; ++c) mx = fmaxf(mx, x[c]);
            mc = fmaxf(mc, __fadd_rn(__fmul_rn(mx, fk), sm.lv[st][c0 / BT]));
          }
          if (!move_to(mc) || !wait_pv()) {
            ok = false;
            break;
          }
          const float base = (m == p_neg_inf()) ? 0.f : m;
#pragma unroll 1
          for (int c0 = 0; c0 < kChunk; c0 += 8) {
            const float lv = sm.lv[st][c0 / BT];
            float x[8], sum = 0.f;
            load8(c0, x);
            uint32_t w[4];
#pragma unroll
            for (int c = 0; c < 8; c += 2) {
              const float e0 = p_exp2(__fadd_rn(__fmul_rn(x[c], fk), lv) - base);
              const float e1 = p_exp2(__fadd_rn(__fmul_rn(x[c + 1], fk), lv) - base);
              sum += e0 + e1;
              w[c >> 1] = pack_f16(e0, e1);
            }
            tc::tmem_st4(p_addr + c0 / 2, w);
            l = fmaf(sum, p_exp2(-lv), l);
          }
          tc::fence_before_sync();
          mbar_arrive(&sm.s_free[h]);
        }
        tc::tmem_st_wait();
        tc::fence_before_sync();    // P, for the tensor core
        mbar_arrive(&sm.p_full[h]);
        if (j == 0) release_stored();
      }
      if (!ok) break;
      // O is complete once the item's last PV is
      if (!mbar_wait_short(&sm.o_full[h], n_o & 1, p.wait_ns)) {
        ok = false;
        break;
      }
      ++n_o;
      tc::fence_after_sync();
      uint32_t ov[kD];
      tc::tmem_ld32(o_addr, *reinterpret_cast<uint32_t(*)[32]>(&ov[0]));
      tc::tmem_ld32(o_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(&ov[32]));
      tc::tmem_ld_wait();
      tc::fence_before_sync();
      mbar_arrive(&sm.o_free[h]);   // the next item's first PV may clear O
      const float inv = factor != factor ? factor : (l > 0.f) ? 1.f / l : 0.f;
      auto row_chunk = [&](int e) {
        const float *f = reinterpret_cast<const float *>(&ov[8 * e]);
        return make_uint4(float2_to_bf16x2(f[0] * inv, f[1] * inv),
                          float2_to_bf16x2(f[2] * inv, f[3] * inv),
                          float2_to_bf16x2(f[4] * inv, f[5] * inv),
                          float2_to_bf16x2(f[6] * inv, f[7] * inv));
      };
      if (rows == kQTok) {
        // a whole half tile: the rows go into the half's part of this item's
        // Q buffer (no MMA reads it any more), in the layout of the output's
        // tensor map (row r, 16-byte chunk e at e ^ (r mod 8)), and leave in
        // one TMA store, whose writes are whole 128-byte lines
        unsigned char *stg = sm.q[qb][h] + r * kTileRowBytes;
#pragma unroll
        for (int e = 0; e < kD / 8; ++e)
          *reinterpret_cast<uint4 *>(stg + ((e ^ (r & 7)) << 4)) = row_chunk(e);
        if (sm.nan_item[qb] == k)   // NaN values that the row sees among the item's last keys
#pragma unroll 1
          for (int d = 0; d < kD; ++d)
            if (sees_nan(sm.nan_from[qb][d], k, qpos))
              *reinterpret_cast<uint16_t *>(stg + (((d >> 3) ^ (r & 7)) << 4) + 2 * (d & 7)) = 0x7fc0;
        fence_proxy_async_smem();
        mbar_arrive(&sm.staged[h]);
        if (r == 0) {
          ok = mbar_wait_short(&sm.staged[h], n_staged & 1, p.wait_ns);
          if (ok) {
            release_stored();
            tma_store_3d(&out_map, sm.q[qb][h], 0, it.g * kGqa, it.row0 + it.t0 + h * kQTok);
            bulk_commit_group();
            pend_qb = qb;
          }
        }
        ++n_staged;
      } else {
        if (tok < rows) {
          uint4 *dst = reinterpret_cast<uint4 *>(
              p.out + ((static_cast<size_t>(it.row0) + it.t0 + h * kQTok + tok) * kHq +
                       it.g * kGqa + hh) * kD);
#pragma unroll
          for (int e = 0; e < kD / 8; ++e) dst[e] = row_chunk(e);
          if (sm.nan_item[qb] == k)
#pragma unroll 1
            for (int d = 0; d < kD; ++d)
              if (sees_nan(sm.nan_from[qb][d], k, qpos)) reinterpret_cast<uint16_t *>(dst)[d] = 0x7fc0;
        }
        // the buffer's NaN record is read by every row before it is released
        mbar_arrive(&sm.staged[h]);
        if (r == 0) {
          ok = mbar_wait_short(&sm.staged[h], n_staged & 1, p.wait_ns);
          release_stored();
          if (ok) mbar_arrive(&sm.q_empty[qb]);
        }
        ++n_staged;
      }
      if (!ok) break;
      gc += it.n_chunks;
    }
    if (!ok) report(p.err, PA_DEV_TIMEOUT);
    release_stored();
    if (r == 0) bulk_wait_group0();   // the output stores are complete
  }
  // every TMEM read and MMA is done (or given up on) before the columns go back
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace

// Tensor map over the 8-bit pool: dims (d 64, kv head 8, token bt, K|V 2,
// block), box (64, 1, bt, 1, 1): one kv head's K or V rows of a page, as they
// are.
static int make_q8_rows_map(CUtensorMap *map, const void *kv_cache, int num_blocks, int bt) {
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
  const cuuint64_t row = kQ8TokBytes;
  const cuuint64_t dims[5] = {kD, kHkv, static_cast<cuuint64_t>(bt), 2,
                              static_cast<cuuint64_t>(num_blocks)};
  const cuuint64_t strides[4] = {kQ8HeadBytes, row, row * bt, row * bt * 2};
  const cuuint32_t box[5] = {kD, 1, static_cast<cuuint32_t>(bt), 1, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void *>(kv_cache), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa

using namespace pa;

namespace {

template <int BT>
int prefill_q8_impl(uint16_t *out, const uint16_t *q, int total_tokens, const int32_t *cu_tokens,
                    const uint8_t *kv_cache, const float *kv_scales, int num_blocks,
                    const int32_t *block_table, int n_layers, int max_blocks_per_seq,
                    const int32_t *context_lens, int num_seqs, int layer, float scale,
                    int32_t *err, void *stream) {
  if (num_seqs < 0 || num_seqs > kMaxSeqsP || total_tokens < 0 || num_blocks <= 0 ||
      n_layers <= 0 || max_blocks_per_seq <= 0)
    return PA_ERR_ARG;
  if (static_cast<long long>(max_blocks_per_seq) * BT > INT_MAX) return PA_ERR_ARG;
  if (layer < 0 || layer >= n_layers) return PA_ERR_LAYER;
  if (num_seqs == 0 || total_tokens == 0) return PA_OK;
  if (!out || !q || !cu_tokens || !kv_cache || !kv_scales || !block_table || !context_lens || !err)
    return PA_ERR_NULL;
  if (!aligned16(out) || !aligned16(q) || !aligned16(kv_cache) || !aligned16(kv_scales))
    return PA_ERR_ALIGN;
  if (!(scale > 0.f) || scale > 3.0e38f) return PA_ERR_ARG;   // the row maximum is taken before scaling
  DeviceInfo di;
  int rc = current_device(&di);
  if (rc != PA_OK) return rc;
  const size_t smem = sizeof(QSmem) + 1024;
  if (cudaFuncSetAttribute(prefill_attention_q8_kernel<BT>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(smem)) != cudaSuccess)
    return PA_ERR_CUDA;
  alignas(64) CUtensorMap kv_map, q_map, out_map;
  rc = make_q8_rows_map(&kv_map, kv_cache, num_blocks, BT);
  if (rc == PA_OK) rc = make_q_map(&q_map, q, total_tokens);
  if (rc == PA_OK) rc = make_q_map(&out_map, out, total_tokens);   // out has q's layout
  if (rc != PA_OK) return rc;
  // every sequence's chunk ends in at most one partial tile; one CTA per SM
  // works through the (tile, kv head) items
  const long long tiles = (static_cast<long long>(total_tokens) + kCtaTok - 1) / kCtaTok + num_seqs;
  const int grid = static_cast<int>(min(static_cast<long long>(di.sm_count), tiles * kHkv));
  if (tiles * kHkv + 2LL * grid > INT_MAX) return PA_ERR_ARG;   // item positions stay in int
  PrefillParams prm;
  prm.out = reinterpret_cast<__nv_bfloat16 *>(out);
  prm.cu_tokens = cu_tokens;
  prm.block_table = block_table;
  prm.context_lens = context_lens;
  prm.err = err;
  prm.num_blocks = num_blocks;
  prm.n_layers = n_layers;
  prm.max_blocks = max_blocks_per_seq;
  prm.num_seqs = num_seqs;
  prm.layer = layer;
  prm.total_tokens = total_tokens;
  prm.qscale = scale * kLog2eP;
  prefill_fault(&prm.fault_chunk, &prm.wait_ns);
  return launch_pdl(prefill_attention_q8_kernel<BT>, dim3(static_cast<unsigned>(grid)),
                    dim3(kQThreads), smem, static_cast<cudaStream_t>(stream), kv_map, q_map,
                    out_map, prm, kv_scales) == cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

}  // namespace

extern "C" int pa_prefill_attention_q8(uint16_t *out, const uint16_t *q, int total_tokens,
                                       const int32_t *cu_tokens, const uint8_t *kv_cache,
                                       const float *kv_scales, int num_blocks, int block_tokens,
                                       const int32_t *block_table, int n_layers,
                                       int max_blocks_per_seq, const int32_t *context_lens,
                                       int num_seqs, int layer, float scale, int32_t *err,
                                       void *stream) {
  auto *impl = block_tokens == 8    ? prefill_q8_impl<8>
               : block_tokens == 16 ? prefill_q8_impl<16>
               : block_tokens == 32 ? prefill_q8_impl<32>
                                    : nullptr;
  if (!impl) return PA_ERR_ARG;
  return impl(out, q, total_tokens, cu_tokens, kv_cache, kv_scales, num_blocks, block_table,
              n_layers, max_blocks_per_seq, context_lens, num_seqs, layer, scale, err, stream);
}
