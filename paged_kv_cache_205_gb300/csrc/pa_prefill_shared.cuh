// pa_prefill_shared.cuh -- what the prefill attention kernels over the bf16
// and the 8-bit cache share: the tile geometry, the order in which the CTAs
// work through the (query tile, kv head) items, and small helpers.
#pragma once

#include <climits>
#include <cudaTypedefs.h>

#include "pa_device.cuh"
#include "pa_host.h"
#include "pa_tc.cuh"

namespace pa {
namespace {

constexpr int kQTok = 32;                     // query tokens per half
constexpr int kHalves = 2;
constexpr int kCtaTok = kQTok * kHalves;      // query tokens per CTA
constexpr int kRows = kQTok * kGqa;           // 128 MMA rows per half
constexpr int kChunk = 128;                   // keys per chunk (8 pages of 16 tokens)
constexpr int kQBufs = 2;                     // Q tiles in flight: the next item's loads early
constexpr int kSortTiles = 4096;              // tiles ordered by weight; beyond, by index
constexpr int kWeightBins = 256;              // weight classes (see tile_bin)
constexpr int kSoftThreads = kRows;           // one softmax warpgroup per half
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kTileRowBytes = kHeadRowBytes;             // 128-byte rows
constexpr int kOperandBytes = kChunk * kTileRowBytes;    // 16 KiB: 128 rows x 64 bf16
constexpr uint32_t kTmemCols = 512;                      // S x2 (256) + O x2 (128) + P x2 (128)
constexpr uint32_t kTmemO = 256;
constexpr uint32_t kTmemP = 384;                         // P of half h: 64 columns of bf16 pairs
constexpr int kMaxSeqsP = 2048;
constexpr float kLog2eP = 1.4426950408889634f;

struct PrefillParams {
  __nv_bfloat16 *out;
  const int32_t *cu_tokens;
  const int32_t *block_table;
  const int32_t *context_lens;
  int32_t *err;
  int num_blocks;
  int n_layers;
  int max_blocks;
  int num_seqs;
  int layer;
  int total_tokens;        // rows of q and out
  float qscale;
  // test hook (pa_prefill_set_test_fault): the chunk of CTA 0 whose copies
  // are left out (-1: none), and the limit of every wait
  int fault_chunk;
  unsigned long long wait_ns;
};

__device__ __forceinline__ float p_neg_inf() { return -__int_as_float(0x7f800000); }

__device__ __forceinline__ float p_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// max(a, b, c) in one instruction
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// Packed two-lane fp32 add.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long ra, rb, rd;
  asm("mov.b64 %0, {%1, %2};" : "=l"(ra) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(rb) : "f"(b.x), "f"(b.y));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(rd) : "l"(ra), "l"(rb));
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(rd));
  return d;
}

__device__ __forceinline__ void tma_load_3d(void *smem_dst, const void *tmap, int c0, int c1,
                                            int c2, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}

// Shared -> global 3-D tiled tensor copy (TMA store) in the thread's bulk
// async-group.
__device__ __forceinline__ void tma_store_3d(const void *tmap, const void *smem_src, int c0, int c1,
                                             int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
          reinterpret_cast<uint64_t>(tmap)),
      "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(smem_src))
      : "memory");
}
__device__ __forceinline__ void bulk_commit_group() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// The thread's bulk stores have read their shared-memory source.
__device__ __forceinline__ void bulk_wait_group_read0() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
// ... and have completed.
__device__ __forceinline__ void bulk_wait_group0() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// A work item is (64-token query tile, kv head).  The tiles are ordered by
// weight class (the weight: the 128-key chunks its two halves go through),
// heaviest first, ties in tile order (a stable counting sort every CTA
// computes alike); with more than kSortTiles tiles, by tile index from the
// last (the last tiles of a sequence see the most keys).  The items of that order are dealt out in
// rounds of G, every other round backwards (CTA b takes positions b,
// 2G - 1 - b, 2G + b, ...), so that each CTA's sum of weights comes close to
// the mean; a CTA keeps its pipeline running from one item into the next.
struct Item {
  int g;                    // kv head
  int ctx, row0, t0;        // the tile's sequence: cached tokens, first row; tile start
  int rows0, rows1;         // query tokens of half 0 / half 1 (<= 0: no work)
  int halves;
  int n_keys0, n_keys;      // keys half 0 / the whole tile sees
  int n_chunks, nc0, nc1;   // 128-key chunks: the tile's, half 0's, half 1's
  int s;
};

// The sequence s whose tiles hold tile t: prefix[s] <= t < prefix[s+1].
template <class Sm>
__device__ __forceinline__ int tile_seq(const Sm &sm, int num_seqs, int t) {
  int lo = 0, hi = num_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sm.tile_prefix[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Sort bin of tile t: kWeightBins - 1 - the class of its weight w, so that
// bins in ascending order hold the tiles heaviest first.  The class is w
// itself below 16 and w's leading four bits with its exponent above (classes
// at most 1/8 wide): a class then holds several tiles of one long sequence,
// which stay in tile order, so the CTAs of one round share more K/V in L2.
template <class Sm>
__device__ __forceinline__ int tile_bin(const Sm &sm, const PrefillParams &p, int t) {
  const int s = tile_seq(sm, p.num_seqs, t);
  const long long t0 = static_cast<long long>(t - sm.tile_prefix[s]) * kCtaTok;
  const long long ctx = __ldg(p.context_lens + s);
  const long long n = __ldg(p.cu_tokens + s + 1) - __ldg(p.cu_tokens + s);
  const long long r0 = min(static_cast<long long>(kQTok), n - t0);
  const long long r1 = min(static_cast<long long>(kQTok), n - t0 - kQTok);
  long long w = (ctx + t0 + r0 + kChunk - 1) / kChunk;
  if (r1 > 0) w += (ctx + t0 + kQTok + r1 + kChunk - 1) / kChunk;
  w = max(w, 1LL);
  const int e = 63 - __clzll(w);                        // w < 2^62: e <= 61
  const int cls = e < 3 ? static_cast<int>(w) : 8 * (e - 3) + static_cast<int>(w >> (e - 3));
  return kWeightBins - 1 - min(cls, kWeightBins - 1);
}

// Position in the work order of this CTA's k-th item, or -1 past the end.
__device__ __forceinline__ int item_position(int k, int n_items) {
  // the walks stop at the first position past the end, so pos <= n_items +
  // 2 G, which the launch keeps below INT_MAX
  const int G = gridDim.x, b = blockIdx.x;
  const int pos = k * G + ((k & 1) ? G - 1 - b : b);
  return pos < n_items ? pos : -1;
}

// The item at position k of this CTA's walk: its place in the work order,
// tile and sequence, and the sequence's three values in global memory.  The
// roles that are on the pipeline's path fetch the next item while the
// current one runs, so that the loads' latency is not paid between items.
struct ItemRef {
  int i;                      // position in the work order; -1 past the end
  int t, s;                   // tile, sequence
  int ctx, row0, row_end;     // cached tokens; the sequence's rows [row0, row_end)
};

// A load that stays where it is written (the compiler may move a read-only
// __ldg down to its first use, which would put its latency back between
// the items).
__device__ __forceinline__ int load_early(const int32_t *ptr) {
  int v;
  asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(v) : "l"(ptr));
  return v;
}

template <class Sm>
__device__ __forceinline__ ItemRef fetch_item(const Sm &sm, const PrefillParams &p,
                                              int total_tiles, bool sorted, int k, int n_items) {
  ItemRef r;
  r.i = item_position(k, n_items);
  r.t = r.s = r.ctx = r.row0 = r.row_end = 0;
  if (r.i < 0) return r;
  const int rank = r.i / kHkv;
  r.t = sorted ? static_cast<int>(sm.order[rank]) : total_tiles - 1 - rank;
  r.s = tile_seq(sm, p.num_seqs, r.t);
  // (read-only for the kernel's lifetime: through the non-coherent path)
  r.ctx = load_early(p.context_lens + r.s);
  r.row0 = load_early(p.cu_tokens + r.s);
  r.row_end = load_early(p.cu_tokens + r.s + 1);
  return r;
}

template <class Sm>
__device__ __forceinline__ Item decode_item(const Sm &sm, const ItemRef &r) {
  Item it;
  it.g = r.i % kHkv;
  it.s = r.s;
  it.t0 = (r.t - sm.tile_prefix[r.s]) * kCtaTok;
  it.ctx = r.ctx;
  it.row0 = r.row0;
  const int n = r.row_end - r.row0;
  it.rows0 = min(kQTok, n - it.t0);
  it.rows1 = min(kQTok, n - it.t0 - kQTok);
  it.halves = it.rows1 > 0 ? 2 : 1;
  it.n_keys0 = it.ctx + it.t0 + it.rows0;
  it.n_keys = it.halves == 2 ? it.ctx + it.t0 + kQTok + it.rows1 : it.n_keys0;
  it.n_chunks = (it.n_keys + kChunk - 1) / kChunk;
  it.nc0 = (it.n_keys0 + kChunk - 1) / kChunk;
  it.nc1 = it.halves == 2 ? it.n_chunks : 0;
  return it;
}

// Pages of BT tokens: a chunk spans kChunk / BT pages; bit l of a stage's
// pmask says whether its page l was loaded.
template <int BT>
struct PageGeom {
  static constexpr int kPages = kChunk / BT;
  static constexpr int kAll = (1 << kPages) - 1;
};

// Query tiles per sequence laid end to end (sm.tile_prefix; sequences whose
// chunk is refused have none), and, up to kSortTiles tiles, their order by
// weight (sm.order).  Every thread of the CTA calls it; returns the number of
// tiles.
template <int BT, int kThreads, int kSort, class Sm>
__device__ __forceinline__ int order_tiles(Sm &sm, const PrefillParams &p, int tid, int warp,
                                           int lane) {
  const long long cap = static_cast<long long>(p.max_blocks) * BT;
  int carry = 0;
  for (int base = 0; base < p.num_seqs; base += kThreads) {
    const int i = base + tid;
    int tiles = 0;
    if (i < p.num_seqs) {
      const int ctx = p.context_lens[i];
      const int c0 = p.cu_tokens[i], c1 = p.cu_tokens[i + 1];
      const int n = c1 - c0;
      // a chunk that does not fit its table, or rows outside [0, total_tokens), is refused
      if (ctx >= 0 && n >= 0 && c0 >= 0 && c1 <= p.total_tokens &&
          static_cast<long long>(ctx) + n <= cap)
        tiles = (n + kCtaTok - 1) / kCtaTok;
      else if (blockIdx.x == 0)
        report(p.err, PA_DEV_CTX_RANGE);
    }
    int incl = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) sm.warp_sum[warp] = incl;
    __syncthreads();
    int before = 0, chunk = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      const int v = sm.warp_sum[w];
      if (w < warp) before += v;
      chunk += v;
    }
    if (i < p.num_seqs) sm.tile_prefix[i + 1] = carry + before + incl;
    carry += chunk;
    __syncthreads();
  }
  if (tid == 0) sm.tile_prefix[0] = 0;
  const int total_tiles = carry;
  __syncthreads();
  if (static_cast<int>(blockIdx.x) >= total_tiles * kHkv) return total_tiles;

  // ---- the tiles heaviest first: a stable counting sort by weight
  const bool sorted = total_tiles <= kSort;
  if (sorted) {
    for (int b = tid; b < kWeightBins; b += kThreads) sm.bin_start[b] = 0;
    __syncthreads();
    for (int t = tid; t < total_tiles; t += kThreads) {
      const int bn = tile_bin(sm, p, t);
      sm.tile_bins[t] = static_cast<uint8_t>(bn);
      atomicAdd(&sm.bin_start[bn], 1);
    }
    __syncthreads();
    if (warp == 0) {
      // exclusive prefix sum over the bins (16 consecutive bins per lane)
      constexpr int kPer = kWeightBins / 32;
      int cnt[kPer];
      int sum = 0;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        cnt[e] = sm.bin_start[lane * kPer + e];
        sum += cnt[e];
      }
      int incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      int run = incl - sum;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        sm.bin_start[lane * kPer + e] = run;
        run += cnt[e];
      }
      __syncwarp();
      // 32 tiles at a time in tile order: a tile's place is its bin's next
      // free place plus the number of lower lanes with the same bin
      for (int base = 0; base < total_tiles; base += 32) {
        const int t = base + lane;
        const int bn = t < total_tiles ? static_cast<int>(sm.tile_bins[t]) : -1;
        const unsigned peers = __match_any_sync(0xffffffffu, bn);
        const int rank = __popc(peers & ((1u << lane) - 1u));
        const int at = t < total_tiles ? sm.bin_start[bn] + rank : 0;
        __syncwarp();
        if (t < total_tiles) {
          sm.order[at] = static_cast<uint16_t>(t);
          if (rank == 0) sm.bin_start[bn] += __popc(peers);
        }
        __syncwarp();
      }
    }
    __syncthreads();
  }
  return total_tiles;
}

// Tensor map over q [total_tokens][32][64] bf16: box (64, 4 heads, 32 tokens)
// = one GQA group's rows of a half tile, 128-byte swizzle; rows past the
// end read as zeros.
int make_q_map(CUtensorMap *map, const void *q, int total_tokens) {
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
  const cuuint64_t dims[3] = {kD, kHq, static_cast<cuuint64_t>(total_tokens)};
  const cuuint64_t strides[2] = {kHeadRowBytes, static_cast<cuuint64_t>(kHq) * kHeadRowBytes};
  const cuuint32_t box[3] = {kD, kGqa, kQTok};
  const cuuint32_t estr[3] = {1, 1, 1};
  CUresult rr = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(q), dims, strides,
                   box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return rr == CUDA_SUCCESS ? PA_OK : PA_ERR_CUDA;
}

}  // namespace
}  // namespace pa
