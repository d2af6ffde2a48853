// pa_append_q8.cu -- KV append with Llama-3-scaled RoPE into the 8-bit cache
// (pa_q8.cuh has the format).
//
// Both entry points run the page allocation kernel of the bf16 appends, then
// a store kernel launched with programmatic dependent launch:
//   append_store_q8_kernel   one CTA per sequence: rotates q and k, quantises
//                            k and v to the page's scale; where the new token
//                            needs a larger scale than the page has, the
//                            page's earlier tokens are brought to it.
//   prefill_store_q8_kernel  one CTA per page that the call's rows touch, half
//                            its warps on k and v, half on q; a page's values
//                            stay in registers between the maximum that sets
//                            the scale and the rounding.
// Both are bound by memory (large) or latency (small): a row costs 2 KiB of k
// and v read, 1 KiB of bytes written, 4 KiB of q read and 4 KiB written.
#include <cuda_fp16.h>

#include "pa_append_shared.cuh"
#include "pa_q8.cuh"

namespace pa {
namespace {

struct Q8Out {
  uint16_t *q_out;   // where rotated q goes (may be q itself)
  float *scales;
};

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
  if (tid < kD / 2) cs[tid] = rope_cos_sin(pos, p.freqs.f[tid]);
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

// The pairs (lo, hi) of one bf16 word each, rotated by (x, y) and (z, w).
__device__ __forceinline__ void rotate2(uint32_t *lo, uint32_t *hi, float4 cs) {
  const float2 a = bf16x2_to_float2(*lo), b = bf16x2_to_float2(*hi);
  *lo = float_to_bf16_bits(fmaf(a.x, cs.x, -b.x * cs.y)) |
        (float_to_bf16_bits(fmaf(a.y, cs.z, -b.y * cs.w)) << 16);
  *hi = float_to_bf16_bits(fmaf(b.x, cs.x, a.x * cs.y)) |
        (float_to_bf16_bits(fmaf(b.y, cs.z, a.y * cs.w)) << 16);
}

// 16 bytes (8 bf16) of one half of a head row, rotated against the other half.
__device__ __forceinline__ void rotate8(uint4 *lo, uint4 *hi, const RowAngles &r, int c) {
  rotate2(&lo->x, &hi->x, r.a[c]);
  rotate2(&lo->y, &hi->y, r.a[4 + c]);
  rotate2(&lo->z, &hi->z, r.a[8 + c]);
  rotate2(&lo->w, &hi->w, r.a[12 + c]);
}

__device__ __forceinline__ uint32_t q8_top4(uint4 w, uint32_t top) {
  return q8_top(w.w, q8_top(w.z, q8_top(w.y, q8_top(w.x, top))));
}

// A CTA takes the rows of one call that fall into one page.  Sequence s owns
// CTAs cu_tokens[s] / BT + 2 s and up: n rows touch at most n / BT + 2 pages, so
// the ranges do not meet, and total_tokens / BT + 2 num_seqs CTAs hold them all.
// Half its warps take k and v (two rows of each a warp, held in registers
// between the maximum that sets the scale and the rounding), half q; the angles
// (fp64, a tenth of the instructions but a quarter of the time on that pipe) are
// worked out once for both.  64 registers let two CTAs of 512 threads, 128 KiB of
// loads, be on the way per SM.  8 x 2048 tokens take 36.5 us, 184 MB at 5.1 TB/s
// (a CTA per window of rows with every warp on k, v and q in turn, 104 registers
// and one CTA an SM: 53 us); 31 tokens 8.9 us, the allocation and the loads one
// after another.
template <int BT>
struct StoreGeom {
  static constexpr int kThreads = 32 * BT;
  static constexpr int kRole = kThreads / 2;         // threads for k and v, threads for q
  static constexpr int kPassRows = kRole / 32;       // 4 threads per kv head and row
  static constexpr int kPasses = 2;
  static constexpr int kQBatch = 4;                  // parts of q rows a thread holds
  static constexpr int kQBatches = 2;
  static_assert(kPassRows * kPasses == BT && kRole * kQBatch * kQBatches == BT * kHq * 4, "");
};

template <int BT>
__global__ void __launch_bounds__(StoreGeom<BT>::kThreads, 1024 / StoreGeom<BT>::kThreads)
prefill_store_q8_kernel(PrefillAppendParams p, Q8Out o) {
  using G = StoreGeom<BT>;
  constexpr size_t kHalfPage = static_cast<size_t>(BT) * kQ8TokBytes;
  __shared__ RowAngles cs[BT];
  __shared__ int owner_s, ctx_s, n_s, row0_s;   // the sequence, its context, rows and first row
  __shared__ uint32_t top_s[2][kHkv];
  __shared__ int e_s[2][kHkv], held_s[2][kHkv];   // held: exponent of the page's scale so far
  __shared__ int blk_s;
  pdl_launch_dependents();   // the next kernel may start its own set-up
  const int tid = threadIdx.x;
  if (tid == 0) owner_s = -1;
  if (tid < 2 * kHkv) top_s[tid >> 3][tid & 7] = 0u;
  __syncthreads();
  int mine = -1, my_ctx = 0, my_n = 0;
  for (int s = tid; s < p.num_seqs; s += G::kThreads) {
    int ctx, n;
    // (a refused chunk is reported by the allocation kernel)
    if (!chunk_fits<BT>(p, s, &ctx, &n) || n == 0) continue;
    const long long j = static_cast<long long>(blockIdx.x) - (p.cu_tokens[s] / BT + 2ll * s);
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
  const int page_at = ctx / BT + static_cast<int>(blockIdx.x) - (row0_s / BT + 2 * seq);
  const int pos0 = max(ctx, page_at * BT);
  const int len = min(ctx + n_s, page_at * BT + BT) - pos0;
  const size_t first = static_cast<size_t>(row0_s) + (pos0 - ctx);   // packed row of pos0
  const int c = tid & 3;
  auto angles = [&]() {   // one pair a thread
    const int t = tid / (kD / 2), d = tid % (kD / 2);
    if (t < len) cs[t].set(d, rope_cos_sin(pos0 + t, p.freqs.f[d]));
  };

  if (tid >= G::kRole) {
    // ------------------------------------------------------------------- q
    const int qt = tid - G::kRole;
    uint4 lo[G::kQBatch], hi[G::kQBatch];
    auto q_at = [&](int i) -> size_t {   // item i of the thread: row, head, part c
      const int item = qt + i * G::kRole;
      return ((first + (item >> 7)) * kHq + ((item >> 2) & 31)) * kD + 8 * c;
    };
    auto held = [&](int i) { return p.q && ((qt + i * G::kRole) >> 7) < len; };
    auto load = [&](int base) {
#pragma unroll
      for (int i = 0; i < G::kQBatch; ++i) {
        lo[i] = hi[i] = make_uint4(0, 0, 0, 0);
        if (held(base + i)) {
          const uint16_t *row = p.q + q_at(base + i);
          lo[i] = *reinterpret_cast<const uint4 *>(row);
          hi[i] = *reinterpret_cast<const uint4 *>(row + kD / 2);
        }
      }
    };
    load(0);
    angles();
    __syncthreads();
#pragma unroll
    for (int b = 0; b < G::kQBatches; ++b) {
      if (b > 0) load(b * G::kQBatch);
#pragma unroll
      for (int i = 0; i < G::kQBatch; ++i) {
        const int it = b * G::kQBatch + i;
        if (!held(it)) continue;
        rotate8(&lo[i], &hi[i], cs[(qt + it * G::kRole) >> 7], c);
        uint16_t *row = o.q_out + q_at(it);
        *reinterpret_cast<uint4 *>(row) = lo[i];
        *reinterpret_cast<uint4 *>(row + kD / 2) = hi[i];
      }
    }
    pdl_wait_primary();
    return;
  }

  // -------------------------------------------------------------- k and v
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
  angles();
  // ---- the largest magnitudes of each head's keys (before the rotation) and values
  uint32_t top_k = 0, top_v = 0;
#pragma unroll
  for (int i = 0; i < G::kPasses; ++i) {
    top_k = q8_top4(khi[i], q8_top4(klo[i], top_k));
    top_v = q8_top4(v1[i], q8_top4(v0[i], top_v));
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
#pragma unroll
  for (int i = 0; i < G::kPasses; ++i) {   // (meanwhile)
    const int t = krow + i * G::kPassRows;
    if (t < len) rotate8(&klo[i], &khi[i], cs[t], c);
  }
  asm volatile("bar.sync 1, %0;" ::"n"(G::kRole) : "memory");
  if (blk_s >= 0) {
    unsigned char *page = p.kv + static_cast<size_t>(blk_s) * 2 * kHalfPage;
    // ---- tokens that the page holds already are brought to its new scale
    for (int x = tid; x < slot0 * 64; x += G::kRole) {   // 16-byte parts: 32 of K, 32 of V a token
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
        *reinterpret_cast<uint2 *>(row + 8 * c) =
            make_uint2(bf16x4_to_e4m3x4(klo[i].x, klo[i].y, inv_k),
                       bf16x4_to_e4m3x4(klo[i].z, klo[i].w, inv_k));
        *reinterpret_cast<uint2 *>(row + kD / 2 + 8 * c) =
            make_uint2(bf16x4_to_e4m3x4(khi[i].x, khi[i].y, inv_k),
                       bf16x4_to_e4m3x4(khi[i].z, khi[i].w, inv_k));
      }
      if (held_s[1][khead] >= kMinExp)
        *reinterpret_cast<uint4 *>(row + kHalfPage + 16 * c) =
            make_uint4(bf16x4_to_e4m3x4(v0[i].x, v0[i].y, inv_v),
                       bf16x4_to_e4m3x4(v0[i].z, v0[i].w, inv_v),
                       bf16x4_to_e4m3x4(v1[i].x, v1[i].y, inv_v),
                       bf16x4_to_e4m3x4(v1[i].z, v1[i].w, inv_v));
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
  const Q8Out o{q_out, kv_scales};
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
  if (num_seqs > (1 << 29)) return PA_ERR_ARG;   // the grid, total_tokens / BT + 2 num_seqs
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
  const Q8Out o{q_out, kv_scales};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (launch_pdl(prefill_alloc_kernel<BT>, dim3(1), dim3(kScanCta), 0, st, prm) != cudaSuccess)
    return PA_ERR_CUDA;
  if (launch_pdl(prefill_store_q8_kernel<BT>, dim3(total_tokens / BT + 2 * num_seqs),
                 dim3(StoreGeom<BT>::kThreads), 0, st, prm, o) != cudaSuccess)
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
