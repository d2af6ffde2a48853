// pa_append_q8.cu -- KV append with Llama-3-scaled RoPE into the 8-bit cache
// (pa_q8.cuh has the format).
//
// Both entry points run the page allocation kernel of the bf16 appends, then
// a store kernel launched with programmatic dependent launch:
//   append_store_q8_kernel   one CTA per sequence: rotates q and k, quantises
//                            k and v to the page's scale; where the new token
//                            needs a larger scale than the page has, the
//                            page's earlier tokens are brought to it.
//   prefill_store_q8_kernel  one CTA per window of BT packed rows: the runs of
//                            rows that fall into one page ("segments", as a
//                            rule one) are taken in turn; a segment's values
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
// 16 bytes (8 bf16) of one half of a head row, rotated against the other half.
__device__ __forceinline__ void rotate8(uint4 *lo, uint4 *hi, const float2 *cs, int c) {
  uint2 l0 = make_uint2(lo->x, lo->y), l1 = make_uint2(lo->z, lo->w);
  uint2 h0 = make_uint2(hi->x, hi->y), h1 = make_uint2(hi->z, hi->w);
  rotate4(l0, h0, cs, 2 * c, &l0, &h0);
  rotate4(l1, h1, cs, 2 * c + 1, &l1, &h1);
  *lo = make_uint4(l0.x, l0.y, l1.x, l1.y);
  *hi = make_uint4(h0.x, h0.y, h1.x, h1.y);
}

__device__ __forceinline__ uint32_t q8_top4(uint4 w, uint32_t top) {
  return q8_top(w.w, q8_top(w.z, q8_top(w.y, q8_top(w.x, top))));
}

// Threads of the prefill store: 32 (4 per kv head) for each row of a pass.
template <int BT>
struct StoreGeom {
  static constexpr int kThreads = BT == 8 ? 256 : 512;
  static constexpr int kPassRows = kThreads / 32;        // rows of k (and of v) a pass takes
  static constexpr int kPasses = BT / kPassRows;         // 1, 1, 2
  static constexpr int kQItems = BT * kHq * 4 / kThreads;   // 4, 4, 8 parts of q rows a thread
};

template <int BT>
__global__ void __launch_bounds__(StoreGeom<BT>::kThreads) prefill_store_q8_kernel(
    PrefillAppendParams p, Q8Out o) {
  using G = StoreGeom<BT>;
  constexpr size_t kHalfPage = static_cast<size_t>(BT) * kQ8TokBytes;
  __shared__ float2 cs[BT][kD / 2];
  __shared__ int row_seq[BT], row_pos[BT], row_len[BT];
  __shared__ uint32_t starts_s;
  __shared__ uint32_t top_s[2][kHkv];
  __shared__ int e_s[2][kHkv], held_s[2][kHkv];   // held: exponent of the page's scale so far
  __shared__ int blk_s;
  pdl_launch_dependents();   // the next kernel may start its own set-up
  const int tid = threadIdx.x;
  const int r0 = blockIdx.x * BT;
  // lane i: row r0 + i's sequence (the largest s with cu_tokens[s] <= r: an
  // empty chunk's start equals the next one's, so the search passes over it),
  // position, and whether a segment (a run of rows in one page) starts there
  if (tid < 32) {
    bool start = false;
    if (tid < BT) {
      const int r = r0 + tid;
      int seq = 0, pos = 0, len = 0;
      if (r < p.total_tokens) {
        int lo = 0, hi = p.num_seqs - 1;
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (p.cu_tokens[mid] <= r) lo = mid;
          else hi = mid - 1;
        }
        int ctx, n;
        const int c0 = p.cu_tokens[lo], c1 = p.cu_tokens[lo + 1];
        // a refused chunk is reported by the allocation kernel
        if (chunk_fits<BT>(p, lo, &ctx, &n) && r >= c0 && r < c1) {
          seq = lo;
          pos = ctx + (r - c0);
          start = r == c0 || pos % BT == 0;
          len = min(BT - pos % BT, c1 - r);
        }
      }
      row_seq[tid] = seq;
      row_pos[tid] = pos;
      row_len[tid] = len;
    }
    const unsigned m = __ballot_sync(0xffffffffu, start);
    if (tid == 0) starts_s = m;
  }
  __syncthreads();
  const int krow = tid >> 5, khead = (tid >> 2) & 7, c = tid & 3;
  for (unsigned left = starts_s; left; left &= left - 1) {
    const int at = __ffs(left) - 1;
    const int len = row_len[at], pos0 = row_pos[at], seq = row_seq[at];
    const size_t first = static_cast<size_t>(r0) + at;
    // every load of the segment is in flight before anything waits on one
    uint4 klo[G::kPasses], khi[G::kPasses], v0[G::kPasses], v1[G::kPasses];
    uint32_t top_k = 0, top_v = 0;
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
    uint4 qlo[4], qhi[4];
    auto load_q = [&](int base) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int item = tid + (base + i) * G::kThreads;
        const int t = item >> 7, h = (item >> 2) & 31;
        qlo[i] = qhi[i] = make_uint4(0, 0, 0, 0);
        if (p.q && t < len) {
          const uint16_t *row = p.q + ((first + t) * kHq + h) * kD;
          qlo[i] = *reinterpret_cast<const uint4 *>(row + 8 * c);
          qhi[i] = *reinterpret_cast<const uint4 *>(row + kD / 2 + 8 * c);
        }
      }
    };
    auto store_q = [&](int base) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int item = tid + (base + i) * G::kThreads;
        const int t = item >> 7, h = (item >> 2) & 31;
        if (p.q && t < len) {
          rotate8(&qlo[i], &qhi[i], cs[t], c);
          uint16_t *row = o.q_out + ((first + t) * kHq + h) * kD;
          *reinterpret_cast<uint4 *>(row + 8 * c) = qlo[i];
          *reinterpret_cast<uint4 *>(row + kD / 2 + 8 * c) = qhi[i];
        }
      }
    };
    load_q(0);
    if (tid < 2 * kHkv) top_s[tid >> 3][tid & 7] = 0u;
    for (int x = tid; x < len * (kD / 2); x += G::kThreads) {
      const int t = x / (kD / 2), d = x % (kD / 2);
      cs[t][d] = rope_cos_sin(pos0 + t, p.freqs.f[d]);
    }
    __syncthreads();
    // ---- the largest magnitudes of each head's keys and values
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
    // (q of the first rows while the table is read)
    store_q(0);
    __syncthreads();
    // ---- the page and its scales
    const int slot0 = pos0 % BT;
    if (tid < 2 * kHkv) {
      const bool opened = slot0 == 0;   // this call opens the page
      if (opened) pdl_wait_primary();   // its entry comes from the allocation kernel
      const int blk =
          p.block_table[table_row(seq, p.n_layers, p.layer, p.max_blocks) + pos0 / BT];
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
    __syncthreads();
    if (blk_s >= 0) {
      unsigned char *page = p.kv + static_cast<size_t>(blk_s) * 2 * kHalfPage;
      // ---- tokens that the page holds already are brought to its new scale
      if (slot0 != 0) {
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
      }
      const float inv_k = pow2(-e_s[0][khead]), inv_v = pow2(-e_s[1][khead]);
#pragma unroll
      for (int i = 0; i < G::kPasses; ++i) {
        const int t = krow + i * G::kPassRows;
        if (t >= len) continue;
        unsigned char *row = page + (slot0 + t) * kQ8TokBytes + khead * kQ8HeadBytes;
        if (held_s[0][khead] >= kMinExp) {
          rotate8(&klo[i], &khi[i], cs[t], c);
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
#pragma unroll
    for (int base = 4; base < G::kQItems; base += 4) {
      load_q(base);
      store_q(base);
    }
    __syncthreads();   // cs, top_s and the exponents are reused
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
  if (launch_pdl(prefill_store_q8_kernel<BT>, dim3((total_tokens + BT - 1) / BT),
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
