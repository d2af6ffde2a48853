// pa_append_shared.cuh -- what the bf16 and the 8-bit cache appends share: the
// page allocation kernels (decode and prefill) and the Llama-3-scaled RoPE
// (frequencies, angle, rotation of one head row).
#pragma once

#include <climits>
#include <cmath>

#include "pa_device.cuh"
#include "pa_host.h"

namespace pa {
namespace {

constexpr int kScanCta = 1024;

// Llama-3-scaled RoPE inverse frequencies of the 32 pairs, computed on the
// host in fp64 and passed by value (no device memory involved).
struct RopeFreqs {
  double f[PA_HEAD_DIM / 2];
};

struct AppendParams {
  RopeFreqs freqs;
  const uint16_t *k_new;
  const uint16_t *v_new;
  uint16_t *q;                 // may be null
  unsigned char *kv;
  int32_t *block_table;
  const int32_t *context_lens;
  int32_t *free_list;
  int32_t *free_count;
  int32_t *err;
  int num_blocks;
  int n_layers;
  int max_blocks;
  int num_seqs;
  int layer;
};

__device__ __forceinline__ size_t table_row(int s, int n_layers, int layer, int max_blocks) {
  return (static_cast<size_t>(s) * n_layers + layer) * static_cast<size_t>(max_blocks);
}

// Exclusive prefix count of `flag` over a 1024-thread CTA; also returns the
// CTA total.  `tot` is 32 ints of shared scratch.
__device__ __forceinline__ int cta_exclusive_count(bool flag, int *tot, int *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned bal = __ballot_sync(0xffffffffu, flag);
  const int before_in_warp = __popc(bal & ((1u << lane) - 1u));
  if (lane == 0) tot[warp] = __popc(bal);
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < kScanCta / 32; ++w) {
    const int t = tot[w];
    if (w < warp) before += t;
    all += t;
  }
  __syncthreads();
  *total = all;
  return before + before_in_warp;
}

template <int BT>
__global__ void __launch_bounds__(kScanCta) append_alloc_kernel(AppendParams p) {
  __shared__ int tot[kScanCta / 32];
  pdl_wait_primary();        // the table and free list may come from the previous kernel
  pdl_launch_dependents();   // the store kernel may start its rotations now
  const int cap = p.max_blocks * BT;
  // a count outside [0, num_blocks] never indexes past the free list
  const int fc0 = min(max(*p.free_count, 0), p.num_blocks);
  int served = 0;
  for (int base = 0; base < p.num_seqs; base += kScanCta) {
    const int i = base + threadIdx.x;
    int pos = 0;
    bool need = false;
    if (i < p.num_seqs) {
      pos = p.context_lens[i];
      const bool in_range = pos >= 0 && pos < cap;
      if (!in_range) report(p.err, PA_DEV_CTX_RANGE);
      need = in_range && (pos % BT == 0);
    }
    int chunk = 0;
    const int rank = served + cta_exclusive_count(need, tot, &chunk);
    if (need) {
      int32_t *entry = p.block_table + table_row(i, p.n_layers, p.layer, p.max_blocks) + pos / BT;
      if (rank < fc0) {
        const int blk = p.free_list[fc0 - 1 - rank];
        *entry = blk;
        if (blk < 0 || blk >= p.num_blocks) report(p.err, PA_DEV_BAD_BLOCK);
      } else {
        *entry = -1;   // refused: the page stays unassigned
        report(p.err, PA_DEV_FREE_UNDERFLOW);
      }
    }
    served += chunk;
  }
  if (threadIdx.x == 0) *p.free_count = max(fc0 - served, 0);
}

// Llama 3 rescaling of the RoPE inverse frequency of pair i (head_dim 64):
// theta 500000, factor 32, low_freq_factor 1, high_freq_factor 4, original
// context 8192.  Wavelengths under 8192/4 keep their frequency, those over
// 8192/1 are slowed by the factor, and the band between blends the two
// linearly in 8192/wavelength.  Host code, run once.
RopeFreqs llama3_freqs() {
  RopeFreqs r;
  const double theta = 500000.0, factor = 32.0, low = 1.0, high = 4.0, orig = 8192.0;
  const double two_pi = 6.283185307179586476925;
  for (int i = 0; i < kD / 2; ++i) {
    const double f = std::pow(theta, -static_cast<double>(2 * i) / kD);
    const double wavelen = two_pi / f;
    if (wavelen < orig / high) {
      r.f[i] = f;
    } else if (wavelen > orig / low) {
      r.f[i] = f / factor;
    } else {
      const double w = (orig / wavelen - low) / (high - low);
      r.f[i] = (1.0 - w) * (f / factor) + w * f;
    }
  }
  return r;
}

__device__ __forceinline__ float bf16_bits_to_float(uint32_t b) { return __uint_as_float(b << 16); }

__device__ __forceinline__ uint32_t float_to_bf16_bits(float x) {
  __nv_bfloat16 h = __float2bfloat16_rn(x);
  return *reinterpret_cast<uint16_t *>(&h);
}

// Rotate 4 consecutive pairs (d, d + 32), d = 4j..4j+3, of one head row.
__device__ __forceinline__ void rotate4(uint2 lo, uint2 hi, const float2 *cs, int j, uint2 *out_lo,
                                        uint2 *out_hi) {
  const uint32_t lw[2] = {lo.x, lo.y}, hw[2] = {hi.x, hi.y};
  uint32_t ol[2], oh[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    uint32_t rl = 0, rh = 0;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const float a = bf16_bits_to_float((lw[w] >> (16 * half)) & 0xffffu);
      const float b = bf16_bits_to_float((hw[w] >> (16 * half)) & 0xffffu);
      const float2 c = cs[4 * j + 2 * w + half];   // (cos, sin)
      const float ra = fmaf(a, c.x, -b * c.y);
      const float rb = fmaf(b, c.x, a * c.y);
      rl |= float_to_bf16_bits(ra) << (16 * half);
      rh |= float_to_bf16_bits(rb) << (16 * half);
    }
    ol[w] = rl;
    oh[w] = rh;
  }
  *out_lo = make_uint2(ol[0], ol[1]);
  *out_hi = make_uint2(oh[0], oh[1]);
}

// (cos, sin) of the angle pos * f.  The angle is formed and reduced modulo
// 2*pi in fp64, so that positions in the tens of thousands keep their phase.
// The reduction is Cody and Waite's (W. J. Cody, W. Waite, "Software Manual
// for the Elementary Functions", 1980): 2*pi is split into a double head and
// the double nearest to the rest, and k*2*pi is taken off in two fused
// multiply-adds, head first.  The reduced angle (|r| <= pi) goes through
// fp32 sincosf, with a first-order correction for the part of it fp32 could
// not hold.
__device__ __forceinline__ float2 rope_cos_sin(int pos, double f) {
  const double two_pi_hi = 6.283185307179586232, two_pi_lo = 2.4492935982947064e-16;
  const double a = static_cast<double>(pos) * f;
  const double k = rint(a * 0.15915494309189533577);
  const double red = fma(-k, two_pi_lo, fma(-k, two_pi_hi, a));
  const float rf = static_cast<float>(red);
  const float rerr = static_cast<float>(red - static_cast<double>(rf));   // |rerr| <= 2^-23
  float sn, cn;
  sincosf(rf, &sn, &cn);
  return make_float2(fmaf(-sn, rerr, cn), fmaf(cn, rerr, sn));
}

// ------------------------------------------------------------------ prefill
// A prompt chunk per sequence: the tokens of sequence s are rows
// cu_tokens[s] .. cu_tokens[s+1]-1, at positions context_lens[s] + i.

struct PrefillAppendParams {
  RopeFreqs freqs;
  const uint16_t *k_new;
  const uint16_t *v_new;
  uint16_t *q;                 // may be null
  unsigned char *kv;
  int32_t *block_table;
  const int32_t *cu_tokens;
  const int32_t *context_lens;
  int32_t *free_list;
  int32_t *free_count;
  int32_t *err;
  int total_tokens;
  int num_blocks;
  int n_layers;
  int max_blocks;
  int num_seqs;
  int layer;
};

// Whether sequence s's chunk is accepted: it fits the sequence's table (of
// max_blocks pages of BT tokens) and its rows lie inside [0, total_tokens).
// Sets the context and chunk length.
template <int BT>
__device__ __forceinline__ bool chunk_fits(const PrefillAppendParams &p, int s, int *ctx, int *n) {
  const int c0 = p.cu_tokens[s], c1 = p.cu_tokens[s + 1];
  *ctx = p.context_lens[s];
  *n = c1 - c0;
  return *ctx >= 0 && *n >= 0 && c0 >= 0 && c1 <= p.total_tokens &&
         static_cast<long long>(*ctx) + *n <= static_cast<long long>(p.max_blocks) * BT;
}

template <int BT>
__global__ void __launch_bounds__(kScanCta) prefill_alloc_kernel(PrefillAppendParams p) {
  __shared__ int tot[kScanCta / 32];
  __shared__ int incl_s[kScanCta];    // pages of the batch's sequences up to and including each
  __shared__ int first_s[kScanCta];   // each sequence's first new page
  pdl_wait_primary();        // the table and free list may come from the previous kernel
  pdl_launch_dependents();   // the store kernel may start its rotations now
  const int fc0 = min(max(*p.free_count, 0), p.num_blocks);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int served = 0;
  for (int base = 0; base < p.num_seqs; base += kScanCta) {
    const int s = base + threadIdx.x;
    int ctx = 0, n = 0, first = 0, pages = 0;
    if (s < p.num_seqs) {
      if (!chunk_fits<BT>(p, s, &ctx, &n)) {
        report(p.err, PA_DEV_CTX_RANGE);
      } else {
        first = (ctx + BT - 1) / BT;                 // pages already open
        pages = (ctx + n + BT - 1) / BT - first;     // pages this chunk opens
      }
    }
    // pages are ranked over the sequences in order: a prefix sum
    int incl = pages;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) tot[warp] = incl;
    __syncthreads();
    int before = 0, chunk = 0;
    for (int w = 0; w < kScanCta / 32; ++w) {
      const int t = tot[w];
      if (w < warp) before += t;
      chunk += t;
    }
    incl_s[threadIdx.x] = before + incl;
    first_s[threadIdx.x] = first;
    __syncthreads();
    // every thread takes pages e, e + 1024, ... of the batch: page e belongs
    // to the first sequence k of the batch with incl_s[k] > e
    for (int e = threadIdx.x; e < chunk; e += kScanCta) {
      int lo = 0, hi = kScanCta - 1;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (incl_s[mid] > e) hi = mid;
        else lo = mid + 1;
      }
      const int j = e - (lo > 0 ? incl_s[lo - 1] : 0);
      int32_t *entry =
          p.block_table + table_row(base + lo, p.n_layers, p.layer, p.max_blocks) + first_s[lo] + j;
      const int rank = served + e;
      if (rank < fc0) {
        const int blk = p.free_list[fc0 - 1 - rank];
        *entry = blk;
        if (blk < 0 || blk >= p.num_blocks) report(p.err, PA_DEV_BAD_BLOCK);
      } else {
        *entry = -1;   // refused: the page stays unassigned
        report(p.err, PA_DEV_FREE_UNDERFLOW);
      }
    }
    served += chunk;
    __syncthreads();
  }
  if (threadIdx.x == 0) *p.free_count = max(fc0 - served, 0);
}

}  // namespace
}  // namespace pa
