// Paged caches: what the append, read and attention kernels share.
#pragma once

#include "dd_internal.cuh"

namespace dd {
namespace paged {

// Multiprocessors of the card this is written for: work is cut by it (and
// not by the device in use, so that workspace sizes need none).
constexpr int kSms = 152;

// Resolved shape of a paged cache.
struct Dims {
  int B, Hq, Hkv, G, d, page, log2_page, n_pages, max_pages, dtype, format;
  int elt;              // bytes of an element of q, k, v, out and plain pages
  int row_bytes;        // bytes of one position's row in a block (codes only in 4-bit pages)
  size_t block_bytes;   // bytes of one (page, KV head) block
  int cap;              // positions a page table row covers
};

dd_status resolve(const dd_paged_shape* s, Dims* out);

// The device arrays of a call, as the kernels take them.
struct Seqs {
  const int32_t* q_start;
  const int32_t* seq_len;
  const int32_t* table;
  unsigned char* k;
  unsigned char* v;
  int B, n_tokens, log2_page, n_pages, max_pages, cap;
  size_t block_bytes;
};

struct AppendArgs {
  const void *q, *k, *v;
  void* q_out;
  int64_t q_stride, k_stride, v_stride;  // bytes
  const float* rope;
  int rope_len, rot_dim, interleaved;
};
// CTAs that a call takes; the launches need kMaxBlocks at most.
constexpr long long kMaxBlocks = 0x7FFFFFFF;
long long append_blocks(const Dims& d, int n_tokens, bool with_q);
long long read_blocks(const Dims& d, int count);
cudaError_t launch_append(const Dims& d, const Seqs& s, const AppendArgs& a, cudaStream_t st);

cudaError_t launch_read(const Dims& d, const Seqs& s, int first, int count, void* k_out,
                        void* v_out, cudaStream_t st);

// Attention of one call.  Partials of a split call: part_o
// [nsplit][n_tokens][H_q][d] and part_ml [nsplit][n_tokens][H_q] as (max, sum),
// or NULL where the splits are a cluster that merges them itself.
struct AttnArgs {
  const void* q;
  int64_t q_stride;  // bytes
  void* out;
  float* lse;  // may be NULL
  float* part_o;
  float2* part_ml;
  int max_q, window, sinks, nsplit;
};
// Which kernel computes a call and how far it is split over the keys.
enum Path { kDecode, kPrefill };
constexpr int kMaxSplits = 128;
constexpr int kClusterSplits = 8;  // the largest cluster every device setting allows
struct Plan {
  Path path;
  int nsplit;
  bool merged;  // by a second kernel, through the workspace
};
Plan attn_plan(const Dims& d, int max_q, int max_kv, int window, int sinks);
cudaError_t launch_attn_decode(const Dims& d, const Seqs& s, const AttnArgs& a, cudaStream_t st);
cudaError_t launch_attn_prefill(const Dims& d, const Seqs& s, const AttnArgs& a, cudaStream_t st);
int prefill_rows(const Dims& d);          // rows of a CTA
int decode_ctas(const Dims& d, int nr);   // CTAs of an SM (8 nr rows each)
cudaError_t launch_attn_merge(const Dims& d, const Seqs& s, const AttnArgs& a, cudaStream_t st);

// ----------------------------------------------------------------- device

// A sequence's part of the call.
struct Seq {
  int q0, nq;  // its tokens
  int pos0;    // position of the first of them (negative: before the sequence's start)
  int len;     // positions with a table entry
};
constexpr int kMaxLen = 1 << 30;

__device__ __forceinline__ Seq load_seq(const Seqs& s, int b) {
  Seq r;
  const int a = __ldg(s.q_start + b), e = __ldg(s.q_start + b + 1);
  const int n = min(max(__ldg(s.seq_len + b), 0), kMaxLen);
  r.q0 = min(max(a, 0), s.n_tokens);
  r.nq = min(max(e, r.q0), s.n_tokens) - r.q0;
  r.pos0 = n - r.nq;
  r.len = min(n, s.cap);
  return r;
}

// The page of position pos of sequence b, or -1 if it has none (0 <= pos < cap).
__device__ __forceinline__ int page_of(const Seqs& s, int b, int pos) {
  const int p = __ldg(s.table + (size_t)b * s.max_pages + (pos >> s.log2_page));
  return (unsigned)p < (unsigned)s.n_pages ? p : -1;
}

// The tiles of BN keys that a run of tokens at positions [pa, pb] reads: those
// of the sinks before the oldest window, then those from the window's start on.
struct KeyTiles {
  int lo, hi;    // positions [lo, hi) and [0, sinks) are visible to some token of the run
  int n_sink;    // sink tiles: 0 .. n_sink - 1
  int first;     // then tiles first .. first + n - n_sink - 1
  int n;
  __device__ __forceinline__ int tile(int i) const { return i < n_sink ? i : first + i - n_sink; }
  __device__ __forceinline__ bool any(int j, int sinks) const {
    return j < hi && (j >= lo || j < sinks);
  }
};
template <int BN>
__device__ __forceinline__ KeyTiles key_tiles(int pa, int pb, int len, int window, int sinks) {
  KeyTiles t;
  t.hi = max(0, min(pb + 1, len));
  t.lo = window > 0 ? min(max(0, pa - window + 1), t.hi) : 0;
  t.first = t.lo / BN;
  t.n_sink = min((min(sinks, t.lo) + BN - 1) / BN, t.first);
  t.n = t.n_sink + (t.hi + BN - 1) / BN - t.first;
  return t;
}
// Whether the token at position p sees position j.
__device__ __forceinline__ bool sees(int p, int j, int window, int sinks) {
  return j <= p && (window == 0 || j > p - window || j < sinks);
}

// m + s c, the value of a code, in fp32.
__device__ __forceinline__ float q4_value(float m, float s, uint32_t c) {
  return fmaf(s, (float)c, m);
}

// Two fp32 rounded to bf16, the first in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace paged
}  // namespace dd
