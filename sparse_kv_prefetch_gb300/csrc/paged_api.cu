// C ABI of the paged cache: argument checks and launches of dd_paged_*.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "paged.cuh"

namespace dd {
namespace paged {

dd_status resolve(const dd_paged_shape* s, Dims* o) {
  if (!s || !o) return DD_ERR_INVALID_ARG;
  if (s->batch < 1 || s->n_q_heads < 1 || s->n_kv_heads < 1 || s->head_dim < 1 ||
      s->page_size < 1 || s->n_pages < 1 || s->max_pages < 1)
    return DD_ERR_INVALID_ARG;
  if (s->n_q_heads % s->n_kv_heads != 0) return DD_ERR_INVALID_ARG;
  if (s->dtype != DD_F32 && s->dtype != DD_BF16) return DD_ERR_UNSUPPORTED;
  if (s->format != DD_PAGES_PLAIN && s->format != DD_PAGES_Q4) return DD_ERR_UNSUPPORTED;
  if (s->format == DD_PAGES_Q4 && s->dtype != DD_BF16) return DD_ERR_UNSUPPORTED;
  const int G = s->n_q_heads / s->n_kv_heads;
  if (G != 1 && G != 2 && G != 4 && G != 8) return DD_ERR_UNSUPPORTED;
  if (s->head_dim != 64 && s->head_dim != 128 &&
      !(s->head_dim == 256 && s->dtype == DD_BF16))
    return DD_ERR_UNSUPPORTED;
  if (s->page_size != 16 && s->page_size != 32 && s->page_size != 64 && s->page_size != 128)
    return DD_ERR_UNSUPPORTED;
  if ((long long)s->max_pages * s->page_size > (1 << 30) ||
      (long long)s->n_pages * s->n_kv_heads > (1 << 30) / s->page_size)
    return DD_ERR_UNSUPPORTED;
  if ((long long)s->batch * s->n_kv_heads > (1 << 24)) return DD_ERR_UNSUPPORTED;
  Dims d;
  d.B = s->batch;
  d.Hq = s->n_q_heads;
  d.Hkv = s->n_kv_heads;
  d.G = G;
  d.d = s->head_dim;
  d.page = s->page_size;
  d.log2_page = ilog2(d.page);
  d.n_pages = s->n_pages;
  d.max_pages = s->max_pages;
  d.dtype = s->dtype;
  d.format = s->format;
  d.elt = s->dtype == DD_BF16 ? 2 : 4;
  d.row_bytes = s->format == DD_PAGES_Q4 ? d.d / 2 : d.d * d.elt;
  d.block_bytes = (size_t)d.page * (s->format == DD_PAGES_Q4 ? d.d / 2 + d.d / 8 : d.d * d.elt);
  d.cap = d.max_pages * d.page;
  *o = d;
  return DD_OK;
}

Plan attn_plan(const Dims& d, int max_q, int max_kv, int window, int sinks) {
  const long long rows = (long long)max_q * d.G;
  max_kv = std::min(max_kv, 1 << 30);  // positions end there
  Plan p;
  // At most 16 rows share a key: reading the keys bounds the call.  More: the
  // products do.  4-bit pages stay with the kernel for few rows up to 32, 16 at a
  // time (4 x 5 tokens, 32 / 8 heads, over 65536 keys: 330 to 350 us against 364 on
  // tcgen05, over 4000 keys 31 against 42; with 12 tokens 387 and 369; bf16 188
  // and 179), and fp32 always: its products do not run on tcgen05.  (On the CUDA
  // cores, 64 rows to a CTA, 2048 and 700 tokens took 1402 us with d = 128 and 691
  // with d = 64, where this takes 1450 and 503; 980 tokens of 4 heads 260 and 122,
  // here 68 and 31.)
  const bool q4 = d.format == DD_PAGES_Q4;
  p.path = d.dtype == DD_F32 || rows <= (q4 ? 32 : 16) ? kDecode : kPrefill;
  // How far the keys are split, by an estimate in ns from rates (bytes of keys and
  // values a ns) that were measured with d = 128 and 32 query heads on 8 KV heads,
  // and are taken for the other shapes too:
  //   plain pages: the card's 6500, or a CTA's 64 where its share takes longer (so
  //     too for fp32 calls of many rows, which arithmetic bounds);
  //   4-bit pages: 21 an SM, 16 for a CTA alone on one, the fullest SM counting;
  //   many rows a key: 13 ns a key for a CTA's 256 rows, 34 over 4-bit pages;
  //   a wave of CTAs takes 4000 more (8000 with many rows), a second kernel 5500
  //     and the partials.
  // Of the splits within 4 % of the cheapest the most: sequences are shorter than
  // max_kv by their own measure, and many CTAs even them out.  Measured with the
  // number given by hand: 8 x 131072 keys, 4 splits (one cluster each) 500 us, 8
  // 512, 19 510, 38 512 (the rule takes 22), but 1 of 8 sequences that long 263,
  // 138, 90, 90; in 4 bits 480, 392, 352, 329; 32 x 4100 keys 97, 111, 108, 143,
  // and unsplit 83 (the rule leaves them whole).
  const bool decode = p.path == kDecode;
  const int cta_rows = p.path == kPrefill ? prefill_rows(d) : rows <= 8 ? 8 : 16;
  const long long at_once = (long long)kSms * (decode ? decode_ctas(d, rows <= 8 ? 1 : 2) : 1);
  const long long ctas = (long long)d.B * d.Hkv * ((rows + cta_rows - 1) / cta_rows);
  const double key_bytes = 2.0 * (double)d.block_bytes / d.page;
  const long long least = decode ? 128 : 1024;
  auto cost = [&](long long keys, long long n) {
    const double share = (double)((keys + n - 1) / n);
    const double waves = (double)((ctas * n + at_once - 1) / at_once);
    const double an_sm = (double)((ctas * n + kSms - 1) / kSms);
    double ns;
    if (!decode)
      ns = waves * (share * (q4 ? 34 : 13) + 8000);
    else if (q4)
      ns = an_sm * share * key_bytes / (an_sm > 1 ? 21 : 16) + 4000 * waves;
    else
      ns = std::max(ctas * (double)keys * key_bytes / 6500, share * key_bytes / 64) + 4000 * waves;
    if (n > 1 && !(decode && n <= kClusterSplits))
      ns += 5500 + (double)n * d.B * max_q * d.Hq * d.d * 8 / 5000;
    return ns;
  };
  // How many keys one split takes at most, whatever that costs.  A tensor core adds
  // each term to a sum with what the sum's last place (and two bits more) leaves of it,
  // cut, so an accumulator loses some 2^-27.5 of itself a key: 0.08 % measured after
  // 2^17 keys of equal weights, 0.6 % after 2^20, 2.5 % after 2^22.  2^18 for the prompt
  // kernel's one accumulator, 2^20 for the four warps' of the other; fp32 adds round
  // instead, and 2^17 keys are 2^11 of them for a warp, 2e-5 measured.
  const long long longest = !decode ? 1 << 18 : d.dtype == DD_F32 ? 1 << 17 : 1 << 20;
  // Tried: every number up to 16, then each some 1/8 above the last.
  auto split = [&](long long keys, int most) {
    const int need = (int)((keys + longest - 1) / longest);
    if (need > kMaxSplits) return need;
    const int top = (int)std::max(1ll, std::min((long long)most, (keys + least - 1) / least));
    int tried[64], k = 0;
    double ns[64], best = 0;
    for (int n = 1; n <= top; n += n < 16 ? 1 : n / 8, ++k) {
      tried[k] = n;
      ns[k] = cost(keys, n);
      if (k == 0 || ns[k] < best) best = ns[k];
    }
    while (ns[--k] > 1.04 * best) {
    }
    return std::max(tried[k], need);
  };
  p.nsplit = split(max_kv, kMaxSplits);
  // A window leaves fewer keys; never more splits, for the workspace's sake.
  if (window > 0)
    p.nsplit = split(std::min((long long)max_kv, (long long)window + max_q + sinks), p.nsplit);
  p.merged = p.nsplit > 1 && !(p.path == kDecode && p.nsplit <= kClusterSplits);
  return p;
}

}  // namespace paged
}  // namespace dd

using namespace dd;
using dd::paged::AppendArgs;
using dd::paged::AttnArgs;
using dd::paged::Seqs;

namespace {

constexpr int kMaxTokens = 1 << 30;

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
dd_status cuda_status(cudaError_t e) { return e == cudaSuccess ? DD_OK : DD_ERR_CUDA; }
size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// The device arrays of a call; q_start may be absent where it is not read.
dd_status resolve_seqs(const paged::Dims& d, const dd_paged_seqs* s, int n_tokens, bool need_q,
                       Seqs* o) {
  if (!s || !s->seq_len || !s->page_table || !s->k_pages || !s->v_pages) return DD_ERR_INVALID_ARG;
  if (need_q && !s->q_start) return DD_ERR_INVALID_ARG;
  if (!aligned16(s->k_pages) || !aligned16(s->v_pages) || !aligned4(s->q_start) ||
      !aligned4(s->seq_len) || !aligned4(s->page_table))
    return DD_ERR_INVALID_ARG;
  if (!all_device({s->seq_len, s->page_table, s->k_pages, s->v_pages})) return DD_ERR_INVALID_ARG;
  if (need_q && !is_device_ptr(s->q_start)) return DD_ERR_INVALID_ARG;
  *o = Seqs{s->q_start, s->seq_len, s->page_table, static_cast<unsigned char*>(s->k_pages),
            static_cast<unsigned char*>(s->v_pages), d.B, n_tokens, d.log2_page, d.n_pages,
            d.max_pages, d.cap, d.block_bytes};
  return DD_OK;
}

// A token stride in elements: at least the heads' elements, whole 16-byte pieces.
bool stride_ok(int64_t stride, int heads, const paged::Dims& d) {
  return stride >= (int64_t)heads * d.d && stride < (1ll << 38) && stride * d.elt % 16 == 0;
}

struct AttnWs {
  size_t ml, total;
};
AttnWs attn_ws(const paged::Dims& d, int n_tokens, const paged::Plan& p) {
  if (!p.merged) return AttnWs{0, 0};
  const size_t rows = (size_t)p.nsplit * n_tokens * d.Hq;
  AttnWs w;
  w.ml = align256(rows * d.d * sizeof(float));
  w.total = w.ml + align256(rows * sizeof(float2));
  return w;
}

}  // namespace

extern "C" {

dd_status dd_paged_pool_bytes(const dd_paged_shape* shape, size_t* bytes) {
  if (!bytes) return DD_ERR_INVALID_ARG;
  paged::Dims d;
  const dd_status st = paged::resolve(shape, &d);
  if (st != DD_OK) return st;
  *bytes = (size_t)d.n_pages * d.Hkv * d.block_bytes;
  return DD_OK;
}

dd_status dd_paged_append(const dd_paged_shape* shape, const dd_paged_seqs* seqs,
                          int32_t n_tokens, const void* q, const void* k, const void* v,
                          int64_t q_stride, int64_t k_stride, int64_t v_stride, void* q_out,
                          const float* rope, int32_t rope_len, int32_t rot_dim, int interleaved,
                          dd_stream_t stream) {
  paged::Dims d;
  dd_status st = paged::resolve(shape, &d);
  if (st != DD_OK) return st;
  if (n_tokens < 0 || n_tokens > kMaxTokens) return DD_ERR_INVALID_ARG;
  if (interleaved != 0 && interleaved != 1) return DD_ERR_INVALID_ARG;
  if (rope ? (rope_len < 1 || rot_dim < 1 || rot_dim > d.d) : (rope_len != 0 || rot_dim != 0))
    return DD_ERR_INVALID_ARG;
  if (rot_dim % 16 != 0) return DD_ERR_UNSUPPORTED;
  if (n_tokens == 0) return DD_OK;
  if (!k || !v || (q == nullptr) != (q_out == nullptr)) return DD_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(rope))
    return DD_ERR_INVALID_ARG;
  if ((q && !stride_ok(q_stride, d.Hq, d)) || !stride_ok(k_stride, d.Hkv, d) ||
      !stride_ok(v_stride, d.Hkv, d))
    return DD_ERR_INVALID_ARG;
  if (q && q == q_out && q_stride != (int64_t)d.Hq * d.d) return DD_ERR_INVALID_ARG;
  if (paged::append_blocks(d, n_tokens, q != nullptr) > paged::kMaxBlocks)
    return DD_ERR_UNSUPPORTED;
  Seqs s;
  st = resolve_seqs(d, seqs, n_tokens, true, &s);
  if (st != DD_OK) return st;
  if (!all_device({q, k, v, q_out, rope})) return DD_ERR_INVALID_ARG;
  const AppendArgs a{q, k, v, q_out, q_stride * d.elt, k_stride * d.elt, v_stride * d.elt, rope,
                     rope_len, rot_dim, interleaved};
  return cuda_status(launch_append(d, s, a, reinterpret_cast<cudaStream_t>(stream)));
}

dd_status dd_paged_read(const dd_paged_shape* shape, const dd_paged_seqs* seqs, int32_t first,
                        int32_t count, void* k_out, void* v_out, dd_stream_t stream) {
  paged::Dims d;
  dd_status st = paged::resolve(shape, &d);
  if (st != DD_OK) return st;
  if (first < 0 || count < 0 || first > kMaxTokens || count > kMaxTokens) return DD_ERR_INVALID_ARG;
  if (count == 0) return DD_OK;
  if (!k_out || !v_out || !aligned16(k_out) || !aligned16(v_out)) return DD_ERR_INVALID_ARG;
  if (paged::read_blocks(d, count) > paged::kMaxBlocks) return DD_ERR_UNSUPPORTED;
  Seqs s;
  st = resolve_seqs(d, seqs, 0, false, &s);
  if (st != DD_OK) return st;
  if (!all_device({k_out, v_out})) return DD_ERR_INVALID_ARG;
  return cuda_status(launch_read(d, s, first, count, k_out, v_out,
                                 reinterpret_cast<cudaStream_t>(stream)));
}

dd_status dd_paged_attn_workspace_size(const dd_paged_shape* shape, int32_t n_tokens,
                                       int32_t max_q_len, int32_t max_kv_len, size_t* bytes) {
  if (!bytes) return DD_ERR_INVALID_ARG;
  paged::Dims d;
  const dd_status st = paged::resolve(shape, &d);
  if (st != DD_OK) return st;
  if (n_tokens < 0 || n_tokens > kMaxTokens || max_q_len < 1 || max_kv_len < 0)
    return DD_ERR_INVALID_ARG;
  *bytes = attn_ws(d, n_tokens, paged::attn_plan(d, max_q_len, max_kv_len, 0, 0)).total;
  return DD_OK;
}

dd_status dd_paged_attn(const dd_paged_shape* shape, const dd_paged_seqs* seqs, int32_t n_tokens,
                        const void* q, int64_t q_stride, int32_t max_q_len, int32_t max_kv_len,
                        int32_t window, int32_t sinks, void* out, float* lse_out,
                        void* workspace, size_t ws_bytes, dd_stream_t stream) {
  paged::Dims d;
  dd_status st = paged::resolve(shape, &d);
  if (st != DD_OK) return st;
  if (n_tokens < 0 || n_tokens > kMaxTokens || max_q_len < 1 || max_kv_len < 0 || window < 0 ||
      sinks < 0)
    return DD_ERR_INVALID_ARG;
  if (n_tokens == 0) return DD_OK;
  if (!q || !out || !aligned16(q) || !aligned16(out) || !aligned4(lse_out) ||
      !aligned16(workspace) || !stride_ok(q_stride, d.Hq, d))
    return DD_ERR_INVALID_ARG;
  // Positions end below 2^30, so a wider window hides nothing.
  window = std::min(window, 1 << 30);
  sinks = std::min(sinks, 1 << 30);
  const paged::Plan p = paged::attn_plan(d, max_q_len, max_kv_len, window, sinks);
  if (p.merged && (long long)n_tokens * d.Hq > paged::kMaxBlocks) return DD_ERR_UNSUPPORTED;
  const AttnWs w = attn_ws(d, n_tokens, p);
  if (w.total > 0 && (!workspace || ws_bytes < w.total)) return DD_ERR_INVALID_ARG;
  Seqs s;
  st = resolve_seqs(d, seqs, n_tokens, true, &s);
  if (st != DD_OK) return st;
  if (!all_device({q, out, lse_out, workspace})) return DD_ERR_INVALID_ARG;
  char* ws = static_cast<char*>(workspace);
  const AttnArgs a{q, q_stride * d.elt, out, lse_out,
                   p.merged ? reinterpret_cast<float*>(ws) : nullptr,
                   p.merged ? reinterpret_cast<float2*>(ws + w.ml) : nullptr, max_q_len,
                   window, sinks, p.nsplit};
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = p.path == paged::kPrefill ? launch_attn_prefill(d, s, a, cs)
                                            : launch_attn_decode(d, s, a, cs);
  if (e == cudaSuccess && p.merged) e = launch_attn_merge(d, s, a, cs);
  return cuda_status(e);
}

}  // extern "C"
