// The merge of a split dd_paged_attn call whose partials went through the
// workspace: out = sum_x e^(m_x - M) o_x / sum_x e^(m_x - M) l_x, M = max m_x,
// lse = M + log of the denominator.
#include <math.h>

#include "paged.cuh"

namespace dd {
namespace paged {
namespace {

// One CTA per (token, query head): the log-sum-exp merge of its partials.  The
// warps take every fourth split each, so that many loads are in flight: 256 rows
// of 22 splits 7.4 us, 25984 rows of 8 splits 38 us.
template <typename T, int D>
__global__ void __launch_bounds__(128)
    attn_merge_kernel(Seqs s, AttnArgs a, int Hq, long long rows) {
  __shared__ float o_sm[4][D];
  __shared__ float l_sm[4];
  const long long row = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = (int)(row / Hq);
  if (t < __ldg(s.q_start) || t >= __ldg(s.q_start + s.B)) return;
  float M = -INFINITY;
  for (int x = lane; x < a.nsplit; x += 32) M = fmaxf(M, a.part_ml[x * rows + row].x);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  const float base = M == -INFINITY ? 0.f : M;
  float L = 0.f;
  float acc[D / 32];
#pragma unroll
  for (int c = 0; c < D / 32; ++c) acc[c] = 0.f;
#pragma unroll 4
  for (int x = warp; x < a.nsplit; x += 4) {
    const float2 ml = a.part_ml[x * rows + row];
    const float* o = a.part_o + (x * rows + row) * D;
    const float w = ml.y == 0.f ? 0.f : __expf(ml.x - base);
    L = ml.y == 0.f ? L : fmaf(w, ml.y, L);
#pragma unroll
    for (int c = 0; c < D / 32; c += 2) {
      const float2 v = *reinterpret_cast<const float2*>(o + 32 * c + 2 * lane);
      acc[c] = ml.y == 0.f ? acc[c] : fmaf(w, v.x, acc[c]);  // nothing seen: o may be anything
      acc[c + 1] = ml.y == 0.f ? acc[c + 1] : fmaf(w, v.y, acc[c + 1]);
    }
  }
#pragma unroll
  for (int c = 0; c < D / 32; c += 2)
    *reinterpret_cast<float2*>(&o_sm[warp][32 * c + 2 * lane]) = make_float2(acc[c], acc[c + 1]);
  if (lane == 0) l_sm[warp] = L;
  __syncthreads();
  L = (l_sm[0] + l_sm[1]) + (l_sm[2] + l_sm[3]);
  const float inv = L == 0.f ? 0.f : 1.f / L;
  for (int d = 2 * threadIdx.x; d < D; d += 256) {
    float2 v = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      v.x += o_sm[w][d];
      v.y += o_sm[w][d + 1];
    }
    const size_t at = (size_t)row * D + d;
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<float2*>(static_cast<float*>(a.out) + at) =
          make_float2(v.x * inv, v.y * inv);
    else
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + at) =
          pack_bf16(v.x * inv, v.y * inv);
  }
  if (a.lse && threadIdx.x == 0) a.lse[row] = L == 0.f ? -INFINITY : M + logf(L);
}

template <typename T, int D>
cudaError_t launch(const Dims& d, const Seqs& s, const AttnArgs& a, cudaStream_t st) {
  static unsigned long long prepared = 0;
  cudaError_t e = prepare_kernel(attn_merge_kernel<T, D>, &prepared, 0);
  if (e != cudaSuccess) return e;
  const long long rows = (long long)s.n_tokens * d.Hq;
  attn_merge_kernel<T, D><<<(unsigned)rows, 128, 0, st>>>(s, a, d.Hq, rows);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_merge(const Dims& d, const Seqs& s, const AttnArgs& a, cudaStream_t st) {
  if (d.dtype == DD_BF16) {
    if (d.d == 64) return launch<bf16_t, 64>(d, s, a, st);
    if (d.d == 128) return launch<bf16_t, 128>(d, s, a, st);
    if (d.d == 256) return launch<bf16_t, 256>(d, s, a, st);
  } else {
    if (d.d == 64) return launch<float, 64>(d, s, a, st);
    if (d.d == 128) return launch<float, 128>(d, s, a, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace paged
}  // namespace dd
