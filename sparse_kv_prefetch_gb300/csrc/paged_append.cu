// dd_paged_append: rotate new queries and keys by their positions, store keys
// and values in the pages.
//
// A pair (a, b) of a head becomes (a cos - b sin, b cos + a sin) with the
// cosines and sines of the token's position read from a table.  Every product
// and sum is rounded by itself (no fused multiply-add), so that a result, and
// with it a 4-bit code at the border of two, is the same whoever computes it.
//
// The kernel moves bytes: per token (H_q + 2 H_kv) d elements are read and as
// many written, and one row of angles is shared by all heads.  A warp works on
// one token and one of its three parts (queries, keys, values).  A lane takes
// two 16-byte pieces of a head that are turned together (of a row that is
// stored in 4 bits one piece, four lanes a group of 32), the same ones in up to
// kHeads heads, so that their angles are read once; it asks for all of them
// before anything else, and only then follows the chain token -> sequence ->
// position -> page.  The token's sequence is found by all lanes at once: the
// number of sequences that end at or before it, counted by ballots over q_start.
//
// Measured (32 query heads on 8 KV heads, d = 128): 16384 tokens of bf16 74 us,
// 5.5 TB/s of the bytes that have to move (6.8 is what a copy reaches); with one
// head to a lane 89 us, with four 80.  8192 tokens into 4-bit pages 44 us, bound
// by the arithmetic of the codes (58 us with a division for each).  32 tokens
// 4.6 us, the chain of loads.
#include "paged.cuh"

namespace dd {
namespace paged {
namespace {

constexpr int kWarps = 4;
constexpr int kHeads = 2;  // heads a lane takes, kHeads apart by a warp's worth

template <typename T, int D>
struct Geo {
  static constexpr int VEC = Elem<T>::kVec;
  static constexpr int kPieces = D / VEC;      // 16-byte pieces of a head
  static constexpr int kUnits = kPieces / 2;   // pairs of them
};

struct Where {
  int b, pos;  // b < 0: the token belongs to no sequence
};
__device__ __forceinline__ Where find_token(const Seqs& s, int t, int lane) {
  int b = 0;
  for (int base = 0; base < s.B; base += 32) {
    const int i = base + lane;
    const int end = i < s.B ? __ldg(s.q_start + i + 1) : 0x7fffffff;
    const int n = __popc(__ballot_sync(0xffffffffu, end <= t));
    b += n;
    if (n < 32) break;
  }
  if (b >= s.B || t < __ldg(s.q_start)) return Where{-1, 0};
  const int len = min(max(__ldg(s.seq_len + b), 0), kMaxLen);
  return Where{b, len - (min(__ldg(s.q_start + b + 1), s.n_tokens) - t)};
}

__device__ __forceinline__ void turn(float a, float b, float c, float s, float& x, float& y) {
  x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  y = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}

__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                    pack_bf16(f[6], f[7]));
}
__device__ __forceinline__ uint4 pack(const float (&f)[4]) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                    __float_as_uint(f[3]));
}
template <int N>
__device__ __forceinline__ void load_f(const float* p, float (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p + i));
    f[i] = v.x;
    f[i + 1] = v.y;
    f[i + 2] = v.z;
    f[i + 3] = v.w;
  }
}

// Turn a unit's two pieces.  Half pairing: element i of the first piece with
// element i of the second.  Interleaved: neighbours, within each piece.
template <int VEC>
__device__ __forceinline__ void turn_unit(uint4& p0, uint4& p1, const float (&c)[VEC],
                                          const float (&s)[VEC], bool interleaved) {
  float a[VEC], b[VEC], x[VEC], y[VEC];
  unpack(p0, a);
  unpack(p1, b);
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      turn(a[2 * i], a[2 * i + 1], c[i], s[i], x[2 * i], x[2 * i + 1]);
      turn(b[2 * i], b[2 * i + 1], c[VEC / 2 + i], s[VEC / 2 + i], y[2 * i], y[2 * i + 1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) turn(a[i], b[i], c[i], s[i], x[i], y[i]);
  }
  p0 = pack(x);
  p1 = pack(y);
}

// One lane's 8 elements of a bf16 row (a key's turned), values of a 4-bit
// group shared by 4 neighbouring lanes.
template <int D>
__device__ __forceinline__ void store_q4(const float (&x)[8], unsigned char* block, int page,
                                         int row, int piece, bool keep) {
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
  }
#pragma unroll
  for (int off = 1; off < 4; off <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
  }
  // The lowest value is a bf16 already; the step is rounded to one.
  const uint32_t sm = pack_bf16(__fdiv_rn(__fsub_rn(hi, lo), 15.f), lo);
  const float s = __uint_as_float(sm << 16);
  // round(d / s), d = x - lo, ties to even.  An approximate quotient gives an
  // integer k with k <= d / s <= k + 1 up to its error, and the comparison of d
  // with (k + 1/2) s, which is exact (4 + 8 bits), says which of the two it is; a
  // tie goes up if k is odd, as if (k + 1/2) s were one bit less.  The rounded
  // quotient d / s lies on a half only if the exact one does: next to a half the
  // floats d lie at least as far apart, relative to d, as half a step of the
  // quotient.  Adding 1.5 2^23 leaves an integer in the low bits.
  constexpr float kRound = 12582912.f;
  const float half = 0.5f * s;
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float d = __fsub_rn(x[i], lo);
    const float t = fmaf(d, inv, -0.5f) + kRound;
    const uint32_t k = __float_as_uint(t);
    const uint32_t b = __float_as_uint(fmaf(t - kRound, s, half)) - (k & 1u);
    codes |= ((k & 15u) + (d > __uint_as_float(b) ? 1u : 0u)) << (4 * i);
  }
  // Steps whose reciprocal is not a normal number, and 0.
  if (!(s > 1e-30f && s < 1e30f)) {
    codes = 0;
    if (s > 0.f) {
#pragma unroll 1
      for (int i = 7; i >= 0; --i) {
        float xi = x[0];
#pragma unroll
        for (int k = 1; k < 8; ++k) xi = i == k ? x[k] : xi;
        const float c = rintf(__fdiv_rn(__fsub_rn(xi, lo), s));
        codes = codes << 4 | (uint32_t)fminf(fmaxf(c, 0.f), 15.f);
      }
    }
  }
  if (!keep) return;
  *reinterpret_cast<uint32_t*>(block + (size_t)row * (D / 2) + 4 * piece) = codes;
  if ((piece & 3) == 0)
    *reinterpret_cast<uint32_t*>(block + (size_t)page * (D / 2) + (size_t)row * (D / 8) + piece) =
        sm;
}

template <typename T, int D, bool Q4>
__global__ void __launch_bounds__(kWarps * 32)
    append_kernel(Seqs s, AppendArgs a, int Hq, int Hkv, int wq, int wk) {
  using G = Geo<T, D>;
  constexpr int VEC = G::VEC, NP = G::kPieces, NU = G::kUnits;
  const int lane = threadIdx.x & 31;
  const int per_token = wq + 2 * wk;
  const long long w = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int t = (int)(w / per_token);
  if (t >= s.n_tokens) return;
  int part = (int)(w - (long long)t * per_token);
  const int kind = part < wq ? 0 : part < wq + wk ? 1 : 2;  // queries, keys, values
  part -= kind == 0 ? 0 : kind == 1 ? wq : wq + wk;
  const unsigned char* src =
      kind == 0 ? static_cast<const unsigned char*>(a.q) + (size_t)t * a.q_stride
      : kind == 1 ? static_cast<const unsigned char*>(a.k) + (size_t)t * a.k_stride
                  : static_cast<const unsigned char*>(a.v) + (size_t)t * a.v_stride;
  const uint4* rows = reinterpret_cast<const uint4*>(src);
  const int heads = kind == 0 ? Hq : Hkv;
  const int rot = kind == 2 ? 0 : a.rot_dim;
  const int half = rot / 2, hp = half / VEC;  // in elements, in pieces
  const int page = 1 << s.log2_page;

  if (Q4 && kind != 0) {
    if constexpr (Q4) {
      constexpr int kStep = 32 / NP;  // heads a warp covers at once
      const int piece = lane % NP, h0 = part * (kHeads * kStep) + lane / NP;
      // The piece that this one is turned with (half pairing).
      const bool first = piece < hp, turned = piece * VEC < rot;
      const bool paired = turned && !a.interleaved;
      const int partner = first ? piece + hp : piece - hp;
      uint4 own[kHeads], other[kHeads];
#pragma unroll
      for (int i = 0; i < kHeads; ++i) {
        const int h = h0 + i * kStep;
        own[i] = h < heads ? __ldg(rows + h * NP + piece) : make_uint4(0, 0, 0, 0);
        if (paired) other[i] = h < heads ? __ldg(rows + h * NP + partner) : own[i];
      }
      const Where at = find_token(s, t, lane);
      if (at.b < 0 || at.pos < 0 || (a.rope && at.pos >= a.rope_len)) return;
      const int pg = at.pos < s.cap ? page_of(s, at.b, at.pos) : -1;
      if (pg < 0) return;
      float c[8], sn[8];
      if (turned) {
        const float* cs = a.rope + (size_t)at.pos * rot;
        if (a.interleaved) {
          float c4[4], s4[4];
          load_f(cs + piece * 4, c4);
          load_f(cs + half + piece * 4, s4);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            c[i] = c4[i];
            sn[i] = s4[i];
          }
        } else {
          const int j = (first ? piece : partner) * 8;
          load_f(cs + j, c);
          load_f(cs + half + j, sn);
#pragma unroll
          for (int i = 0; i < 8; ++i) sn[i] = first ? -sn[i] : sn[i];
        }
      }
#pragma unroll
      for (int i = 0; i < kHeads; ++i) {
        const int h = h0 + i * kStep;
        if (part * (kHeads * kStep) + i * kStep >= heads) break;  // no lane has a head
        float x[8];
        unpack(own[i], x);
        if (turned) {
          if (a.interleaved) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float u = x[2 * e], v = x[2 * e + 1];
              turn(u, v, c[e], sn[e], x[2 * e], x[2 * e + 1]);
            }
          } else {
            float y[8];  // own cos -+ other sin
            unpack(other[i], y);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              x[e] = __fadd_rn(__fmul_rn(x[e], c[e]), __fmul_rn(y[e], sn[e]));
          }
          unpack(pack(x), x);  // the bf16 that a plain page would hold
        }
        unsigned char* block = (kind == 1 ? s.k : s.v) +
                               ((size_t)pg * Hkv + (h < heads ? h : 0)) * s.block_bytes;
        store_q4<D>(x, block, page, at.pos & (page - 1), piece, h < heads);
      }
    }
    return;
  }

  constexpr int kStep = 32 / NU;
  const int u = lane % NU, h0 = part * (kHeads * kStep) + lane / NU;
  // The unit's pieces: a turned pair, or two neighbours.
  int i0 = 2 * u, i1 = 2 * u + 1;
  if (!a.interleaved && u < hp) {
    i0 = u;
    i1 = u + hp;
  }
  const bool turned = u * VEC < half;
  uint4 p0[kHeads], p1[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int h = h0 + i * kStep;
    if (h < heads) {
      p0[i] = __ldcs(rows + h * NP + i0);
      p1[i] = __ldcs(rows + h * NP + i1);
    }
  }
  const Where at = find_token(s, t, lane);
  if (at.b < 0 || at.pos < 0 || (a.rope && at.pos >= a.rope_len)) return;
  uint4* dst;
  size_t step = NP;  // between heads, in pieces
  if (kind == 0) {
    dst = static_cast<uint4*>(a.q_out) + (size_t)t * Hq * NP;
  } else {
    const int pg = at.pos < s.cap ? page_of(s, at.b, at.pos) : -1;
    if (pg < 0) return;
    step = s.block_bytes / 16;
    dst = reinterpret_cast<uint4*>((kind == 1 ? s.k : s.v) + (size_t)pg * Hkv * s.block_bytes) +
          (at.pos & (page - 1)) * NP;
  }
  float c[VEC], sn[VEC];
  if (turned) {
    const float* cs = a.rope + (size_t)at.pos * rot;
    load_f(cs + u * VEC, c);
    load_f(cs + half + u * VEC, sn);
  }
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int h = h0 + i * kStep;
    if (h >= heads) break;
    if (turned) turn_unit<VEC>(p0[i], p1[i], c, sn, a.interleaved != 0);
    dst[h * step + i0] = p0[i];
    dst[h * step + i1] = p1[i];
  }
}

// Warps for a token's queries and for its keys (as many for its values): heads by
// the lanes that share one.
struct Warps {
  int q, k;
};
Warps warps_of(const Dims& d, bool with_q) {
  const int pieces = d.d * d.elt / 16;
  const int hq = kHeads * (32 / (pieces / 2));
  const int hk = d.format == DD_PAGES_Q4 ? kHeads * (32 / pieces) : hq;
  return Warps{with_q ? (d.Hq + hq - 1) / hq : 0, (d.Hkv + hk - 1) / hk};
}

template <typename T, int D, bool Q4>
cudaError_t launch(const Dims& d, const Seqs& s, const AppendArgs& a, cudaStream_t st) {
  static unsigned long long prepared = 0;
  cudaError_t e = prepare_kernel(append_kernel<T, D, Q4>, &prepared, 0);
  if (e != cudaSuccess) return e;
  const Warps w = warps_of(d, a.q != nullptr);
  append_kernel<T, D, Q4>
      <<<(unsigned)append_blocks(d, s.n_tokens, a.q != nullptr), kWarps * 32, 0, st>>>(
          s, a, d.Hq, d.Hkv, w.q, w.k);
  return cudaGetLastError();
}

}  // namespace

long long append_blocks(const Dims& d, int n_tokens, bool with_q) {
  const Warps w = warps_of(d, with_q);
  return ((long long)n_tokens * (w.q + 2 * w.k) + kWarps - 1) / kWarps;
}

cudaError_t launch_append(const Dims& d, const Seqs& s, const AppendArgs& a, cudaStream_t st) {
  if (d.format == DD_PAGES_Q4) {
    if (d.d == 64) return launch<bf16_t, 64, true>(d, s, a, st);
    if (d.d == 128) return launch<bf16_t, 128, true>(d, s, a, st);
    if (d.d == 256) return launch<bf16_t, 256, true>(d, s, a, st);
  } else if (d.dtype == DD_BF16) {
    if (d.d == 64) return launch<bf16_t, 64, false>(d, s, a, st);
    if (d.d == 128) return launch<bf16_t, 128, false>(d, s, a, st);
    if (d.d == 256) return launch<bf16_t, 256, false>(d, s, a, st);
  } else {
    if (d.d == 64) return launch<float, 64, false>(d, s, a, st);
    if (d.d == 128) return launch<float, 128, false>(d, s, a, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace paged
}  // namespace dd
