// dd_paged_read: positions first .. first + count - 1 of every sequence out of
// the pages into dense [B][H_kv][count][d] keys and values.
//
// The kernel moves bytes: rows are read once and written once.  A thread
// takes kPer 16-byte pieces of the output of each tensor and asks for all of
// them before it writes the first; neighbouring threads take neighbouring
// pieces, so a warp reads and writes runs of 512 bytes (of 4-bit pages it
// reads 128 bytes of codes and their steps).  Measured (8 KV heads, d = 128): eight
// contexts of up to 32768 positions 304 us, 6.3 TB/s read and written (8 pieces
// at a time: 326); 8192 4-bit positions 14 us.
#include "paged.cuh"

namespace dd {
namespace paged {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 2;

template <typename T, int D, bool Q4>
__device__ __forceinline__ uint4 load_piece(const unsigned char* block, int page, int row,
                                            int piece) {
  constexpr int NP = D / Elem<T>::kVec;
  if constexpr (Q4) {
    const uint32_t c = __ldg(reinterpret_cast<const uint32_t*>(block + row * (D / 2)) + piece);
    const uint32_t sm = __ldg(
        reinterpret_cast<const uint32_t*>(block + page * (D / 2) + row * (D / 8)) + (piece >> 2));
    const float s = __uint_as_float(sm << 16), m = __uint_as_float(sm & 0xFFFF0000u);
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r[i] = pack_bf16(q4_value(m, s, (c >> (8 * i)) & 15u),
                       q4_value(m, s, (c >> (8 * i + 4)) & 15u));
    return make_uint4(r[0], r[1], r[2], r[3]);
  } else {
    return __ldg(reinterpret_cast<const uint4*>(block) + row * NP + piece);
  }
}

template <typename T, int D, bool Q4>
__global__ void __launch_bounds__(kThreads)
    read_kernel(Seqs s, int Hkv, int first, int count, int tiles, uint4* __restrict__ k_out,
                uint4* __restrict__ v_out) {
  constexpr int NP = D / Elem<T>::kVec;
  const int unit = blockIdx.x / tiles, tile = blockIdx.x - unit * tiles;
  const int b = unit / Hkv, h = unit - b * Hkv;
  const int len = min(min(max(__ldg(s.seq_len + b), 0), kMaxLen), s.cap);
  const int page = 1 << s.log2_page;
  const long long n = (long long)count * NP;
  const size_t out0 = (size_t)unit * count * NP;
  uint4 kv[kPer], vv[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const long long x = (long long)tile * (kThreads * kPer) + i * kThreads + threadIdx.x;
    kv[i] = vv[i] = make_uint4(0, 0, 0, 0);
    const long long pos = first + x / NP;
    if (x < n && pos < len) {
      const int pg = page_of(s, b, (int)pos);
      if (pg >= 0) {
        const size_t off = ((size_t)pg * Hkv + h) * s.block_bytes;
        const int row = (int)pos & (page - 1), piece = (int)(x % NP);
        kv[i] = load_piece<T, D, Q4>(s.k + off, page, row, piece);
        vv[i] = load_piece<T, D, Q4>(s.v + off, page, row, piece);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const long long x = (long long)tile * (kThreads * kPer) + i * kThreads + threadIdx.x;
    if (x < n) {
      k_out[out0 + x] = kv[i];
      v_out[out0 + x] = vv[i];
    }
  }
}

// CTAs of one (sequence, KV head).
int tiles_of(const Dims& d, int count) {
  const long long n = (long long)count * (d.d * d.elt / 16);
  return (int)((n + kThreads * kPer - 1) / (kThreads * kPer));
}

template <typename T, int D, bool Q4>
cudaError_t launch(const Dims& d, const Seqs& s, int first, int count, void* k_out, void* v_out,
                   cudaStream_t st) {
  static unsigned long long prepared = 0;
  cudaError_t e = prepare_kernel(read_kernel<T, D, Q4>, &prepared, 0);
  if (e != cudaSuccess) return e;
  read_kernel<T, D, Q4><<<(unsigned)read_blocks(d, count), kThreads, 0, st>>>(
      s, d.Hkv, first, count, tiles_of(d, count), static_cast<uint4*>(k_out),
      static_cast<uint4*>(v_out));
  return cudaGetLastError();
}

}  // namespace

long long read_blocks(const Dims& d, int count) {
  return (long long)tiles_of(d, count) * d.B * d.Hkv;
}

cudaError_t launch_read(const Dims& d, const Seqs& s, int first, int count, void* k_out,
                        void* v_out, cudaStream_t st) {
  if (d.format == DD_PAGES_Q4) {
    if (d.d == 64) return launch<bf16_t, 64, true>(d, s, first, count, k_out, v_out, st);
    if (d.d == 128) return launch<bf16_t, 128, true>(d, s, first, count, k_out, v_out, st);
    if (d.d == 256) return launch<bf16_t, 256, true>(d, s, first, count, k_out, v_out, st);
  } else if (d.dtype == DD_BF16) {
    if (d.d == 64) return launch<bf16_t, 64, false>(d, s, first, count, k_out, v_out, st);
    if (d.d == 128) return launch<bf16_t, 128, false>(d, s, first, count, k_out, v_out, st);
    if (d.d == 256) return launch<bf16_t, 256, false>(d, s, first, count, k_out, v_out, st);
  } else {
    if (d.d == 64) return launch<float, 64, false>(d, s, first, count, k_out, v_out, st);
    if (d.d == 128) return launch<float, 128, false>(d, s, first, count, k_out, v_out, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace paged
}  // namespace dd
