// dd_paged_attn for few tokens of a sequence: a decode step, or a few
// speculated tokens.
//
// The kernel is bound by reading every visible key and value once.  Up to 8 NR
// rows ((token, query head of the group) pairs) share each row of the cache; a
// call is split over the keys until the card is full, every CTA is four warps (six
// for more than 8 fp32 rows of 512 bytes), and every warp walks over its own tiles
// of 16 keys (a tile lies in one page) with a ring of its own, filled by
// asynchronous 16-byte copies, and a softmax of its own.  Nothing synchronises the
// warps before their results are merged.
// Up to eight splits are a cluster, which merges them in its shared memory and
// writes the result; more go through the workspace and a second kernel.
// Measured (32 query heads on 8 KV heads, d = 128), of the bytes that have to be
// read: bf16, 8 contexts of up to 131072 506 us, 7.2 TB/s (a copy reaches 6.8; the
// short contexts stay in L2 between calls); a window of 4096 over 32 requests 80
// us, 6.7 TB/s; fp32, 4 contexts of 92000 457 us, 6.6 TB/s.
//
// The products run on warp-level matrix instructions with the keys (then the
// head's elements) as the 16 rows of A and the queries as the 8 columns of B:
//   S^T[16 keys][8 rows] = K Q^T,   O^T[16 elements][8 rows] += V^T P^T.
// P^T leaves the first product in the layout that a transposed 8 x 8 fragment
// of the second needs (movmatrix).  Weights use a maximum that follows the
// running one lazily, when a logit is 2^8 above it, so that the usual tile
// needs no reduction over lanes.  They are rounded to bf16 for the second
// product (2^-8 relative at most); their sum is not.
//
// 4-bit pages are never widened to values.  With x = m + s c per group of 32:
//   S   = sum_groups 16 s (q . (1 + c / 16)) + (m - 16 s) sum q:
//         1 + c / 16 is a bf16 whose mantissa holds the code, so a code costs a
//         shift and a logic operation; the second term is one more matrix
//         instruction over the (s, m) pairs as they lie in memory, sum q being
//         split into three bf16;
//   O^T = sum_groups (c - 8) (P s) + sum P m + 8 sum P s: P s is formed in fp32
//         and rounded once, c - 8 is exact, and centring the codes keeps that
//         rounding in proportion to the value; the last two are again one
//         matrix instruction over the pairs.
// 8 contexts of up to 131072 take 331 us, 3.4 TB/s, two thirds of the bf16 pages'
// time: some 560 instructions for a tile of 16 keys.  No unit is full (issue slots
// 64 %, the integer pipe 63 %, DRAM 44 %); what holds the rest up is not settled.
// Two tiles share the tests of one (365 us without), and four CTAs of 128 threads
// share an SM.
//
// fp32 pages: the same products on tf32 (11 bits of the mantissa) would lose
// half the digits, so every operand is split into what tf32 holds and the rest,
// and a product is hi hi + hi lo + lo hi: 2^-21 relative, of the order of the
// fp32 sums' own rounding.  P goes to the second product over shuffles.  fp32
// calls of many tokens run here too, 16 rows at a time: 2048 and 700 tokens (32 /
// 8 heads, d = 128) 1.45 ms, 26 TFLOP/s, bound by the splitting's instructions.
// Infinities do not split: rows that meet one are computed again in plain fp32.
#include <math.h>

#include "paged.cuh"

namespace dd {
namespace paged {
namespace {

constexpr float kLazy = 8.f;  // in log2

// D[16x8] += A[16x16] B[16x8], bf16 in, fp32 out.
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// D = A B.
__device__ __forceinline__ void mma_new(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// D[16x8] = C + A[16x8] B[8x8], tf32 in (the low bits of an fp32 are dropped), fp32 out.
// Fragments (g = lane / 4, c = lane % 4): a0 = A[g][c], a1 = A[g + 8][c], a2 = A[g][c + 4],
// a3 = A[g + 8][c + 4]; b0 = B[c][g], b1 = B[c + 4][g].
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1, float c0, float c1, float c2, float c3) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2),
        "f"(c3));
}
// hi is rounded, not cut, so that lo and what is dropped of it have either sign.
__device__ __forceinline__ void split(uint32_t x, uint32_t& hi, uint32_t& lo) {
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi) : "f"(__uint_as_float(x)));
  lo = __float_as_uint(__uint_as_float(x) - __uint_as_float(hi));
}
// d(t) += A b(t, .) in three tf32 products, for each of NR columns of tiles.  The
// matrix unit cuts its sums where fp32 additions round, and over a long chain
// that adds up (2e-6 of a result where it was measured), so each step starts
// from zero, the small terms first, and is added in fp32.
template <int NR, typename Acc, typename B>
__device__ __forceinline__ void mma_f32(Acc d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        B b) {
  uint32_t hi[4], lo[4];
  split(a0, hi[0], lo[0]);
  split(a1, hi[1], lo[1]);
  split(a2, hi[2], lo[2]);
  split(a3, hi[3], lo[3]);
#pragma unroll
  for (int t = 0; t < NR; ++t) {
    uint32_t bh0, bl0, bh1, bl1;
    split(b(t, 0), bh0, bl0);
    split(b(t, 1), bh1, bl1);
    float x[4], y[4];
    mma_tf32(x, lo, bh0, bh1, 0.f, 0.f, 0.f, 0.f);
    mma_tf32(y, hi, bl0, bl1, x[0], x[1], x[2], x[3]);
    mma_tf32(x, hi, bh0, bh1, y[0], y[1], y[2], y[3]);
#pragma unroll
    for (int e = 0; e < 4; ++e) d(t)[e] += x[e];
  }
}
// Four 8 x 8 tiles of 16-bit elements; lane i gives the address of row i % 8 of tile i / 8.
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// N bytes global -> shared, or N zero bytes.
template <int N>
__device__ __forceinline__ void copy_to(uint32_t dst, const void* src, bool there) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(there ? 16 : 0)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N),
                 "r"(there ? N : 0)
                 : "memory");
}
template <int N>
__device__ __forceinline__ void copy_all(uint32_t dst, const void* src) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Clusters: all CTAs of one, and another CTA's shared memory.
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
__device__ __forceinline__ uint32_t of_cta(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
               : "=f"(v.x), "=f"(v.y)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
// The (s, m) pairs of a row of 32 N elements.
template <int N>
__device__ __forceinline__ void lds_pairs(uint32_t (&r)[N], uint32_t a) {
  if constexpr (N == 2) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(a) : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint4 v = lds128(a + 4 * i);
      r[i] = v.x;
      r[i + 1] = v.y;
      r[i + 2] = v.z;
      r[i + 3] = v.w;
    }
  }
}
__device__ __forceinline__ float exp2a(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float bf_lo(uint32_t x) { return __uint_as_float(x << 16); }

// Four codes of two keys, as bf16 pairs 1 + c / 16: nibble i of each half of x.
__device__ __forceinline__ uint32_t code_pair(uint32_t x, int i) {
  const uint32_t y = i == 0 ? x << 3 : x >> (4 * i - 3);
  return (y & 0x00780078u) | 0x3F803F80u;
}
// ... and as c - 8, scaled by 1/16: (1 + c / 16) - 1.5, exact.
__device__ __forceinline__ uint32_t centred(uint32_t x) {
  uint32_t r;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(0xBFC0BFC0u));
  return r;
}

// What the pages hold.
enum Kind { kBf16, kQ4, kF32 };

template <int D, Kind K>
struct Geo {
  static constexpr bool Q4 = K == kQ4;
  // fp32 rows of 512 bytes: one CTA fills an SM, of four warps with three stages
  // for 8 rows, which reading bounds, of six with two for more.
  static constexpr bool kWide = K == kF32 && D == 128;
  __host__ __device__ static constexpr int warps(int nr) { return kWide && nr > 1 ? 6 : 4; }
  static constexpr int kRow = Q4 ? D / 2 : K == kF32 ? 4 * D : 2 * D;  // bytes of a row (its codes)
  static constexpr int kGroups = D / 32;
  static constexpr int kPairs = Q4 ? kGroups * 4 : 0;       // bytes of a row's (s, m) pairs
  static constexpr int kTensor = 16 * (kRow + kPairs);      // a tile's keys or values
  static constexpr int kStage = 2 * kTensor;
  // About 24 KB of ring to a warp, two CTAs to an SM (rows of 512 bytes: 48 KB, one).
  __host__ __device__ static constexpr int stages(int nr) {
    return Q4 ? (D == 64 ? 8 : 4) : K == kBf16 && D == 64 ? 6 : kWide && nr > 1 ? 2 : 3;
  }
  static constexpr int kPieces = kRow / 16;                 // 16-byte pieces of a row
  // Tiles a warp computes at once, and CTAs to an SM: 4-bit pages are bound by
  // instructions, share the tests of two tiles, and want warps.
  __host__ __device__ static constexpr int at_once(int nr) { return Q4 && nr == 1 ? 2 : 1; }
  __host__ __device__ static constexpr int ctas(int nr) {
    return Q4 && nr == 1 && D < 256 ? 4 : D == 256 || (kWide) ? 1 : 2;
  }
};

// Where piece p of row r lies in a tile: the pieces of neighbouring rows are
// exchanged so that the eight rows a fragment reads lie in different banks.
template <int D, Kind K>
__device__ __forceinline__ uint32_t piece_at(int r, int p) {
  using G = Geo<D, K>;
  if (K == kF32) return r * G::kRow + 16 * (p ^ (((r & 1) << 2) | (r & 2)));
  constexpr int kRowsPerLine = G::kRow >= 128 ? 1 : 128 / G::kRow;
  constexpr int kMask = (G::kPieces < 8 ? G::kPieces : 8) - 1;
  return r * G::kRow + 16 * (p ^ ((r / kRowsPerLine) & kMask));
}

// A warp's part of fp32 rows again, for sums that the split products left without a
// finite value: an infinity has no finite rest (and the largest fp32 round to one in
// tf32), so there it becomes NaN.  A key and a row at a time; rows of D + 4 into po,
// (max, sum) into pml.  Where the warp's keys lie is found again, so that the kernel
// keeps no registers for it; as a function of its own it costs calls of many rows of
// 512 bytes 3 % (1404 us without, 1450 with, 1506 inlined), of 256 bytes 1 % (497,
// 503 and 519), of few rows nothing.
template <int D>
__device__ __noinline__ void in_plain_fp32(Seqs s, AttnArgs a, int Hkv, int G, int warps,
                                           long long r0, int nr, float k1, float* po,
                                           float2* pml) {
  constexpr int E = D / 32;  // elements of a lane
  const int b = blockIdx.x / Hkv, hk = blockIdx.x - b * Hkv, split = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, page = 1 << s.log2_page;
  const Seq q = load_seq(s, b);
  const KeyTiles kt = key_tiles<16>(q.pos0 + (int)(r0 / G), q.pos0 + (int)((r0 + nr - 1) / G),
                                    q.len, a.window, a.sinks);
  const int i0 = (int)((long long)kt.n * split / a.nsplit);
  const int i1 = (int)((long long)kt.n * (split + 1) / a.nsplit);
#pragma unroll 1
  for (int r = 0; r < nr; ++r) {
    const int token = (int)((r0 + r) / G), p = q.pos0 + token;
    const float* qr =
        reinterpret_cast<const float*>(static_cast<const unsigned char*>(a.q) +
                                       (size_t)(q.q0 + token) * a.q_stride) +
        (hk * G + (int)((r0 + r) % G)) * D + E * lane;
    float acc[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 1
    for (int x = 16 * (i0 + warp); x < 16 * i1; x += (x & 15) < 15 ? 1 : 16 * warps - 15) {
      const int j = kt.tile(x >> 4) * 16 + (x & 15);
      const int pg = page_of(s, b, j);
      if (pg < 0 || !sees(p, j, a.window, a.sinks)) continue;
      const size_t at = ((size_t)pg * Hkv + hk) * s.block_bytes +
                        (size_t)((j & (page - 1)) * D + E * lane) * 4;
      const float* kr = reinterpret_cast<const float*>(s.k + at);
      const float* vr = reinterpret_cast<const float*>(s.v + at);
      float y = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) y = fmaf(__ldg(qr + e), __ldg(kr + e), y);
#pragma unroll
      for (int z = 16; z > 0; z >>= 1) y += __shfl_xor_sync(0xffffffffu, y, z);
      const float to = fmaxf(m, y);
      const float f = to == -INFINITY ? 1.f : exp2a((m - to) * k1);
      const float w = y == -INFINITY ? 0.f : exp2a((y - to) * k1);
      m = to;
      l = fmaf(l, f, w);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(acc[e], f, w * __ldg(vr + e));
    }
    if (lane == 0) pml[r] = make_float2(m, l);
#pragma unroll
    for (int e = 0; e < E; ++e) po[r * (D + 4) + E * lane + e] = acc[e];
  }
}

template <int D, Kind K, int NR>
__global__ void __launch_bounds__((32 * Geo<D, K>::warps(NR)), (Geo<D, K>::ctas(NR)))
    decode_kernel(Seqs s, AttnArgs a, int Hq, int Hkv, int G, float scale) {
  using Ge = Geo<D, K>;
  constexpr bool Q4 = K == kQ4;
  constexpr int kWarps = Ge::warps(NR), kThreads = 32 * kWarps, kStages = Ge::stages(NR);
  constexpr int kElt = K == kF32 ? 4 : 2;
  constexpr int NK = D / 16;  // contraction steps of S, row tiles of O^T
  constexpr int KT = Ge::at_once(NR);
  static_assert(kStages % KT == 0 && kStages >= 2 * KT, "ring");
  extern __shared__ __align__(128) unsigned char smem[];
  const int b = blockIdx.x / Hkv, hk = blockIdx.x - b * Hkv, split = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const Seq q = load_seq(s, b);
  const long long rows = (long long)q.nq * G;
  const int page = 1 << s.log2_page;
  const uint32_t ring = smem_addr(smem) + warp * kStages * Ge::kStage;
  // The weight of a logit is 2^(x k1); 4-bit logits are held over 16.
  const float k1 = scale * 1.4426950408889634f * (Q4 ? 16.f : 1.f);

  for (long long r0 = (long long)blockIdx.y * (8 * NR); r0 < rows;
       r0 += (long long)gridDim.y * (8 * NR)) {
    const int nr = (int)min((long long)(8 * NR), rows - r0);
    const int pos_a = q.pos0 + (int)(r0 / G), pos_b = q.pos0 + (int)((r0 + nr - 1) / G);
    const KeyTiles kt = key_tiles<16>(pos_a, pos_b, q.len, a.window, a.sinks);
    const int i0 = (int)((long long)kt.n * split / a.nsplit);
    const int i1 = (int)((long long)kt.n * (split + 1) / a.nsplit);
    // Tiles of this warp: i0 + warp, + kWarps, ...
    const int n = i1 - i0 > warp ? (i1 - i0 - warp + kWarps - 1) / kWarps : 0;

    // Pages of 32 tiles of this warp from x on, lane by lane.
    auto load_pages = [&](int x) {
      return x + lane < n ? page_of(s, b, kt.tile(i0 + warp + (x + lane) * kWarps) * 16) : -1;
    };
    int pages = -1;
    uint32_t dst = ring;  // the stage that is filled next
    // Copies of tile x; rows that no token sees become zeros.  The pieces of a
    // tile's rows lie on end: piece y is 16 y bytes from the first.
    constexpr int kPart = Ge::kPairs < 16 ? 8 : 16;  // of a row's pairs: 8, 16 or 2 x 16
    constexpr int kParts = Q4 ? 16 * Ge::kPairs / kPart : 0;
    auto fetch = [&](int x) {
      if (x < (n + KT - 1) / KT * KT) {  // tiles computed beside the last one are zeros
        if ((x & 31) == 0) pages = load_pages(x);
        const int pg = __shfl_sync(0xffffffffu, pages, x & 31);
        const int j0 = x < n ? kt.tile(i0 + warp + x * kWarps) * 16 : 0;
        const size_t off = ((size_t)max(pg, 0) * Hkv + hk) * s.block_bytes;
        const int row0 = j0 & (page - 1);
        const size_t at = off + (size_t)(row0 * Ge::kRow + 16 * lane);
        const size_t pair_at = off + (size_t)(page * Ge::kRow + row0 * Ge::kPairs + kPart * lane);
        if (pg >= 0 && j0 + 16 <= kt.hi && (j0 >= kt.lo || j0 + 16 <= a.sinks)) {
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const unsigned char* src = (kv ? s.v : s.k) + at;
#pragma unroll
            for (int i = 0; i < Ge::kPieces / 2; ++i) {
              const int y = lane + 32 * i;
              copy_all<16>(dst + kv * Ge::kTensor + piece_at<D, K>(y / Ge::kPieces, y % Ge::kPieces),
                           src + 512 * i);
            }
            if (Q4 && (kParts >= 32 || lane < kParts))
              copy_all<kPart>(dst + kv * Ge::kTensor + 16 * Ge::kRow + kPart * lane,
                              (kv ? s.v : s.k) + pair_at);
          }
        } else {
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv) {
            const unsigned char* src = (kv ? s.v : s.k) + at;
#pragma unroll 1
            for (int i = 0; i < Ge::kPieces / 2; ++i) {
              const int y = lane + 32 * i, r = y / Ge::kPieces;
              copy_to<16>(dst + kv * Ge::kTensor + piece_at<D, K>(r, y % Ge::kPieces),
                          src + 512 * i, pg >= 0 && kt.any(j0 + r, a.sinks));
            }
            if (Q4 && (kParts >= 32 || lane < kParts))
              copy_to<kPart>(dst + kv * Ge::kTensor + 16 * Ge::kRow + kPart * lane,
                             (kv ? s.v : s.k) + pair_at,
                             pg >= 0 && kt.any(j0 + kPart * lane / max(Ge::kPairs, 1), a.sinks));
          }
        }
      }
      dst = dst + Ge::kStage == ring + kStages * Ge::kStage ? ring : dst + Ge::kStage;
      if (x % KT == KT - 1) copies_commit();
    };
#pragma unroll 1
    for (int x = 0; x < kStages - KT; ++x) fetch(x);
    int live = pages;   // pages of the tiles being computed (fetch runs ahead)
    uint32_t kb = ring;  // the stage that is read next

    // Queries as B: column g is row r0 + 8 t + g.
    uint32_t qb[NR][NK][K == kF32 ? 4 : 2];
    uint32_t qs[NR][Q4 ? (Ge::kGroups + 3) / 4 : 1][3];  // their sums, by groups (4-bit)
#pragma unroll
    for (int t = 0; t < NR; ++t) {
      const int r = 8 * t + g;
      const long long rr = r0 + (r < nr ? r : 0);
      const unsigned char* src = static_cast<const unsigned char*>(a.q) +
                                 (size_t)(q.q0 + (int)(rr / G)) * a.q_stride +
                                 (size_t)(hk * G + (int)(rr % G)) * (kElt * D);
      if constexpr (K == kF32) {
#pragma unroll
        for (int k = 0; k < NK; ++k) {  // elements 16 k + 4 c + (0 .. 3)
          const uint4 v = ld_ro(src + 64 * k + 16 * c);
          qb[t][k][0] = v.x;
          qb[t][k][1] = v.y;
          qb[t][k][2] = v.z;
          qb[t][k][3] = v.w;
        }
      } else if constexpr (!Q4) {
#pragma unroll
        for (int k = 0; k < NK; ++k) {
          qb[t][k][0] = __ldg(reinterpret_cast<const uint32_t*>(src + 32 * k + 4 * c));
          qb[t][k][1] = __ldg(reinterpret_cast<const uint32_t*>(src + 32 * k + 16 + 4 * c));
        }
      } else {
#pragma unroll
        for (int x = 0; x < (Ge::kGroups + 3) / 4; ++x) qs[t][x][0] = qs[t][x][1] = qs[t][x][2] = 0;
        // Word c of group k: elements 32 k + 8 c + (0 .. 7), paired i with i + 4 as
        // the codes come out of a word.
#pragma unroll
        for (int k = 0; k < Ge::kGroups; ++k) {
          const uint4 v = ld_ro(src + 64 * k + 16 * c);
          qb[t][2 * k][0] = __byte_perm(v.x, v.z, 0x5410);
          qb[t][2 * k][1] = __byte_perm(v.x, v.z, 0x7632);
          qb[t][2 * k + 1][0] = __byte_perm(v.y, v.w, 0x5410);
          qb[t][2 * k + 1][1] = __byte_perm(v.y, v.w, 0x7632);
          float f[8], sum = 0.f;
          unpack(v, f);
#pragma unroll
          for (int e = 0; e < 8; ++e) sum += f[e];
          sum += __shfl_xor_sync(0xffffffffu, sum, 1);
          sum += __shfl_xor_sync(0xffffffffu, sum, 2);
          if (c == (k & 3)) {  // B[2c] meets s, B[2c + 1] meets m; all over 16
            float rest = sum;  // in three bf16, which hold an fp32
#pragma unroll
            for (int y = 0; y < 3; ++y) {
              qs[t][k / 4][y] = pack_bf16(-rest, rest * 0.0625f);
              rest += bf_lo(qs[t][k / 4][y]);
            }
          }
        }
      }
    }

    float o[NR][NK][4];
    float os[NR][4];                 // 4-bit: sums of P m and P s by group
    float m[NR][2], l[NR][2];        // of rows 8 t + 2 c and + 1
    float off[NR][2], lim[NR][2];    // -m k1, and the logit above which m has to move
    const float lazy = kLazy / k1;
    int pos[NR][2];
#pragma unroll
    for (int t = 0; t < NR; ++t) {
#pragma unroll
      for (int k = 0; k < NK; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][k][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) os[t][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[t][e] = lim[t][e] = -INFINITY;
        l[t][e] = off[t][e] = 0.f;
        pos[t][e] = q.pos0 + (int)((r0 + 8 * t + 2 * c + e) / G);
      }
    }

#pragma unroll 1
    for (int x = 0; x < n; x += KT) {
      if ((x & 31) == 0 && x > 0) live = load_pages(x);
      copies_wait<kStages / KT - 2>();
      __syncwarp();
      // Into the stages of the tiles before, which every lane is done with.
#pragma unroll
      for (int u = 0; u < KT; ++u) fetch(x + u + kStages - KT);
      bool there = false;
      int j0[KT];  // a tile without a page, or behind the last one: past every position
#pragma unroll
      for (int u = 0; u < KT; ++u) {
        const bool page_there = __shfl_sync(0xffffffffu, live, (x + u) & 31) >= 0;
        j0[u] = page_there ? kt.tile(i0 + warp + (x + u) * kWarps) * 16 : kMaxLen;
        there |= page_there;
      }
      if (there) {
        float st[KT][NR][4];  // S^T: keys g, g + 8 by rows 2 c, 2 c + 1
#pragma unroll
        for (int u = 0; u < KT; ++u) {
          const uint32_t kbu = kb + u * Ge::kStage;
          if constexpr (K == kF32) {
#pragma unroll
            for (int t = 0; t < NR; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e) st[u][t][e] = 0.f;
            auto st_of = [&](int t) -> float(&)[4] { return st[u][t]; };
#pragma unroll
            for (int k = 0; k < NK; ++k) {
              const uint4 x0 = lds128(kbu + piece_at<D, K>(g, 4 * k + c));
              const uint4 x1 = lds128(kbu + piece_at<D, K>(g + 8, 4 * k + c));
              mma_f32<NR>(st_of, x0.x, x1.x, x0.y, x1.y, [&](int t, int e) { return qb[t][k][e]; });
              mma_f32<NR>(st_of, x0.z, x1.z, x0.w, x1.w,
                          [&](int t, int e) { return qb[t][k][2 + e]; });
            }
          } else if constexpr (!Q4) {
            const int r = (lane & 7) + (lane & 8), p = lane >> 4;
#pragma unroll
            for (int k = 0; k < NK; ++k) {
              uint32_t f[4];
              ldsm4(f, kbu + piece_at<D, K>(r, 2 * k + p));
#pragma unroll
              for (int t = 0; t < NR; ++t) {
                if (k == 0)
                  mma_new(st[u][t], f[0], f[1], f[2], f[3], qb[t][k][0], qb[t][k][1]);
                else
                  mma(st[u][t], f[0], f[1], f[2], f[3], qb[t][k][0], qb[t][k][1]);
              }
            }
          } else {
            const uint32_t kp = kbu + 16 * Ge::kRow;
            uint32_t sm0[Ge::kGroups], sm1[Ge::kGroups];  // pairs of keys g and g + 8
            lds_pairs(sm0, kp + g * Ge::kPairs);
            lds_pairs(sm1, kp + (g + 8) * Ge::kPairs);
#pragma unroll
            for (int x4 = 0; x4 < (Ge::kGroups + 3) / 4; ++x4) {
              const bool in = 4 * x4 + c < Ge::kGroups;
              const uint32_t w0 = in ? lds32(kp + g * Ge::kPairs + 16 * x4 + 4 * c) : 0u;
              const uint32_t w1 = in ? lds32(kp + (g + 8) * Ge::kPairs + 16 * x4 + 4 * c) : 0u;
#pragma unroll
              for (int t = 0; t < NR; ++t) {
                if (x4 == 0)
                  mma_new(st[u][t], w0, w1, w0, w1, qs[t][x4][0], qs[t][x4][1]);
                else
                  mma(st[u][t], w0, w1, w0, w1, qs[t][x4][0], qs[t][x4][1]);
                mma(st[u][t], w0, w1, 0u, 0u, qs[t][x4][2], 0u);
              }
            }
#pragma unroll
            for (int k = 0; k < Ge::kGroups; ++k) {
              const uint32_t w0 = lds32(kbu + piece_at<D, K>(g, k) + 4 * c);
              const uint32_t w1 = lds32(kbu + piece_at<D, K>(g + 8, k) + 4 * c);
              uint32_t f0[4], f1[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                f0[i] = code_pair(w0, i);
                f1[i] = code_pair(w1, i);
              }
              const float s0 = bf_lo(sm0[k]), s1 = bf_lo(sm1[k]);
#pragma unroll
              for (int t = 0; t < NR; ++t) {
                float acc[4];
                mma_new(acc, f0[0], f1[0], f0[1], f1[1], qb[t][2 * k][0], qb[t][2 * k][1]);
                mma(acc, f0[2], f1[2], f0[3], f1[3], qb[t][2 * k + 1][0], qb[t][2 * k + 1][1]);
                st[u][t][0] = fmaf(s0, acc[0], st[u][t][0]);
                st[u][t][1] = fmaf(s0, acc[1], st[u][t][1]);
                st[u][t][2] = fmaf(s1, acc[2], st[u][t][2]);
                st[u][t][3] = fmaf(s1, acc[3], st[u][t][3]);
              }
            }
          }
        }
        bool all = true;
#pragma unroll
        for (int u = 0; u < KT; ++u)
          all = all && j0[u] + 15 <= pos_a &&
                (a.window == 0 || j0[u] > pos_b - a.window || j0[u] + 16 <= a.sinks);
        if (!all) {
#pragma unroll
          for (int u = 0; u < KT; ++u)
#pragma unroll
            for (int t = 0; t < NR; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int j = j0[u] + g + 8 * (e >> 1);
                if (j0[u] == kMaxLen || !sees(pos[t][e & 1], j, a.window, a.sinks))
                  st[u][t][e] = -INFINITY;
              }
        }
        bool grow = false;
        float top[NR][2];
#pragma unroll
        for (int t = 0; t < NR; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            top[t][e] = fmaxf(st[0][t][e], st[0][t][e + 2]);
            if (KT == 2) top[t][e] = fmaxf(top[t][e], fmaxf(st[KT - 1][t][e], st[KT - 1][t][e + 2]));
            grow |= top[t][e] > lim[t][e];
          }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int t = 0; t < NR; ++t) {
            float f[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float to = fmaxf(m[t][e], top[t][e]);
#pragma unroll
              for (int y = 4; y < 32; y <<= 1)
                to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, y));
              f[e] = to == -INFINITY ? 1.f : exp2a((m[t][e] - to) * k1);
              m[t][e] = to;
              off[t][e] = to == -INFINITY ? 0.f : -to * k1;
              lim[t][e] = to + lazy;
              l[t][e] *= f[e];
            }
            // O^T has the same columns: rows 2 c and 2 c + 1.
#pragma unroll
            for (int k = 0; k < NK; ++k)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[t][k][e] *= f[e & 1];
#pragma unroll
            for (int e = 0; e < 4; ++e) os[t][e] *= f[e & 1];
          }
        }
#pragma unroll
        for (int u = 0; u < KT; ++u) {
          const uint32_t vb = kb + u * Ge::kStage + Ge::kTensor;
          uint32_t pb[NR][K == kF32 ? 4 : 2];  // P^T as B (unscaled)
#pragma unroll
          for (int t = 0; t < NR; ++t) {
#pragma unroll
            for (int e = 0; e < 4; ++e) st[u][t][e] = exp2a(fmaf(st[u][t][e], k1, off[t][e & 1]));
            l[t][0] += st[u][t][0] + st[u][t][2];
            l[t][1] += st[u][t][1] + st[u][t][3];
            if constexpr (K == kF32) {
              // Keys c, c + 4 and c + 8, c + 12 of row g, from the lanes that have them.
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int from = ((e & 1) * 4 + c) * 4 + (g >> 1);
                const float x0 = __shfl_sync(0xffffffffu, st[u][t][(e >> 1) * 2], from);
                const float x1 = __shfl_sync(0xffffffffu, st[u][t][(e >> 1) * 2 + 1], from);
                pb[t][e] = __float_as_uint((g & 1) ? x1 : x0);
              }
            } else {
              pb[t][0] = transpose8(pack_bf16(st[u][t][0], st[u][t][1]));
              pb[t][1] = transpose8(pack_bf16(st[u][t][2], st[u][t][3]));
            }
          }
          if constexpr (K == kF32) {
            // Piece 8 y + g of a key's row: elements e of pieces 16 x + g and 16 x + 8 + g
            // are rows g and g + 8 of tile 4 x + e.
#pragma unroll
            for (int h = 0; h < 2; ++h)  // keys 8 h + c, 8 h + c + 4
#pragma unroll
              for (int x = 0; x < NK / 4; ++x) {
                const uint4 v0 = lds128(vb + piece_at<D, K>(8 * h + c, 16 * x + g));
                const uint4 v1 = lds128(vb + piece_at<D, K>(8 * h + c, 16 * x + 8 + g));
                const uint4 v2 = lds128(vb + piece_at<D, K>(8 * h + c + 4, 16 * x + g));
                const uint4 v3 = lds128(vb + piece_at<D, K>(8 * h + c + 4, 16 * x + 8 + g));
                auto p = [&](int t, int e) { return pb[t][2 * h + e]; };
                auto acc = [&](int e) {
                  return [&, e](int t) -> float(&)[4] { return o[t][4 * x + e]; };
                };
                mma_f32<NR>(acc(0), v0.x, v1.x, v2.x, v3.x, p);
                mma_f32<NR>(acc(1), v0.y, v1.y, v2.y, v3.y, p);
                mma_f32<NR>(acc(2), v0.z, v1.z, v2.z, v3.z, p);
                mma_f32<NR>(acc(3), v0.w, v1.w, v2.w, v3.w, p);
              }
          } else if constexpr (!Q4) {
            // V^T tiles: rows are elements, so keys' rows are read transposed.
            const int r = (lane & 7) + (lane >> 4) * 8, p = (lane >> 3) & 1;
#pragma unroll
            for (int k = 0; k < NK; ++k) {
              uint32_t f[4];
              ldsm4_t(f, vb + piece_at<D, K>(r, 2 * k + p));
#pragma unroll
              for (int t = 0; t < NR; ++t) mma(o[t][k], f[0], f[1], f[2], f[3], pb[t][0], pb[t][1]);
            }
          } else {
            const uint32_t vp = vb + 16 * Ge::kRow;
            // Row g of A: m of group g (g < groups), then s; keys 2 c, 2 c + 1, 2 c + 8, 2 c + 9.
            auto pair_row = [&](int r) -> uint2 {
              const bool in = r < 2 * Ge::kGroups;
              const uint32_t at = vp + (in ? r % Ge::kGroups : 0) * 4 + 2 * c * Ge::kPairs;
              const uint32_t sel = r < Ge::kGroups ? 0x7632 : 0x5410;
              const uint32_t x0 = lds32(at), x1 = lds32(at + Ge::kPairs);
              const uint32_t x2 = lds32(at + 8 * Ge::kPairs), x3 = lds32(at + 9 * Ge::kPairs);
              return in ? make_uint2(__byte_perm(x0, x1, sel), __byte_perm(x2, x3, sel))
                        : make_uint2(0, 0);
            };
            const uint2 ra = pair_row(g), rb = Ge::kGroups > 4 ? pair_row(g + 8) : make_uint2(0, 0);
#pragma unroll
            for (int t = 0; t < NR; ++t) mma(os[t], ra.x, rb.x, ra.y, rb.y, pb[t][0], pb[t][1]);
            // Codes: lane g takes word g % 4 of the group, the half g / 4 of it; of its
            // nibbles n, rows g and g + 8 of tile 2 k + (n >> 1) are 0, 1 and 2, 3.
            const uint32_t sel = (g & 4) ? 0x7632 : 0x5410;
            uint32_t sm0[Ge::kGroups], sm1[Ge::kGroups];
            lds_pairs(sm0, vp + g * Ge::kPairs);
            lds_pairs(sm1, vp + (g + 8) * Ge::kPairs);
#pragma unroll
            for (int k = 0; k < Ge::kGroups; ++k) {
              const float s0 = bf_lo(sm0[k]), s1 = bf_lo(sm1[k]);
              uint32_t sb[NR][2];
#pragma unroll
              for (int t = 0; t < NR; ++t) {
                sb[t][0] = transpose8(pack_bf16(st[u][t][0] * s0, st[u][t][1] * s0));
                sb[t][1] = transpose8(pack_bf16(st[u][t][2] * s1, st[u][t][3] * s1));
              }
              uint32_t w[2];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int r = 2 * c + 8 * h;
                w[h] = __byte_perm(lds32(vb + piece_at<D, K>(r, k) + 4 * (g & 3)),
                                   lds32(vb + piece_at<D, K>(r + 1, k) + 4 * (g & 3)), sel);
              }
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const uint32_t f0 = centred(code_pair(w[0], 2 * y));
                const uint32_t f1 = centred(code_pair(w[0], 2 * y + 1));
                const uint32_t f2 = centred(code_pair(w[1], 2 * y));
                const uint32_t f3 = centred(code_pair(w[1], 2 * y + 1));
#pragma unroll
                for (int t = 0; t < NR; ++t)
                  mma(o[t][2 * k + y], f0, f1, f2, f3, sb[t][0], sb[t][1]);
              }
            }
          }
        }
      }
      kb = kb + KT * Ge::kStage == ring + kStages * Ge::kStage ? ring : kb + KT * Ge::kStage;
    }
    copies_wait<0>();

    // Merge the warps: O^T, m, l of each in shared memory (the rings are done).
    __syncthreads();
    float* po = reinterpret_cast<float*>(smem);  // [warp][8 NR][D + 4]
    constexpr int LD = D + 4;
    float2* pml = reinterpret_cast<float2*>(smem + kWarps * 8 * NR * LD * 4);  // [warp][8 NR]
#pragma unroll
    for (int t = 0; t < NR; ++t) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int y = 4; y < 32; y <<= 1) l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], y);
        const int r = 8 * t + 2 * c + e;
        if (g == 0) pml[warp * 8 * NR + r] = make_float2(m[t][e], l[t][e]);
        float* dst = po + (warp * 8 * NR + r) * LD;
        if constexpr (K == kF32) {
#pragma unroll
          for (int x = 0; x < NK / 4; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              dst[4 * (16 * x + g) + y] = o[t][4 * x + y][e];
              dst[4 * (16 * x + 8 + g) + y] = o[t][4 * x + y][e + 2];
            }
        } else if constexpr (!Q4) {
#pragma unroll
          for (int k = 0; k < NK; ++k) {
            dst[16 * k + g] = o[t][k][e];
            dst[16 * k + g + 8] = o[t][k][e + 2];
          }
        } else {
          // Sums by group: row of m for group x, row of s for group x, column r.
#pragma unroll
          for (int k = 0; k < Ge::kGroups; ++k) {
            const int rm = k, rs = Ge::kGroups + k;  // rows of the pairs' product
            const float sm =
                __shfl_sync(0xffffffffu, rm < 8 ? os[t][e] : os[t][e + 2], (rm & 7) * 4 + c);
            const float ss =
                __shfl_sync(0xffffffffu, rs < 8 ? os[t][e] : os[t][e + 2], (rs & 7) * 4 + c);
            const float add = fmaf(8.f, ss, sm);
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                // Tile 2 k + y, row g + 8 h: nibble 2 y + h of half g / 4 of word g % 4.
                const int d = 32 * k + 8 * (g & 3) + (g & 4) + 2 * y + h;
                dst[d] = fmaf(16.f, o[t][2 * k + y][e + 2 * h], add);
              }
          }
        }
      }
    }
    __syncthreads();
    float* res = po + kWarps * 8 * NR * (LD + 2);  // [8 NR][D]: what a cluster's CTAs read
    float2* res_ml = reinterpret_cast<float2*>(res + 8 * NR * D);
    auto finish = [&](int r, int d, float M, float L, const float4& v) {
      const long long rr = r0 + r;
      const size_t row = (size_t)(q.q0 + (int)(rr / G)) * Hq + hk * G + (int)(rr % G);
      const float inv = L == 0.f ? 0.f : 1.f / L;
      if constexpr (K == kF32)
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + row * D + d) =
            make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
      else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * D + d) =
            make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
      if (a.lse && d == 0)
        a.lse[row] = L == 0.f ? -INFINITY : M * (scale * (Q4 ? 16.f : 1.f)) + logf(L);
    };
    // Add a partial (ml, v) to (L, acc) for the maximum `base`.
    auto add = [&](const float2& ml, const float4& x, float base, float& L, float4& acc) {
      if (ml.y == 0.f) return;  // nothing seen
      const float f = exp2a((ml.x - base) * k1);
      L = fmaf(f, ml.y, L);
      acc.x = fmaf(f, x.x, acc.x);
      acc.y = fmaf(f, x.y, acc.y);
      acc.z = fmaf(f, x.z, acc.z);
      acc.w = fmaf(f, x.w, acc.w);
    };
#pragma unroll 1
    for (bool last = K != kF32;; last = true) {
      float worst = 0.f;  // NaN if a sum is not finite
      for (int y = threadIdx.x; y < nr * (D / 4); y += kThreads) {
        const int r = y / (D / 4), d = 4 * (y % (D / 4));
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, pml[w * 8 * NR + r].x);
        const float base = M == -INFINITY ? 0.f : M;
        float L = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
          add(pml[w * 8 * NR + r],
              *reinterpret_cast<const float4*>(po + (w * 8 * NR + r) * LD + d), base, L, v);
        if (K == kF32)
          worst = fmaf(v.x, 0.f, fmaf(v.y, 0.f, fmaf(v.z, 0.f, fmaf(v.w, 0.f, fmaf(L, 0.f, worst)))));
        if (a.nsplit == 1) {
          finish(r, d, M, L, v);
        } else if (a.part_o) {
          const long long rr = r0 + r;
          const size_t row = (size_t)(q.q0 + (int)(rr / G)) * Hq + hk * G + (int)(rr % G);
          const size_t at = (size_t)split * s.n_tokens * Hq + row;
          *reinterpret_cast<float4*>(a.part_o + at * D + d) = v;
          if (d == 0) a.part_ml[at] = make_float2(M * (scale * (Q4 ? 16.f : 1.f)), L);
        } else {
          *reinterpret_cast<float4*>(res + r * D + d) = v;
          if (d == 0) res_ml[r] = make_float2(M, L);
        }
      }
      if (last || !__syncthreads_or(worst != 0.f)) break;
      in_plain_fp32<D>(s, a, Hkv, G, kWarps, r0, nr, k1, po + warp * 8 * NR * LD,
                       pml + warp * 8 * NR);
      __syncthreads();
    }
    if (a.nsplit > 1 && !a.part_o) {
      cluster_sync();  // every CTA's sums are there
      for (int y = split * kThreads + threadIdx.x; y < nr * (D / 4); y += a.nsplit * kThreads) {
        const int r = y / (D / 4), d = 4 * (y % (D / 4));
        const uint32_t ml_at = smem_addr(res_ml + r), v_at = smem_addr(res + r * D + d);
        float M = -INFINITY;
        for (int x = 0; x < a.nsplit; ++x) M = fmaxf(M, ld_cluster2(of_cta(ml_at, x)).x);
        const float base = M == -INFINITY ? 0.f : M;
        float L = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int x = 0; x < a.nsplit; ++x)
          add(ld_cluster2(of_cta(ml_at, x)), ld_cluster4(of_cta(v_at, x)), base, L, v);
        finish(r, d, M, L, v);
      }
      cluster_sync();  // and read by every CTA
    }
    __syncthreads();  // the next rows' copies land where these sums were
  }
}

template <int D, Kind K, int NR>
cudaError_t launch_nr(const Dims& d, const Seqs& s, const AttnArgs& a, cudaStream_t st) {
  static unsigned long long prepared = 0;
  using Ge = Geo<D, K>;
  constexpr int kThreads = 32 * Ge::warps(NR);
  constexpr int ring = Ge::warps(NR) * Ge::stages(NR) * Ge::kStage;
  constexpr int merge =
      Ge::warps(NR) * 8 * NR * ((D + 4) * 4 + 8) + 8 * NR * (D * 4 + 8);
  constexpr int smem = ring > merge ? ring : merge;
  cudaError_t e = prepare_kernel(decode_kernel<D, K, NR>, &prepared, smem);
  if (e != cudaSuccess) return e;
  const long long chunks = ((long long)min(a.max_q, s.n_tokens) * d.G + 8 * NR - 1) / (8 * NR);
  const dim3 grid((unsigned)(d.B * d.Hkv), (unsigned)(chunks < 65535 ? chunks : 65535),
                  (unsigned)a.nsplit);
  cudaLaunchAttribute cluster;
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim = {1, 1, (unsigned)a.nsplit};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &cluster;
  cfg.numAttrs = a.nsplit > 1 && !a.part_o ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, decode_kernel<D, K, NR>, s, a, d.Hq, d.Hkv, d.G,
                            1.f / sqrtf((float)D));
}
template <int D, Kind K>
cudaError_t launch(const Dims& d, const Seqs& s, const AttnArgs& a, cudaStream_t st) {
  if ((long long)a.max_q * d.G <= 8) return launch_nr<D, K, 1>(d, s, a, st);
  return launch_nr<D, K, 2>(d, s, a, st);
}

}  // namespace

int decode_ctas(const Dims& d, int nr) {
  if (d.format == DD_PAGES_Q4)
    return d.d == 64    ? Geo<64, kQ4>::ctas(nr)
           : d.d == 128 ? Geo<128, kQ4>::ctas(nr)
                        : Geo<256, kQ4>::ctas(nr);
  if (d.dtype == DD_BF16)
    return d.d == 64    ? Geo<64, kBf16>::ctas(nr)
           : d.d == 128 ? Geo<128, kBf16>::ctas(nr)
                        : Geo<256, kBf16>::ctas(nr);
  return d.d == 64 ? Geo<64, kF32>::ctas(nr) : Geo<128, kF32>::ctas(nr);
}

cudaError_t launch_attn_decode(const Dims& d, const Seqs& s, const AttnArgs& a, cudaStream_t st) {
  if (d.format == DD_PAGES_Q4) {
    if (d.d == 64) return launch<64, kQ4>(d, s, a, st);
    if (d.d == 128) return launch<128, kQ4>(d, s, a, st);
    if (d.d == 256) return launch<256, kQ4>(d, s, a, st);
  } else if (d.dtype == DD_BF16) {
    if (d.d == 64) return launch<64, kBf16>(d, s, a, st);
    if (d.d == 128) return launch<128, kBf16>(d, s, a, st);
    if (d.d == 256) return launch<256, kBf16>(d, s, a, st);
  } else {
    if (d.d == 64) return launch<64, kF32>(d, s, a, st);
    if (d.d == 128) return launch<128, kF32>(d, s, a, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace paged
}  // namespace dd
