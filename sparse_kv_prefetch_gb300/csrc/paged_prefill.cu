// dd_paged_attn for many tokens of a sequence, bf16 and 4-bit pages: both
// products on the tensor cores (tcgen05).
//
// Rows are (token, query head of the group) pairs of one KV head, NT tiles of
// 128 to a CTA; keys come in tiles of BN.  For each tile of keys
//   S = Q K^T           fp32 in tensor memory, one 128-lane row per thread,
//   P = 2^(c S - c m)   bf16, written back over S (c = log2 e / sqrt(d)),
//   O += P V            fp32 in tensor memory,
// with the running maximum m and sum l of each row in its thread's registers.
// O is rescaled only when a row's maximum has grown by more than 2^8 since the
// last time (the weights are then at most 2^8, far inside fp32 and, since
// rounding is relative, without loss in bf16), so it is hardly ever touched.
// Rounding P to bf16 (2^-8 relative at most per weight) is what the tensor
// cores take; l sums the unrounded weights.
//
// What bounds it: the two products, 4 BN 128 D operations a tile, against an
// exponential for each of its BN 128 logits.  So the roles are warps of their
// own, with mbarriers between them: one warp copies pages into a ring of
// 128-byte-swizzled tiles (TMA), one thread issues every matrix instruction,
// and a warpgroup per row tile does the softmax.  With NT = 2 the tensor cores
// work on one row tile while the other is in its softmax; with NT = 1 (d = 256,
// where two accumulators do not fit) two S buffers let the next Q K^T run
// beside the softmax.
//
// CTAs differ by their number of keys, and one fills an SM.  So a CTA goes on
// with the work of CTAs that have not started (cluster launch control hands it
// their places one at a time): the card stays full to the end, and the next Q, K
// and V are on their way, and S is computed, while the last rows are still being
// written.  Places are handed out from the highest row tile of the grid down: of
// prompts without a cached context that is the longest work first.  A sequence
// with few new tokens has only low row tiles, so its places come last however
// long its context is (a prompt of 2048 beside seven single tokens over 131072
// keys takes 982 us, the two apart 44 and 527).
//
// Measured (32 query heads, d = 128): prompts of 8192 and 3001 tokens on 8 KV
// heads 400 us with pauses between calls, 1559 TFLOP/s (a bf16 matrix product of
// 8192 reaches 1939), and 432 back to back, where power holds the clock; of 8192
// and 5000 with a window of 1024 on 32 KV heads 231 and 237 us, where a CTA has
// some ten tiles of keys, half of them cut by the mask.  With pauses, too: before
// the rows left through TMA 416 us, and 382 of them with the exponentials left
// out; issuing the products from `lane == 0` instead of an elected thread 570 and
// 339 us, and one CTA to each place of the grid 441 and 279.  On 8 KV heads back to
// back 337 us with d = 64, 1020 with d = 256.
//
// 4-bit pages: m + s c has more bits than a bf16, and rounding it would move
// the logits by 2^-9 of their terms.  Four warps widen each tile of codes into
// two bf16 tiles, the rounded values and what the rounding left (together good
// to 2^-17), and every product is issued for both: twice the work on the tensor
// cores, in tiles of 64 keys.  512 and 300 tokens over 32768 and 20011 positions
// 673 us, 38 of them the merge of eight splits.  Neither the widening bounds it
// (left out: 623 us) nor the products (the first of the two alone: 703): what is
// left is the chain of one tile, S, a softmax of only 64 columns, P V, with a
// barrier between each.
#include <math.h>

#include <type_traits>

#include "paged.cuh"
#include "tcgen05.cuh"

namespace dd {
namespace paged {
namespace {

__device__ unsigned int g_prefill_status = 0;

// Warps: 8 for the softmax; plain pages: one for the copies, the matrix warp, the
// one that asks for work, one idle; 4-bit pages: four that widen (eight measured
// no faster, 711 us), the matrix warp, the asking one, two idle.  Registers move
// from the other warpgroups to the softmax: 256 x 216 + 128 x 72 of the 384 x 168
// of the launch, 256 x 168 + 128 x 104 + 128 x 72 of 512 x 128.
template <bool Q4>
struct Roles {
  static constexpr int kThreads = Q4 ? 512 : 384;
  static constexpr int kCopyWarp = 8, kCopyWarps = Q4 ? 4 : 1, kMmaWarp = Q4 ? 12 : 9,
                       kAskWarp = kMmaWarp + 1;
  static constexpr int kSoftmaxRegs = Q4 ? 168 : 216, kCopyRegs = Q4 ? 104 : 72, kMmaRegs = 72;
};
constexpr uint32_t kTmemCols = 512;
constexpr float kLazy = 8.f;  // log2 of the growth that forces a rescale

template <int D, int NT, int BN, bool Q4>
struct Geo {
  static constexpr int kRows = NT * 128;
  static constexpr int kPanels = D / 64;
  static constexpr int kQTile = 128 * D * 2;
  static constexpr int kTile = BN * D * 2;
  static constexpr int kStage = kTile * (Q4 ? 2 : 1);
  static constexpr int kStages = (200 * 1024 - NT * kQTile) / kStage < 6
                                     ? (200 * 1024 - NT * kQTile) / kStage
                                     : 6;
  // 4-bit pages: codes and pairs on their way, kAhead - 1 tiles deep; each of the
  // 128 widening threads has kUnits groups of 32 (20 bytes) of a tile.
  static constexpr int kUnits = Q4 ? BN * D / 32 / 128 : 0;
  static constexpr int kAhead = D == 256 ? 3 : 6;
  static constexpr int kCodes = kUnits * 128 * 20;
  // Plain pages: 32 rows of a panel to each softmax warp, from where they are
  // stored (TMA) while the warp goes on.
  static constexpr int kOut = Q4 ? 0 : 32 * 128;
  static constexpr int kSmem =
      NT * kQTile + kStages * kStage + kAhead * kCodes + 4 * NT * kOut + 1024;
  static_assert(kSmem <= 226 * 1024, "shared memory");
  // Tensor memory columns: two S buffers (P over them), then the accumulators.
  static constexpr uint32_t kS = 0, kO = 2 * BN;
  static_assert(kO + NT * D <= kTmemCols, "tensor memory");
  static_assert(kStages >= (NT == 2 ? 4 : 2),
                "the ring must hold a tile of values and the next of keys");
};

struct Bars {
  uint64_t q_full, q_free;
  uint64_t full[6], empty[6];
  uint64_t s_full[2], p_ready[2];  // by S buffer
  uint64_t pv_done;                // NT = 1: after every P V
  uint64_t fix;                    // copies of a tile that is cleared before use
  uint64_t o_full[2];              // by row tile
  uint64_t given, taken;           // the next CTA's place: answered, read by every role
  uint4 answer;
  uint32_t tmem;
  uint32_t failed;                 // a role has given up
};

// The lowest n of 32 bits.
__device__ __forceinline__ uint32_t below(int n) {
  return n >= 32 ? ~0u : (1u << max(n, 0)) - 1u;
}

// N bytes global -> shared, or N zero bytes.
template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N),
               "r"(there ? N : 0)
               : "memory");
}
// 16 + nibble i of w.
__device__ __forceinline__ float code_16(uint32_t w, int i) {
  const uint32_t y = i < 5 ? w << (19 - 4 * i) : w >> (4 * i - 19);
  return __uint_as_float((y & 0x00780000u) | 0x41800000u);
}

__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}
// A wait that lasts as long as other roles' work, which grows with the number of
// keys: it ends with that work, or when a role whose waits are for single tiles
// (two seconds each) has given up and says so.
__device__ __forceinline__ bool wait_for_roles(uint64_t* bar, uint32_t parity,
                                               const uint32_t* failed) {
  for (uint32_t n = 0; !mbar_try_wait_sleep(bar, parity, 1000); ++n)
    if (*const_cast<const volatile uint32_t*>(failed) != 0 || n >= (1u << 30)) return false;
  return true;
}

template <int D, int NT, int BN, bool Q4>
__global__ void __launch_bounds__(Roles<Q4>::kThreads, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap q_map,
                   const __grid_constant__ CUtensorMap k_map,
                   const __grid_constant__ CUtensorMap v_map,
                   const __grid_constant__ CUtensorMap o_map, Seqs s, AttnArgs a, int Hq, int Hkv,
                   int G, float scale) {
  using Ge = Geo<D, NT, BN, Q4>;
  using Ro = Roles<Q4>;
  extern __shared__ unsigned char raw[];
  __shared__ Bars bars;
  unsigned char* q_sm = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
  unsigned char* ring = q_sm + NT * Ge::kQTile;
  unsigned char* out_sm = ring + Ge::kStages * Ge::kStage;  // plain pages
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == Ro::kMmaWarp) {
    if (lane == 0) {
      mbar_init(&bars.q_full, 1);
      mbar_init(&bars.q_free, 1);
      for (int i = 0; i < Ge::kStages; ++i) {
        mbar_init(&bars.full[i], Ro::kCopyWarps);
        mbar_init(&bars.empty[i], 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bars.s_full[i], 1);
        mbar_init(&bars.p_ready[i], 4);
        mbar_init(&bars.o_full[i], 1);
      }
      mbar_init(&bars.pv_done, 1);
      mbar_init(&bars.fix, 1);
      mbar_init(&bars.given, 1);
      bars.failed = 0;
      mbar_init(&bars.taken, Ro::kCopyWarps + 1 + 4 * NT);
      mbar_fence_init();
    }
    __syncwarp();
    tc::tmem_alloc(&bars.tmem, kTmemCols);
    tc::fence_before();
  }
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = bars.tmem;

  const int page = 1 << s.log2_page;
  const int sub = min(page, BN);  // rows of a box
  const int log2_sub = min(s.log2_page, ilog2(BN));
  const int nsub = BN >> log2_sub;
  bool ok = true;

  // The CTA's work: its own place in the grid, then those it is given.  A place
  // is a (sequence, KV head), a split, and row tiles from the last one on (the
  // one that sees the most keys; the grid is launched in that order), every
  // gridDim.y-th.  Every role walks over the same runs.
  struct Run {
    int b, hk, split;
    Seq q;
    long long rows, r0;
    int t0, i0, n;
    KeyTiles kt;
  };
  // body(run) returns false to stop.  `single`: called by one thread, else by a warp.
  auto each_run = [&](auto single, auto&& body) {
    int x = blockIdx.x, y = blockIdx.y, z = blockIdx.z;
    for (uint32_t phase = 0;; phase ^= 1) {
      Run r;
      r.b = x / Hkv;
      r.hk = x - r.b * Hkv;
      r.split = z;
      r.q = load_seq(s, r.b);
      r.rows = (long long)r.q.nq * G;
      for (long long tile = (int)gridDim.y - 1 - y; tile * Ge::kRows < r.rows; tile += gridDim.y) {
        r.r0 = tile * Ge::kRows;
        r.t0 = (int)(r.r0 / G);
        const int t1 = (int)((min(r.rows, r.r0 + Ge::kRows) - 1) / G);
        r.kt = key_tiles<BN>(r.q.pos0 + r.t0, r.q.pos0 + t1, r.q.len, a.window, a.sinks);
        r.i0 = (int)((long long)r.kt.n * z / a.nsplit);
        r.n = (int)((long long)r.kt.n * (z + 1) / a.nsplit) - r.i0;
        if (!body(r)) {
          ok = false;
          return;
        }
      }
      // A role without work in its last places (a row tile without rows) waits here
      // for those of the others.
      ok = wait_for_roles(&bars.given, phase, &bars.failed);
      if constexpr (!decltype(single)::value) ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      const bool more = tc::work_given(&bars.answer, x, y, z);
      tc::fence_async_smem();  // read before the next answer is written
      if constexpr (decltype(single)::value) {
        mbar_arrive(&bars.taken);
      } else {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.taken);
      }
      if (!more) return;
    }
  };
  const auto warp_wide = std::false_type{};
  // The key tiles that some row of row tile t sees (NT = 2): those that reach
  // into positions lo to hi, and those of the sinks.  `some`: the run has one.
  struct Active {
    int lo, hi, sinks;
    bool some;
    __device__ __forceinline__ bool at(int j) const {
      return j < hi && (j + BN > lo || j < sinks);
    }
  };
  auto active = [&](const Run& r, int t) {
    Active x{0, 0, 0, false};
    const long long rt = r.r0 + t * 128;
    if (rt >= r.rows) return x;
    x.hi = max(0, min(r.q.pos0 + (int)((min(r.rows, rt + 128) - 1) / G) + 1, r.kt.hi));
    x.lo = a.window > 0 ? min(max(0, r.q.pos0 + (int)(rt / G) - a.window + 1), x.hi) : 0;
    x.sinks = a.sinks;
    // In the run's numbering of tiles: [0, n_sink), then tile first + i - n_sink.
    auto meets = [&](int from, int to) { return max(from, r.i0) < min(to, r.i0 + r.n); };
    const int shift = r.kt.n_sink - r.kt.first, last = (x.hi + BN - 1) / BN + shift;
    const int sink_end = (int)min(((long long)a.sinks + BN - 1) / BN + shift, (long long)last);
    x.some = x.hi > 0 && (meets(0, r.kt.n_sink) || meets(r.kt.n_sink, sink_end) ||
                          meets(max(x.lo / BN, r.kt.first) + shift, last));
    return x;
  };

  if (warp == Ro::kAskWarp) {
    // -------------------------------------------------------------- more work
    tc::fewer_registers<Ro::kMmaRegs>();
    if (tc::elect_one()) {
      for (uint32_t phase = 0;; phase ^= 1) {
        mbar_arrive_expect_tx(&bars.given, 16);
        tc::ask_for_work(&bars.answer, &bars.given);
        if (!(ok = mbar_wait(&bars.given, phase))) break;
        int x, y, z;
        if (!tc::work_given(&bars.answer, x, y, z)) break;
        // Not asked again before every role has gone on to this one, which takes as
        // long as the work before it.
        if (!(ok = wait_for_roles(&bars.taken, phase, &bars.failed))) break;
      }
    }
    __syncwarp();
  } else if (!Q4 && warp == Ro::kCopyWarp) {
    // ---------------------------------------------------------------- copies
    tc::fewer_registers<Ro::kCopyRegs>();
    if (lane == 0) {
      tc::prefetch_map(&q_map);
      tc::prefetch_map(&k_map);
      tc::prefetch_map(&v_map);
    }
    int n_stage = 0, n_run = 0, n_fix = 0;
    each_run(warp_wide, [&](const Run& r) {
      const Seq& q = r.q;
      const int b = r.b, hk = r.hk;
      // Positions that no token of the sequence sees: from len on, and between
      // the sinks and the first token's window.
      const int lo_seq = a.window > 0 ? min(max(0, q.pos0 - a.window + 1), q.len) : 0;
      if (r.n == 0) return true;
      if (n_run > 0 && !wait_all(&bars.q_free, (n_run - 1) & 1)) return false;
      ++n_run;
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars.q_full, NT * Ge::kQTile);
        for (int t = 0; t < NT; ++t)
          for (int p = 0; p < Ge::kPanels; ++p)
            tc::tma_load_3d(q_sm + t * Ge::kQTile + p * (128 * 128), &q_map, 64 * p, hk * G,
                            q.q0 + r.t0 + t * (128 / G), &bars.q_full);
      }
      for (int i = 0; i < r.n; ++i) {
        const int j0 = r.kt.tile(r.i0 + i) * BN;
        // Lane x looks up box x's block; a box without one reads zeros.
        int z = s.n_pages * Hkv;
        if (lane < nsub && j0 + lane * sub < q.len) {
          const int pg = page_of(s, b, j0 + lane * sub);
          if (pg >= 0) z = pg * Hkv + hk;
        }
        const int y = j0 & (page - 1);  // nonzero only where a page has more than BN rows
        for (int kv = 0; kv < 2; ++kv, ++n_stage) {
          const int st = n_stage % Ge::kStages;
          if (n_stage >= Ge::kStages &&
              !wait_all(&bars.empty[st], (n_stage / Ge::kStages - 1) & 1))
            return false;
          unsigned char* dst = ring + st * Ge::kStage;
          // Values that no token sees may be anything, and 0 times them is not
          // 0: such a tile is copied, cleared there and only then handed on.
          const int end = min(max(q.len - j0, 0), BN);
          const int gap0 = min(max(a.sinks - j0, 0), BN), gap1 = min(max(lo_seq - j0, 0), BN);
          const bool clear = kv == 1 && (end < BN || gap0 < gap1);
          uint64_t* bar = clear ? &bars.fix : &bars.full[st];
          if (lane == 0) mbar_arrive_expect_tx(bar, Ge::kStage);
          __syncwarp();
          if (lane < nsub)
            for (int p = 0; p < Ge::kPanels; ++p)
              tc::tma_load_3d(dst + p * (BN * 128) + lane * sub * 128, kv ? &v_map : &k_map,
                              64 * p, y, z, bar);
          if (clear) {
            if (!wait_all(&bars.fix, n_fix & 1)) return false;
            ++n_fix;
            for (int x = lane; x < BN * Ge::kPanels * 8; x += 32) {
              const int row = (x >> 3) % BN;
              if (row >= end || (row >= gap0 && row < gap1))
                reinterpret_cast<uint4*>(dst)[x] = make_uint4(0, 0, 0, 0);
            }
            tc::fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.full[st]);
          }
        }
      }
      return true;
    });
  } else if (Q4 && warp >= Ro::kCopyWarp && warp < Ro::kCopyWarp + 4) {
    // --------------------------------------------------------------- widening
    tc::fewer_registers<Ro::kCopyRegs>();
    if constexpr (Q4) {
      constexpr int kUnits = Ge::kUnits;
      const unsigned char* codes = ring + Ge::kStages * Ge::kStage;
      static_assert(128 % BN == 0, "a thread's groups must be of one row");
      const int th = threadIdx.x - 32 * Ro::kCopyWarp;
      int n_stage = 0, n_run = 0;
      each_run(warp_wide, [&](const Run& r) {
        const Seq& q = r.q;
        const int b = r.b, hk = r.hk;
        const int lo_seq = a.window > 0 ? min(max(0, q.pos0 - a.window + 1), q.len) : 0;
        if (r.n == 0) return true;
        if (n_run > 0 && !wait_all(&bars.q_free, (n_run - 1) & 1)) return false;
        ++n_run;
        if (th == 0) {
          mbar_arrive_expect_tx(&bars.q_full, NT * Ge::kQTile);
          for (int t = 0; t < NT; ++t)
            for (int p = 0; p < Ge::kPanels; ++p)
              tc::tma_load_3d(q_sm + t * Ge::kQTile + p * (128 * 128), &q_map, 64 * p, hk * G,
                              q.q0 + r.t0 + t * (128 / G), &bars.q_full);
        }
        __syncwarp();
        // Stage 2 i has the keys of tile i, 2 i + 1 its values; of each a thread
        // widens groups th + 128 y: group u / BN of row u % BN, so that neighbouring
        // lanes store to neighbouring rows of the swizzled tile.  The groups are of
        // one row, whose page is looked up a tile ahead of its codes.
        auto find = [&](int i) {
          if (i >= r.n) return -1;
          const int j = r.kt.tile(r.i0 + i) * BN + th % BN;
          return j < q.len && (j < a.sinks || j >= lo_seq) ? page_of(s, b, j) : -1;
        };
        int pg = find(0), pg_next = find(1);
        auto fetch = [&](int x) {
          if (x < 2 * r.n) {
            if (x > 0 && !(x & 1)) {
              pg = pg_next;
              pg_next = find((x >> 1) + 1);
            }
            const int pr = (r.kt.tile(r.i0 + (x >> 1)) * BN + th % BN) & (page - 1);
            const unsigned char* blk =
                ((x & 1) ? s.v : s.k) + ((size_t)max(pg, 0) * Hkv + hk) * s.block_bytes;
            const uint32_t to = smem_addr(codes) + (x % Ge::kAhead) * Ge::kCodes;
#pragma unroll
            for (int i = 0; i < kUnits; ++i) {
              const int grp = (th + 128 * i) / BN;
              // Rows that no token of the sequence sees become zeros.
              copy_async<16>(to + 16 * (th + 128 * i), blk + pr * (D / 2) + 16 * grp, pg >= 0);
              copy_async<4>(to + 16 * 128 * kUnits + 4 * (th + 128 * i),
                            blk + page * (D / 2) + pr * (D / 8) + 4 * grp, pg >= 0);
            }
          }
          asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll 1
        for (int x = 0; x < Ge::kAhead - 1; ++x) fetch(x);
#pragma unroll 1
        for (int x = 0; x < 2 * r.n; ++x, ++n_stage) {
          const int st = n_stage % Ge::kStages;
          // A thread reads what it copied itself.
          asm volatile("cp.async.wait_group %0;" ::"n"(Ge::kAhead - 2) : "memory");
          const unsigned char* from = codes + (x % Ge::kAhead) * Ge::kCodes;
          uint4 now[kUnits];
          uint32_t sm[kUnits];
#pragma unroll
          for (int i = 0; i < kUnits; ++i) {
            now[i] = *reinterpret_cast<const uint4*>(from + 16 * (th + 128 * i));
            sm[i] = *reinterpret_cast<const uint32_t*>(from + 16 * 128 * kUnits + 4 * (th + 128 * i));
          }
          fetch(x + Ge::kAhead - 1);
          if (n_stage >= Ge::kStages &&
              !wait_all(&bars.empty[st], (n_stage / Ge::kStages - 1) & 1))
            return false;
          unsigned char* dst = ring + st * Ge::kStage;
#pragma unroll
          for (int i = 0; i < kUnits; ++i) {
            const int u = th + 128 * i, row = u % BN, grp = u / BN;
            const float step = __uint_as_float(sm[i] << 16);
            // m + s c = (m - 16 s) + s (16 + c): 16 + c is an fp32 with the code in its
            // mantissa, and m - 16 s loses no more than fp32 does.
            const float low = fmaf(-16.f, step, __uint_as_float(sm[i] & 0xFFFF0000u));
            const uint32_t w[4] = {now[i].x, now[i].y, now[i].z, now[i].w};
            unsigned char* to = dst + (grp / 2) * (BN * 128) + row * 128;
#pragma unroll
            for (int e = 0; e < 4; ++e) {  // word e: 8 codes, a 16-byte piece of each tile
              uint32_t hi[4], lo[4];
#pragma unroll
              for (int h = 0; h < 4; ++h) {
                const float v0 = fmaf(step, code_16(w[e], 2 * h), low);
                const float v1 = fmaf(step, code_16(w[e], 2 * h + 1), low);
                hi[h] = pack_bf16(v0, v1);
                lo[h] = pack_bf16(v0 - __uint_as_float(hi[h] << 16),
                                  v1 - __uint_as_float(hi[h] & 0xFFFF0000u));
              }
              const int piece = ((grp & 1) * 4 + e) ^ (row & 7);
              *reinterpret_cast<uint4*>(to + 16 * piece) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
              *reinterpret_cast<uint4*>(to + Ge::kTile + 16 * piece) =
                  make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
          }
          tc::fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars.full[st]);
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        return true;
      });
    }
  } else if (warp == Ro::kMmaWarp) {
    // ------------------------------------------------------ matrix instructions
    tc::fewer_registers<Ro::kMmaRegs>();
    if (tc::elect_one()) {
      constexpr uint32_t kIdescS = tc::instr_bf16(128, BN, false);
      constexpr uint32_t kIdescO = tc::instr_bf16(128, D, true);
      const uint64_t q_desc = tc::desc_k(smem_addr(q_sm));
      const uint64_t k_desc = tc::desc_k(smem_addr(ring));
      const uint64_t v_desc = tc::desc_mn(smem_addr(ring), BN * 128);
      // Contraction steps of 16: along the panels for S, along the keys for O; `at` is
      // the stage's offset in the ring.
      auto issue_s = [&](int t, uint32_t d, uint32_t at) {
        const uint64_t qd = tc::further(q_desc, t * Ge::kQTile), kd = tc::further(k_desc, at);
#pragma unroll
        for (int h = 0; h < (Q4 ? 2 : 1); ++h)
#pragma unroll
          for (int e = 0; e < D / 16; ++e)
            tc::mma_ss(d, tc::further(qd, (e / 4) * (128 * 128) + (e % 4) * 32),
                       tc::further(kd, h * Ge::kTile + (e / 4) * (BN * 128) + (e % 4) * 32),
                       kIdescS, h > 0 || e > 0);
      };
      auto issue_o = [&](uint32_t d, uint32_t p, uint32_t at, bool add) {
        const uint64_t vd = tc::further(v_desc, at);
#pragma unroll
        for (int h = 0; h < (Q4 ? 2 : 1); ++h)
#pragma unroll
          for (int e = 0; e < BN / 16; ++e)
            tc::mma_ts(d, p + 8 * e, tc::further(vd, h * Ge::kTile + e * 2048), kIdescO,
                       add || h > 0 || e > 0);
      };
      int n_stage = 0, n_run = 0;  // next stage to take
      int phase[2] = {0, 0};       // of p_ready, by S buffer
      auto take = [&](int x) {     // wait for stage number x of the ring
        return mbar_wait(&bars.full[x % Ge::kStages], (x / Ge::kStages) & 1);
      };
      auto addr = [&](int x) { return (uint32_t)(x % Ge::kStages) * Ge::kStage; };
      auto free_stage = [&](int x) { tc::commit(&bars.empty[x % Ge::kStages]); };
      each_run(std::true_type{}, [&](const Run& r) {
        if (r.n == 0) return true;
        if (!mbar_wait(&bars.q_full, n_run & 1)) return false;
        ++n_run;
        // Stage numbers of tile i: keys base + 2 i, values base + 2 i + 1.
        const int base = n_stage;
        n_stage += 2 * r.n;
        if (!take(base)) return false;
        tc::fence_after();
        if constexpr (NT == 1) {
          issue_s(0, tmem + Ge::kS, addr(base));
          tc::commit(&bars.s_full[0]);
          free_stage(base);
          if (r.n == 1) tc::commit(&bars.q_free);
          for (int i = 0; i < r.n; ++i) {
            const int kx = base + 2 * (i + 1), vx = base + 2 * i + 1;
            if (i + 1 < r.n) {  // the next S beside this one's softmax
              if (!take(kx)) return false;
              issue_s(0, tmem + Ge::kS + ((i + 1) & 1) * BN, addr(kx));
              tc::commit(&bars.s_full[(i + 1) & 1]);
              free_stage(kx);
              if (i + 2 == r.n) tc::commit(&bars.q_free);
            }
            if (!take(vx) || !mbar_wait(&bars.p_ready[i & 1], phase[i & 1])) return false;
            phase[i & 1] ^= 1;
            tc::fence_after();
            issue_o(tmem + Ge::kO, tmem + Ge::kS + (i & 1) * BN, addr(vx), i > 0);
            tc::commit(&bars.pv_done);
            if (i + 1 == r.n) tc::commit(&bars.o_full[0]);
            free_stage(vx);
          }
        } else {
          // A row tile skips key tiles that none of its rows sees.
          const Active act0 = active(r, 0), act1 = active(r, 1);
          bool any0 = false, any1 = false;
          if (act0.at(r.kt.tile(r.i0) * BN)) {
            issue_s(0, tmem + Ge::kS, addr(base));
            tc::commit(&bars.s_full[0]);
          }
          if (act1.at(r.kt.tile(r.i0) * BN)) {
            issue_s(1, tmem + Ge::kS + BN, addr(base));
            tc::commit(&bars.s_full[1]);
          }
          free_stage(base);
          if (r.n == 1) tc::commit(&bars.q_free);
          for (int i = 0; i < r.n; ++i) {
            const bool more = i + 1 < r.n;
            const int kx = base + 2 * (i + 1), vx = base + 2 * i + 1;
            const int j = r.kt.tile(r.i0 + i) * BN;
            const int jn = more ? r.kt.tile(r.i0 + i + 1) * BN : 0;
            if (!take(vx)) return false;
            if (act0.at(j)) {
              if (!mbar_wait(&bars.p_ready[0], phase[0])) return false;
              phase[0] ^= 1;
              tc::fence_after();
              issue_o(tmem + Ge::kO, tmem + Ge::kS, addr(vx), any0);
              any0 = true;
            }
            if (more) {
              if (!take(kx)) return false;
              if (act0.at(jn)) {
                issue_s(0, tmem + Ge::kS, addr(kx));
                tc::commit(&bars.s_full[0]);
              }
            } else if (act0.some) {
              tc::commit(&bars.o_full[0]);
            }
            if (act1.at(j)) {
              if (!mbar_wait(&bars.p_ready[1], phase[1])) return false;
              phase[1] ^= 1;
              tc::fence_after();
              issue_o(tmem + Ge::kO + D, tmem + Ge::kS + BN, addr(vx), any1);
              any1 = true;
            }
            free_stage(vx);
            if (more) {
              if (act1.at(jn)) {
                issue_s(1, tmem + Ge::kS + BN, addr(kx));
                tc::commit(&bars.s_full[1]);
              }
              free_stage(kx);
              if (i + 2 == r.n) tc::commit(&bars.q_free);
            } else if (act1.some) {
              tc::commit(&bars.o_full[1]);
            }
          }
        }
        return true;
      });
    }
    __syncwarp();
  } else if (warp < 4 * NT) {
    // ---------------------------------------------------------------- softmax
    tc::more_registers<Ro::kSoftmaxRegs>();
    const int t = warp >> 2;                      // row tile
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // the warp's 32 lanes
    const int row = (warp & 3) * 32 + lane;
    const float c = scale * 1.4426950408889634f;
    int s_phase[2] = {0, 0}, o_phase = 0, pv_phase = 0;
    each_run(warp_wide, [&](const Run& r) {
      const Seq& q = r.q;
      const int b = r.b, hk = r.hk, split = r.split;
      const long long rt = r.r0 + t * 128;  // first row of the tile
      if (rt >= r.rows) return true;
      const Active act = active(r, t);
      const int pos = q.pos0 + (int)((rt + row) / G);
      const int pos_min = q.pos0 + (int)(rt / G), pos_max = q.pos0 + (int)((rt + 127) / G);
      float m = -INFINITY, l = 0.f;
      bool first = true;
      for (int i = 0; i < r.n; ++i) {
        const int j0 = r.kt.tile(r.i0 + i) * BN;
        if (NT == 2 && !act.at(j0)) continue;
        const int buf = NT == 1 ? (i & 1) : t;
        // Which boxes of the tile have a page.
        const bool has = lane < nsub && j0 + lane * sub < q.len && page_of(s, b, j0 + lane * sub) >= 0;
        const uint32_t pages = __ballot_sync(0xffffffffu, has);
        if (!wait_all(&bars.s_full[buf], s_phase[buf])) return false;
        s_phase[buf] ^= 1;
        tc::fence_after();
        uint32_t x[BN];
        const uint32_t s_addr = tmem + lanes + Ge::kS + buf * BN;
#pragma unroll
        for (int k = 0; k < BN; k += 32) tc::tmem_ld32(s_addr + k, x + k);
        tc::tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < BN; k += 32) tc::tmem_loaded32(x + k);
        const bool all = j0 + BN - 1 <= pos_min && pages == (nsub == 32 ? ~0u : (1u << nsub) - 1u) &&
                         (a.window == 0 || j0 > pos_max - a.window || j0 + BN <= a.sinks);
        if (!all) {
          // Columns [0, sink) and (first, last] of this row are visible.
          const int last = pos - j0, sink = min(a.sinks, pos + 1) - j0;
          const int first = a.window > 0 ? last - a.window : -1;
#pragma unroll
          for (int k = 0; k < BN; k += 32) {
            uint32_t keep = (below(last + 1 - k) & ~below(first + 1 - k)) | below(sink - k);
            if (log2_sub >= 5) {
              if (!((pages >> (k >> log2_sub)) & 1u)) keep = 0;
            } else {
              const uint32_t two = pages >> (k >> 4);
              keep &= ((two & 1u) ? 0xFFFFu : 0u) | ((two & 2u) ? 0xFFFF0000u : 0u);
            }
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(keep & (1u << e))) x[k + e] = 0xff800000u;
          }
        }
        float top[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) top[e] = __uint_as_float(x[e]);
#pragma unroll
        for (int k = 4; k + 8 <= BN; k += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            top[e] = tc::max3(top[e], __uint_as_float(x[k + 2 * e]), __uint_as_float(x[k + 2 * e + 1]));
#pragma unroll
        for (int e = 0; e < 4; ++e) top[e] = fmaxf(top[e], __uint_as_float(x[BN - 4 + e]));
        const float tm = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        const bool grow = (tm - m) * c > kLazy || (m == -INFINITY && tm > m);
        if (first) {
          m = tm;
          first = false;
        } else if (__any_sync(0xffffffffu, grow)) {
          // S of this tile was computed after the last P V of this row tile
          // (NT = 2), or the barrier says that it is done (NT = 1).
          if constexpr (NT == 1) {
            if (!wait_all(&bars.pv_done, pv_phase ^ 1)) return false;
            tc::fence_after();
          }
          const float f = grow ? tc::ex2((m - tm) * c) : 1.f;
          if (grow) m = tm;
          l *= f;
          const uint32_t o_addr = tmem + lanes + Ge::kO + t * D;
#pragma unroll 1
          for (int k = 0; k < D; k += 32) {
            uint32_t o[32];
            tc::tmem_ld32(o_addr + k, o);
            tc::tmem_wait_ld();
            tc::tmem_loaded32(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tc::tmem_st32(o_addr + k, o);
          }
        }
        if constexpr (NT == 1) pv_phase ^= 1;
        const float off = m == -INFINITY ? 0.f : -m * c;
        uint64_t sum[4] = {0, 0, 0, 0};
        const uint64_t c2 = tc::pair(c, c), off2 = tc::pair(off, off);
#pragma unroll
        for (int k = 0; k < BN; k += 64) {
          uint32_t pk[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float p0, p1;
            tc::unpair(tc::fma2(tc::pair(__uint_as_float(x[k + 2 * e]),
                                         __uint_as_float(x[k + 2 * e + 1])),
                                c2, off2),
                       p0, p1);
            p0 = tc::ex2(p0);
            p1 = tc::ex2(p1);
            sum[e & 3] = tc::add2(sum[e & 3], tc::pair(p0, p1));
            pk[e] = pack_bf16(p0, p1);
          }
          tc::tmem_st32(s_addr + k / 2, pk);
        }
        tc::tmem_wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.p_ready[buf]);
        float s0, s1;
        tc::unpair(tc::add2(tc::add2(sum[0], sum[1]), tc::add2(sum[2], sum[3])), s0, s1);
        l += s0 + s1;
      }
      const bool some = NT == 1 ? r.n > 0 : act.some;
      if (some) {
        if (!wait_all(&bars.o_full[t], o_phase)) return false;
        o_phase ^= 1;
        tc::fence_after();
      }
      const long long rr = rt + row;
      const bool mine = rr < r.rows;
      const size_t at = mine ? (size_t)(q.q0 + (int)(rr / G)) * Hq + hk * G + (int)(rr % G) : 0;
      const bool empty = l == 0.f;
      const float inv = empty ? 0.f : 1.f / l;
      const uint32_t o_addr = tmem + lanes + Ge::kO + t * D;
      const size_t pat = (size_t)split * s.n_tokens * Hq + at;
      // Whole warps of rows leave through shared memory, 64 elements at a time.
      const bool staged = !Q4 && a.nsplit == 1 && rt + 32 * (warp & 3) + 32 <= r.rows;
      if (staged) {
        unsigned char* stage = out_sm + warp * Ge::kOut;
        const int token = q.q0 + (int)((rt + 32 * (warp & 3)) / G);
#pragma unroll 1
        for (int p = 0; p < Ge::kPanels; ++p) {
          uint32_t o[64];
          if (some) {
            tc::tmem_ld32(o_addr + 64 * p, o);
            tc::tmem_ld32(o_addr + 64 * p + 32, o + 32);
            tc::tmem_wait_ld();
            tc::tmem_loaded32(o);
            tc::tmem_loaded32(o + 32);
          }
          if (!some || empty) {
#pragma unroll
            for (int e = 0; e < 64; ++e) o[e] = 0;
          }
          if (lane == 0) bulk_wait_read_all();  // the panel before has been read
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            uint32_t w[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
              w[u] = pack_bf16(__uint_as_float(o[8 * e + 2 * u]) * inv,
                               __uint_as_float(o[8 * e + 2 * u + 1]) * inv);
            *reinterpret_cast<uint4*>(stage + lane * 128 + 16 * (e ^ (lane & 7))) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
          tc::fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            tc::tma_store_3d(&o_map, stage, 64 * p, hk * G, token);
            bulk_commit();
          }
        }
      }
#pragma unroll 1
      for (int k = staged ? D : 0; k < D; k += 32) {
        uint32_t o[32];
        __syncwarp();
        if (some) {
          tc::tmem_ld32(o_addr + k, o);
          tc::tmem_wait_ld();
          tc::tmem_loaded32(o);
        }
        if (!some || empty) {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0;
        }
        if (mine && a.nsplit > 1) {
          uint4* dst = reinterpret_cast<uint4*>(a.part_o + pat * D + k);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            dst[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        } else if (mine) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at * D + k);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t w[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
              w[u] = pack_bf16(__uint_as_float(o[8 * e + 2 * u]) * inv,
                               __uint_as_float(o[8 * e + 2 * u + 1]) * inv);
            dst[e] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      if (mine) {
        if (a.nsplit > 1)
          a.part_ml[pat] = make_float2(empty ? -INFINITY : m * scale, l);
        else if (a.lse)
          a.lse[at] = empty ? -INFINITY : m * scale + logf(l);
      }
      tc::fence_before();  // the next run's P V overwrites O after p_ready
      return true;
    });
    if (lane == 0) bulk_wait_all();  // the last rows have left
    __syncwarp();
  } else {
    if (warp < 8 || !Q4)
      tc::fewer_registers<Ro::kCopyRegs>();
    else
      tc::fewer_registers<Ro::kMmaRegs>();
  }
  // A wait that gave up leaves its role and says so, and every role behind it gives up
  // in its turn, seconds after the last copy or product has landed.
  if (!ok) {
    *const_cast<volatile uint32_t*>(&bars.failed) = 1;
    g_prefill_status = 1;
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  if (warp == Ro::kMmaWarp) {
    tc::fence_after();
    tc::tmem_free(tmem, kTmemCols);
  }
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// A map of bf16 [n2][n1][d], boxes of 64 elements by b1 by b2.
bool make_map(CUtensorMap* m, const void* p, uint64_t d, uint64_t n1, uint64_t n2, uint64_t stride1,
              uint64_t stride2, uint32_t b1, uint32_t b2) {
  const EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {d, n1, n2};
  const cuuint64_t strides[2] = {stride1, stride2};
  const cuuint32_t box[3] = {64, b1, b2}, step[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int NT, int BN, bool Q4>
cudaError_t launch(const Dims& d, const Seqs& s, const AttnArgs& a, cudaStream_t st) {
  using Ge = Geo<D, NT, BN, Q4>;
  static unsigned long long prepared = 0;
  cudaError_t e = prepare_kernel(prefill_kernel<D, NT, BN, Q4>, &prepared, Ge::kSmem);
  if (e != cudaSuccess) return e;
  CUtensorMap qm, km, vm;
  const uint64_t row = (uint64_t)D * 2;
  const int sub = d.page < BN ? d.page : BN;
  if (!make_map(&qm, a.q, D, d.Hq, s.n_tokens, row, a.q_stride, d.G, 128 / d.G))
    return cudaErrorInvalidValue;
  CUtensorMap om;
  if (Q4)
    km = vm = om = qm;  // not used
  else if (!make_map(&om, a.out, D, d.Hq, s.n_tokens, row, row * d.Hq, d.G, 32 / d.G) ||
           !make_map(&km, s.k, D, d.page, (uint64_t)d.n_pages * d.Hkv, row, row * d.page, sub, 1) ||
           !make_map(&vm, s.v, D, d.page, (uint64_t)d.n_pages * d.Hkv, row, row * d.page, sub, 1))
    return cudaErrorInvalidValue;
  const long long tiles =
      ((long long)min(a.max_q, s.n_tokens) * d.G + Ge::kRows - 1) / Ge::kRows;
  const dim3 grid((unsigned)(d.B * d.Hkv), (unsigned)(tiles < 65535 ? tiles : 65535),
                  (unsigned)a.nsplit);
  prefill_kernel<D, NT, BN, Q4><<<grid, Roles<Q4>::kThreads, Ge::kSmem, st>>>(
      qm, km, vm, om, s, a, d.Hq, d.Hkv, d.G, 1.f / sqrtf((float)D));
  return cudaGetLastError();
}

}  // namespace

int prefill_rows(const Dims& d) { return d.d == 256 ? 128 : 256; }

cudaError_t launch_attn_prefill(const Dims& d, const Seqs& s, const AttnArgs& a, cudaStream_t st) {
  if (d.format == DD_PAGES_Q4) {
    if (d.d == 64) return launch<64, 2, 64, true>(d, s, a, st);
    if (d.d == 128) return launch<128, 2, 64, true>(d, s, a, st);
    if (d.d == 256) return launch<256, 1, 64, true>(d, s, a, st);
  } else {
    if (d.d == 64) return launch<64, 2, 128, false>(d, s, a, st);
    if (d.d == 128) return launch<128, 2, 128, false>(d, s, a, st);
    if (d.d == 256) return launch<256, 1, 64, false>(d, s, a, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace paged

unsigned int take_prefill_status() {
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, paged::g_prefill_status, sizeof v) != cudaSuccess) return 0;
  if (v) cudaMemcpyToSymbol(paged::g_prefill_status, &zero, sizeof zero);
  return v;
}

}  // namespace dd
