// decode_shared.cu -- the shared-prefix decode: one query per (sequence, head)
// against a prefix that the whole batch shares and the sequence's own cache rows,
// joined in one softmax:
//   s_j = <q P_h, K~_j> / sqrt(m),  O = sum_j softmax(s)_j V_j
// over rows 0 .. plen-1 of the prefix cache and 0 .. lens[b]-1 of the
// sequence's; query heads h*G .. h*G+G-1 share key head h.  This file: the prefix
// kernel and the layout of a call; the other kernels are in decode_own.cu.
//
// The prefix kernel is persistent, one CTA per SM.  Work is cut into segments, a
// row tile of queries against a run of 128-key tiles:
//   prefix   all rows of the tile; segments go round robin with the row tiles
//            fastest, so that CTAs side by side stream the same keys and all but
//            one read them from L2
//   own      (groups of more than 32 heads) one group against its sequence's rows,
//            an equal share of all own tiles for every CTA
// Sixteen warps in four warpgroups:
//   warps 0-3, 4-7   softmax of the tiles of even / odd number (two streams)
//   warps 8-11       output: a finished segment's sums, both streams joined
//   warp  12         the list of segments (the divisions and the sequences' lengths
//                    are its work alone) and their V tiles, by TMA into a ring
//   warp  13         tensor-memory allocation, q~ tiles, tcgen05.mma issue
//   warps 14, 15     K~ tiles, each warp every other one, by TMA into a ring of its
//                    own: a tile's multipliers become one range for its rows
// The streams alternate tile by tile, each with scores and sums of its own in
// tensor memory (S0 | S1 | O0 | O1), so that the products of one run while the
// other is exponentiated.
//
// Scores.  q~ comes split into two fp16 parts (22 bits), so the scores carry
// fp32's precision.  The cache rows are fp16 with a power of two each; a warp
// brings the rows of a tile to the largest multiplier of them in shared memory, and
// the tile's common factor joins the row's.  A row's largest entry is 2^13 or more, so
// down to a factor of 2^-14 its entries lose less than 2^-24 of it (what falls below
// fp16's 2^-24 is rounded); where a tile's multipliers are further apart, as beside a
// row of zeros, whose multiplier is 1, the rows stay as they are and the softmax takes
// each score by its own key's.  (That for every tile, read from shared memory, made the
// softmax of a tile 600 cycles longer, of 2200.)  K~ and V have rings of their own
// because a K~ slot is free again once the scores are formed; with both in one slot
// the way from a free slot to scores that can be formed took 3500 cycles, and with
// the three slots that fit at m = 64 a tile took 2300.
// Probabilities are rounded to bf16 for the value product (2^-8 relative, each key's
// by itself: with the output's own rounding an output is off by 0.0023 in the mean,
// for 0.0017 with the output's alone); their sums, and the weights that are
// accumulated, take them in fp32.  With the parts that bf16 leaves as a second value
// product, as the kernel of the own rows has it, 65536 keys for 512 rows of 8 key
// heads took 323 us for 251 in the whole call and 32768 keys for 128 rows 55 for 46:
// the tensor pipe and the softmax are what bounds this kernel, so one part it is.
//
// Softmax in base 2 with the running maximum moved only when a row's tile sum
// exceeds 2^40, as in the forward.  Key columns behind a length are replaced
// by -inf after the product, and value rows behind it are zeroed in shared
// memory up to the 16 rows that one MMA step reads: what they hold (NaN too)
// is never used.  A segment's sums start afresh, so that one sequence's values
// never meet another's rows.
//
// What bounds it.  65536 keys against 512 rows of each of 8 key heads (m = 64, d_v =
// 128): 155 us, 2570 cycles per tile and row tile; the products alone would take 1070
// (the score product's K is 2 m for the two parts of q~).  A tile moves 176 KB through
// the SM's shared memory, 1400 cycles at 128 bytes a cycle: both operands of the score
// product, V, what TMA writes and the range pass.  The issuer is held up by the tensor
// pipe for 1600 cycles of a tile and waits for probabilities for 630 (clocks of a build
// without the check of a tile's range, whose tiles took 2450).  32768 keys against 128
// rows (m = 32): 29.5 us, 1750 cycles per tile, which is the memory bandwidth, and
// 10000 + 6000 cycles of start and end.  One score buffer that both
// streams read into registers, with the probabilities beside it and the scores three
// tiles ahead, took the softmax out of the way between two score products, and the
// large case took 266 us for 251 then: the issuer then waited for nothing, and each product
// took longer.
//
// Every wait is bounded; a role that gives up sets the CTA's abort flag and
// the device error word, and all roles leave after their own operations in
// flight have ended.
#include <math.h>

#include <cstddef>

#include "decode_shared.cuh"
#include "ptx.cuh"
#include "waits.cuh"

namespace spa {
using namespace ds;
namespace {

using namespace ptx;

constexpr int kThreads = 512;
constexpr uint32_t kRegSoftmax = 168, kRegOutput = 104, kRegControl = 72;
static_assert(128 * (2 * kRegSoftmax + kRegOutput + kRegControl) <= kThreads * 128,
              "register split exceeds the launch");
constexpr int kLoadWarp = 12, kMmaWarp = 13;
constexpr int kSegs = 8;               // segments the scheduler may be ahead
constexpr int kSegReaders = 1 + 2 + 4 + 8;  // issuer, multipliers, output warps, softmax warps
constexpr float kSumLimit = 1099511627776.f;  // 2^40
constexpr int kMaxDynSmem = 227 * 1024 - 10 * 1024;
constexpr float kRange = 1.f / 16384.f;  // 2^-14: what the rows of a tile may be apart for one range

constexpr int cmax(int a, int b) { return a > b ? a : b; }

template <int M, int DV>
struct Plan {
  static constexpr int kKBytes = kTile * M * 2, kVBytes = kTile * DV * 2;
  static constexpr int kKRow = M < 64 ? M * 2 : 128;  // bytes of a K~ row in shared memory (a box)
  static constexpr int kQBytes = kTile * 4 * M;
  static constexpr int kQ = 0, kOut = kQBytes;
  static constexpr int kKs = kOut + 4 * 4096;  // a box of 32 x 32 sums per output warp
  static constexpr int kKStages = M == 128 ? 1 : M == 64 ? 2 : 3;  // of each of the two K~ rings
  static constexpr int kVs = kKs + 2 * kKStages * kKBytes;
  static constexpr int kFit = (kMaxDynSmem - 1024 - kVs) / kVBytes;
  static constexpr int kVStages = kFit > 4 ? 4 : kFit;
  static constexpr int kBytes = kVs + kVStages * kVBytes + 1024;
  // one CTA per SM: a second one would wait in tcgen05.alloc for the 512 columns
  static constexpr int kLaunch = cmax(kBytes, 120 * 1024);
  static_assert(kVStages >= 2 && kLaunch <= kMaxDynSmem, "shared-memory plan");
  static constexpr uint32_t kColS = 0, kColO = 256;
};

// A run of key tiles for rows lo .. hi-1 of one row tile.
struct alignas(16) Seg {
  int own, qnew, hk, rt;
  int lo, hi;
  int plane, key0;   // tensor-map coordinates of the first key
  int tiles, keys;   // tiles = 0: the end
  int row;           // partial result of lane r: row + r
  int srow;          // own: score row of lane r: srow + r
};

struct Shared {
  uint64_t v_full[4], v_empty[4];
  uint64_t k_full[2][3], k_empty[2][3], k_ready[2][3];  // ready: the tile's rows are in one range
  uint64_t s_full[2], p_full[2], o_final[2], o_empty[2];
  uint64_t q_empty, q_full, drain;
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint32_t tmem;
  volatile int abort;
  Seg seg[kSegs];
  float stat_l[2][2][kTile], stat_m[2][2][kTile];
  // by the tile's number: a K~ slot is filled again once the scores of the tile that was
  // in it are formed, six tiles behind at most, and those wait until the softmax is done
  // with the tile two in front; so no reader is eight tiles behind
  alignas(16) float mul[8][kTile];
  float kscale[8];  // 0: the rows of the tile keep their own multipliers
};
static_assert(offsetof(Shared, seg) % 16 == 0 && alignof(Shared) >= 16, "vector loads from shared memory");
static_assert(sizeof(Shared) <= 10 * 1024 - 256, "static shared memory");
static_assert(offsetof(Shared, mul) % 16 == 0, "vector loads from shared memory");

// The CTA's segments in order, then the end: told to the other roles, then given
// to `load`.
template <class Load>
__device__ __forceinline__ void run_segments(const Params& a, Shared& sh, const WaitCtl& ctl, Load load) {
  const Geo& g = a.g;
  const int lane = threadIdx.x & 31, B = a.p.B;
  int k = 0, last = -1;
  auto emit = [&](Seg s) -> bool {
    const int slot = k % kSegs;
    if (k >= kSegs && !__all_sync(0xffffffffu, wait_or_abort(&sh.seg_empty[slot], (k / kSegs - 1) & 1, ctl)))
      return false;
    const int q = s.hk * g.RT + s.rt;
    s.qnew = q != last;
    last = q;
    if (lane == 0) {
      sh.seg[slot] = s;
      mbar_arrive(&sh.seg_full[slot]);
    }
    ++k;
    return s.tiles == 0 || load(s);
  };
  for (int unit = blockIdx.x; unit < g.units; unit += g.grid) {
    Seg s{};
    const int us = g.dRT(unit);
    s.rt = unit - us * g.RT;
    s.hk = g.dS(us);
    const int split = us - s.hk * g.S;
    s.row = ((s.hk * g.RT + s.rt) * g.S + split) * g.rows;
    s.hi = g.parts > 1 ? min(kTile, a.p.G - (s.rt - g.dparts(s.rt) * g.parts) * kTile)
                       : min(g.spt, B - s.rt * g.spt) * a.p.G;
    s.plane = s.hk;
    s.key0 = split * g.chunk * kTile;
    s.tiles = min(g.chunk, g.PT - split * g.chunk);
    s.keys = min(s.tiles * kTile, a.p.plen - s.key0);
    if (!emit(s)) return;
  }
  wait_for_previous();
  let_next_start();
  if (!g.warp_own && a.p.cap > 0) {
    const int head = a.w.off[B] * g.oparts;
    const Deal deal(head * a.p.Hk, g);
    int o = deal.start(blockIdx.x);
    const int o1 = deal.start(blockIdx.x + 1);
    if (o < o1) {
      int hk = o / head, left = o - hk * head;
      int b = find_sequence(a, g.doparts(left));
      left -= a.w.off[b] * g.oparts;
      int len = length_of(a, b), nt = (len + kTile - 1) / kTile;
      int part = left / nt, tile = left - part * nt;
#pragma unroll 1
      while (o < o1) {
        if (nt > 0) {
          Seg s{};
          s.own = 1;
          s.hk = hk;
          s.tiles = min(nt - tile, o1 - o);
          s.key0 = tile * kTile;
          s.keys = min(s.tiles * kTile, len - s.key0);
          s.plane = b * a.p.Hk + hk;
          const int slot = (hk * B + b) * g.oparts + part + blockIdx.x;
          int row;
          s.rt = row_tile(g, a.p.G, b, part * kTile, &row);
          s.lo = row;
          s.hi = row + min(g.orows, a.p.G - part * kTile);
          s.row = slot * g.orows - s.lo;
          s.srow = b * a.p.H + hk * a.p.G + part * kTile - s.lo;
          if (!emit(s)) return;
          o += s.tiles;
          tile += s.tiles;
          if (tile < nt) break;  // the share ends inside the sequence
          tile = 0;
          if (++part < g.oparts) continue;
        }
        part = 0;
        if (++b == B) {
          b = 0;
          ++hk;
        }
        len = length_of(a, b);
        nt = (len + kTile - 1) / kTile;
      }
    }
  }
  emit(Seg{});
}

// The next segment for a role; false at the end or after an abort.
struct Segments {
  int k = 0;
  // one thread
  __device__ __forceinline__ bool next(Shared& sh, const WaitCtl& ctl, Seg& s, bool& ok) {
    const int slot = k % kSegs;
    if (!(ok = wait_or_abort(&sh.seg_full[slot], (k / kSegs) & 1, ctl))) return false;
    s = sh.seg[slot];
    mbar_arrive(&sh.seg_empty[slot]);
    ++k;
    return s.tiles > 0;
  }
  // a whole warp
  __device__ __forceinline__ bool next_warp(Shared& sh, const WaitCtl& ctl, Seg& s, bool& ok) {
    const int slot = k % kSegs;
    ok = __all_sync(0xffffffffu, wait_or_abort(&sh.seg_full[slot], (k / kSegs) & 1, ctl));
    if (!ok) return false;
    s = sh.seg[slot];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&sh.seg_empty[slot]);
    ++k;
    return s.tiles > 0;
  }
};

// ------------------------------------------------------------------ loader
// `n` rows of a tile in boxes of 64 features: one copy each, or 16 rows at a time, so
// that nothing behind the last step of 16 is read.
template <int FEATURES>
__device__ __forceinline__ void load_rows(const CUtensorMap* maps, uint8_t* to, uint64_t* bar, int plane, int key,
                                          int n) {
  constexpr int kBoxes = (FEATURES + 63) / 64, kRow = FEATURES < 64 ? FEATURES * 2 : 128;
  if (n == kTile) {
    mbar_arrive_expect_tx(bar, kTile * FEATURES * 2);
#pragma unroll
    for (int h = 0; h < kBoxes; ++h) tma_load_3d(to + h * 16384, &maps[0], h * 64, key, plane, bar);
  } else {
    const int steps = (n + 15) / 16;
    mbar_arrive_expect_tx(bar, steps * 16 * FEATURES * 2);
#pragma unroll 1
    for (int s = 0; s < steps; ++s)
#pragma unroll
      for (int h = 0; h < kBoxes; ++h)
        tma_load_3d(to + h * 16384 + s * 16 * kRow, &maps[1], h * 64, key + 16 * s, plane, bar);
  }
}

template <int M, int DV>
__global__ void __launch_bounds__(kThreads, 1)
    decode_prefix_kernel(const __grid_constant__ Params a, const __grid_constant__ Maps maps) {
  using P = Plan<M, DV>;
  constexpr int VS = P::kVStages, KS = P::kKStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const WaitCtl ctl{&sh.abort, a.err, a.limit_ns};
  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - smem_u32(smem_raw));

  if (warp == kMmaWarp) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int s = 0; s < VS; ++s) {
      mbar_init(&sh.v_full[s], 1);
      mbar_init(&sh.v_empty[s], 1);
    }
    for (int s = 0; s < 2 * KS; ++s) {
      mbar_init(&sh.k_full[s / KS][s % KS], 1);
      mbar_init(&sh.k_empty[s / KS][s % KS], 1);
      mbar_init(&sh.k_ready[s / KS][s % KS], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sh.s_full[t], 1);
      mbar_init(&sh.p_full[t], 4);  // one arrival per warp of the warpgroup
      mbar_init(&sh.o_final[t], 1);
      mbar_init(&sh.o_empty[t], 4);
    }
    for (int k = 0; k < kSegs; ++k) {
      mbar_init(&sh.seg_full[k], 1);
      mbar_init(&sh.seg_empty[k], kSegReaders);
    }
    mbar_init(&sh.q_empty, 1);
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.drain, 1);
    sh.abort = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = sh.tmem;
  Segments segs;
  Seg s{};
  bool ok = true;

  if (warp >= 12) {
    setmaxnreg_dec<kRegControl>();
    if (warp == kLoadWarp) {
      // -------------------------------------------------------------- loader
      int i = 0;
      run_segments(a, sh, ctl, [&](const Seg& x) -> bool {
        bool good = true;
        if (elect_one_sync()) {
          for (int j = 0; j < x.tiles; ++j, ++i) {
            const int slot = i % VS;
            if (i >= VS && !(good = wait_or_abort(&sh.v_empty[slot], (i / VS - 1) & 1, ctl))) break;
            load_rows<DV>(maps.v[x.own], smem + P::kVs + slot * P::kVBytes, &sh.v_full[slot], x.plane,
                          x.key0 + j * kTile, min(kTile, x.keys - j * kTile));
          }
        }
        return __all_sync(0xffffffffu, good);
      });
      // every copy that was started lands before the memory is given up (i: the
      // elected lane knows how far it came)
      for (int k = max(0, i - VS); k < i; ++k) mbar_wait(&sh.v_full[k % VS], (k / VS) & 1, ctl.limit_ns);
    } else if (warp != kMmaWarp) {
      // ---------------------------------------------------------- K~ tiles
      // The multipliers come by copies that a fence does not wait for (loads in flight
      // at the fence below cost each tile their latency).
      const int mine = warp & 1;
      uint8_t* const ring = smem + P::kKs + mine * KS * P::kKBytes;
      int j = 0, at = 0, done = 0, issued = 0;  // tile in its segment and in all, own tiles finished and copied
      bool end = false, between = true;         // in front of a segment
      // Starts the next own tile's copies.  Where that needs a segment that is not
      // told yet, or a slot, it only waits if it must: others may wait for tiles that
      // this warp has not finished.
      auto fetch = [&](bool must) -> bool {
        while (!end) {
          if (between) {
            if (!must && !__all_sync(0xffffffffu, mbar_test_wait(&sh.seg_full[segs.k % kSegs], (segs.k / kSegs) & 1)))
              return false;
            end = !segs.next_warp(sh, ctl, s, ok);
            between = false;
            continue;
          }
          const bool own_tile = (at & 1) == mine;
          if (own_tile) {
            const int slot = issued % KS;
            if (issued >= KS) {
              uint64_t* bar = &sh.k_empty[mine][slot];
              const uint32_t parity = (issued / KS - 1) & 1;
              if (must) {
                ok = __all_sync(0xffffffffu, wait_or_abort(bar, parity, ctl));
                if (!ok) return false;
              } else if (!__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) {
                return false;
              }
            }
            const int key = s.key0 + j * kTile, n = s.keys - j * kTile;
            if (elect_one_sync())
              load_rows<M>(maps.k[s.own], ring + slot * P::kKBytes, &sh.k_full[mine][slot], s.plane, key, min(kTile, n));
            __syncwarp();
            const float* from = (s.own ? a.p.kc_mul : a.p.pkc_mul) +
                                static_cast<size_t>(s.plane) * (s.own ? a.p.cap : a.p.pcap) + key;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int k = lane + 32 * c;
              float* to = &sh.mul[at % 8][k];
              if (k < n)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(to)), "l"(from + k) : "memory");
              else
                *to = 0.f;
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            ++issued;
          }
          ++at;
          if (++j == s.tiles) {
            j = 0;
            between = true;
          }
          if (own_tile) return true;
        }
        return false;
      };
      for (;; ++done) {
        if (issued == done && !fetch(true)) break;
        while (issued < done + KS && fetch(false)) {
        }
        const int slot = done % KS, tile = (2 * done + mine) % 8;
        if (issued == done + 3)
          asm volatile("cp.async.wait_group 2;" ::: "memory");
        else if (issued == done + 2)
          asm volatile("cp.async.wait_group 1;" ::: "memory");
        else
          asm volatile("cp.async.wait_group 0;" ::: "memory");
        float x[4];  // each lane reads what it copied
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] = sh.mul[tile][lane + 32 * c];
        // rows behind the length have the multiplier 0 here; 1 where there is none
        // (positive floats are in the order of their bits)
        int most = 0;
        uint32_t least = ~0u;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          most = max(most, __float_as_int(x[c]));
          least = min(least, __float_as_uint(x[c]) - 1u);  // 0 is no multiplier
        }
        const float top = __int_as_float(__reduce_max_sync(0xffffffffu, most));
        const float low = __uint_as_float(__reduce_min_sync(0xffffffffu, least) + 1u);
        const bool narrow = low >= top * kRange;
        const float scale = top > 0.f ? top : 1.f, inv = __frcp_rn(scale);
        if (!__all_sync(0xffffffffu, wait_or_abort(&sh.k_full[mine][slot], (done / KS) & 1, ctl))) break;
        // the lanes' rows lie 32, 64 or 128 bytes apart: each starts at another piece of
        // its row, so that they meet all banks
        const int turn = M >= 64 ? lane & 7 : M == 32 ? (lane >> 1) & 3 : (lane >> 2) & 1;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float f = x[c] * inv;
          if (narrow && __any_sync(0xffffffffu, f != 1.f)) {  // row lane + 32 c, all of it by one factor
            const __half2 h = __float2half2_rn(f);
            uint8_t* row = ring + slot * P::kKBytes + (lane + 32 * c) * P::kKRow;
            constexpr int kBatch = M / 8 < 8 ? M / 8 : 8;  // 16-byte pieces in flight
#pragma unroll 1
            for (int box = 0; box < M / 8 / kBatch; ++box) {
              uint4* w = reinterpret_cast<uint4*>(row + box * 16384);
              uint4 v[kBatch];
#pragma unroll
              for (int e = 0; e < kBatch; ++e) v[e] = w[e ^ turn];
#pragma unroll
              for (int e = 0; e < kBatch; ++e) {
                __half2* u = reinterpret_cast<__half2*>(&v[e]);
#pragma unroll
                for (int k = 0; k < 4; ++k) u[k] = __hmul2(u[k], h);
              }
#pragma unroll
              for (int e = 0; e < kBatch; ++e) w[e ^ turn] = v[e];
            }
          }
        }
        if (lane == 0) sh.kscale[tile] = narrow ? scale : 0.f;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.k_ready[mine][slot]);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      for (int k = max(0, issued - KS); k < issued; ++k)
        mbar_wait(&sh.k_full[mine][k % KS], (k / KS) & 1, ctl.limit_ns);
    } else if (elect_one_sync()) {
      // ----------------------------------------------------------- MMA issue
      // One elected thread; scores run two tiles ahead of the value products.
      constexpr uint32_t kIdS = idesc_f16(128, 128, kFmtF16, 0, 0);
      constexpr uint32_t kIdPV = idesc_f16(128, DV, kFmtBF16, 0, 1);
      // rows as TMA left them: 32-, 64- or 128-byte swizzle by their width
      constexpr uint32_t kLayout = M == 16 ? 6 : M == 32 ? 4 : kLayoutSwizzle128;
      const uint64_t qa = smem_desc(sbase + P::kQ, 2048, 128, kLayoutInterleave);
      const uint64_t k0d = smem_desc(sbase + P::kKs, 16, 8 * P::kKRow, kLayout);
      const uint64_t v0d = smem_desc(sbase + P::kVs, 16384, 1024, kLayoutSwizzle128);
      int j = 0, is = 0, ip = 0;        // tile in its segment; next score and value products
      int nq = 0;                       // row tiles so far
      int nd0 = 0, nd1 = 0;             // segments finished by each stream
      int pend0 = 0, pend1 = 0;         // the streams' pending tiles: keys | first << 8 | last << 9
      int kslot = 0, kphase = 0, vslot = 0, vphase = 0;  // ring places of is (in its stream's ring) and ip
      // the q~ tile of the next segment's rows
      auto load_q = [&]() -> bool {
        if (nq > 0) {  // the old one has been read
          mma_commit(&sh.q_empty);
          if (!wait_or_abort(&sh.q_empty, (nq - 1) & 1, ctl)) return false;
        }
        mbar_arrive_expect_tx(&sh.q_full, P::kQBytes);
        bulk_g2s(smem + P::kQ, a.w.qt + (static_cast<size_t>(s.hk) * a.g.RT + s.rt) * (kTile * 2 * M), P::kQBytes,
                 &sh.q_full);
        // its own copy: waited for even where another role has given up
        if (!mbar_wait(&sh.q_full, nq & 1, ctl.limit_ns)) {
          sh.abort = 1;
          atomicExch(a.err, 1);
          return false;
        }
        ++nq;
        return true;
      };
      wait_for_previous();
      bool more = segs.next(sh, ctl, s, ok), newq = more && s.qnew;
      while (ok) {
        // a new row tile waits until the value products of the old one are on their way
        if (more && (newq ? is == ip : is < ip + 2)) {
          if (newq) {
            if (!(ok = load_q())) break;
            newq = false;
          }
          const int t = is & 1;
          if (!(ok = wait_or_abort(&sh.k_ready[t][kslot], kphase, ctl))) break;
          tc_fence_after();
          const uint32_t d = tb + P::kColS + t * 128;
          const uint64_t kb = k0d + static_cast<uint64_t>((t * KS + kslot) * (P::kKBytes >> 4));
#pragma unroll
          for (int k = 0; k < 2 * M / 16; ++k) {
            // low parts of q~ first, while the sums are small, then high parts
            const int kk = k % (M / 16), part = (k + M / 16) % (2 * M / 16);
            mma_ss(d, qa + (part * 4096 >> 4), kb + (((kk >> 2) * 16384 + (kk & 3) * 32) >> 4), kIdS, k > 0);
          }
          // a failure-detection test withholds the first "scores ready"
          if (!(a.inject_stall && is == 0)) mma_commit(&sh.s_full[t]);
          mma_commit(&sh.k_empty[t][kslot]);
          const int what = min(kTile, s.keys - j * kTile) | (j < 2) << 8 | (j + 2 >= s.tiles) << 9;
          if (t) pend1 = what; else pend0 = what;
          if ((++is & 1) == 0 && ++kslot == KS) {
            kslot = 0;
            kphase ^= 1;
          }
          if (++j == s.tiles) {
            j = 0;
            more = segs.next(sh, ctl, s, ok);
            newq = more && s.qnew;
          }
        } else if (ip < is) {
          const int t = ip & 1, what = t ? pend1 : pend0, nd = t ? nd1 : nd0;
          const bool first = what >> 8 & 1;
          if (!(ok = wait_or_abort(&sh.p_full[t], (ip / 2) & 1, ctl) && wait_or_abort(&sh.v_full[vslot], vphase, ctl) &&
                     (!first || nd == 0 || wait_or_abort(&sh.o_empty[t], (nd - 1) & 1, ctl))))
            break;
          tc_fence_after();
          const uint32_t pa = tb + P::kColS + t * 128, d = tb + P::kColO + t * DV;
          const uint64_t vb = v0d + static_cast<uint64_t>(vslot * (P::kVBytes >> 4));
          const int keys = what & 255;
          mma_ts(d, pa, vb, kIdPV, !first);
          if (keys > kTile - 16) {
#pragma unroll
            for (int k = 1; k < 8; ++k) mma_ts(d, pa + k * 8, vb + (k * 2048 >> 4), kIdPV, 1u);
          } else {
#pragma unroll 1
            for (int k = 1; k * 16 < keys; ++k)
              mma_ts(d, pa + k * 8, vb + static_cast<uint64_t>(k * 2048 >> 4), kIdPV, 1u);
          }
          mma_commit(&sh.v_empty[vslot]);
          if (what >> 9 & 1) {
            mma_commit(&sh.o_final[t]);
            if (t) ++nd1; else ++nd0;
          }
          ++ip;
          if (++vslot == VS) {
            vslot = 0;
            vphase ^= 1;
          }
        } else {
          break;
        }
      }
      mma_commit(&sh.drain);
      mbar_wait(&sh.drain, 0, ctl.limit_ns);  // own products in flight
    }
  } else if (warp >= 8) {
    // ---------------------------------------------------------------- output
    setmaxnreg_dec<kRegOutput>();
    const int r = tid & 127, w0 = r & ~31;
    const uint32_t lanes = tb + (static_cast<uint32_t>(w0) << 16);
    uint8_t* box = smem + P::kOut + w0 * 128;  // 32 rows of 128 bytes, 16-byte piece q of row x at q ^ (x % 8)
    int nd[2] = {0, 0}, i0 = 0;
    while (segs.next_warp(sh, ctl, s, ok)) {
      // streams of this segment: the tiles of number i0 .. i0 + tiles - 1
      const bool in0 = s.tiles > 1 || (i0 & 1) == 0, in1 = s.tiles > 1 || (i0 & 1) == 1;
      i0 += s.tiles;
      float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
      if (in0) {
        ok = __all_sync(0xffffffffu, wait_or_abort(&sh.o_final[0], nd[0] & 1, ctl));
        m0 = sh.stat_m[0][nd[0] & 1][r];
        l0 = sh.stat_l[0][nd[0] & 1][r];
      }
      if (ok && in1) {
        ok = __all_sync(0xffffffffu, wait_or_abort(&sh.o_final[1], nd[1] & 1, ctl));
        m1 = sh.stat_m[1][nd[1] & 1][r];
        l1 = sh.stat_l[1][nd[1] & 1][r];
      }
      if (!ok) break;
      tc_fence_after();
      if (w0 < s.hi && w0 + 32 > s.lo) {  // warp-uniform: rows of the segment here
        const float top = fmaxf(m0, m1);
        const float f0 = in0 ? ex2(m0 - top) : 0.f, f1 = in1 ? ex2(m1 - top) : 0.f;
        if (r >= s.lo && r < s.hi) {
          float* ml = (s.own ? a.w.oml : a.w.pml) + static_cast<size_t>(s.row + r) * 2;
          *reinterpret_cast<float2*>(ml) = make_float2(top, f0 * l0 + f1 * l1);
        }
        float* o = (s.own ? a.w.oo : a.w.po) + (static_cast<long long>(s.row) + w0) * DV;
#pragma unroll 1
        for (int c = 0; c < DV; c += 32) {
          uint32_t x[32], y[32];
          if (in0) tmem_ld32(lanes + P::kColO + c, x);
          if (in1) tmem_ld32(lanes + P::kColO + DV + c, y);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            float v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              v[q] = in0 ? f0 * __uint_as_float(x[e + q]) : 0.f;
              if (in1) v[q] = fmaf(f1, __uint_as_float(y[e + q]), v[q]);
            }
            *reinterpret_cast<float4*>(box + lane * 128 + (((e >> 2) ^ (lane & 7)) << 4)) =
                make_float4(v[0], v[1], v[2], v[3]);
          }
          __syncwarp();
          // eight lanes write the 32 columns of a row
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int x = 4 * e + (lane >> 3), q = lane & 7;
            const float4 v = *reinterpret_cast<const float4*>(box + x * 128 + ((q ^ (x & 7)) << 4));
            if (w0 + x >= s.lo && w0 + x < s.hi) *reinterpret_cast<float4*>(o + x * DV + c + 4 * q) = v;
          }
          __syncwarp();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (in0) {
        if (lane == 0) mbar_arrive(&sh.o_empty[0]);
        ++nd[0];
      }
      if (in1) {
        if (lane == 0) mbar_arrive(&sh.o_empty[1]);
        ++nd[1];
      }
    }
  } else {
    // --------------------------------------------------------------- softmax
    setmaxnreg_inc<kRegSoftmax>();
    const int t = warp >> 2, r = tid & 127, w0 = r & ~31;
    const uint32_t lanes = tb + (static_cast<uint32_t>(w0) << 16);
    const uint32_t tS = lanes + P::kColS + t * 128, tO = lanes + P::kColO + t * DV;
    int i = 0, ndone = 0;
    float qm = 0.f;

    wait_for_previous();
    while (segs.next_warp(sh, ctl, s, ok)) {
      if (s.qnew) qm = a.w.qmul[(static_cast<size_t>(s.hk) * a.g.RT + s.rt) * kTile + r];
      const bool here = w0 < s.hi && w0 + 32 > s.lo;  // warp-uniform
      const bool mine = r >= s.lo && r < s.hi;
      float m_run = -INFINITY, l_run = 0.f;
      const int i1 = i + s.tiles;
      int at = i + ((i & 1) != t);  // this stream's first tile
      float* srow = nullptr;
      if (s.own && mine && a.w.scores)
        srow = a.w.scores + static_cast<size_t>(s.srow + r) * a.g.capr + s.key0;
#pragma unroll 1
      for (; at < i1; at += 2) {
        const int j = at - i, n = min(kTile, s.keys - j * kTile);
        if (!(ok = __all_sync(0xffffffffu, wait_or_abort(&sh.s_full[t], (at / 2) & 1, ctl)))) break;
        tc_fence_after();
        if (n & 15) {  // value rows up to the next step of 16: zero
          if (!(ok = __all_sync(0xffffffffu, wait_or_abort(&sh.v_full[at % VS], (at / VS) & 1, ctl)))) break;
          uint8_t* vd = smem + P::kVs + at % VS * P::kVBytes;
          const int words = (16 - (n & 15)) * (DV / 8);
#pragma unroll 1
          for (int c = r; c < words; c += 128) {
            const int row = n + c / (DV / 8), part = c % (DV / 8);
            *reinterpret_cast<uint4*>(vd + (part >> 3) * 16384 + row * 128 + (part & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        if (here) {
          const float ks = sh.kscale[at % 8];
          if (ks == 0.f) {  // each key's own multiplier
            const float4* km = reinterpret_cast<const float4*>(sh.mul[at % 8]);
#pragma unroll 1
            for (int c = 0; c < 128; c += 32) {
              uint32_t v[32];
              tmem_ld32(tS + c, v);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 f = km[(c + e) / 4];
                v[e] = __float_as_uint(__uint_as_float(v[e]) * (qm * f.x));
                v[e + 1] = __float_as_uint(__uint_as_float(v[e + 1]) * (qm * f.y));
                v[e + 2] = __float_as_uint(__uint_as_float(v[e + 2]) * (qm * f.z));
                v[e + 3] = __float_as_uint(__uint_as_float(v[e + 3]) * (qm * f.w));
              }
              tmem_st32(tS + c, v);
            }
            tmem_wait_st();
          }
          float x[128];
          {
            uint32_t v0[32], v1[32], v2[32], v3[32];
            tmem_ld32(tS, v0);
            tmem_ld32(tS + 32, v1);
            tmem_ld32(tS + 64, v2);
            tmem_ld32(tS + 96, v3);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              x[c] = __uint_as_float(v0[c]);
              x[32 + c] = __uint_as_float(v1[c]);
              x[64 + c] = __uint_as_float(v2[c]);
              x[96 + c] = __uint_as_float(v3[c]);
            }
          }
          const float mult = ks == 0.f ? 1.f : qm * ks;  // > 0
          if (n < kTile) {
#pragma unroll
            for (int c = 0; c < 128; ++c) x[c] = c < n ? x[c] : -INFINITY;
          }
          if (srow) {
            float* to = srow + j * kTile;
#pragma unroll
            for (int c = 0; c < 128; c += 4)
              *reinterpret_cast<float4*>(to + c) = make_float4(x[c] * mult, x[c + 1] * mult, x[c + 2] * mult, x[c + 3] * mult);
          }
          // The stream's first tile of the segment takes the maximum; a later one
          // is exponentiated against the running one, and again after taking its
          // maximum where the row's sum says that it has moved.
          const bool fresh = j < 2;
          bool take = fresh, grow = false;
          float alpha = 1.f, lsum;
#pragma unroll 1
          while (true) {
            if (take) {
              float mx[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                float mi = max3(x[16 * k], x[16 * k + 1], x[16 * k + 2]);
#pragma unroll
                for (int c = 3; c < 15; c += 2) mi = max3(mi, x[16 * k + c], x[16 * k + c + 1]);
                mx[k] = fmaxf(mi, x[16 * k + 15]);
              }
              const float top = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])) * mult;
              grow = top > m_run + kGrow;
              if (grow) {
                alpha = ex2(m_run - top);  // 0 at the row's first tile
                m_run = top;
              }
            }
            const uint64_t q2 = pack_f32x2(mult, mult), negm = pack_f32x2(-m_run, -m_run);
            uint64_t sum[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              uint32_t pk[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const int c = h * 32 + 2 * e;
                float y0, y1;
                unpack_f32x2(fma_f32x2(pack_f32x2(x[c], x[c + 1]), q2, negm), y0, y1);
                const float e0 = ex2(y0), e1 = ex2(y1);
                sum[e & 3] = add_f32x2(sum[e & 3], pack_f32x2(e0, e1));
                pk[e] = pack_bf16x2(e0, e1);
              }
              tmem_st16(tS + h * 16, pk);
            }
            lsum = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float u, v;
              unpack_f32x2(sum[e], u, v);
              lsum += u + v;
            }
            if (take || !__any_sync(0xffffffffu, mine && !(lsum <= kSumLimit))) break;
            take = true;
          }
          // the row's sums follow the maximum: the stream's last value product is
          // complete (covered by this tile's scores), the next waits for p_full
          if (!fresh && __any_sync(0xffffffffu, grow)) {
#pragma unroll 1
            for (int c = 0; c < DV; c += 32) {
              uint32_t o[32];
              tmem_ld32(tO + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st32(tO + c, o);
            }
          }
          l_run = l_run * alpha + lsum;
          tmem_wait_st();
        }
        if (at + 2 >= i1) {
          // The row's statistics, in front of the arrival that leads to the last
          // value product and so to o_final.  The slot's last reader is done:
          // this tile's scores were issued behind the stream's value products of
          // the segment between, and those behind o_empty.
          sh.stat_l[t][ndone & 1][r] = l_run;
          sh.stat_m[t][ndone & 1][r] = m_run;
          ++ndone;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[t]);
      }
      if (!ok) break;
      i = i1;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tb, 512);
}

// -------------------------------------------------------------------- host
Geo geometry(const DecodeSharedParams& p, int sms) {
  Geo g{};
  const int most = sms < kMaxCtas ? sms : kMaxCtas;
  g.spt = p.G <= kTile ? kTile / p.G : 1;
  g.parts = (p.G + kTile - 1) / kTile;
  g.RT = g.parts > 1 ? p.B * g.parts : (p.B + g.spt - 1) / g.spt;
  g.rows = g.parts > 1 ? kTile : (p.B < g.spt ? p.B : g.spt) * p.G;
  g.PT = (p.plen + kTile - 1) / kTile;
  g.capr = (p.cap + kTile - 1) / kTile * kTile;
  g.warp_own = p.G <= kDecodeOwnGroup;
  g.ounit = g.warp_own ? kStep : kTile;
  const int opart = g.warp_own ? kStep : kTile;  // rows of an own part
  g.oparts = (p.G + opart - 1) / opart;
  g.orows = p.G < opart ? p.G : opart;
  const long long rowtiles = static_cast<long long>(p.Hk) * g.RT;
  const long long own = static_cast<long long>(p.Hk) * p.B * g.oparts * ((p.cap + g.ounit - 1LL) / g.ounit);
  const long long all = rowtiles * g.PT + (g.warp_own ? 0 : own);
  g.grid = static_cast<int>(all < 1 ? 1 : all < most ? all : most);
  // the split of the prefix with the shortest schedule, in cycles: rounds of segments,
  // each its tiles and about two tiles' time of start and end, and the partial sums'
  // way to memory and back (65536 keys for 512 rows of 8 key heads: 4, 9, 14, 19, 28
  // segments per row tile 258, 251, 256, 259, 270 us for the whole call, of a build that
  // takes 262 now).  Cycles per tile were measured for m = 32 and 64 with d_v = 128; the
  // one for m = 128 is an estimate.
  if (g.PT > 0) {
    const long long tile = p.m <= 32 ? 1750 : p.m == 64 ? 2400 : 3500;
    const long long sums = rowtiles * g.rows * p.dv * 8 / 3500;
    long long best = -1;
    long long limit = kPrefixSlots / rowtiles;
    limit = limit < 1 ? 1 : limit > g.PT ? g.PT : limit;
    for (int s = 1; s <= limit; ++s) {
      const int chunk = (g.PT + s - 1) / s, S = (g.PT + chunk - 1) / chunk;
      const long long cost = (rowtiles * S + g.grid - 1) / g.grid * (chunk + 2) * tile + S * sums;
      if (best < 0 || cost < best) {
        best = cost;
        g.S = S;
        g.chunk = chunk;
      }
    }
  }
  g.units = static_cast<int>(rowtiles * g.S);
  if (g.warp_own) {
    const long long ctas = (own + kOwnWarps - 1) / kOwnWarps;
    g.workers = kOwnWarps * static_cast<int>(ctas < 1 ? 1 : ctas < most ? ctas : most);
  } else {
    g.workers = g.grid;
    g.extra = g.units % g.grid;
    g.pre = g.units / g.grid * g.chunk;
  }
  g.dRT.set(g.RT);
  g.dS.set(g.S);
  g.dG.set(p.G);
  g.dH.set(p.H);
  g.dHk.set(p.Hk);
  g.dspt.set(g.spt);
  g.dparts.set(g.parts);
  g.doparts.set(g.oparts);
  g.dworkers.set(g.workers);
  g.dextra.set(g.extra);
  g.drest.set(g.workers - g.extra);
  return g;
}

// The layout holds for every grid up to kMaxCtas: its size is the same on every machine.
size_t layout(const DecodeSharedParams& p, const Geo& g, char* ws, Work* w) {
  size_t o = 0;
  auto take = [&](size_t bytes) {
    char* at = ws + o;
    o = (o + bytes + 255) & ~static_cast<size_t>(255);
    return at;
  };
  const size_t rowtiles = static_cast<size_t>(p.Hk) * g.RT;
  size_t most = kPrefixSlots / rowtiles;
  most = most < 1 ? 1 : most > static_cast<size_t>(g.PT) ? g.PT : most;
  const size_t prows = g.PT > 0 ? rowtiles * most * g.rows : 0;
  const size_t workers = g.warp_own ? kMaxCtas * kOwnWarps : kMaxCtas;
  const size_t orows = p.cap > 0 ? (static_cast<size_t>(p.Hk) * p.B * g.oparts + workers) * g.orows : 0;
  Work x{};
  x.off = reinterpret_cast<int*>(take((static_cast<size_t>(p.B) + 1) * sizeof(int)));
  x.qt = reinterpret_cast<uint16_t*>(take(rowtiles * kTile * 2 * p.m * sizeof(uint16_t)));
  x.qmul = reinterpret_cast<float*>(take(rowtiles * kTile * sizeof(float)));
  x.po = reinterpret_cast<float*>(take(prows * p.dv * sizeof(float)));
  x.pml = reinterpret_cast<float*>(take(prows * 2 * sizeof(float)));
  x.oo = reinterpret_cast<float*>(take(orows * p.dv * sizeof(float)));
  x.oml = reinterpret_cast<float*>(take(orows * 2 * sizeof(float)));
  if (p.acc_out)
    x.scores = reinterpret_cast<float*>(take(static_cast<size_t>(p.B) * p.H * g.capr * sizeof(float)));
  if (w) *w = x;
  return o;
}

template <int M, int DV>
cudaError_t launch(const Params& a, const Maps& maps, cudaStream_t stream) {
  using P = Plan<M, DV>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(decode_prefix_kernel<M, DV>, P::kLaunch, done);
  if (e != cudaSuccess) return e;
  return launch_after(decode_prefix_kernel<M, DV>, a.g.grid, kThreads, P::kLaunch, stream, a, maps);
}

template <int DV>
cudaError_t launch_m(const Params& a, const Maps& maps, cudaStream_t stream) {
  switch (a.p.m) {
    case 16: return launch<16, DV>(a, maps, stream);
    case 32: return launch<32, DV>(a, maps, stream);
    case 64: return launch<64, DV>(a, maps, stream);
    case 128: return launch<128, DV>(a, maps, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

bool decode_shared_fits(const DecodeSharedParams& p) {
  // counts of tiles and rows of partial results are 30-bit
  const Geo g = geometry(p, kMaxCtas);
  const long long own = static_cast<long long>(p.Hk) * p.B * g.oparts, rows = static_cast<long long>(p.Hk) * g.RT;
  const long long tiles = own * ((p.cap + g.ounit - 1LL) / g.ounit) + 2 * rows * g.PT;
  return tiles < (1LL << 30) && (own + kMaxCtas * kOwnWarps) * g.orows < (1LL << 30) &&
         (rows + kPrefixSlots) * kTile < (1LL << 30);
}

size_t decode_shared_workspace(const DecodeSharedParams& p) {
  return layout(p, geometry(p, kMaxCtas), nullptr, nullptr);
}

cudaError_t launch_decode_shared(const DecodeSharedParams& p, const DecodeSharedRun& run, cudaStream_t stream) {
  Params a{};
  a.p = p;
  a.g = geometry(p, run.sms);
  layout(p, a.g, p.ws, &a.w);
  a.err = run.err;
  a.limit_ns = run.limit_ns;
  a.inject_stall = run.inject_stall;
  Maps maps{};
  for (int own = 0; own < 2; ++own)
    for (int small = 0; small < 2; ++small) {
      maps.k[own][small] = run.k[own][small];
      maps.v[own][small] = run.v[own][small];
    }
  cudaError_t e = launch_query(a, stream);
  if (e == cudaSuccess && (a.g.units > 0 || (!a.g.warp_own && p.cap > 0)))
    e = p.dv == 64 ? launch_m<64>(a, maps, stream) : launch_m<128>(a, maps, stream);
  if (e == cudaSuccess && a.g.warp_own && p.cap > 0) e = launch_own(a, maps, stream);
  return e == cudaSuccess ? launch_combine(a, stream) : e;
}

}  // namespace spa
