// decode_shared.cu -- one query per (sequence, head) against a prefix that the
// whole batch shares and the sequence's own cache rows, joined in one softmax:
//   s_j = <q P_h, K~_j> / sqrt(m),  O = sum_j softmax(s)_j V_j
// over rows 0 .. plen-1 of the prefix cache and 0 .. lens[b]-1 of the
// sequence's; query heads h*G .. h*G+G-1 share key head h.
//
// The queries of one key head are the rows (b, g) of a matrix, cut into tiles
// of up to 128 rows that hold whole groups (a group of more than 128 heads is
// cut into parts).  Work is cut into segments of 128-key tiles:
//   prefix   one row tile against a range of prefix keys: all its rows
//   own      one (sequence, key head) against a range of its own keys: the
//            group's rows of the row tile, the others idle
// A prefix tile is read once per row tile (from L2 beyond the first), an own
// tile once.  Every segment leaves its rows' unnormalised sums, maxima and
// weights' sums in the workspace; the combine kernel joins them.
//
// The main kernel is persistent, one CTA per SM: prefix segments round robin
// with the row tiles fastest, so that CTAs side by side stream the same keys,
// then an equal share of all own tiles (counted on the device from lens).
// Sixteen warps in four warpgroups:
//   warps 0-3, 4-7   softmax of the tiles of even / odd number (two streams)
//   warps 8-11       output: a finished segment's sums, both streams joined
//   warp  12         K~ and V tiles by TMA into a ring of slots
//   warp  13         tensor-memory allocation and tcgen05.mma issue
//   warp  14         the keys' multipliers into the ring
//   warp  15         the list of segments, a few ahead of the other roles: the
//                    divisions and the sequences' lengths are its work alone
// The streams alternate tile by tile, each with scores and sums of its own in
// tensor memory (S0 | S1 | O0 | O1), so that the products of one run while the
// other is exponentiated.
//
// Scores.  q~ = q P_h comes from the tensor cores (exact products, fp32 sums)
// at each change of the row tile, scaled by a power of two per row and split
// into two fp16 parts (22 bits); the cache rows are fp16 as they are, so the
// scores carry fp32's precision.  The multiplier of a key scales its column.
// Probabilities are rounded to bf16 for the value product (2^-8 relative,
// averaged over the keys); their sums, and the weights that are accumulated,
// take them in fp32.
//
// Softmax in base 2 with the running maximum moved only when a row's tile sum
// exceeds 2^40, as in the forward.  Key columns behind a length are replaced
// by -inf after the product, and value rows behind it are zeroed in shared
// memory up to the 16 rows that one MMA step reads: what they hold (NaN too)
// is never used.  A segment's sums start afresh, so that one sequence's values
// never meet another's rows.
//
// Every wait is bounded; a role that gives up sets the CTA's abort flag and
// the device error word, and all roles leave after their own operations in
// flight have ended.
#include <math.h>

#include <cstddef>

#include "kernels.cuh"
#include "ptx.cuh"
#include "waits.cuh"

namespace spa {
namespace {

using namespace ptx;

constexpr int kThreads = 512;
constexpr uint32_t kRegSoftmax = 176, kRegOutput = 88, kRegControl = 72;
static_assert(128 * (2 * kRegSoftmax + kRegOutput + kRegControl) <= kThreads * 128,
              "register split exceeds the launch");
constexpr int kLoadWarp = 12, kMmaWarp = 13, kMulWarp = 14;
constexpr int kTile = 128;             // keys per tile, rows per row tile
constexpr int kSchedWarp = 15;
constexpr int kSegs = 8;               // segments the scheduler may be ahead
constexpr int kSegReaders = 3 + 4 + 8; // loader, issuer, multipliers, output warps, softmax warps
constexpr float kSumLimit = 1099511627776.f;  // 2^40
constexpr float kGrow = 40.f;
constexpr int kMaxCtas = 256;          // grid limit (sizes the workspace)
constexpr int kPrefixSlots = 1024;     // prefix segments per call at most (beyond one per row tile)
constexpr int kMaxDynSmem = 227 * 1024 - 8 * 1024;

// What host and device know of a call's layout.
struct Geo {
  int spt, parts;      // sequences per row tile, parts per group
  int RT;              // row tiles per key head
  int rows;            // rows of a tile that can be in use
  int orows;           // rows of an own segment
  int PT, S, chunk;    // prefix tiles, splits, tiles per split
  int units;           // prefix segments
  int grid;
  int capr;            // keys per row of the score buffer
};

struct Work {
  int* off;            // [B+1] own tiles of one part in front of each sequence
  float *po, *pml;     // prefix segments: [units][rows][dv], [units][rows][2]
  float *oo, *oml;     // own segments
  float* scores;       // [B*H][capr], or NULL
};

struct Maps {
  CUtensorMap k[2][2], v[2][2];  // [own][128-row or 16-row box]
  CUtensorMap P;                 // P as 3-D (m, d, Hk), box (min(m, 64), 64, 1), swizzled like K~
};

struct Params {
  DecodeSharedParams p;
  Geo g;
  Work w;
  int* err;
  unsigned long long limit_ns;
  int inject_stall;
};

constexpr int cmax(int a, int b) { return a > b ? a : b; }

template <int M, int DV>
struct Plan {
  static constexpr int kKBytes = kTile * M * 2, kVBytes = kTile * DV * 2;
  static constexpr int kSlot = kKBytes + kVBytes;
  static constexpr int kKRow = M < 64 ? M * 2 : 128;  // bytes of a K~ row in shared memory (a box)
  // the staging of q and P_h for the projection (two slots of 64 features)
  // lies in the place of the result
  static constexpr int kStageP = 16384, kStage = kStageP + 64 * M * 2;
  static constexpr int kQBytes = cmax(kTile * 4 * M, 2 * kStage);
  static constexpr int kQ = 0, kOut = (kQBytes + 1023) / 1024 * 1024;
  static constexpr int kRing = kOut + 4 * 4096;  // a box of 32 x 32 sums per output warp
  static constexpr int kFit = (kMaxDynSmem - 1024 - kRing) / kSlot;
  static constexpr int kStages = kFit > 4 ? 4 : kFit;
  static constexpr int kBytes = kRing + kStages * kSlot + 1024;
  // one CTA per SM: a second one would wait in tcgen05.alloc for the 512 columns
  static constexpr int kLaunch = cmax(kBytes, 120 * 1024);
  static_assert(kStages >= 2 && kLaunch <= kMaxDynSmem, "shared-memory plan");
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
  uint64_t kv_full[4], kv_empty[4], mul_full[4];
  uint64_t s_full[2], p_full[2], o_final[2], o_empty[2];
  uint64_t q_empty, q_full, stage_full, stage_done, p_map, drain;
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint32_t tmem;
  volatile int abort;
  Seg seg[kSegs];
  float stat_l[2][2][kTile], stat_m[2][2][kTile];
  float qmul[2][kTile];
  alignas(16) float mul[4][kTile];  // read four at a time
};
static_assert(offsetof(Shared, mul) % 16 == 0 && offsetof(Shared, seg) % 16 == 0 && alignof(Shared) >= 16,
              "vector loads from shared memory");
static_assert(sizeof(Shared) <= 8 * 1024 - 256, "static shared memory");

// The own tiles are dealt out in equal runs: `a` tiles to each of the first
// `extra` CTAs, which have one prefix segment more, `b` to each of the others,
// so that all have about the same number of tiles.  CTAs without any lie in
// front or at the end, never between two that have some.  (All counts of tiles
// fit in 31 bits: checked on the host.)
struct Deal {
  int total, extra, a, b;
  __device__ __forceinline__ Deal(int total_, const Geo& g) : total(total_) {
    const int full = g.units / g.grid;
    extra = g.units - full * g.grid;
    const int pre = g.units * g.chunk;
    a = (pre + total + g.grid - 1) / g.grid - (full + 1) * g.chunk;
    if (a < 0 || extra == 0) a = 0;
    if (extra > 0 && a > total / extra) a = total / extra;
    b = (total - a * extra + g.grid - extra - 1) / (g.grid - extra);
  }
  __device__ __forceinline__ int start(int c) const {
    if (c <= extra) return a * c;
    const long long t = a * extra + static_cast<long long>(b) * (c - extra);
    return t < total ? static_cast<int>(t) : total;
  }
  __device__ __forceinline__ int owner(int t) const {
    return t < a * extra ? t / a : extra + (t - a * extra) / b;
  }
};

__device__ __forceinline__ int tiles_of(const Params& a, int b) {
  return b < a.p.B ? (min(max(a.p.lens[b], 0), a.p.cap) + kTile - 1) / kTile : 0;
}

// The scheduler warp: the CTA's segments in order, then the end.
__device__ __forceinline__ void run_scheduler(const Params& a, Shared& sh, const WaitCtl& ctl) {
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
    return true;
  };
  for (int unit = blockIdx.x; unit < g.units; unit += g.grid) {
    Seg s{};
    const int us = unit / g.RT;
    s.rt = unit - us * g.RT;
    s.hk = us / g.S;
    const int split = us - s.hk * g.S;
    s.row = ((s.hk * g.RT + s.rt) * g.S + split) * g.rows;
    s.hi = g.parts > 1 ? min(kTile, a.p.G - (s.rt % g.parts) * kTile)
                       : min(g.spt, B - s.rt * g.spt) * a.p.G;
    s.plane = s.hk;
    s.key0 = split * g.chunk * kTile;
    s.tiles = min(g.chunk, g.PT - split * g.chunk);
    s.keys = min(s.tiles * kTile, a.p.plen - s.key0);
    if (!emit(s)) return;
  }
  if (a.p.cap > 0) {
    // own tiles of the batch; CTA 0 leaves the prefix sums for the combine kernel
    int all = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < B; b0 += 128) {
      int n[4], sum = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) n[e] = tiles_of(a, b0 + 4 * lane + e);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum += n[e];
      int s = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += t;
      }
      if (blockIdx.x == 0) {
        int at = all + s - sum;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (b0 + 4 * lane + e < B) a.w.off[b0 + 4 * lane + e] = at;
          at += n[e];
        }
      }
      all += __shfl_sync(0xffffffffu, s, 31);
    }
    if (blockIdx.x == 0 && lane == 0) a.w.off[B] = all;
    const int head = all * g.parts;
    const Deal deal(head * a.p.Hk, g);
    int o = deal.start(blockIdx.x);
    const int o1 = deal.start(blockIdx.x + 1);
    if (o < o1) {
      int hk = o / head, left = o - hk * head;
      // the sequence that holds tile `left` of the key head: 32 at a time
      int b0 = 0, n, s, before = 0;
#pragma unroll 1
      while (true) {
        n = tiles_of(a, b0 + lane) * g.parts;
        s = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int t = __shfl_up_sync(0xffffffffu, s, d);
          if (lane >= d) s += t;
        }
        const int sum = __shfl_sync(0xffffffffu, s, 31);
        if (left < before + sum) break;
        before += sum;
        b0 += 32;
      }
      int l = __ffs(__ballot_sync(0xffffffffu, left < before + s)) - 1;  // lane = sequence b0 + l
      left -= before + __shfl_sync(0xffffffffu, s - n, l);
      n /= g.parts;
      int nt = __shfl_sync(0xffffffffu, n, l);
      int part = left / nt, tile = left - part * nt;
#pragma unroll 1
      while (o < o1) {
        if (nt > 0) {
          const int b = b0 + l;
          Seg s{};
          s.own = 1;
          s.hk = hk;
          s.tiles = min(nt - tile, o1 - o);
          s.key0 = tile * kTile;
          s.keys = min(s.tiles * kTile, min(a.p.lens[b], a.p.cap) - s.key0);
          s.plane = b * a.p.Hk + hk;
          const int slot = (hk * B + b) * g.parts + part + blockIdx.x;
          if (g.parts > 1) {
            s.rt = b * g.parts + part;
            s.hi = min(kTile, a.p.G - part * kTile);
          } else {
            s.rt = b / g.spt;
            s.lo = (b - s.rt * g.spt) * a.p.G;
            s.hi = s.lo + a.p.G;
          }
          s.row = slot * g.orows - s.lo;
          s.srow = b * a.p.H + hk * a.p.G + part * kTile - s.lo;
          if (!emit(s)) return;
          o += s.tiles;
          tile += s.tiles;
          if (tile < nt) break;  // the share ends inside the sequence
          tile = 0;
          if (++part < g.parts) continue;
        }
        part = 0;
        if (++l == 32 || b0 + l == B) {
          b0 = b0 + l == B ? 0 : b0 + 32;
          hk += b0 == 0;
          l = 0;
          n = tiles_of(a, b0 + lane);
        }
        nt = __shfl_sync(0xffffffffu, n, l);
      }
    }
  } else if (blockIdx.x == 0) {
    for (int b = lane; b <= B; b += 32) a.w.off[b] = 0;
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

// The query row of lane r of row tile (hk, rt), or NULL.
__device__ __forceinline__ const __nv_bfloat16* query_row(const Params& a, int hk, int rt, int r) {
  int b, g;
  if (a.g.parts > 1) {
    b = rt / a.g.parts;
    g = (rt - b * a.g.parts) * kTile + r;
    if (g >= a.p.G) return nullptr;
  } else {
    const int i = r / a.p.G;
    b = rt * a.g.spt + i;
    g = r - i * a.p.G;
    if (i >= a.g.spt || b >= a.p.B) return nullptr;
  }
  return a.p.q + (static_cast<size_t>(b) * a.p.H + hk * a.p.G + g) * a.p.d;
}

__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ uint32_t bits_at(const __nv_bfloat16* x, int k, int d) {
  return k < d ? __bfloat16_as_ushort(x[k]) : 0u;
}

// ------------------------------------------------------------------ loader
template <class P, int M, int DV>
__device__ __forceinline__ void load_tile(const Maps& maps, uint8_t* slot, uint64_t* bar, int own, int plane,
                                          int key, int n) {
  const CUtensorMap* km = maps.k[own];
  const CUtensorMap* vm = maps.v[own];
  uint8_t* kd = slot;
  uint8_t* vd = slot + P::kKBytes;
  constexpr int kKBoxes = M > 64 ? 2 : 1;
  if (n == kTile) {
    mbar_arrive_expect_tx(bar, P::kSlot);
#pragma unroll
    for (int h = 0; h < kKBoxes; ++h) tma_load_3d(kd + h * 16384, &km[0], h * 64, key, plane, bar);
#pragma unroll
    for (int h = 0; h < DV / 64; ++h) tma_load_3d(vd + h * 16384, &vm[0], h * 64, key, plane, bar);
  } else {  // 16 rows at a time: nothing behind the last step is read
    const int steps = (n + 15) / 16;
    mbar_arrive_expect_tx(bar, steps * 16 * 2 * (M + DV));
    for (int s = 0; s < steps; ++s) {
#pragma unroll
      for (int h = 0; h < kKBoxes; ++h)
        tma_load_3d(kd + h * 16384 + s * 16 * P::kKRow, &km[1], h * 64, key + 16 * s, plane, bar);
#pragma unroll
      for (int h = 0; h < DV / 64; ++h)
        tma_load_3d(vd + h * 16384 + s * 2048, &vm[1], h * 64, key + 16 * s, plane, bar);
    }
  }
}

template <int M, int DV>
__global__ void __launch_bounds__(kThreads, 1)
    decode_shared_kernel(const __grid_constant__ Params a, const __grid_constant__ Maps maps) {
  using P = Plan<M, DV>;
  constexpr int ST = P::kStages;
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
    for (int s = 0; s < ST; ++s) {
      mbar_init(&sh.kv_full[s], 1);
      mbar_init(&sh.kv_empty[s], 1);
      mbar_init(&sh.mul_full[s], 1);
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
    mbar_init(&sh.q_full, 4);
    mbar_init(&sh.stage_full, 4);
    mbar_init(&sh.stage_done, 1);
    mbar_init(&sh.p_map, 1);
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
    if (warp == kSchedWarp) {
      run_scheduler(a, sh, ctl);
    } else if (warp == kLoadWarp) {
      // -------------------------------------------------------------- loader
      if (elect_one_sync()) {
        int i = 0;
        while (segs.next(sh, ctl, s, ok)) {
          for (int j = 0; j < s.tiles; ++j, ++i) {
            const int slot = i % ST;
            if (i >= ST && !(ok = wait_or_abort(&sh.kv_empty[slot], (i / ST - 1) & 1, ctl))) break;
            load_tile<P, M, DV>(maps, smem + P::kRing + slot * P::kSlot, &sh.kv_full[slot], s.own, s.plane,
                                s.key0 + j * kTile, min(kTile, s.keys - j * kTile));
          }
          if (!ok) break;
        }
        // every copy that was started lands before the memory is given up
        for (int k = max(0, i - ST); k < i; ++k) mbar_wait(&sh.kv_full[k % ST], (k / ST) & 1, ctl.limit_ns);
      }
    } else if (warp == kMulWarp) {
      // -------------------------------------------------- keys' multipliers
      const float* from = nullptr;
      int j = 0, i = 0;
      bool more = segs.next_warp(sh, ctl, s, ok);
      auto fetch = [&](float (&x)[4]) {  // the next tile's, a tile ahead of its slot
        if (j == 0)
          from = s.own ? a.p.kc_mul + static_cast<size_t>(s.plane) * a.p.cap + s.key0
                       : a.p.pkc_mul + static_cast<size_t>(s.plane) * a.p.pcap + s.key0;
        const int n = s.keys - j * kTile;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int k = lane + 32 * c;
          x[c] = k < n ? __ldg(from + j * kTile + k) : 0.f;
        }
        if (++j == s.tiles) {
          j = 0;
          more = segs.next_warp(sh, ctl, s, ok);
        }
      };
      float x[4], y[4];
      bool have = more;
      if (have) fetch(x);
      while (have && ok) {
        const bool next = more;
        if (next) fetch(y);
        const int slot = i % ST;
        if (i >= ST && !__all_sync(0xffffffffu, wait_or_abort(&sh.kv_empty[slot], (i / ST - 1) & 1, ctl))) break;
#pragma unroll
        for (int c = 0; c < 4; ++c) sh.mul[slot][lane + 32 * c] = x[c];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.mul_full[slot]);
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] = y[c];
        have = next;
        ++i;
      }
    } else {
      // ----------------------------------------------------------- MMA issue
      // The whole warp runs the role, converged and on votes alone, and elects
      // the issuing lane: descriptors then stay in uniform registers.  (Issued
      // by one lane of a diverged warp, each MMA took about 200 cycles.)
      constexpr uint32_t kIdS = idesc_f16(128, 128, kFmtF16, 0, 0);
      constexpr uint32_t kIdPV = idesc_f16(128, DV, kFmtBF16, 0, 1);
      constexpr uint32_t kIdQ = idesc_f16(128, M, kFmtBF16, 0, 1);
      // rows as TMA left them: 32-, 64- or 128-byte swizzle by their width
      constexpr uint32_t kLayout = M == 16 ? 6 : M == 32 ? 4 : kLayoutSwizzle128;
      const uint64_t qa = smem_desc(sbase + P::kQ, 2048, 128, kLayoutInterleave);
      const uint64_t k0d = smem_desc(sbase + P::kRing, 16, 8 * P::kKRow, kLayout);
      const uint64_t v0d = smem_desc(sbase + P::kRing + P::kKBytes, 16384, 1024, kLayoutSwizzle128);
      int j = 0, is = 0, ip = 0;        // tile in its segment; next score and value products
      int nq = 0, np = 0;               // row tiles and projection passes so far
      int nd0 = 0, nd1 = 0;             // segments finished by each stream
      int pend0 = 0, pend1 = 0;         // the streams' pending tiles: keys | first << 8 | last << 9
      bool held = false, newq = false, more = false;
      auto ready = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_test_wait(bar, parity)) != 0;
      };
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_or_abort(bar, parity, ctl)) != 0;
      };
      auto next_seg = [&]() {
        more = segs.next_warp(sh, ctl, s, ok);
        more = __any_sync(0xffffffffu, more) != 0;
        ok = __all_sync(0xffffffffu, ok) != 0;
        newq = __any_sync(0xffffffffu, more && s.qnew) != 0;
      };
      // q~ = q P_h for the next tile's rows into the scores' columns d; the
      // stream's warpgroup brings q and takes the result
      auto project = [&](uint32_t d) -> bool {
        if (nq > 0) {  // the old q~ has been read
          if (elect_one_sync()) mma_commit(&sh.q_empty);
          __syncwarp();
          if (!wait(&sh.q_empty, (nq - 1) & 1)) return false;
        }
#pragma unroll 1
        for (int k0 = 0; k0 < a.p.d; k0 += 128, ++np) {
          const int chunks = a.p.d - k0 > 64 ? 2 : 1;
          if (k0 > 0 && !wait(&sh.stage_done, (np - 1) & 1)) return false;
          if (elect_one_sync()) {
            mbar_arrive_expect_tx(&sh.p_map, chunks * 128 * M);
#pragma unroll 1
            for (int c = 0; c < chunks; ++c)
#pragma unroll
              for (int h = 0; h < (M + 63) / 64; ++h)
                tma_load_3d(smem + P::kQ + c * P::kStage + P::kStageP + h * 8192, &maps.P, h * 64, k0 + 64 * c, s.hk,
                            &sh.p_map);
          }
          __syncwarp();
          const bool both = wait(&sh.stage_full, np & 1);
          if (!__all_sync(0xffffffffu, mbar_wait(&sh.p_map, np & 1, ctl.limit_ns)) || !both) return false;
          tc_fence_after();
          if (elect_one_sync()) {
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
              const uint32_t st = sbase + P::kQ + c * P::kStage;
              const uint64_t qd = smem_desc(st, 2048, 128, kLayoutInterleave);
              const uint64_t pd = smem_desc(st + P::kStageP, 8192, 8 * P::kKRow, kLayout);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_ss(d, qd + (k * 4096 >> 4), pd + (k * 16 * P::kKRow >> 4), kIdQ, k0 > 0 || c > 0 || k > 0);
            }
            mma_commit(&sh.stage_done);
          }
          __syncwarp();
        }
        if (!wait(&sh.q_full, nq & 1)) return false;
        tc_fence_after();
        ++nq;
        return true;
      };
      next_seg();
      uint64_t idle = 0;
      while (ok && (more || ip < is)) {
        bool did = false;
        // a new row tile waits until the value products of the old one are on their way
        if (more && (newq ? is == ip : is < ip + 2)) {
          const int slot = is % ST, t = is & 1;
          const uint32_t d = tb + P::kColS + t * 128;
          if (newq) {
            if (!(ok = project(d))) break;
            newq = false;
          }
          if (ready(&sh.kv_full[slot], (is / ST) & 1) && ready(&sh.mul_full[slot], (is / ST) & 1)) {
            tc_fence_after();
            const uint64_t kb = k0d + static_cast<uint64_t>(slot * (P::kSlot >> 4));
            // a failure-detection test withholds the first "scores ready"
            const bool tell = !(a.inject_stall && !held);
            if (elect_one_sync()) {
#pragma unroll
              for (int k = 0; k < 2 * M / 16; ++k) {  // high parts, then low parts of q~
                const int kk = k % (M / 16);
                mma_ss(d, qa + (k * 4096 >> 4), kb + (((kk >> 2) * 16384 + (kk & 3) * 32) >> 4), kIdS, k > 0);
              }
              if (tell) mma_commit(&sh.s_full[t]);
            }
            __syncwarp();
            held = true;
            const int what = __shfl_sync(0xffffffffu, min(kTile, s.keys - j * kTile) | (j < 2) << 8 |
                                                          (j + 2 >= s.tiles) << 9, 0);
            if (t) pend1 = what; else pend0 = what;
            ++is;
            ++j;
            if (__any_sync(0xffffffffu, j == s.tiles)) {
              j = 0;
              next_seg();
            }
            did = true;
          }
        }
        if (!did && ip < is) {
          const int slot = ip % ST, t = ip & 1, what = t ? pend1 : pend0, nd = t ? nd1 : nd0;
          const bool first = what >> 8 & 1;
          if (ready(&sh.p_full[t], (ip / 2) & 1) && (!first || nd == 0 || ready(&sh.o_empty[t], (nd - 1) & 1))) {
            tc_fence_after();
            const uint32_t pa = tb + P::kColS + t * 128, d = tb + P::kColO + t * DV;
            const uint64_t vb = v0d + static_cast<uint64_t>(slot * (P::kSlot >> 4));
            const int keys = what & 255;
            if (elect_one_sync()) {
              mma_ts(d, pa, vb, kIdPV, !first);
              if (keys > kTile - 16) {
#pragma unroll
                for (int k = 1; k < 8; ++k) mma_ts(d, pa + k * 8, vb + (k * 2048 >> 4), kIdPV, 1u);
              } else {
#pragma unroll 1
                for (int k = 1; k * 16 < keys; ++k)
                  mma_ts(d, pa + k * 8, vb + static_cast<uint64_t>(k * 2048 >> 4), kIdPV, 1u);
              }
              mma_commit(&sh.kv_empty[slot]);
              if (what >> 9 & 1) mma_commit(&sh.o_final[t]);
            }
            __syncwarp();
            if (what >> 9 & 1) {
              if (t) ++nd1; else ++nd0;
            }
            ++ip;
            did = true;
          }
        }
        if (did) {
          idle = 0;
        } else if (__any_sync(0xffffffffu, sh.abort != 0)) {
          ok = false;
        } else if (idle == 0) {
          idle = globaltimer();
        } else if (__any_sync(0xffffffffu, globaltimer() - idle > ctl.limit_ns)) {
          if (lane == 0) {
            sh.abort = 1;
            atomicExch(a.err, 1);
          }
          ok = false;
        }
      }
      if (elect_one_sync()) mma_commit(&sh.drain);
      __syncwarp();
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
          uint32_t x[32], y[16];
          if (in0) tmem_ld32(lanes + P::kColO + c, x);
#pragma unroll
          for (int h = 0; h < 32; h += 16) {
            if (in1) tmem_ld16(lanes + P::kColO + DV + c + h, y);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              float v[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                v[q] = in0 ? f0 * __uint_as_float(x[h + e + q]) : 0.f;
                if (in1) v[q] = fmaf(f1, __uint_as_float(y[e + q]), v[q]);
              }
              *reinterpret_cast<float4*>(box + lane * 128 + ((((h + e) >> 2) ^ (lane & 7)) << 4)) =
                  make_float4(v[0], v[1], v[2], v[3]);
            }
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
    const int passes = (a.p.d + 127) / 128;
    int i = 0, ndone = 0, nq = 0, np = 0;
    float qm = 0.f;

    // q~ of the segment's row tile: staging, then the split result (this
    // warpgroup's stream has the segment's first tile)
    auto project = [&]() -> bool {
      const __nv_bfloat16* q = query_row(a, s.hk, s.rt, r);
      const int d = a.p.d;
      if (nq > 0 && !__all_sync(0xffffffffu, wait_or_abort(&sh.q_empty, (nq - 1) & 1, ctl))) return false;
      int c = np;
      uint8_t* to = smem + P::kQ + (r >> 3) * 128 + (r & 7) * 16;
#pragma unroll 1
      for (int k0 = 0; k0 < d; k0 += 128, ++c) {
        if (k0 > 0 && !__all_sync(0xffffffffu, wait_or_abort(&sh.stage_done, (c - 1) & 1, ctl))) return false;
        if (d % 8 == 0) {  // 8 features per load, all in flight
          uint4 x[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            x[e] = q && k0 + 8 * e < d ? __ldg(reinterpret_cast<const uint4*>(q + k0 + 8 * e)) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            *reinterpret_cast<uint4*>(to + (e >> 3) * P::kStage + (e & 7) * 2048) = x[e];
        } else {
#pragma unroll 1
          for (int e = 0; e < 16; ++e) {
            uint32_t x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int k = k0 + 8 * e + 2 * u;
              x[u] = q ? bits_at(q, k, d) | bits_at(q, k + 1, d) << 16 : 0u;
            }
            *reinterpret_cast<uint4*>(to + (e >> 3) * P::kStage + (e & 7) * 2048) = make_uint4(x[0], x[1], x[2], x[3]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.stage_full);
      }
      if (!__all_sync(0xffffffffu, wait_or_abort(&sh.stage_done, (c - 1) & 1, ctl))) return false;
      tc_fence_after();
      float x[M];
#pragma unroll
      for (int k = 0; k < M; k += 16) {
        uint32_t v[16];
        tmem_ld16(tS + k, v);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) x[k + e] = __uint_as_float(v[e]) * a.p.qscale;
      }
      float top = 0.f;
#pragma unroll
      for (int k = 0; k < M; ++k) top = fmaxf(top, fabsf(x[k]));
      int e = 0;
      if (top > 0.f && isfinite(top)) {  // the largest magnitude into [2^13, 2^14)
        frexpf(top, &e);
        e = max(-125, min(125, e - 14));
      }
      const float down = __int_as_float((127 - e) << 23);
#pragma unroll
      for (int k = 0; k < M; k += 8) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float x0 = x[k + 2 * u] * down, x1 = x[k + 2 * u + 1] * down;
          const __half2 h = __floats2half2_rn(x0, x1);
          const float2 f = __half22float2(h);
          const __half2 g = __floats2half2_rn(x0 - f.x, x1 - f.y);
          hi[u] = *reinterpret_cast<const uint32_t*>(&h);
          lo[u] = *reinterpret_cast<const uint32_t*>(&g);
        }
        *reinterpret_cast<uint4*>(to + (k >> 3) * 2048) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(to + ((M + k) >> 3) * 2048) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
      sh.qmul[nq & 1][r] = __int_as_float((127 + e) << 23);
      tc_fence_before();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_full);
      return true;
    };

    while (segs.next_warp(sh, ctl, s, ok)) {
      if (s.qnew) {
        // the other warpgroup waits for it, so that neither runs a row tile ahead
        ok = (i & 1) == t ? project() : __all_sync(0xffffffffu, wait_or_abort(&sh.q_full, nq & 1, ctl));
        if (!ok) break;
        qm = sh.qmul[nq & 1][r];
        ++nq;
        np += passes;
      }
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
        const int j = at - i, n = min(kTile, s.keys - j * kTile), slot = at % ST;
        if (!(ok = __all_sync(0xffffffffu, wait_or_abort(&sh.s_full[t], (at / 2) & 1, ctl)))) break;
        tc_fence_after();
        if (n & 15) {  // value rows up to the next step of 16: zero
          uint8_t* vd = smem + P::kRing + slot * P::kSlot + P::kKBytes;
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
          const float* mul = sh.mul[slot];
#pragma unroll
          for (int c = 0; c < 128; c += 4) {
            const float4 k = *reinterpret_cast<const float4*>(mul + c);
            unpack_f32x2(mul_f32x2(pack_f32x2(x[c], x[c + 1]), pack_f32x2(k.x, k.y)), x[c], x[c + 1]);
            unpack_f32x2(mul_f32x2(pack_f32x2(x[c + 2], x[c + 3]), pack_f32x2(k.z, k.w)), x[c + 2], x[c + 3]);
          }
          if (n < kTile) {
#pragma unroll
            for (int c = 0; c < 128; ++c) x[c] = c < n ? x[c] : -INFINITY;
          }
          if (srow) {
            float* to = srow + j * kTile;
#pragma unroll
            for (int c = 0; c < 128; c += 4)
              *reinterpret_cast<float4*>(to + c) = make_float4(x[c] * qm, x[c + 1] * qm, x[c + 2] * qm, x[c + 3] * qm);
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
              const float top = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])) * qm;
              grow = top > m_run + kGrow;
              if (grow) {
                alpha = ex2(m_run - top);  // 0 at the row's first tile
                m_run = top;
              }
            }
            const uint64_t q2 = pack_f32x2(qm, qm), negm = pack_f32x2(-m_run, -m_run);
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

// ----------------------------------------------------------------- combine
constexpr int kCombineThreads = 256;

// The partial results of row (b, h): np prefix segments, then own segments; rows
// of the partial buffers.
struct Parts {
  int np, n;
  int prow, orow;
};

__device__ __forceinline__ Parts parts_of(const Params& a, int b, int h) {
  const Geo& g = a.g;
  const int hk = h / a.p.G, gg = h - hk * a.p.G;
  const int part = g.parts > 1 ? gg / kTile : 0;
  const int rt = g.parts > 1 ? b * g.parts + part : b / g.spt;
  const int lane = g.parts > 1 ? gg - part * kTile : (b - rt * g.spt) * a.p.G + gg;
  Parts x;
  x.np = g.S;
  x.prow = (hk * g.RT + rt) * g.S * g.rows + lane;
  x.n = x.np;
  x.orow = 0;
  const int off = a.w.off[b], n = a.w.off[b + 1] - off, all = a.w.off[a.p.B];
  if (n > 0) {
    const Deal deal(all * g.parts * a.p.Hk, g);
    const int t0 = hk * (all * g.parts) + off * g.parts + part * n;
    const int c0 = deal.owner(t0);  // the CTAs with the first and the last tile
    x.orow = ((hk * a.p.B + b) * g.parts + part + c0) * g.orows + gg - part * kTile;
    x.n += deal.owner(t0 + n - 1) - c0 + 1;
  }
  return x;
}

// Maximum and sum of a row over its partial results, by one warp.
__device__ __forceinline__ float2 stats_of(const Params& a, const Parts& x, int i) {
  const float* p = i < x.np ? a.w.pml + static_cast<size_t>(x.prow + i * a.g.rows) * 2
                            : a.w.oml + static_cast<size_t>(x.orow + (i - x.np) * a.g.orows) * 2;
  return i < x.n ? *reinterpret_cast<const float2*>(p) : make_float2(-INFINITY, 0.f);
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A warp per row of the output (the first `oblocks` blocks), a lane per DV/32 of
// its columns.  The other blocks: the weights of 1024 keys of a (sequence, key head).
template <int DV>
__global__ void __launch_bounds__(kCombineThreads)
    decode_combine_kernel(const __grid_constant__ Params a, int oblocks, int kblocks) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (static_cast<int>(blockIdx.x) < oblocks) {
    const int row = blockIdx.x * (kCombineThreads / 32) + warp;
    if (row >= a.p.B * a.p.H) return;
    const int b = row / a.p.H;
    const Parts x = parts_of(a, b, row - b * a.p.H);
    float top = -INFINITY, sum = 0.f;
    constexpr int C = DV / 32;
    float o[C];
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] = 0.f;
#pragma unroll 1
    for (int i0 = 0; i0 < x.n; i0 += 32) {
      const float2 st = stats_of(a, x, i0 + lane);
      const float now = fmaxf(top, warp_max(st.x));
      const float old = ex2(top - now);  // 0 at first
      const float w = st.y > 0.f ? ex2(st.x - now) : 0.f;
      top = now;
      sum = sum * old + warp_sum(w * st.y);
#pragma unroll
      for (int c = 0; c < C; ++c) o[c] *= old;
      const int n = min(32, x.n - i0);
#pragma unroll 8
      for (int k = 0; k < n; ++k) {
        const int i = i0 + k;
        const float* p = i < x.np ? a.w.po + static_cast<size_t>(x.prow + i * a.g.rows) * DV
                                  : a.w.oo + static_cast<size_t>(x.orow + (i - x.np) * a.g.orows) * DV;
        const float wk = __shfl_sync(0xffffffffu, w, k);
        if constexpr (C == 4) {
          const float4 v = *reinterpret_cast<const float4*>(p + 4 * lane);
          o[0] = fmaf(wk, v.x, o[0]);
          o[1] = fmaf(wk, v.y, o[1]);
          o[2] = fmaf(wk, v.z, o[2]);
          o[3] = fmaf(wk, v.w, o[3]);
        } else {
          const float2 v = *reinterpret_cast<const float2*>(p + 2 * lane);
          o[0] = fmaf(wk, v.x, o[0]);
          o[1] = fmaf(wk, v.y, o[1]);
        }
      }
    }
    const float inv = x.n > 0 ? 1.f / sum : 0.f;  // a row without keys: 0
    uint32_t* out = reinterpret_cast<uint32_t*>(a.p.out + static_cast<size_t>(row) * DV) + lane * (C / 2);
    if constexpr (C == 4)
      *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
    else
      *out = pack_bf16x2(o[0] * inv, o[1] * inv);
    return;
  }
  const int w = blockIdx.x - oblocks, bh = w / kblocks, b = bh / a.p.Hk, hk = bh - b * a.p.Hk;
  const int n = min(max(a.p.lens[b], 0), a.p.cap);
  const int k0 = (w - bh * kblocks) * 1024;
  if (k0 >= n) return;
  __shared__ float lse[128];
  constexpr int E = 1024 / kCombineThreads;
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 1
  for (int g0 = 0; g0 < a.p.G; g0 += 128) {
    const int gn = min(128, a.p.G - g0);
    __syncthreads();
#pragma unroll 1
    for (int g = warp; g < gn; g += kCombineThreads / 32) {
      const Parts x = parts_of(a, b, hk * a.p.G + g0 + g);
      float top = -INFINITY, sum = 0.f;
#pragma unroll 1
      for (int i0 = 0; i0 < x.n; i0 += 32) {
        const float2 st = stats_of(a, x, i0 + lane);
        const float now = fmaxf(top, warp_max(st.x));
        sum = sum * ex2(top - now) + warp_sum(st.y > 0.f ? ex2(st.x - now) * st.y : 0.f);
        top = now;
      }
      if (lane == 0) lse[g] = top + log2f(sum);
    }
    __syncthreads();
    const float* s = a.w.scores + (static_cast<size_t>(b) * a.p.H + hk * a.p.G + g0) * a.g.capr + k0 + tid;
#pragma unroll 2
    for (int g = 0; g < gn; ++g, s += a.g.capr) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (k0 + tid + e * kCombineThreads < n) acc[e] += ex2(s[e * kCombineThreads] - lse[g]);
    }
  }
  const size_t at = static_cast<size_t>(bh) * a.p.cap + k0 + tid;
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (k0 + tid + e * kCombineThreads < n) {
      const size_t k = at + e * kCombineThreads;
      a.p.acc_out[k] = a.p.acc[k] + acc[e];
    }
}

// -------------------------------------------------------------------- host
Geo geometry(const DecodeSharedParams& p, int sms) {
  Geo g{};
  g.spt = p.G <= kTile ? kTile / p.G : 1;
  g.parts = (p.G + kTile - 1) / kTile;
  g.RT = g.parts > 1 ? p.B * g.parts : (p.B + g.spt - 1) / g.spt;
  g.rows = g.parts > 1 ? kTile : (p.B < g.spt ? p.B : g.spt) * p.G;
  g.orows = p.G < kTile ? p.G : kTile;
  g.PT = (p.plen + kTile - 1) / kTile;
  g.capr = (p.cap + kTile - 1) / kTile * kTile;
  const long long rowtiles = static_cast<long long>(p.Hk) * g.RT;
  const long long own = static_cast<long long>(p.Hk) * p.B * g.parts * ((p.cap + kTile - 1) / kTile);
  const int most = sms < kMaxCtas ? sms : kMaxCtas;
  const long long all = own + rowtiles * g.PT;
  g.grid = static_cast<int>(all < 1 ? 1 : all < most ? all : most);
  // the split of the prefix with the shortest schedule: rounds of segments,
  // each its tiles and about one tile's time of start and end
  g.S = g.chunk = 0;
  if (g.PT > 0) {
    long long best = -1;
    long long limit = kPrefixSlots / rowtiles;
    limit = limit < 1 ? 1 : limit > g.PT ? g.PT : limit;
    for (int s = 1; s <= limit; ++s) {
      const int chunk = (g.PT + s - 1) / s, S = (g.PT + chunk - 1) / chunk;
      const long long cost = (rowtiles * S + g.grid - 1) / g.grid * (chunk + 1);
      if (best < 0 || cost < best) {
        best = cost;
        g.S = S;
        g.chunk = chunk;
      }
    }
  }
  g.units = static_cast<int>(rowtiles * g.S);
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
  const size_t orows = p.cap > 0 ? (static_cast<size_t>(p.Hk) * p.B * g.parts + kMaxCtas) * g.orows : 0;
  Work x{};
  x.off = reinterpret_cast<int*>(take((static_cast<size_t>(p.B) + 1) * sizeof(int)));
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
  cudaError_t e = cudaFuncSetAttribute(decode_shared_kernel<M, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       P::kLaunch);
  if (e != cudaSuccess) return e;
  decode_shared_kernel<M, DV><<<a.g.grid, kThreads, P::kLaunch, stream>>>(a, maps);
  return cudaGetLastError();
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
  // counts of tiles and rows of partial results are 31-bit
  const Geo g = geometry(p, kMaxCtas);
  const long long own = static_cast<long long>(p.Hk) * p.B * g.parts, rows = static_cast<long long>(p.Hk) * g.RT;
  const long long tiles = own * ((p.cap + kTile - 1LL) / kTile) + rows * g.PT;
  return tiles < (1LL << 30) && (own + kMaxCtas) * g.orows < (1LL << 30) &&
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
  maps.P = run.P;
  cudaError_t e = p.dv == 64 ? launch_m<64>(a, maps, stream) : launch_m<128>(a, maps, stream);
  if (e != cudaSuccess) return e;
  const int kblocks = p.acc_out ? (p.cap + 1023) / 1024 : 0;
  const int oblocks = (p.B * p.H + kCombineThreads / 32 - 1) / (kCombineThreads / 32);
  const long long blocks = oblocks + static_cast<long long>(p.B) * p.Hk * kblocks;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (p.dv == 64)
    decode_combine_kernel<64><<<static_cast<unsigned>(blocks), kCombineThreads, 0, stream>>>(a, oblocks, kblocks);
  else
    decode_combine_kernel<128><<<static_cast<unsigned>(blocks), kCombineThreads, 0, stream>>>(a, oblocks, kblocks);
  return cudaGetLastError();
}

}  // namespace spa
