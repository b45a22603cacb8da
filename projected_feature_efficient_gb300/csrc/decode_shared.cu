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
constexpr uint32_t kRegSoftmax = 184, kRegOther = 72;
static_assert(128 * (2 * kRegSoftmax + 2 * kRegOther) <= kThreads * 128, "register split exceeds the launch");
constexpr int kLoadWarp = 12, kMmaWarp = 13, kMulWarp = 14;
constexpr int kTile = 128;             // keys per tile, rows per row tile
constexpr int kLenCache = 1024;        // sequences whose lengths fit in shared memory
constexpr float kSumLimit = 1099511627776.f;  // 2^40
constexpr float kGrow = 40.f;
constexpr int kMaxCtas = 256;          // grid limit (sizes the workspace)
constexpr int kPrefixSlots = 1024;     // prefix segments per call at most (beyond one per row tile)
constexpr int kMaxDynSmem = 227 * 1024 - 14 * 1024;

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
  long long* off;      // [B+1] own tiles of one part in front of each sequence
  float *po, *pml;     // prefix segments: [units][rows][dv], [units][rows][2]
  float *oo, *oml;     // own segments
  float* scores;       // [B*H][capr], or NULL
};

struct Maps {
  CUtensorMap k[2][2], v[2][2];  // [own][128-row or 16-row box]
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
  // the staging of q and P_h for the projection lies in the place of the result
  static constexpr int kStageP = 16384;
  static constexpr int kQBytes = cmax(kTile * 4 * M, kStageP + 64 * M * 2);
  static constexpr int kQ = 0, kRing = (kQBytes + 1023) / 1024 * 1024;
  static constexpr int kFit = (kMaxDynSmem - 1024 - kRing) / kSlot;
  static constexpr int kStages = kFit > 4 ? 4 : kFit;
  static constexpr int kBytes = kRing + kStages * kSlot + 1024;
  // one CTA per SM: a second one would wait in tcgen05.alloc for the 512 columns
  static constexpr int kLaunch = cmax(kBytes, 120 * 1024);
  static_assert(kStages >= 2 && kLaunch <= kMaxDynSmem, "shared-memory plan");
  static constexpr uint32_t kColS = 0, kColO = 256;
  static constexpr int kKRow = M < 64 ? M * 2 : 128;  // bytes of a K~ row in shared memory (a box)
};

struct Shared {
  uint64_t kv_full[4], kv_empty[4], mul_full[4];
  uint64_t s_full[2], p_full[2], o_final[2], o_empty[2], stats_full[2];
  uint64_t q_empty, q_full, stage_full, stage_done, drain;
  uint32_t tmem;
  volatile int abort;
  long long own0, own1, per_head;  // this CTA's own tiles, own tiles per key head
  int hk, b, part, tile;           // where they start
  long long red[kThreads / 32];
  float stat_l[2][2][kTile], stat_m[2][2][kTile];
  float qmul[2][kTile];
  alignas(16) float mul[4][kTile];  // read four at a time
  int len[kLenCache];
};
static_assert(offsetof(Shared, mul) % 16 == 0 && alignof(Shared) >= 16, "vector loads of the multipliers");

__device__ __forceinline__ int read_length(const Params& a, int b) {
  return a.p.cap > 0 ? min(max(a.p.lens[b], 0), a.p.cap) : 0;
}
__device__ __forceinline__ int length_of(const Params& a, const Shared& sh, int b) {
  return a.p.B <= kLenCache ? sh.len[b] : read_length(a, b);
}

// A run of key tiles for rows lo .. hi-1 of one row tile.
struct Seg {
  bool own, qnew;
  int hk, rt, b;
  int lo, hi;
  int plane, key0;   // tensor-map coordinates of the first key
  int tiles, keys;
  long long slot;
};

// The segments of a CTA in order.
struct Walker {
  int unit;
  long long o;
  int hk, b, part, tile, last;
  __device__ __forceinline__ Walker(const Shared& sh)
      : unit(blockIdx.x), o(sh.own0), hk(sh.hk), b(sh.b), part(sh.part), tile(sh.tile), last(-1) {}
  __device__ __forceinline__ bool next(const Params& a, const Shared& sh, Seg& s) {
    const Geo& g = a.g;
    if (unit < g.units) {
      s.own = false;
      s.rt = unit % g.RT;
      const int split = (unit / g.RT) % g.S;
      s.hk = unit / (g.RT * g.S);
      s.slot = (static_cast<long long>(s.hk) * g.RT + s.rt) * g.S + split;
      s.lo = 0;
      s.hi = g.parts > 1 ? min(kTile, a.p.G - (s.rt % g.parts) * kTile)
                         : min(g.spt, a.p.B - s.rt * g.spt) * a.p.G;
      s.plane = s.hk;
      s.key0 = split * g.chunk * kTile;
      s.tiles = min(g.chunk, g.PT - split * g.chunk);
      s.keys = min(s.tiles * kTile, a.p.plen - s.key0);
      s.b = -1;
      unit += gridDim.x;
    } else {
      if (o >= sh.own1) return false;
      int len = length_of(a, sh, b), n = (len + kTile - 1) / kTile;
      while (n == 0) {  // a sequence without own rows
        step(a);
        len = length_of(a, sh, b);
        n = (len + kTile - 1) / kTile;
      }
      s.own = true;
      s.hk = hk;
      s.b = b;
      s.tiles = static_cast<int>(min(static_cast<long long>(n - tile), sh.own1 - o));
      s.key0 = tile * kTile;
      s.keys = min(s.tiles * kTile, len - s.key0);
      s.plane = b * a.p.Hk + hk;
      s.slot = (static_cast<long long>(hk) * a.p.B + b) * g.parts + part + blockIdx.x;
      if (g.parts > 1) {
        s.rt = b * g.parts + part;
        s.lo = 0;
        s.hi = min(kTile, a.p.G - part * kTile);
      } else {
        s.rt = b / g.spt;
        s.lo = (b - s.rt * g.spt) * a.p.G;
        s.hi = s.lo + a.p.G;
      }
      o += s.tiles;
      tile += s.tiles;
      if (tile == n) {
        tile = 0;
        if (++part == g.parts) step(a);
      }
    }
    const int q = s.hk * g.RT + s.rt;
    s.qnew = q != last;
    last = q;
    return true;
  }
  __device__ __forceinline__ void step(const Params& a) {
    part = 0;
    if (++b == a.p.B) {
      b = 0;
      ++hk;
    }
  }
};

// The own tiles are dealt out in equal runs: `a` tiles to each of the first
// `extra` CTAs, which have one prefix segment more, `b` to each of the others,
// so that all have about the same number of tiles.  CTAs without any lie in
// front or at the end, never between two that have some.
struct Deal {
  long long total;
  int extra;
  long long a, b;
  __host__ __device__ __forceinline__ Deal(long long total_, const Geo& g) : total(total_) {
    const int full = g.units / g.grid;
    extra = g.units % g.grid;
    const long long all = static_cast<long long>(g.units) * g.chunk + total;
    a = (all + g.grid - 1) / g.grid - static_cast<long long>(full + 1) * g.chunk;
    if (a < 0 || extra == 0) a = 0;
    if (a * extra > total) a = total / extra;
    b = (total - a * extra + g.grid - extra - 1) / (g.grid - extra);
  }
  __host__ __device__ __forceinline__ long long start(int c) const {
    if (c <= extra) return a * c;
    const long long t = a * extra + b * (c - extra);
    return t < total ? t : total;
  }
  __host__ __device__ __forceinline__ int owner(long long t) const {
    return static_cast<int>(t < a * extra ? t / a : extra + (t - a * extra) / b);
  }
};

// Own tiles of the batch: prefix sums over the sequences, this CTA's share and
// where it starts.  All threads.
__device__ __forceinline__ void make_schedule(const Params& a, Shared& sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = a.p.B, per = (B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, B), b1 = min(b0 + per, B);
  long long sum = 0;
  for (int b = b0; b < b1; ++b) {
    const int len = read_length(a, b);
    if (B <= kLenCache) sh.len[b] = len;
    sum += (len + kTile - 1) / kTile;
  }
  long long s = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += t;
  }
  if (lane == 31) sh.red[warp] = s;
  __syncthreads();
  long long base = 0, all = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) base += sh.red[w];
    all += sh.red[w];
  }
  const long long before = base + s - sum;
  const long long head = all * a.g.parts, total = head * a.p.Hk;
  const Deal deal(total, a.g);
  const long long o0 = deal.start(blockIdx.x), o1 = deal.start(blockIdx.x + 1);
  if (tid == 0) {
    sh.own0 = o0;
    sh.own1 = o1;
    sh.per_head = head;
    sh.hk = sh.b = sh.part = sh.tile = 0;
  }
  __syncthreads();
  if (o0 < o1) {
    const int hk = static_cast<int>(o0 / head);
    const long long at = o0 - hk * head;  // within the key head, parts counted
    if (at >= before * a.g.parts && at < (before + sum) * a.g.parts) {
      long long left = at - before * a.g.parts;
      for (int b = b0; b < b1; ++b) {
        const int n = (read_length(a, b) + kTile - 1) / kTile;
        const long long here = static_cast<long long>(n) * a.g.parts;
        if (left < here) {
          sh.hk = hk;
          sh.b = b;
          sh.part = static_cast<int>(left / n);
          sh.tile = static_cast<int>(left % n);
          break;
        }
        left -= here;
      }
    }
  }
  if (blockIdx.x == 0) {  // for the combine kernel
    long long at = before;
    for (int b = b0; b < b1; ++b) {
      a.w.off[b] = at;
      at += (read_length(a, b) + kTile - 1) / kTile;
    }
    if (tid == 0) a.w.off[B] = all;
  }
  __syncthreads();
}

// The query row of lane r of row tile (hk, rt), or NULL.
__device__ __forceinline__ const __nv_bfloat16* query_row(const Params& a, int hk, int rt, int r) {
  int b, g;
  if (a.g.parts > 1) {
    b = rt / a.g.parts;
    g = (rt % a.g.parts) * kTile + r;
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
__device__ __forceinline__ void load_tile(const Maps& maps, uint8_t* slot, uint64_t* bar, bool own, int plane,
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
      mbar_init(&sh.stats_full[t], 4);
    }
    mbar_init(&sh.q_empty, 1);
    mbar_init(&sh.q_full, 4);
    mbar_init(&sh.stage_full, 4);
    mbar_init(&sh.stage_done, 1);
    mbar_init(&sh.drain, 1);
    sh.abort = 0;
    fence_mbar_init();
  }
  make_schedule(a, sh);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = sh.tmem;

  if (warp >= 12) {
    setmaxnreg_dec<kRegOther>();
    if (warp == kLoadWarp) {
      // -------------------------------------------------------------- loader
      if (lane == 0) {
        Walker w(sh);
        Seg s{};
        int i = 0;
        bool ok = true;
        while (ok && w.next(a, sh, s)) {
          for (int j = 0; j < s.tiles; ++j, ++i) {
            const int slot = i % ST;
            if (i >= ST && !(ok = wait_or_abort(&sh.kv_empty[slot], (i / ST - 1) & 1, ctl))) break;
            load_tile<P, M, DV>(maps, smem + P::kRing + slot * P::kSlot, &sh.kv_full[slot], s.own, s.plane,
                                s.key0 + j * kTile, min(kTile, s.keys - j * kTile));
          }
        }
        // every copy that was started lands before the memory is given up
        for (int k = max(0, i - ST); k < i; ++k) mbar_wait(&sh.kv_full[k % ST], (k / ST) & 1, ctl.limit_ns);
      }
    } else if (warp == kMulWarp) {
      // -------------------------------------------------- keys' multipliers
      Walker w(sh);
      Seg s{};
      const float* from = nullptr;
      int j = 0, i = 0;
      bool more = w.next(a, sh, s);
      auto fetch = [&](float (&x)[4]) {  // the next tile's, a tile ahead of its slot
        if (j == 0) {
          const size_t row = static_cast<size_t>(s.plane) * (s.own ? a.p.cap : a.p.pcap) + s.key0;
          from = (s.own ? a.p.kc_mul : a.p.pkc_mul) + row;
        }
        const int n = s.keys - j * kTile;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int k = lane + 32 * c;
          x[c] = k < n ? __ldg(from + j * kTile + k) : 0.f;
        }
        if (++j == s.tiles) {
          j = 0;
          more = w.next(a, sh, s);
        }
      };
      float x[4];
      bool have = more;
      if (have) fetch(x);
      while (have) {
        float y[4];
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
    } else if (warp == kMmaWarp) {
      // ----------------------------------------------------------- MMA issue
      if (lane == 0) {
        constexpr uint32_t kIdS = idesc_f16(128, 128, kFmtF16, 0, 0);
        constexpr uint32_t kIdPV = idesc_f16(128, DV, kFmtBF16, 0, 1);
        constexpr uint32_t kIdQ = idesc_f16(128, M, kFmtBF16, 0, 0);
        // K~ rows as TMA left them: 32-, 64- or 128-byte swizzle by their width
        constexpr uint32_t kKLayout = M == 16 ? 6 : M == 32 ? 4 : kLayoutSwizzle128;
        constexpr uint32_t kKSbo = 8 * P::kKRow;
        Walker w(sh);
        Seg s{};
        int j = 0, is = 0, ip = 0;        // tile in its segment; next score and value products
        int nq = 0, sc = 0;               // row tiles and projection chunks so far
        int ndone[2] = {0, 0};            // segments finished by each stream
        int keys[2] = {0, 0};             // the pending tile of each stream
        bool first[2] = {false, false}, fin[2] = {false, false};
        bool more = w.next(a, sh, s), ok = true, held = false;
        auto project = [&](uint32_t d) -> bool {
          if (nq > 0) mma_commit(&sh.q_empty);  // the old q~ has been read
          for (int c = 0; c < (a.p.d + 63) / 64; ++c, ++sc) {
            if (!wait_or_abort(&sh.stage_full, sc & 1, ctl)) return false;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ss(d, smem_desc(sbase + P::kQ + k * 4096, 2048, 128, kLayoutInterleave),
                     smem_desc(sbase + P::kQ + P::kStageP + k * 2 * (M / 8) * 128, (M / 8) * 128, 128,
                               kLayoutInterleave),
                     kIdQ, c > 0 || k > 0);
            mma_commit(&sh.stage_done);
          }
          if (!wait_or_abort(&sh.q_full, nq & 1, ctl)) return false;
          tc_fence_after();
          ++nq;
          return true;
        };
        uint64_t idle = 0;
        while (ok && (more || ip < is)) {
          bool did = false;
          if (more && is < ip + 2) {
            const int slot = is % ST, t = is & 1;
            if (mbar_test_wait(&sh.kv_full[slot], (is / ST) & 1) &&
                mbar_test_wait(&sh.mul_full[slot], (is / ST) & 1)) {
              const uint32_t d = tb + P::kColS + t * 128;
              if (j == 0 && s.qnew && !(ok = project(d))) break;
              tc_fence_after();
              const uint32_t kb = sbase + P::kRing + slot * P::kSlot;
#pragma unroll
              for (int k = 0; k < 2 * M / 16; ++k) {  // high parts, then low parts of q~
                const int kk = k % (M / 16);
                mma_ss(d, smem_desc(sbase + P::kQ + k * 4096, 2048, 128, kLayoutInterleave),
                       smem_desc(kb + (kk >> 2) * 16384 + (kk & 3) * 32, 16, kKSbo, kKLayout), kIdS, k > 0);
              }
              // a failure-detection test withholds the first "scores ready"
              if (!(a.inject_stall && !held)) mma_commit(&sh.s_full[t]);
              held = true;
              keys[t] = min(kTile, s.keys - j * kTile);
              first[t] = j < 2;
              fin[t] = j + 2 >= s.tiles;
              ++is;
              if (++j == s.tiles) {
                j = 0;
                more = w.next(a, sh, s);
              }
              did = true;
            }
          }
          if (!did && ip < is) {
            const int slot = ip % ST, t = ip & 1;
            if (mbar_test_wait(&sh.p_full[t], (ip / 2) & 1) &&
                (!first[t] || ndone[t] == 0 || mbar_test_wait(&sh.o_empty[t], (ndone[t] - 1) & 1))) {
              tc_fence_after();
              const uint32_t pa = tb + P::kColS + t * 128, d = tb + P::kColO + t * DV;
              const uint32_t vb = sbase + P::kRing + slot * P::kSlot + P::kKBytes;
              const int steps = (keys[t] + 15) / 16;
              for (int k = 0; k < steps; ++k)
                mma_ts(d, pa + k * 8, smem_desc(vb + k * 2048, 16384, 1024, kLayoutSwizzle128), kIdPV,
                       !(first[t] && k == 0));
              mma_commit(&sh.kv_empty[slot]);
              if (fin[t]) {
                mma_commit(&sh.o_final[t]);
                ++ndone[t];
              }
              ++ip;
              did = true;
            }
          }
          if (did) {
            idle = 0;
          } else if (sh.abort) {
            ok = false;
          } else if (idle == 0) {
            idle = globaltimer();
          } else if (globaltimer() - idle > ctl.limit_ns) {
            sh.abort = 1;
            atomicExch(a.err, 1);
            ok = false;
          }
        }
        mma_commit(&sh.drain);
        mbar_wait(&sh.drain, 0, ctl.limit_ns);  // own products in flight
      }
    }
  } else if (warp >= 8) {
    // ---------------------------------------------------------------- output
    setmaxnreg_dec<kRegOther>();
    const int r = tid & 127;
    const uint32_t lanes = tb + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    int nd[2] = {0, 0}, i0 = 0;
    Walker w(sh);
    Seg s{};
    bool ok = true;
    while (ok && w.next(a, sh, s)) {
      // streams of this segment: the tiles of number i0 .. i0 + tiles - 1
      const bool in[2] = {s.tiles > 1 || (i0 & 1) == 0, s.tiles > 1 || (i0 & 1) == 1};
      i0 += s.tiles;
      float mx[2], l[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        mx[t] = -INFINITY;
        l[t] = 0.f;
        if (!in[t]) continue;
        ok = ok && __all_sync(0xffffffffu, wait_or_abort(&sh.o_final[t], nd[t] & 1, ctl) &&
                                               wait_or_abort(&sh.stats_full[t], nd[t] & 1, ctl));
        if (!ok) break;
        mx[t] = sh.stat_m[t][nd[t] & 1][r];
        l[t] = sh.stat_l[t][nd[t] & 1][r];
      }
      if (!ok) break;
      tc_fence_after();
      const int w0 = (warp & 3) * 32;
      if (w0 < s.hi && w0 + 32 > s.lo) {  // warp-uniform: rows of the segment here
        const bool mine = r >= s.lo && r < s.hi;
        const float top = fmaxf(mx[0], mx[1]);
        const float f0 = in[0] ? ex2(mx[0] - top) : 0.f, f1 = in[1] ? ex2(mx[1] - top) : 0.f;
        const long long row = s.own ? s.slot * a.g.orows + (r - s.lo) : s.slot * a.g.rows + r;
        float* o = (s.own ? a.w.oo : a.w.po) + row * DV;
        if (mine) {
          float2* ml = reinterpret_cast<float2*>((s.own ? a.w.oml : a.w.pml) + row * 2);
          *ml = make_float2(top, f0 * l[0] + f1 * l[1]);
        }
#pragma unroll 1
        for (int c = 0; c < DV; c += 16) {
          uint32_t x[16], y[16];
          if (in[0]) tmem_ld16(lanes + P::kColO + c, x);
          if (in[1]) tmem_ld16(lanes + P::kColO + DV + c, y);
          tmem_wait_ld();
          if (mine) {
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              float v[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                v[q] = in[0] ? f0 * __uint_as_float(x[e + q]) : 0.f;
                if (in[1]) v[q] = fmaf(f1, __uint_as_float(y[e + q]), v[q]);
              }
              *reinterpret_cast<float4*>(o + c + e) = make_float4(v[0], v[1], v[2], v[3]);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (!in[t]) continue;
        if (lane == 0) mbar_arrive(&sh.o_empty[t]);
        ++nd[t];
      }
    }
  } else {
    // --------------------------------------------------------------- softmax
    setmaxnreg_inc<kRegSoftmax>();
    const int t = warp >> 2, r = tid & 127;
    const uint32_t lanes = tb + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t tS = lanes + P::kColS + t * 128, tO = lanes + P::kColO + t * DV;
    int i = 0, ndone = 0, nq = 0, sc = 0, seen = -1;
    float qm = 0.f;
    Walker w(sh);
    Seg s{};
    bool ok = true;

    // q~ of the segment's row tile: staging, then the split result (this
    // warpgroup's stream has the segment's first tile)
    auto project = [&]() -> bool {
      if (nq > 0 && !__all_sync(0xffffffffu, wait_or_abort(&sh.q_empty, (nq - 1) & 1, ctl))) return false;
      const __nv_bfloat16* q = query_row(a, s.hk, s.rt, r);
      const __nv_bfloat16* Ph = a.p.P + static_cast<size_t>(s.hk) * a.p.d * M;
      const int d = a.p.d;
      int c = sc;
      for (int k0 = 0; k0 < d; k0 += 64, ++c) {
        if (k0 > 0 && !__all_sync(0xffffffffu, wait_or_abort(&sh.stage_done, (c - 1) & 1, ctl))) return false;
#pragma unroll
        for (int e = 0; e < 8; ++e) {  // row r of q: 8 features per store
          uint4 x = make_uint4(0u, 0u, 0u, 0u);
          const int k = k0 + 8 * e;
          if (q && k < d) {
            if (d % 8 == 0) {
              x = __ldg(reinterpret_cast<const uint4*>(q + k));
            } else {
              x.x = bits_at(q, k, d) | bits_at(q, k + 1, d) << 16;
              x.y = bits_at(q, k + 2, d) | bits_at(q, k + 3, d) << 16;
              x.z = bits_at(q, k + 4, d) | bits_at(q, k + 5, d) << 16;
              x.w = bits_at(q, k + 6, d) | bits_at(q, k + 7, d) << 16;
            }
          }
          *reinterpret_cast<uint4*>(smem + P::kQ + (e * 16 + (r >> 3)) * 128 + (r & 7) * 16) = x;
        }
        for (int task = r; task < 8 * M; task += 128) {  // P_h transposed: 8 features of column n
          const int e = task / M, n = task % M, k = k0 + 8 * e;
          uint32_t x[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint32_t lo = k + 2 * u < d ? __bfloat16_as_ushort(Ph[static_cast<size_t>(k + 2 * u) * M + n]) : 0u;
            const uint32_t hi = k + 2 * u + 1 < d ? __bfloat16_as_ushort(Ph[static_cast<size_t>(k + 2 * u + 1) * M + n]) : 0u;
            x[u] = lo | hi << 16;
          }
          *reinterpret_cast<uint4*>(smem + P::kQ + P::kStageP + (e * (M / 8) + (n >> 3)) * 128 + (n & 7) * 16) =
              make_uint4(x[0], x[1], x[2], x[3]);
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
        uint8_t* to = smem + P::kQ + ((k >> 3) * 16 + (r >> 3)) * 128 + (r & 7) * 16;
        *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(to + (M >> 3) * 16 * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
      sh.qmul[nq & 1][r] = __int_as_float((127 + e) << 23);
      tc_fence_before();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_full);
      return true;
    };

    while (ok && w.next(a, sh, s)) {
      if (s.qnew) {
        // the other warpgroup waits for it, so that neither runs a row tile ahead
        ok = (i & 1) == t ? project() : __all_sync(0xffffffffu, wait_or_abort(&sh.q_full, nq & 1, ctl));
        if (!ok) break;
        ++nq;
        sc += (a.p.d + 63) / 64;
      }
      const int w0 = (warp & 3) * 32;
      const bool here = w0 < s.hi && w0 + 32 > s.lo;  // warp-uniform
      const bool mine = r >= s.lo && r < s.hi;
      float m_run = -INFINITY, l_run = 0.f;
      const int i1 = i + s.tiles;
      int at = i + ((i & 1) != t);  // this stream's first tile
      bool any = at < i1;
      float* srow = nullptr;
      if (s.own && mine && a.w.scores) {
        const int g = (a.g.parts > 1 ? (s.rt % a.g.parts) * kTile : 0) + r - s.lo;
        srow = a.w.scores + (static_cast<size_t>(s.b) * a.p.H + s.hk * a.p.G + g) * a.g.capr + s.key0;
      }
      for (; at < i1; at += 2) {
        const int j = at - i, n = min(kTile, s.keys - j * kTile), slot = at % ST;
        if (!(ok = __all_sync(0xffffffffu, wait_or_abort(&sh.s_full[t], (at / 2) & 1, ctl)))) break;
        tc_fence_after();
        if (seen != nq) {
          qm = sh.qmul[(nq - 1) & 1][r];
          seen = nq;
        }
        if (n & 15) {  // value rows up to the next step of 16: zero
          uint8_t* vd = smem + P::kRing + slot * P::kSlot + P::kKBytes;
          const int rows = 16 - (n & 15), words = rows * (DV / 8);
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
          float alpha = 1.f;
          bool grow = false;
          auto take_max = [&]() {
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
          };
          auto exps = [&]() -> float {
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
            float ls = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float u, v;
              unpack_f32x2(sum[e], u, v);
              ls += u + v;
            }
            return ls;
          };
          const bool fresh = j < 2;  // the stream's first tile of the segment
          if (fresh) take_max();
          float lsum = exps();
          if (!fresh && __any_sync(0xffffffffu, mine && !(lsum <= kSumLimit))) {
            take_max();
            if (__any_sync(0xffffffffu, grow)) lsum = exps();
            if (__any_sync(0xffffffffu, grow)) {  // the row's sums follow the maximum
#pragma unroll
              for (int c = 0; c < DV; c += 32) {
                uint32_t o[32];
                tmem_ld32(tO + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                tmem_st32(tO + c, o);
              }
            }
          }
          l_run = l_run * alpha + lsum;
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[t]);
      }
      if (!ok) break;
      i = i1;
      if (any) {
        // the output has taken the stream's last statistics: a segment of one
        // tile could otherwise be two phases of stats_full ahead of its waiters
        ok = ndone == 0 || __all_sync(0xffffffffu, wait_or_abort(&sh.o_empty[t], (ndone - 1) & 1, ctl));
        if (!ok) break;
        sh.stat_l[t][ndone & 1][r] = l_run;
        sh.stat_m[t][ndone & 1][r] = m_run;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.stats_full[t]);
        ++ndone;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tb, 512);
}

// ----------------------------------------------------------------- combine
constexpr int kCombineThreads = 128;

// The partial results of row (b, h): prefix segments, then own segments.
struct Parts {
  const float *po, *pml, *oo, *oml;
  int np, n;                 // prefix segments, all
  size_t pstep, ostep;       // rows between consecutive ones
  __device__ __forceinline__ float2 ml(int i) const {
    return *reinterpret_cast<const float2*>(i < np ? pml + i * pstep * 2 : oml + (i - np) * ostep * 2);
  }
  __device__ __forceinline__ const float* o(int i, int dv) const {
    return i < np ? po + i * pstep * dv : oo + (i - np) * ostep * dv;
  }
};

__device__ __forceinline__ Parts parts_of(const Params& a, int b, int h) {
  const Geo& g = a.g;
  const int hk = h / a.p.G, gg = h - hk * a.p.G;
  const int part = g.parts > 1 ? gg / kTile : 0;
  const int rt = g.parts > 1 ? b * g.parts + part : b / g.spt;
  const int lane = g.parts > 1 ? gg - part * kTile : (b - rt * g.spt) * a.p.G + gg;
  Parts x;
  x.np = g.PT > 0 ? g.S : 0;
  const size_t prow = (static_cast<size_t>(hk) * g.RT + rt) * g.S * g.rows + lane;
  x.pml = a.w.pml + prow * 2;
  x.po = a.w.po + prow * a.p.dv;
  x.pstep = g.rows;
  x.ostep = g.orows;
  x.n = x.np;
  x.oml = x.oo = nullptr;
  const long long off = a.w.off[b], n = a.w.off[b + 1] - off, all = a.w.off[a.p.B];
  if (n > 0) {
    const long long head = all * g.parts, total = head * a.p.Hk;
    const long long t0 = hk * head + off * g.parts + part * n, t1 = t0 + n - 1;
    const Deal deal(total, g);
    const int c0 = deal.owner(t0), c1 = deal.owner(t1);
    const size_t slot = (static_cast<size_t>(hk) * a.p.B + b) * g.parts + part + c0;
    const size_t orow = slot * g.orows + (gg - part * kTile);
    x.oml = a.w.oml + orow * 2;
    x.oo = a.w.oo + orow * a.p.dv;
    x.n += c1 - c0 + 1;
  }
  return x;
}

// Maximum and sum of a row over its partial results, by one warp.
__device__ __forceinline__ void join(const Parts& x, int lane, float& top, float& sum) {
  top = -INFINITY;
  for (int i = lane; i < x.n; i += 32) top = fmaxf(top, x.ml(i).x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  sum = 0.f;
  for (int i = lane; i < x.n; i += 32) {
    const float2 v = x.ml(i);
    sum = fmaf(exp2f(v.x - top), v.y, sum);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
}

// Blocks 0 .. B*H-1: a row of the output.  The others: the weights of 1024
// keys of a (sequence, key head).
__global__ void __launch_bounds__(kCombineThreads) decode_combine_kernel(const __grid_constant__ Params a, int kblocks) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rows = a.p.B * a.p.H;
  const int blk = blockIdx.x;
  if (blk < rows) {
    const int b = blk / a.p.H, h = blk % a.p.H, dv = a.p.dv;
    const Parts x = parts_of(a, b, h);
    float top, sum;
    join(x, lane, top, sum);
    __shared__ float half[64];
    const int groups = kCombineThreads / dv, g = tid / dv, c = tid % dv;
    float o = 0.f;
#pragma unroll 4
    for (int i = g; i < x.n; i += groups) o = fmaf(exp2f(x.ml(i).x - top), x.o(i, dv)[c], o);
    if (groups == 2) {
      if (g == 1) half[c] = o;
      __syncthreads();
      if (g == 0) o += half[c];
    }
    if (g == 0) a.p.out[static_cast<size_t>(blk) * dv + c] = __float2bfloat16_rn(x.n > 0 ? o / sum : 0.f);
    return;
  }
  const int w = blk - rows, bh = w / kblocks, b = bh / a.p.Hk, hk = bh % a.p.Hk;
  const int n = min(max(a.p.lens[b], 0), a.p.cap);
  const int k0 = (w % kblocks) * 1024;
  if (k0 >= n) return;
  __shared__ float lse[128];
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.f;
  for (int g0 = 0; g0 < a.p.G; g0 += 128) {
    const int gn = min(128, a.p.G - g0);
    __syncthreads();
    for (int g = warp; g < gn; g += kCombineThreads / 32) {
      float top, sum;
      join(parts_of(a, b, hk * a.p.G + g0 + g), lane, top, sum);
      if (lane == 0) lse[g] = top + log2f(sum);
    }
    __syncthreads();
    const float* s = a.w.scores + (static_cast<size_t>(b) * a.p.H + hk * a.p.G + g0) * a.g.capr + k0;
    for (int g = 0; g < gn; ++g, s += a.g.capr) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int k = tid + e * kCombineThreads;
        if (k0 + k < n) acc[e] += ex2(s[k] - lse[g]);
      }
    }
  }
  const size_t at = static_cast<size_t>(bh) * a.p.cap + k0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int k = tid + e * kCombineThreads;
    if (k0 + k < n) a.p.acc_out[at + k] = a.p.acc[at + k] + acc[e];
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
  x.off = reinterpret_cast<long long*>(take((static_cast<size_t>(p.B) + 1) * sizeof(long long)));
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
  cudaError_t e = p.dv == 64 ? launch_m<64>(a, maps, stream) : launch_m<128>(a, maps, stream);
  if (e != cudaSuccess) return e;
  const int kblocks = p.acc_out ? (p.cap + 1023) / 1024 : 0;
  const long long blocks = static_cast<long long>(p.B) * p.H + static_cast<long long>(p.B) * p.Hk * kblocks;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  decode_combine_kernel<<<static_cast<unsigned>(blocks), kCombineThreads, 0, stream>>>(a, kblocks > 0 ? kblocks : 1);
  return cudaGetLastError();
}

}  // namespace spa
