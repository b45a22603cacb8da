// decode_shared.cuh -- what the kernels of the shared-prefix decode have in common:
// the layout of a call and of its workspace.
//
// The queries of one key head are the rows (b, g) of a matrix, cut into row
// tiles of up to 128 rows that hold whole groups (a group of more than 128 heads
// is cut into parts).  A call runs
//   decode_query_kernel   q~ = q P_h of every row, split for the tensor cores,
//                         and the own tiles in front of each sequence
//   decode_prefix_kernel  row tiles against ranges of the prefix (and, for groups
//                         of more than 32 heads, against the sequences' own rows)
//   decode_own_kernel     groups of up to 32 heads against the own rows
//   decode_combine_kernel the parts of a row joined; the weights
// Every part of a row's keys leaves unnormalised sums, a maximum and a sum of
// probabilities in the workspace.
#pragma once
#include <atomic>
#include <cstdint>

#include "kernels.cuh"

namespace spa {
namespace ds {

constexpr int kTile = 128;          // keys per tile, rows per row tile
constexpr int kStep = 16;           // keys per step of the own kernel, rows of its products
constexpr int kOwnWarps = 8;        // warps per CTA of the own kernel
constexpr int kMaxCtas = 256;       // grid limit (sizes the workspace)
constexpr int kPrefixSlots = 1024;  // prefix segments per call at most (beyond one per row tile)
constexpr float kGrow = 40.f;       // log2 units that a running maximum may lag behind

// Division of 31-bit numbers by a divisor that the host knows: a multiplication by its
// scaled reciprocal (Granlund and Montgomery, Division by invariant integers using
// multiplication, 1994).
struct FastDiv {
  uint32_t m, s;
  void set(uint32_t d) {
    if (d == 0) d = 1;
    s = 0;
    while (s < 31 && (1u << s) < d) ++s;
    m = static_cast<uint32_t>(((1ull << 32) * ((1ull << s) - d)) / d + 1);
  }
  __device__ __forceinline__ int operator()(int n) const {
    return static_cast<int>((__umulhi(static_cast<uint32_t>(n), m) + static_cast<uint32_t>(n)) >> s);
  }
};

struct Geo {
  int spt, parts;      // sequences per row tile, row tiles per group
  int RT;              // row tiles per key head
  int rows;            // rows of a tile that can be in use
  int PT, S, chunk;    // prefix tiles, splits, tiles per split
  int units;           // prefix segments
  int grid;            // CTAs of the prefix kernel
  int capr;            // keys per row of the score buffer
  int warp_own;        // the own rows run on decode_own_kernel
  int ounit;           // keys per own tile: 16 there, 128 on the prefix kernel
  int oparts, orows;   // parts of a group there and rows per part
  int workers;         // CTAs or warps that share the own tiles
  int extra, pre;      // workers with one prefix segment more; tiles of the others' prefix segments
  FastDiv dRT, dS, dG, dH, dHk, dspt, dparts, doparts, dworkers, dextra, drest;
};

struct Work {
  int* off;            // [B+1] own tiles of one part in front of each sequence
  uint16_t* qt;        // [Hk][RT][128 * 2m] fp16 q~, high and low parts: (r, k) of a tile at
                       // ((k/8)*16 + r/8)*64 + (r%8)*8 + k%8
  float* qmul;         // [Hk][RT][128] row multipliers
  float *po, *pml;     // prefix segments: [units][rows][dv], [units][rows][2]
  float *oo, *oml;     // own segments: [slots][orows][dv], [slots][orows][2]
  float* scores;       // [B*H][capr], or NULL
};

struct Params {
  DecodeSharedParams p;
  Geo g;
  Work w;
  int* err;
  unsigned long long limit_ns;
  int inject_stall;
};

// K~ and V of the prefix [0] and the sequences [1], boxes of 128 and of 16 rows.
struct Maps {
  CUtensorMap k[2][2], v[2][2];
};

// The own tiles are dealt out in equal runs: `a` tiles to each of the first
// `extra` workers, which have one prefix segment more, `b` to each of the others,
// so that all have about the same number of tiles.  Workers without any lie in
// front or at the end, never between two that have some.  (All counts of tiles
// fit in 30 bits: checked on the host.)
struct Deal {
  int total, extra, a, b;
  __device__ __forceinline__ Deal(int total_, const Geo& g) : total(total_), extra(g.extra) {
    a = g.dworkers(g.units * g.chunk + total + g.workers - 1) - g.pre - g.chunk;
    if (a < 0 || extra == 0) a = 0;
    if (extra > 0) a = min(a, g.dextra(total));
    b = g.drest(total - a * extra + g.workers - extra - 1);
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

__device__ __forceinline__ int length_of(const Params& a, int b) {
  return min(max(a.p.lens[b], 0), a.p.cap);
}

// The sequence whose own tiles hold tile `at` of a part (off[b] <= at < off[b+1]),
// by one warp: 32 probes at a time.
__device__ __forceinline__ int find_sequence(const Params& a, int at) {
  int lo = 0, n = a.p.B;
  while (n > 1) {
    const int step = (n + 31) / 32, probe = lo + (threadIdx.x & 31) * step;
    const bool below = probe < lo + n && a.w.off[probe] <= at;
    const int hit = __popc(__ballot_sync(0xffffffffu, below)) - 1;
    const int end = lo + n;
    lo += hit * step;
    n = min(step, end - lo);
  }
  return lo;
}

// Row tile and row of group member g of sequence b.
__device__ __forceinline__ int row_tile(const Geo& g, int G, int b, int m, int* row) {
  if (g.parts > 1) {
    const int part = m / kTile;
    *row = m - part * kTile;
    return b * g.parts + part;
  }
  const int rt = g.dspt(b);
  *row = (b - rt * g.spt) * G + m;
  return rt;
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

// The kernel before this one in the stream may still be running where this one
// starts; its results are there after the wait.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A kernel's dynamic shared memory, set once per device (every launch sets the same).
template <class Kernel>
cudaError_t allow_smem(Kernel kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

template <class... P, class... A>
cudaError_t launch_after(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t stream,
                         A... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

cudaError_t launch_query(const Params& a, cudaStream_t stream);
cudaError_t launch_own(const Params& a, const Maps& maps, cudaStream_t stream);
cudaError_t launch_combine(const Params& a, cudaStream_t stream);

}  // namespace ds
}  // namespace spa
