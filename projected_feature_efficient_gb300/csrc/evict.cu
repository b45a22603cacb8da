// evict.cu -- the rows of smallest accumulated attention weight leave the
// projected key cache, in place.
//
// Of the n rows of a (sequence, head) min(n, budget) stay: first the protected
// ones (the first `sink` token positions and the newest `recent` ones), then
// the others by accumulated weight, ties to the lower row, NaN last.  Rows that
// stay and lie below the new length do not move; the others, in ascending
// order, fill the places of the evicted ones, in ascending order.  Attention
// does not depend on the order of the rows, so a step that drops one row moves
// one row, where a compaction in order would move half of the cache.
// Sources lie at or behind the new length and destinations in front of it: the
// moves of all rows run at once.
//
//   evict_select_kernel  one CTA per (sequence, head): the weight of the last
//                        row that stays by a radix selection (8 bits at a
//                        time) on order-preserving 32-bit keys, then one pass
//                        that pairs the holes with the rows to move
//   evict_move_kernel    the rows' K~, multiplier and V, a warp per row
#include "kernels.cuh"

namespace spa {
namespace {

constexpr int kSelThreads = 1024;

// Keys in the order of the weights: protected rows on top, NaN at the bottom.
__device__ __forceinline__ uint32_t key_of(float w, int pos, int sink, int last) {
  if (pos < sink || pos > last) return 0xffffffffu;
  if (w != w) return 0u;
  w += 0.f;  // -0 ranks with 0
  const uint32_t u = __float_as_uint(w);
  // [-inf, inf] maps to [0x007fffff, 0xff800000]
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix sum over the block of a small value per thread; total in *sum.
__device__ __forceinline__ int block_scan(int v, int* red, int* sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += t;
  }
  if (lane == 31) red[warp] = s;
  __syncthreads();
  if (warp == 0) {
    int w = red[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += t;
    }
    red[lane] = w;
  }
  __syncthreads();
  const int before = (warp ? red[warp - 1] : 0) + s - v;
  *sum = red[31];
  __syncthreads();
  return before;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p) {
  __shared__ int hist[256];
  __shared__ int red[32];
  __shared__ int sh_bin, sh_above;
  const int bh = blockIdx.x, b = bh / p.H, tid = threadIdx.x;
  const int n = min(max(p.lens[b], 0), p.cap);
  const int left = min(n, p.budget);
  const float* acc = p.acc + static_cast<size_t>(bh) * p.cap;
  const int* pos = p.row_pos + static_cast<size_t>(bh) * p.cap;
  float* acc_out = p.acc_out + static_cast<size_t>(bh) * p.cap;
  int* pos_out = p.row_pos_out + static_cast<size_t>(bh) * p.cap;
  int* src = p.src + static_cast<size_t>(bh) * p.budget;
  int* ws = p.ws + static_cast<size_t>(bh) * evict_stride(p.cap, p.budget);
  for (int i = left + tid; i < p.budget; i += kSelThreads) src[i] = -1;
  if (n <= p.budget) {
    for (int i = tid; i < n; i += kSelThreads) {
      src[i] = i;
      if (acc_out != acc) acc_out[i] = acc[i];
      if (pos_out != pos) pos_out[i] = pos[i];
    }
    if (tid == 0) ws[0] = 0;
    return;
  }
  // the newest token position
  int newest = -2147483647 - 1;
  for (int i = tid; i < n; i += kSelThreads) newest = max(newest, pos[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) newest = max(newest, __shfl_xor_sync(0xffffffffu, newest, o));
  if ((tid & 31) == 0) red[tid >> 5] = newest;
  __syncthreads();
  newest = red[0];
  for (int w = 1; w < 32; ++w) newest = max(newest, red[w]);
  __syncthreads();
  // positions above `last` are protected (in 64 bits: `recent` may reach below the lowest)
  const long long last64 = static_cast<long long>(newest) - p.recent;
  const int last = last64 < -2147483647LL - 1 ? -2147483647 - 1 : static_cast<int>(last64);

  // radix selection of the left-th largest key
  uint32_t prefix = 0, mask = 0;
  int want = left;  // this many keys are wanted among those that match the prefix
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kSelThreads) {
      const uint32_t k = key_of(acc[i], pos[i], p.sink, last);
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1);
    }
    __syncthreads();
    // thread t < 256 looks at bin 255 - t: how many keys lie in higher bins
    const int c = tid < 256 ? hist[255 - tid] : 0;
    int total;
    const int above = block_scan(c, red, &total);
    if (tid < 256 && above < want && above + c >= want) {
      sh_bin = 255 - tid;
      sh_above = above;
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(sh_bin) << shift;
    mask |= 255u << shift;
    want -= sh_above;
    __syncthreads();
  }
  // keys above `prefix` stay, and the first `want` rows of those equal to it
  int ties = 0, holes = 0, movers = 0;
  for (int i0 = 0; i0 < n; i0 += kSelThreads) {
    const int i = i0 + tid;
    float a = 0.f;
    int ps = 0;
    uint32_t k = 0;
    if (i < n) {
      a = acc[i];
      ps = pos[i];
      k = key_of(a, ps, p.sink, last);
    }
    const bool tie = i < n && k == prefix;
    int sum;
    const int tr = ties + block_scan(tie, red, &sum);
    ties += sum;
    const bool kept = i < n && (k > prefix || (tie && tr < want));
    // below the new length the places to fill are counted, behind it the rows to move
    const bool hole = i < left && !kept, mover = i >= left && kept;
    const int hr = holes + block_scan(hole, red, &sum);
    holes += sum;
    const int mr = movers + block_scan(mover, red, &sum);
    movers += sum;
    if (hole) ws[4 + 2 * hr] = i;
    __syncthreads();  // the holes come before the rows that fill them
    if (kept && i < left) {
      src[i] = i;
      if (acc_out != acc) acc_out[i] = a;
      if (pos_out != pos) pos_out[i] = ps;
    }
    if (mover) {
      const int to = ws[4 + 2 * mr];
      ws[4 + 2 * mr + 1] = i;
      src[to] = i;
      acc_out[to] = a;
      pos_out[to] = ps;
    }
  }
  if (tid == 0) ws[0] = holes;
}

constexpr int kMoveThreads = 256;

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p, int blocks) {
  const int bh = blockIdx.x / blocks, part = blockIdx.x % blocks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int* ws = p.ws + static_cast<size_t>(bh) * evict_stride(p.cap, p.budget);
  const int moves = ws[0];
  const int kp = p.m / 8, vp = p.dv / 8;  // 16-byte pieces of a row
  uint4* kc = reinterpret_cast<uint4*>(p.kc) + static_cast<size_t>(bh) * p.cap * kp;
  uint4* v = reinterpret_cast<uint4*>(p.v) + static_cast<size_t>(bh) * p.cap * vp;
  float* mul = p.kc_mul + static_cast<size_t>(bh) * p.cap;
  for (int i = part * (kMoveThreads / 32) + warp; i < moves; i += blocks * (kMoveThreads / 32)) {
    const size_t to = ws[4 + 2 * i], from = ws[4 + 2 * i + 1];
    if (lane < kp) kc[to * kp + lane] = kc[from * kp + lane];
    if (lane < vp) v[to * vp + lane] = v[from * vp + lane];
    if (lane == 0) mul[to] = mul[from];
  }
  // one thread per sequence reads its length and writes the new one
  if (part == 0 && bh % p.H == 0 && threadIdx.x == 0) {
    const int b = bh / p.H;
    p.lens_out[b] = min(min(max(p.lens[b], 0), p.cap), p.budget);
  }
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream) {
  evict_select_kernel<<<p.B * p.H, kSelThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int blocks = (152 * 8 + p.B * p.H - 1) / (p.B * p.H);
  evict_move_kernel<<<p.B * p.H * blocks, kMoveThreads, 0, stream>>>(p, blocks);
  return cudaGetLastError();
}

}  // namespace spa
