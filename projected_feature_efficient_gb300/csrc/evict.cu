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
//   evict_select_kernel  one CTA per (sequence, head): the weights once from
//                        memory, as order-preserving 32-bit keys in registers (or
//                        shared memory, by the cache's length); the key of the last
//                        row that stays by a radix selection (or, for a few rows to
//                        drop, those one by one); then the ranks of holes and of rows
//                        to move, a lane per row
//   evict_move_kernel    the rows' K~, multiplier and V, a warp per row; many warps
//                        with a row each in flight beat fewer with more (64 pairs
//                        of up to 16383 rows: 52 us for a call with the caches
//                        flushed before it, two rows 54, four 60, eight 71)
// The first is bound by issued instructions and the latency of its passes, the second
// by memory.  Dropping one of 2049 rows of 512 pairs: selection 9.5 us, move 4.7 us
// (what it cannot do without: 3.1 us of memory traffic); 4096 of up to 16383 rows of
// 64 pairs, which occupy 64 SMs in the selection: 46.7 us a call in a stream of calls,
// selection 26 us, move 15 to 17 us (traffic: 13.8 us).
// Selections that were measured on 512 pairs of 2049 rows: a histogram of 8 bits per
// pass 18 us, equal digits of a warp counted by one lane 39 us, two bits per pass by
// counting keys above three candidates 31 us, the worst row looked for 9.5 us.
#include "decode_shared.cuh"
#include "kernels.cuh"

namespace spa {
namespace {

// Keys in the order of the weights: protected rows on top, NaN at the bottom.
__device__ __forceinline__ uint32_t key_of(float w, int pos, int sink, int last) {
  if (pos < sink || pos > last) return 0xffffffffu;
  if (w != w) return 0u;
  w += 0.f;  // -0 ranks with 0
  const uint32_t u = __float_as_uint(w);
  // [-inf, inf] maps to [0x007fffff, 0xff800000]
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Counts (one per warp, the same in all its lanes) of the warps in front of this one.
template <int THREADS>
__device__ __forceinline__ int2 warps_before(int2 v, int2* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  const int2 w = lane < warp ? red[lane] : make_int2(0, 0);
  return make_int2(__reduce_add_sync(0xffffffffu, w.x), __reduce_add_sync(0xffffffffu, w.y));
}

// Where the keys are between the passes.
enum Keys { kRegisters, kShared, kNowhere };
constexpr int kRegKeys = 16;        // rows per thread that fit in registers
constexpr int kFew = 4;             // rows to drop that are looked for one by one
constexpr int kSharedRows = 49600;  // rows whose keys fit in 200 KB of shared memory

template <int THREADS, Keys KEYS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) evict_select_kernel(const EvictParams p) {
  extern __shared__ uint32_t dyn[];  // a bit per row that stays; kShared: the keys behind them
  constexpr int W = THREADS / 32;
  __shared__ alignas(16) int hist[2][256];
  __shared__ uint64_t found[2][W];
  __shared__ int red[W];
  __shared__ int2 red2[2][W];
  ds::let_next_start();
  const int bh = blockIdx.x, b = bh / p.H, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = min(max(p.lens[b], 0), p.cap);
  const int left = min(n, p.budget);
  const float* acc = p.acc + static_cast<size_t>(bh) * p.cap;
  const int* pos = p.row_pos + static_cast<size_t>(bh) * p.cap;
  float* acc_out = p.acc_out + static_cast<size_t>(bh) * p.cap;
  int* pos_out = p.row_pos_out + static_cast<size_t>(bh) * p.cap;
  int* src = p.src + static_cast<size_t>(bh) * p.budget;
  int* ws = p.ws + static_cast<size_t>(bh) * evict_stride(p.cap, p.budget);
  for (int i = left + tid; i < p.budget; i += THREADS) src[i] = -1;
  if (n <= p.budget) {
    for (int i = tid; i < n; i += THREADS) {
      src[i] = i;
      if (acc_out != acc) acc_out[i] = acc[i];
      if (pos_out != pos) pos_out[i] = pos[i];
    }
    if (tid == 0) ws[0] = 0;
    return;
  }
  // A warp takes a run of 32-row words, w0 .. w1-1, a lane a row of each.
  const int words = (n + 31) / 32, per = (words + W - 1) / W;
  const int w0 = min(warp * per, words), w1 = min(w0 + per, words);
  const int mine = w1 - w0, row0 = 32 * w0 + lane;
  uint32_t* const bits = dyn;
  uint32_t* const keys = dyn + (p.cap + 31) / 32;
  uint32_t reg[KEYS == kRegisters ? kRegKeys : 1];
  float weight[KEYS == kRegisters ? kRegKeys : 1];
  int last = 0;
  // f(word, row, key) for the warp's words; a lane behind the last row has row >= n
  auto each = [&](auto f) {
    if constexpr (KEYS == kRegisters) {
#pragma unroll
      for (int e = 0; e < kRegKeys; ++e)
        if (e < mine) f(w0 + e, row0 + 32 * e, reg[e]);
    } else {
#pragma unroll 4
      for (int w = w0; w < w1; ++w) {
        const int i = 32 * w + lane;
        f(w, i, i >= n ? 0u : KEYS == kShared ? keys[i] : key_of(acc[i], pos[i], p.sink, last));
      }
    }
  };
  // the newest token position
  int newest = -2147483647 - 1;
  if constexpr (KEYS == kRegisters) {
#pragma unroll
    for (int e = 0; e < kRegKeys; ++e) {
      const int i = row0 + 32 * e;
      const bool in = e < mine && i < n;
      const int x = in ? pos[i] : -2147483647 - 1;
      weight[e] = in ? acc[i] : 0.f;
      reg[e] = static_cast<uint32_t>(x);
      newest = max(newest, x);
    }
  } else {
#pragma unroll 8
    for (int w = w0; w < w1; ++w) newest = max(newest, 32 * w + lane < n ? pos[32 * w + lane] : newest);
  }
  newest = __reduce_max_sync(0xffffffffu, newest);
  if (lane == 0) red[warp] = newest;
  __syncthreads();
  newest = __reduce_max_sync(0xffffffffu, red[lane % W]);
  // positions above `last` are protected (in 64 bits: `recent` may reach below the lowest)
  const long long last64 = static_cast<long long>(newest) - p.recent;
  last = last64 < -2147483647LL - 1 ? -2147483647 - 1 : static_cast<int>(last64);
  if constexpr (KEYS == kRegisters) {
#pragma unroll
    for (int e = 0; e < kRegKeys; ++e)
      reg[e] = e < mine && row0 + 32 * e < n ? key_of(weight[e], static_cast<int>(reg[e]), p.sink, last) : 0u;
  } else if constexpr (KEYS == kShared) {
#pragma unroll 8
    for (int w = w0; w < w1; ++w) {
      const int i = 32 * w + lane;
      if (i < n) keys[i] = key_of(acc[i], pos[i], p.sink, last);  // read by this lane alone
    }
  }
  if (n - left <= kFew) {
    // The usual step drops a row: the worst rows one after the other, by smallest
    // key and then last row.
    const int drop = n - left;
    uint64_t gone = ~0ull;  // (key, row from the end) of the last one that went
    int row[kFew];          // the rows that go; none: -1
#pragma unroll
    for (int r = 0; r < kFew; ++r) row[r] = -1;
#pragma unroll 1
    for (int round = 0; round < drop; ++round) {
      uint32_t key = ~0u;
      int at = -1;
      if (round == 0) {
        // a lane meets its rows in ascending order: an equal key goes to the later one
        each([&](int, int i, uint32_t k) {
          if (i < n && k <= key) {
            key = k;
            at = i;
          }
        });
      } else {  // not those that went: smaller keys, and of the same key later rows
        const uint32_t top = static_cast<uint32_t>(gone >> 32);
        each([&](int, int i, uint32_t k) {
          if (i < n && k <= key && (k > top || (k == top && i < row[0]))) {
            key = k;
            at = i;
          }
        });
      }
      uint64_t worst = at < 0 ? ~0ull : static_cast<uint64_t>(key) << 32 | static_cast<uint32_t>(n - 1 - at);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const uint64_t x = __shfl_xor_sync(0xffffffffu, worst, o);
        worst = x < worst ? x : worst;
      }
      if (lane == 0) found[round & 1][warp] = worst;
      __syncthreads();
      worst = found[round & 1][lane % W];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const uint64_t x = __shfl_xor_sync(0xffffffffu, worst, o);
        worst = x < worst ? x : worst;
      }
      gone = worst;
#pragma unroll
      for (int r = kFew - 1; r > 0; --r) row[r] = row[r - 1];  // the newest first
      row[0] = n - 1 - static_cast<int>(worst & 0xffffffffu);
    }
    // Every weight and position has been read.  The last `drop` rows: those of them
    // that stay fill the places of the rows that go in front of them, in order.
    auto goes = [&](int i) {
      bool y = false;
#pragma unroll
      for (int r = 0; r < kFew; ++r) y |= i == row[r];
      return y;
    };
    for (int i = tid; i < left; i += THREADS) {
      if (goes(i)) continue;
      src[i] = i;
      if (acc_out != acc) acc_out[i] = acc[i];
      if (pos_out != pos) pos_out[i] = pos[i];
    }
    if (tid < drop) {
      const int i = left + tid;
      int rank = 0;  // of this row among those to move
      for (int x = left; x < i; ++x) rank += !goes(x);
      if (!goes(i)) {
        int to = -1;  // the place of that rank, in ascending order
#pragma unroll
        for (int r = 0; r < kFew; ++r) {
          int lower = 0;
#pragma unroll
          for (int x = 0; x < kFew; ++x) lower += row[x] >= 0 && row[x] < row[r];
          if (row[r] >= 0 && row[r] < left && lower == rank) to = row[r];
        }
        ws[4 + 2 * rank] = to;
        ws[5 + 2 * rank] = i;
        src[to] = i;
        acc_out[to] = acc[i];
        pos_out[to] = pos[i];
        ++rank;
      }
      if (i == n - 1) ws[0] = rank;
    }
    return;
  }
  // `low` and `want`: the rows of a larger key stay, and of those equal to it the
  // first `want` (all of them: exact = false).
  uint32_t low = 0;
  int want = 0;
  bool exact = true;
  uint32_t keep = ~0u;  // the bits that are compared
  {
    // radix selection of the left-th largest key, 8 bits at a time until all keys of
    // the digit stay; below, keys are compared in the bits that were decided
    uint32_t mask = 0;
    int count = n;
    want = left;
    for (int i = tid; i < 256; i += THREADS) hist[0][i] = 0;
    __syncthreads();
    for (int shift = 24, turn = 0; shift >= 0; shift -= 8, turn ^= 1) {
      each([&](int, int i, uint32_t k) {
        if (i < n && (k & mask) == low) atomicAdd(&hist[turn][(k >> shift) & 255u], 1);
      });
      for (int i = tid; i < 256; i += THREADS) hist[turn ^ 1][i] = 0;
      __syncthreads();
      // lane l of every warp looks at the bins 255 - 8l .. 248 - 8l: how many keys lie above
      const int4 x = reinterpret_cast<const int4*>(hist[turn])[63 - 2 * lane];
      const int4 y = reinterpret_cast<const int4*>(hist[turn])[62 - 2 * lane];
      const int c[8] = {x.w, x.z, x.y, x.x, y.w, y.z, y.y, y.x};
      int sum = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += c[e];
      int before = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += t;
      }
      before -= sum;
      const int l = __ffs(__ballot_sync(0xffffffffu, before < want && before + sum >= want)) - 1;
      int bin = 0, rest = 0, size = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (before < want && before + c[e] >= want) {
          bin = 255 - 8 * lane - e;
          rest = want - before;
          size = c[e];
        }
        before += c[e];
      }
      low |= static_cast<uint32_t>(__shfl_sync(0xffffffffu, bin, l)) << shift;
      mask |= 255u << shift;
      want = __shfl_sync(0xffffffffu, rest, l);
      count = __shfl_sync(0xffffffffu, size, l);
      if (want == count) break;
      __syncthreads();  // this histogram is zeroed in the next pass
    }
    exact = want < count;
    keep = mask;
  }
  const uint32_t lower = (1u << lane) - 1u;
  int ties = 0;
  if (exact) {
    each([&](int, int i, uint32_t k) { ties += __popc(__ballot_sync(0xffffffffu, i < n && (k & keep) == low)); });
    ties = warps_before<THREADS>(make_int2(ties, 0), red2[0]).x;
  }
  int2 moves = make_int2(0, 0);  // below the new length the places to fill, behind it the rows to move
  auto below = [&](int w) {      // rows of the word below the new length
    const int cut = left - 32 * w;
    return cut >= 32 ? 0xffffffffu : cut <= 0 ? 0u : (1u << cut) - 1u;
  };
  each([&](int w, int i, uint32_t k) {
    k &= keep;
    const uint32_t tie = __ballot_sync(0xffffffffu, i < n && k == low);
    const bool stays = i < n && (k > low || (k == low && (!exact || ties + __popc(tie & lower) < want)));
    ties += __popc(tie);
    const uint32_t m = __ballot_sync(0xffffffffu, stays);
    if (lane == 0) bits[w] = m;
    moves.x += __popc(~m & below(w));
    moves.y += __popc(m & ~below(w));
  });
  int2 at = warps_before<THREADS>(moves, red2[1]);
  if (tid == THREADS - 1) ws[0] = at.x + moves.x;
#pragma unroll 4
  for (int w = w0; w < w1; ++w) {
    const uint32_t holes = ~bits[w] & below(w);
    if (holes >> lane & 1u) ws[4 + 2 * (at.x + __popc(holes & lower))] = 32 * w + lane;
    at.x += __popc(holes);
  }
  __syncthreads();  // the holes come before the rows that fill them
  const bool copy_acc = acc_out != acc, copy_pos = pos_out != pos;
  constexpr int E = 4;  // words whose loads are in flight together
#pragma unroll 1
  for (int v = w0; v < w1; v += E) {
    int to[E], slot[E], x[E];
    float a[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int w = v + e, i = 32 * w + lane;
      to[e] = slot[e] = -1;
      if (w >= w1) continue;
      const uint32_t m = bits[w], movers = m & ~below(w);
      if (m >> lane & 1u) {
        const bool moves = movers >> lane & 1u;
        to[e] = i;
        if (moves) {
          slot[e] = 4 + 2 * (at.y + __popc(movers & lower));
          to[e] = ws[slot[e]];
        }
        if (moves || copy_acc) a[e] = acc[i];
        if (moves || copy_pos) x[e] = pos[i];
      }
      at.y += __popc(movers);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i = 32 * (v + e) + lane;
      if (to[e] < 0) continue;
      src[to[e]] = i;
      if (slot[e] >= 0) ws[slot[e] + 1] = i;
      if (slot[e] >= 0 || copy_acc) acc_out[to[e]] = a[e];
      if (slot[e] >= 0 || copy_pos) pos_out[to[e]] = x[e];
    }
  }
}

constexpr int kMoveThreads = 256;

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p, int blocks) {
  ds::wait_for_previous();
  const int bh = blockIdx.x / blocks, part = blockIdx.x % blocks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int* ws = p.ws + static_cast<size_t>(bh) * evict_stride(p.cap, p.budget);
  const int kp = p.m / 8, vp = p.dv / 8;  // 16-byte pieces of a row
  uint4* kc = reinterpret_cast<uint4*>(p.kc) + static_cast<size_t>(bh) * p.cap * kp;
  uint4* v = reinterpret_cast<uint4*>(p.v) + static_cast<size_t>(bh) * p.cap * vp;
  float* mul = p.kc_mul + static_cast<size_t>(bh) * p.cap;
  const int stride = blocks * (kMoveThreads / 32);
  const int moves = ws[0];
  const int2* list = reinterpret_cast<const int2*>(ws + 4);  // destination, source
  int i = part * (kMoveThreads / 32) + warp;
  int2 next = i < moves ? list[i] : make_int2(0, 0);
  for (; i < moves; i += stride) {
    const size_t to = next.x, from = next.y;
    uint4 k, x;
    float f;
    if (lane < kp) k = kc[from * kp + lane];
    if (lane < vp) x = v[from * vp + lane];
    if (lane == 0) f = mul[from];
    if (i + stride < moves) next = list[i + stride];  // while the row is on its way
    if (lane < kp) kc[to * kp + lane] = k;
    if (lane < vp) v[to * vp + lane] = x;
    if (lane == 0) mul[to] = f;
  }
  // one thread per sequence reads its length and writes the new one
  if (part == 0 && bh % p.H == 0 && threadIdx.x == 0) {
    const int b = bh / p.H;
    p.lens_out[b] = min(min(max(p.lens[b], 0), p.cap), p.budget);
  }
}

template <int THREADS, Keys KEYS>
cudaError_t launch_select(const EvictParams& p, cudaStream_t stream) {
  const long long words = (p.cap + 31LL) / 32;
  const int smem = static_cast<int>(4 * (KEYS == kShared ? 33 * words : words));
  if constexpr (KEYS != kRegisters) {
    // the longest cache's for every call: 48 KB without asking count the static part in
    static std::atomic<uint64_t> done{0};
    constexpr int most = KEYS == kShared ? 4 * 33 * ((kSharedRows + 31) / 32) : kEvictMaxRows / 8;
    const cudaError_t e = ds::allow_smem(evict_select_kernel<THREADS, KEYS>, most, done);
    if (e != cudaSuccess) return e;
  }
  evict_select_kernel<THREADS, KEYS><<<p.B * p.H, THREADS, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream) {
  // the smallest CTA whose registers hold the keys; longer caches in shared memory
  // (up to 200 KB), the longest from memory in every pass
  cudaError_t e = p.cap <= 256 * kRegKeys    ? launch_select<256, kRegisters>(p, stream)
                  : p.cap <= 512 * kRegKeys  ? launch_select<512, kRegisters>(p, stream)
                  : p.cap <= 1024 * kRegKeys ? launch_select<1024, kRegisters>(p, stream)
                  : p.cap <= kSharedRows     ? launch_select<1024, kShared>(p, stream)
                                             : launch_select<1024, kNowhere>(p, stream);
  if (e != cudaSuccess) return e;
  const int blocks = (152 * 16 + p.B * p.H - 1) / (p.B * p.H);
  return ds::launch_after(evict_move_kernel, static_cast<unsigned>(p.B * p.H * blocks), kMoveThreads, 0, stream, p, blocks);
}

}  // namespace spa
