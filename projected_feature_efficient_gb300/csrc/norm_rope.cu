// norm_rope.cu -- norms of queries and keys for each head with the rotary positions in
// the same pass, and the gradient.
//
// A row x of d features, weights w [d] of its tensor:
//   r = (mean_i x_i^2 + eps)^(-1/2),   y = R(pos) (w * x r)
// with R as in rope.cu (pairs turned by pos * f_i, features from rot on passed through).
// With the upstream gradient u of y, h = R^T u and t = w * h:
//   dx = r t - x r^3 (sum_i t_i x_i) / d,     dw = sum over rows of h * x r
// The gradient reads x again instead of keeping r: the row is needed for dx anyway.
//
// Bound by memory: every row is read and written once (forward 2, gradient 3 rows' bytes).
// A group of neighbouring lanes holds a row, a lane the same features of every row that it
// sees, so that sines, weights and the sums of dw stay in its registers, and a row's sums
// take a few shuffles.  2 x 8192 tokens of 20 heads, d = 128, bf16: 168 MB, 31 us (5.4 TB/s,
// 25 us at the rate of a copy); the gradient of 4 x 8192: 503 MB, 106 us and 7 for the sums of
// dw (4.8 TB/s; 75 us); 8191 tokens of 16 heads of 96 in fp32: 101 MB, 25 us a call (15 us).  What is left is the instructions: they issue in 59% and 54% of the
// cycles, and 107 registers of the gradient leave room for two blocks per SM.
#include "decode_shared.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "rope.cuh"

namespace spa {
namespace {

constexpr int kThreads = 256;
template <int UPL, bool INTER>
constexpr int kFwdBlocks = UPL > 1 ? 1 : INTER ? 4 : 3;  // blocks per SM that the registers are to leave room for
template <int UPL, bool INTER>
constexpr int kBwdBlocks = UPL > 1 ? 1 : 2;
constexpr int kMaxVec = 16;  // features of a thread at most: UPL * (V, or 2 V of the two halves)
// the gradient's vectors in the half layout: it holds twice the values (8: 142 us for 129 at the time, 4 x 8192 tokens)
constexpr int kMaxHalfVec = 4;

// V features of a row as they lie in memory, in whole registers: a load under a condition
// then writes nothing but its registers and is waited for where the values are used.
// (Held as single bf16 values they were taken apart behind each load, one after the other:
// the gradient of 4 x 8192 rows of 20 heads took 217 us.)  LOOSE: a feature at a time.
template <class T, int V, bool LOOSE>
struct Raw {
  static constexpr bool kPairs = sizeof(T) == 2 && V > 1 && !LOOSE;  // two bf16 values a word
  static constexpr int kWords = kPairs ? V / 2 : V;
  uint32_t w[kWords];

  __device__ __forceinline__ static uint32_t bits(const T* x) {
    if constexpr (sizeof(T) == 4) return *reinterpret_cast<const uint32_t*>(x);
    else return *reinterpret_cast<const uint16_t*>(x);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  __device__ __forceinline__ void load(const T* x, int left) {  // LOOSE: of `left` features
    if constexpr (LOOSE) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < left) w[i] = bits(x + i);
    } else if constexpr (kWords == 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(x);
      w[0] = v.x;
      w[1] = v.y;
      w[2] = v.z;
      w[3] = v.w;
    } else if constexpr (kWords == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(x);
      w[0] = v.x;
      w[1] = v.y;
    } else {
      w[0] = kPairs ? *reinterpret_cast<const uint32_t*>(x) : bits(x);
    }
  }
  __device__ __forceinline__ void store(T* x, int left) const {
    if constexpr (LOOSE) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < left) put(x + i, w[i]);
    } else if constexpr (kWords == 4) {
      *reinterpret_cast<uint4*>(x) = make_uint4(w[0], w[1], w[2], w[3]);
    } else if constexpr (kWords == 2) {
      *reinterpret_cast<uint2*>(x) = make_uint2(w[0], w[1]);
    } else if constexpr (kPairs) {
      *reinterpret_cast<uint32_t*>(x) = w[0];
    } else {
      put(x, w[0]);
    }
  }
  __device__ __forceinline__ static void put(T* x, uint32_t v) {
    if constexpr (sizeof(T) == 4) *reinterpret_cast<uint32_t*>(x) = v;
    else *reinterpret_cast<uint16_t*>(x) = static_cast<uint16_t>(v);
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else if constexpr (kPairs) return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    else return __uint_as_float(w[i] << 16);
  }
  // features i and i + 1 (V = 1: feature i alone)
  __device__ __forceinline__ void set2(int i, float x, float y) {
    if constexpr (sizeof(T) == 4) {
      w[i] = __float_as_uint(x);
      if (V > 1) w[V > 1 ? i + 1 : i] = __float_as_uint(y);
    } else if constexpr (kPairs) {
      w[i / 2] = ptx::pack_bf16x2(x, y);
    } else {
      w[i] = __bfloat16_as_ushort(__float2bfloat16_rn(x));
      if (V > 1) w[V > 1 ? i + 1 : i] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
    }
  }
};

// What a thread holds of a row: UPL units, each V neighbouring features (interleaved
// pairs), or V of each half of the turned features, or of the others (which are turned by
// nothing; the first half of an odd number of those is one longer).
template <class T, int V, bool INTER, int UPL, bool LOOSE>
struct Row {
  using W = Raw<T, V, LOOSE>;
  static constexpr int kPairs = INTER ? V / 2 : V;
  W a[UPL], b[INTER ? 1 : UPL];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < UPL; ++j) {
      a[j].clear();
      if constexpr (!INTER) b[j].clear();
    }
  }
  __device__ __forceinline__ void put(const float (&x)[UPL][kPairs], const float (&y)[UPL][kPairs]) {
#pragma unroll
    for (int j = 0; j < UPL; ++j) {
      if constexpr (INTER) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) a[j].set2(2 * i, x[j][i], y[j][i]);
      } else {
#pragma unroll
        for (int i = 0; i < kPairs; i += 2) {
          const int k = kPairs > 1 ? i + 1 : i;
          a[j].set2(i, x[j][i], x[j][k]);
          b[j].set2(i, y[j][i], y[j][k]);
        }
      }
    }
  }
  // pairs 2 i and 2 i + 1 of unit j
  __device__ __forceinline__ uint64_t a2(int j, int i) const {
    return ptx::pack_f32x2(pa(j, 2 * i), 2 * i + 1 < kPairs ? pa(j, 2 * i + 1 < kPairs ? 2 * i + 1 : 0) : 0.f);
  }
  __device__ __forceinline__ uint64_t b2(int j, int i) const {
    return ptx::pack_f32x2(pb(j, 2 * i), 2 * i + 1 < kPairs ? pb(j, 2 * i + 1 < kPairs ? 2 * i + 1 : 0) : 0.f);
  }
  // pair i of unit j
  __device__ __forceinline__ float pa(int j, int i) const { return a[j].get(INTER ? 2 * i : i); }
  __device__ __forceinline__ float pb(int j, int i) const {
    if constexpr (INTER) return a[j].get(2 * i + 1);
    else return b[j].get(i);
  }
};

// Two pairs' values in one register pair: Blackwell multiplies and adds two fp32 values per
// instruction, and the kernels below are bound by their instructions before memory.
template <int UPL, int PR>
struct Twos {
  static constexpr int N = (PR + 1) / 2;
  uint64_t v[UPL][N];

  __device__ __forceinline__ void set(const float (&x)[UPL][PR]) {
#pragma unroll
    for (int j = 0; j < UPL; ++j)
#pragma unroll
      for (int i = 0; i < N; ++i) v[j][i] = ptx::pack_f32x2(x[j][2 * i], 2 * i + 1 < PR ? x[j][2 * i + 1 < PR ? 2 * i + 1 : 0] : 0.f);
  }
  __device__ __forceinline__ void get(float (&x)[UPL][PR]) const {
#pragma unroll
    for (int j = 0; j < UPL; ++j)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float hi;
        ptx::unpack_f32x2(v[j][i], x[j][2 * i], hi);
        if (2 * i + 1 < PR) x[j][2 * i + 1 < PR ? 2 * i + 1 : 0] = hi;
      }
  }
};
__device__ __forceinline__ uint64_t both_of(float x) { return ptx::pack_f32x2(x, x); }
__device__ __forceinline__ float sum_of(uint64_t x) {
  float a, b;
  ptx::unpack_f32x2(x, a, b);
  return a + b;
}

// Where the units of a thread lie.  EXACT: every lane has all of its units, with both
// halves.
template <class T, int V, bool INTER, int UPL, bool LOOSE, bool EXACT>
struct Place {
  using R = Row<T, V, INTER, UPL, LOOSE>;
  int at[UPL], half[UPL];  // first feature, distance of the second half
  int d;
  unsigned have, both;     // bit j: unit j lies in the row; it has a second half

  __device__ __forceinline__ Place(int lane, int lanes, int units, int turning, int rot, int d_) : d(d_) {
    have = both = 0;
#pragma unroll
    for (int j = 0; j < UPL; ++j) {
      const int u = lane + j * lanes;
      const bool turns = INTER || u < turning;
      at[j] = turns ? u * V : rot + (u - turning) * V;
      half[j] = turns ? rot / 2 : (d - rot + 1) / 2;
      if (u < units) have |= 1u << j;
      if (!INTER && u < units && at[j] + half[j] < d) both |= 1u << j;
    }
  }
  __device__ __forceinline__ bool has(int j) const { return EXACT || (have >> j & 1); }
  __device__ __forceinline__ bool has_both(int j) const { return EXACT || (both >> j & 1); }
  __device__ __forceinline__ void read(const T* x, R& row) const {
#pragma unroll
    for (int j = 0; j < UPL; ++j) {
      if (has(j)) row.a[j].load(x + at[j], d - at[j]);
      if constexpr (!INTER)
        if (has_both(j)) row.b[j].load(x + at[j] + half[j], V);
    }
  }
  __device__ __forceinline__ void write(T* y, const R& row) const {
#pragma unroll
    for (int j = 0; j < UPL; ++j) {
      if (has(j)) row.a[j].store(y + at[j], d - at[j]);
      if constexpr (!INTER)
        if (has_both(j)) row.b[j].store(y + at[j] + half[j], V);
    }
  }
  // f(j, i, index of the pair's first feature, of its second one or -1)
  template <class F>
  __device__ __forceinline__ void pairs(F f) const {
#pragma unroll
    for (int j = 0; j < UPL; ++j)
#pragma unroll
      for (int i = 0; i < R::kPairs; ++i) {
        if constexpr (INTER) {
          const int k = at[j] + 2 * i;
          f(j, i, has(j) ? k : -1, has(j) && (!LOOSE || k + 1 < d) ? k + 1 : -1);
        } else {
          const int k = at[j] + i;
          f(j, i, has(j) ? k : -1, has_both(j) ? k + half[j] : -1);
        }
      }
  }
};

// A group takes items of `per` neighbouring heads of a token; the first `first` blocks take
// tensor 0.
struct Side {
  uint32_t per, chunks;  // heads of an item, items of a token
};
struct Items {
  Side side[2];
  uint32_t first;
};

// Sums over the lanes of a row.
template <int E>
__device__ __forceinline__ void over_lanes(float (&x)[E], int lanes) {
#pragma unroll
  for (int o = 16; o; o >>= 1)
    if (o < lanes) {
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] += __shfl_xor_sync(0xffffffffu, x[e], o);
    }
}

template <class T, int V, bool INTER, int UPL, bool LOOSE, bool EXACT>
__device__ __forceinline__ void angles(const NormRopeParams& p, const Place<T, V, INTER, UPL, LOOSE, EXACT>& pl, int b, int n,
                                       float (&s)[UPL][Row<T, V, INTER, UPL, LOOSE>::kPairs],
                                       float (&c)[UPL][Row<T, V, INTER, UPL, LOOSE>::kPairs]) {
  const int pos = p.rot == 0 || b >= p.B ? 0 : p.pos ? p.pos[static_cast<long long>(b) * p.N + n] : p.pos0 + n;
  pl.pairs([&](int j, int i, int ka, int) {
    const int pair = INTER ? ka / 2 : ka;
    s[j][i] = 0.f;
    c[j][i] = 1.f;
    if (ka >= 0 && ka < p.rot && (INTER || ka < p.rot / 2)) sincos_of(p.table[pair], pos, s[j][i], c[j][i]);
  });
}

// E rows at a time, their loads in flight together.  Rows behind the item's last one are
// computed with what the registers hold and dropped: no lane leaves the shuffles.
template <class T, int V, bool INTER, int UPL, bool LOOSE, bool EXACT, int E>
__global__ void __launch_bounds__(kThreads, kFwdBlocks<UPL, INTER>) norm_rope_kernel(const NormRopeParams p, const Items items,
                                                                                    int lanes, int units, int turning) {
  using R = Row<T, V, INTER, UPL, LOOSE>;
  constexpr int PR = R::kPairs;
  const int t = blockIdx.x >= items.first;
  const Side it = t ? items.side[1] : items.side[0];
  const uint32_t item = (blockIdx.x - (t ? items.first : 0u)) * (kThreads / lanes) + threadIdx.x / lanes;
  const Place<T, V, INTER, UPL, LOOSE, EXACT> pl(threadIdx.x & (lanes - 1), lanes, units, turning, p.rot, p.d);
  const uint32_t tokens = static_cast<uint32_t>(p.B) * p.N, chunk = item / tokens, token = item - chunk * tokens;
  const uint32_t h0 = chunk * it.per;
  const int b = token / p.N, n = token - b * p.N;
  const int rows = chunk < it.chunks ? min(static_cast<int>(it.per), p.H[t] - static_cast<int>(h0)) : 0;
  const long long xs = p.xs[t][1], ys = p.ys[t][1];
  const T* x = static_cast<const T*>(p.x[t]) + b * p.xs[t][0] + n * p.xs[t][2] + h0 * xs;
  T* y = static_cast<T*>(p.y[t]) + b * p.ys[t][0] + n * p.ys[t][2] + h0 * ys;
  R row[E];
  // Places that no load fills hold what the row before left there, where a NaN is one in every
  // place: they are 0 again before each row, or the next row's sum would take them in.
  auto fetch = [&](int left) {
    if constexpr (!EXACT) {
#pragma unroll
      for (int e = 0; e < E; ++e) row[e].clear();
    }
    if (left >= E) {
#pragma unroll
      for (int e = 0; e < E; ++e, x += xs) pl.read(x, row[e]);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e, x += xs)
        if (e < left) pl.read(x, row[e]);
    }
  };
#pragma unroll
  for (int e = 0; e < E; ++e) row[e].clear();
  fetch(rows);
  // y_a = r (a ca - b sb), y_b = r (a sa + b cb): weights and turn in one
  using D = Twos<UPL, PR>;
  D ca, sa, cb, sb;  // sb negated
  {
    float s[UPL][PR], c[UPL][PR], x0[UPL][PR], x1[UPL][PR], x2[UPL][PR], x3[UPL][PR];
    angles(p, pl, b, n, s, c);
    const T* w = static_cast<const T*>(p.w[t]);
    pl.pairs([&](int j, int i, int ka, int kb) {
      const float wa = ka < 0 ? 0.f : w ? up(w[ka]) : 1.f, wb = kb < 0 ? 0.f : w ? up(w[kb]) : 1.f;
      x0[j][i] = wa * c[j][i];
      x1[j][i] = wa * s[j][i];
      x2[j][i] = wb * c[j][i];
      x3[j][i] = -wb * s[j][i];
    });
    ca.set(x0);
    sa.set(x1);
    cb.set(x2);
    sb.set(x3);
  }
  const float mean = 1.f / p.d;
  for (int left = rows, k = it.per;;) {
    float sum[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      uint64_t q = 0;
#pragma unroll
      for (int j = 0; j < UPL; ++j)
#pragma unroll
        for (int i = 0; i < D::N; ++i) {
          const uint64_t a = row[e].a2(j, i), bb = row[e].b2(j, i);
          q = ptx::fma_f32x2(a, a, ptx::fma_f32x2(bb, bb, q));
        }
      sum[e] = sum_of(q);
    }
    over_lanes(sum, lanes);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const uint64_t r = both_of(rsqrtf(fmaf(sum[e], mean, p.eps)));
      D ya, yb;
#pragma unroll
      for (int j = 0; j < UPL; ++j)
#pragma unroll
        for (int i = 0; i < D::N; ++i) {
          const uint64_t a = ptx::mul_f32x2(row[e].a2(j, i), r), bb = ptx::mul_f32x2(row[e].b2(j, i), r);
          ya.v[j][i] = ptx::fma_f32x2(bb, sb.v[j][i], ptx::mul_f32x2(a, ca.v[j][i]));
          yb.v[j][i] = ptx::fma_f32x2(a, sa.v[j][i], ptx::mul_f32x2(bb, cb.v[j][i]));
        }
      float fa[UPL][PR], fb[UPL][PR];
      ya.get(fa);
      yb.get(fb);
      row[e].put(fa, fb);
    }
    if (left >= E) {
#pragma unroll
      for (int e = 0; e < E; ++e, y += ys) pl.write(y, row[e]);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e, y += ys)
        if (e < left) pl.write(y, row[e]);
    }
    left -= E;
    k -= E;
    if (k <= 0) break;
    fetch(left);
  }
}

template <class T, int V, bool INTER, int UPL, bool LOOSE, bool EXACT, int E>
__global__ void __launch_bounds__(kThreads, kBwdBlocks<UPL, INTER>) norm_rope_bwd_kernel(const NormRopeParams p,
                                                                                        const Items items, int lanes,
                                                                                        int units, int turning) {
  using R = Row<T, V, INTER, UPL, LOOSE>;
  constexpr int PR = R::kPairs;
  const int t = blockIdx.x >= items.first;
  const Side it = t ? items.side[1] : items.side[0];
  const uint32_t groups = kThreads / lanes, blocks = t ? gridDim.x - items.first : items.first;
  const uint32_t tokens = static_cast<uint32_t>(p.B) * p.N, count = tokens * it.chunks;
  const Place<T, V, INTER, UPL, LOOSE, EXACT> pl(threadIdx.x & (lanes - 1), lanes, units, turning, p.rot, p.d);
  const long long xs = p.xs[t][1], gs = p.gs[t][1], ys = p.ys[t][1];
  const float mean = 1.f / p.d;
  using D = Twos<UPL, PR>;
  D wa, wb, da, db;
  {
    float x[UPL][PR], z[UPL][PR];
    const T* w = static_cast<const T*>(p.w[t]);
    pl.pairs([&](int j, int i, int ka, int kb) {
      x[j][i] = ka < 0 ? 0.f : w ? up(w[ka]) : 1.f;
      z[j][i] = kb < 0 ? 0.f : w ? up(w[kb]) : 1.f;
    });
    wa.set(x);
    wb.set(z);
    pl.pairs([&](int j, int i, int, int) { x[j][i] = 0.f; });
    da.set(x);
    db.set(x);
  }
  // The rows that are computed, and the next ones, in flight meanwhile, across items too.
  R row[E], gr[E], row1[E], gr1[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    row1[e].clear();
    gr1[e].clear();
  }
  struct At {
    int b, n, rows;
    const T *x, *g;
    T* y;
  };
  auto place = [&](uint32_t item) {
    At at;
    const uint32_t chunk = item / tokens, token = item - chunk * tokens, h0 = chunk * it.per;
    at.b = token / p.N;
    at.n = token - at.b * p.N;
    at.rows = item < count ? min(static_cast<int>(it.per), p.H[t] - static_cast<int>(h0)) : 0;
    at.x = static_cast<const T*>(p.x[t]) + at.b * p.xs[t][0] + at.n * p.xs[t][2] + h0 * xs;
    at.g = static_cast<const T*>(p.g[t]) + at.b * p.gs[t][0] + at.n * p.gs[t][2] + h0 * gs;
    at.y = static_cast<T*>(p.y[t]) + at.b * p.ys[t][0] + at.n * p.ys[t][2] + h0 * ys;
    return at;
  };
  auto fetch = [&](At& at, int left) {
    if (left >= E) {
#pragma unroll
      for (int e = 0; e < E; ++e, at.x += xs, at.g += gs) {
        pl.read(at.x, row1[e]);
        pl.read(at.g, gr1[e]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e, at.x += xs, at.g += gs)
        if (e < left) {
          pl.read(at.x, row1[e]);
          pl.read(at.g, gr1[e]);
        }
    }
  };
  // all groups of a warp run as many rounds: the shuffles are whole warps'
  const uint32_t first = (blockIdx.x - (t ? items.first : 0u)) * groups, group = threadIdx.x / lanes;
  At ahead = place(first + group);
  fetch(ahead, ahead.rows);
  for (uint32_t i0 = first; i0 < count; i0 += blocks * groups) {
    At at = ahead;
    D s, m, c;  // sine, its negative, cosine
    {
      float x[UPL][PR], z[UPL][PR];
      angles(p, pl, at.rows ? at.b : p.B, at.n, x, z);
      s.set(x);
      c.set(z);
      pl.pairs([&](int j, int i, int, int) { x[j][i] = -x[j][i]; });
      m.set(x);
    }
    for (int left = at.rows, k = it.per; k > 0; left -= E, k -= E) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        row[e] = row1[e];
        gr[e] = gr1[e];
      }
      if (k > E) {
        fetch(ahead, left - E);
      } else if (i0 + blocks * groups < count) {
        ahead = place(i0 + blocks * groups + group);
        fetch(ahead, ahead.rows);
      }
      float sum[2 * E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        uint64_t q = 0, d = 0;
#pragma unroll
        for (int j = 0; j < UPL; ++j)
#pragma unroll
          for (int i = 0; i < D::N; ++i) {
            const uint64_t a = row[e].a2(j, i), bb = row[e].b2(j, i), ga = gr[e].a2(j, i), gb = gr[e].b2(j, i);
            const uint64_t ha = ptx::fma_f32x2(gb, s.v[j][i], ptx::mul_f32x2(ga, c.v[j][i]));
            const uint64_t hb = ptx::fma_f32x2(ga, m.v[j][i], ptx::mul_f32x2(gb, c.v[j][i]));
            q = ptx::fma_f32x2(a, a, ptx::fma_f32x2(bb, bb, q));
            d = ptx::fma_f32x2(ptx::mul_f32x2(wa.v[j][i], a), ha, ptx::fma_f32x2(ptx::mul_f32x2(wb.v[j][i], bb), hb, d));
          }
        sum[2 * e] = sum_of(q);
        sum[2 * e + 1] = sum_of(d);
      }
      over_lanes(sum, lanes);
      R z[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        // a row that is not there adds nothing
        const float rr = e < left ? rsqrtf(fmaf(sum[2 * e], mean, p.eps)) : 0.f;
        const uint64_t r = both_of(rr), f = both_of(-rr * rr * (sum[2 * e + 1] * mean));
        D ya, yb;
#pragma unroll
        for (int j = 0; j < UPL; ++j)
#pragma unroll
          for (int i = 0; i < D::N; ++i) {
            const uint64_t a = ptx::mul_f32x2(row[e].a2(j, i), r), bb = ptx::mul_f32x2(row[e].b2(j, i), r);
            const uint64_t ga = gr[e].a2(j, i), gb = gr[e].b2(j, i);
            const uint64_t ha = ptx::fma_f32x2(gb, s.v[j][i], ptx::mul_f32x2(ga, c.v[j][i]));
            const uint64_t hb = ptx::fma_f32x2(ga, m.v[j][i], ptx::mul_f32x2(gb, c.v[j][i]));
            da.v[j][i] = ptx::fma_f32x2(ha, a, da.v[j][i]);
            db.v[j][i] = ptx::fma_f32x2(hb, bb, db.v[j][i]);
            ya.v[j][i] = ptx::fma_f32x2(ptx::mul_f32x2(wa.v[j][i], ha), r, ptx::mul_f32x2(a, f));
            yb.v[j][i] = ptx::fma_f32x2(ptx::mul_f32x2(wb.v[j][i], hb), r, ptx::mul_f32x2(bb, f));
          }
        float fa[UPL][PR], fb[UPL][PR];
        ya.get(fa);
        yb.get(fb);
        z[e].put(fa, fb);
      }
      if (left >= E) {
#pragma unroll
        for (int e = 0; e < E; ++e, at.y += ys) pl.write(at.y, z[e]);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e, at.y += ys)
          if (e < left) pl.write(at.y, z[e]);
      }
    }
  }
  ds::let_next_start();
  if (!p.dw[t]) return;
  // the block's sums of dw: a group after the other, always in the same order
  __shared__ float part[kThreads * kMaxVec];
  float fa[UPL][PR], fb[UPL][PR];
  da.get(fa);
  db.get(fb);
  pl.pairs([&](int j, int i, int ka, int kb) {
    float* to = part + threadIdx.x / lanes * p.d;
    if (ka >= 0) to[ka] = fa[j][i];
    if (kb >= 0) to[kb] = fb[j][i];
  });
  __syncthreads();
  for (int k = threadIdx.x; k < p.d; k += kThreads) {
    float sum = 0.f;
    for (uint32_t q = 0; q < groups; ++q) sum += part[q * p.d + k];
    p.part[static_cast<size_t>(blockIdx.x) * p.d + k] = sum;
  }
}

// dw from the blocks' sums: a warp per feature, always in the same order.
__global__ void __launch_bounds__(kThreads) norm_rope_sum_kernel(const NormRopeParams p, unsigned first, unsigned all,
                                                                 unsigned per_tensor) {
  const int t = blockIdx.x >= per_tensor, lane = threadIdx.x & 31;
  const int k = (blockIdx.x - t * per_tensor) * (kThreads / 32) + threadIdx.x / 32;
  ds::wait_for_previous();
  if (k >= p.d || !p.dw[t]) return;
  const unsigned from = t ? first : 0, to = t ? all : first;
  float sum = 0.f;
  constexpr int kAhead = 10;  // in flight
  for (unsigned i = from + lane; i < to; i += 32 * kAhead) {
    float x[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) x[u] = i + 32 * u < to ? p.part[static_cast<size_t>(i + 32 * u) * p.d + k] : 0.f;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) sum += x[u];
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) p.dw[t][k] = sum;
}

template <bool INTER>
int units_of(const NormRopeParams& p, int v) {
  return INTER ? (p.d + v - 1) / v : p.rot / 2 / v + ((p.d - p.rot + 1) / 2 + v - 1) / v;
}

template <class T, int V, bool INTER, int UPL, bool LOOSE = false, bool EXACT = false>
cudaError_t launch(const NormRopeParams& p, cudaStream_t stream) {
  const int turning = INTER ? 0 : p.rot / 2 / V;
  const int units = units_of<INTER>(p, V);
  int lanes = 1;
  while (lanes < 32 && lanes < units) lanes *= 2;
  static_assert(UPL * V * (INTER ? 1 : 2) <= kMaxVec, "features of a thread");
  const long long tokens = static_cast<long long>(p.B) * p.N;
  const int groups = kThreads / lanes;
  // rows in flight: as many as the registers hold (halves of 8 bf16: four rows 88 us, two 66, for 4 x 8192 tokens)
  constexpr int E = UPL > 1 ? 1 : INTER || V < 8 ? 4 : 2, EB = UPL == 1 ? 2 : 1;
  const bool gradient = p.g[0] || p.g[1];
  const long long most = kNormRopeBlocks, heads = p.H[0] + p.H[1];
  Items it{};
  long long blocks[2] = {0, 0};
  for (int t = 0; t < 2; ++t) {
    if (!p.H[t]) continue;
    // heads that share a thread's sines: up to 8, fewer where that leaves SMs without threads
    int per = p.H[t] < 8 ? p.H[t] : 8;
    while (per > 1 && tokens * lanes * ((p.H[t] + per - 1) / per) < 152LL * 1024) per = (per + 1) / 2;
    it.side[t].per = per;
    it.side[t].chunks = (p.H[t] + per - 1) / per;
    blocks[t] = (tokens * it.side[t].chunks + groups - 1) / groups;
    // two rounds of the two per SM that run at once, shared out by the tensors' heads (one round: 118 us for 116, 4 x
    // 8192 tokens)
    if (gradient) {
      const long long share = most * p.H[t] / heads > 0 ? most * p.H[t] / heads : 1;
      if (blocks[t] > share) blocks[t] = share;
    }
  }
  it.first = static_cast<uint32_t>(blocks[0]);
  const unsigned all = static_cast<unsigned>(blocks[0] + blocks[1]);
  if (!gradient) {
    if (UPL == 1 && it.side[0].per <= 1 && it.side[1].per <= 1) {
      norm_rope_kernel<T, V, INTER, UPL, LOOSE, EXACT, 1><<<all, kThreads, 0, stream>>>(p, it, lanes, units, turning);
      return cudaGetLastError();
    }
    norm_rope_kernel<T, V, INTER, UPL, LOOSE, EXACT, E><<<all, kThreads, 0, stream>>>(p, it, lanes, units, turning);
    return cudaGetLastError();
  }
  if constexpr (!INTER && V > kMaxHalfVec) {  // launch_norm_rope starts at vectors of kMaxHalfVec
    return cudaErrorInvalidValue;
  } else {
    norm_rope_bwd_kernel<T, V, INTER, UPL, LOOSE, EXACT, EB><<<all, kThreads, 0, stream>>>(p, it, lanes, units, turning);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || (!p.dw[0] && !p.dw[1])) return e;
    const unsigned per_tensor = (p.d + kThreads / 32 - 1) / (kThreads / 32);
    return ds::launch_after(norm_rope_sum_kernel, 2 * per_tensor, kThreads, 0, stream, p, it.first, all, per_tensor);
  }
}

// d <= 256: with V features a vector a row has at most 256 / V units (INTER), or 128 / V.
// EXACT where a power of two of lanes holds the row without a place left over: no load or
// store under a condition, which cost the other form about half of its time.
template <class T, int V, bool INTER>
cudaError_t launch_exact(const NormRopeParams& p, cudaStream_t stream) {
  const int units = units_of<INTER>(p, V);
  if (units <= 32 && (units & (units - 1)) == 0) return launch<T, V, INTER, 1, false, true>(p, stream);
  if constexpr (INTER && V == 4)
    if (units > 32) return launch<T, V, INTER, 2>(p, stream);
  return launch<T, V, INTER, 1>(p, stream);
}
template <class T, bool INTER>
cudaError_t launch_v(const NormRopeParams& p, int v, cudaStream_t stream) {
  if constexpr (sizeof(T) == 2)
    if (v == 8) return launch_exact<T, 8, INTER>(p, stream);
  if (v >= 4) return launch_exact<T, 4, INTER>(p, stream);
  if constexpr (INTER) {
    if (v >= 2) return launch<T, 2, INTER, 4>(p, stream);
    return launch<T, 2, true, 4, true>(p, stream);
  } else {
    if (v >= 2) return launch<T, 2, INTER, 2>(p, stream);
    return launch<T, 1, false, 4>(p, stream);
  }
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, cudaStream_t stream) {
  const int size = p.bf16 ? 2 : 4;
  // the widest vector that every address allows: rows, halves and tail
  int v = (p.g[0] || p.g[1]) && !p.interleaved ? kMaxHalfVec : 16 / size;
  auto fits = [&](int w) {
    const uintptr_t bytes = static_cast<uintptr_t>(w) * size;
    if (p.d % w) return false;
    if (!p.interleaved && ((p.rot / 2) % w || (p.d - p.rot) % (2 * w))) return false;
    for (int t = 0; t < 2; ++t) {
      if (p.H[t] == 0) continue;
      if (reinterpret_cast<uintptr_t>(p.x[t]) % bytes || reinterpret_cast<uintptr_t>(p.y[t]) % bytes ||
          reinterpret_cast<uintptr_t>(p.g[t]) % bytes)
        return false;
      for (int i = 0; i < 3; ++i)
        if (p.xs[t][i] % w || p.ys[t][i] % w || p.gs[t][i] % w) return false;
    }
    return true;
  };
  while (v > 1 && !fits(v)) v /= 2;
  if (p.bf16) return p.interleaved ? launch_v<__nv_bfloat16, true>(p, v, stream)
                                   : launch_v<__nv_bfloat16, false>(p, v, stream);
  return p.interleaved ? launch_v<float, true>(p, v, stream) : launch_v<float, false>(p, v, stream);
}

}  // namespace spa
