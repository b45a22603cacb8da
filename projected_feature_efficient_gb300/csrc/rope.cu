// rope.cu -- rotary positions on queries and keys, forward and gradient.
//
// Feature pair i of a row at position n is turned by the angle n * f_i:
//   (a, b) -> scale * (a cos - b sin, a sin + b cos)
// with (a, b) = features (2i, 2i+1) (interleaved) or (i, i + rot/2) (halves);
// features from rot on pass through.  The map is orthogonal up to `scale`, so
// its gradient is the same map with the angle negated (inverse).
//
// The angle never goes through floating point before it is reduced: the table
// holds f_i / 2pi as a 64-bit fraction of a turn, and position * table wraps
// modulo one turn exactly in integer arithmetic.  Its top 48 bits, as a signed
// fraction, are the angle to within 2^-48 of a turn at any position (an fp32
// product is off by 2^-24 of the angle itself: 0.06 rad at position 10^6), so that
// sine and cosine are off by their fp32 arithmetic alone.
//
// Bound by memory: every feature is read and written once.  A thread owns the
// same vector of pairs in several heads of one token, so the sines are formed
// once per thread and used for each of them, four heads' loads in flight.
// 2 x 8192 rows of 20 heads of 128 bf16 features: 29 us, 5.7 TB/s (24.8 us at the
// measured 6.8 TB/s); 8191 rows of 16 heads of 96 fp32 features: 20.6 us a call, 4.9
// TB/s with the launch (the kernel 15.4 us).  With a head at a time and the pairs converted one by one the first took
// 45 us.
#include "kernels.cuh"
#include "rope.cuh"

namespace spa {
namespace {

constexpr int kThreads = 256;

template <class T, int V>
struct alignas(sizeof(T) * V) Vec {
  T e[V];
};

// Two neighbouring elements of a vector at a time: one conversion of a bf16 pair.
template <int V>
__device__ __forceinline__ void put2(Vec<float, V>& w, int i, float x, float y) {
  w.e[i] = x;
  if (V > 1) w.e[V > 1 ? i + 1 : i] = y;
}
template <int V>
__device__ __forceinline__ void put2(Vec<__nv_bfloat16, V>& w, int i, float x, float y) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
  w.e[i] = v.x;
  if (V > 1) w.e[V > 1 ? i + 1 : i] = v.y;
}

// A thread's unit of a row: V elements (V/2 pairs) of an interleaved row, or V
// elements of each half, or V elements of the tail.  LOOSE (interleaved, V = 2):
// odd widths and strides, one feature at a time.
template <class T, int V, bool INTER, bool LOOSE>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p, int units, int turning,
                                                        int per) {
  const long long id = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  const long long token = id / units;
  const int u = static_cast<int>(id - token * units);
  if (token >= static_cast<long long>(p.B) * p.N) return;
  const int b = static_cast<int>(token / p.N), n = static_cast<int>(token - static_cast<long long>(b) * p.N);
  const int heads = p.H[0] + p.H[1];
  const int h0 = blockIdx.y * per, h1 = min(heads, h0 + per);
  const bool turns = u < turning;
  constexpr int kPairs = INTER ? (V + 1) / 2 : V;
  float s[kPairs], c[kPairs];
  if (turns) {
    const int pos = p.pos ? p.pos[token] : p.pos0 + n;
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const int pair = INTER ? u * kPairs + i : u * V + i;
      if (pair < p.rot / 2) {
        sincos_of(p.table[pair], pos, s[i], c[i]);
        s[i] *= p.inverse ? -p.scale : p.scale;
        c[i] *= p.scale;
      } else {
        s[i] = 0.f;
        c[i] = 1.f;
      }
    }
  }
  const int half = p.rot / 2;
  // first element of the unit; the tail of the half layout starts at rot
  const int e0 = INTER ? u * V : turns ? u * V : p.rot + (u - turning) * V;
  using W = Vec<T, V>;
  constexpr int E = 4;  // heads in flight
  constexpr bool kTwo = !INTER;  // a vector of each half
  auto turn = [&](W& wa, W& wb) {
    if constexpr (INTER) {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        if (u * (V / 2) + i < half) {  // a vector may end in the tail: those features stay as they are
          const float a = up(wa.e[2 * i]), bb = up(wa.e[2 * i + 1]);
          put2(wa, 2 * i, a * c[i] - bb * s[i], a * s[i] + bb * c[i]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const int k = V > 1 ? i + 1 : i;
        const float a0 = up(wa.e[i]), b0 = up(wb.e[i]), a1 = up(wa.e[k]), b1 = up(wb.e[k]);
        put2(wa, i, a0 * c[i] - b0 * s[i], a1 * c[k] - b1 * s[k]);
        put2(wb, i, a0 * s[i] + b0 * c[i], a1 * s[k] + b1 * c[k]);
      }
    }
  };
  auto read = [&](const T* x, W& wa, W& wb) {
    if constexpr (LOOSE) {
      wa.e[0] = x[0];
      wa.e[1] = e0 + 1 < p.d ? x[1] : x[0];
    } else {
      wa = *reinterpret_cast<const W*>(x);
      if (kTwo && turns) wb = *reinterpret_cast<const W*>(x + half);
    }
  };
  auto write = [&](T* y, const W& wa, const W& wb) {
    if constexpr (LOOSE) {
      y[0] = wa.e[0];
      if (e0 + 1 < p.d) y[1] = wa.e[1];
    } else {
      *reinterpret_cast<W*>(y) = wa;
      if (kTwo && turns) *reinterpret_cast<W*>(y + half) = wb;
    }
  };
#pragma unroll
  for (int t = 0; t < 2; ++t) {  // heads h0 .. h1-1 of the two tensors' one after the other
    const int from = max(h0 - (t ? p.H[0] : 0), 0), to = min(h1 - (t ? p.H[0] : 0), p.H[t]);
    if (from >= to) continue;
    const long long xs = p.xs[t][1], ys = p.ys[t][1];
    const T* x = static_cast<const T*>(p.x[t]) + b * p.xs[t][0] + n * p.xs[t][2] + from * xs + e0;
    T* y = static_cast<T*>(p.y[t]) + b * p.ys[t][0] + n * p.ys[t][2] + from * ys + e0;
    int left = to - from;
    for (; left >= E; left -= E, x += E * xs, y += E * ys) {
      W wa[E], wb[E];
#pragma unroll
      for (int e = 0; e < E; ++e) read(x + e * xs, wa[e], wb[e]);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (turns) turn(wa[e], wb[e]);
        write(y + e * ys, wa[e], wb[e]);
      }
    }
    for (; left > 0; --left, x += xs, y += ys) {
      W wa, wb;
      read(x, wa, wb);
      if (turns) turn(wa, wb);
      write(y, wa, wb);
    }
  }
}

template <class T, int V, bool INTER, bool LOOSE = false>
cudaError_t launch(const RopeParams& p, cudaStream_t stream) {
  const int turning = INTER ? (p.rot + V - 1) / V : p.rot / 2 / V;
  const int units = INTER ? (p.d + V - 1) / V : turning + (p.d - p.rot) / V;
  const int heads = p.H[0] + p.H[1];
  const long long threads = static_cast<long long>(p.B) * p.N * units;
  int per = 1;
  while (per < 8 && threads * heads / (2 * per) >= 152LL * 2048) per *= 2;
  const dim3 grid(static_cast<unsigned>((threads + kThreads - 1) / kThreads),
                  static_cast<unsigned>((heads + per - 1) / per));
  rope_kernel<T, V, INTER, LOOSE><<<grid, kThreads, 0, stream>>>(p, units, turning, per);
  return cudaGetLastError();
}

template <class T, bool INTER>
cudaError_t launch_v(const RopeParams& p, int v, cudaStream_t stream) {
  if constexpr (sizeof(T) == 2)
    if (v == 8) return launch<T, 8, INTER>(p, stream);
  if (v >= 4) return launch<T, 4, INTER>(p, stream);
  if (v >= 2) return launch<T, 2, INTER>(p, stream);
  if constexpr (INTER) return launch<T, 2, true, true>(p, stream);
  return launch<T, 1, false>(p, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, cudaStream_t stream) {
  const int size = p.bf16 ? 2 : 4;
  // the widest vector that every address allows: rows, halves and tail
  int v = 16 / size;
  auto fits = [&](int w) {
    const long long bytes = static_cast<long long>(w) * size;
    if (p.d % w) return false;
    if (!p.interleaved && ((p.rot / 2) % w || (p.d - p.rot) % w)) return false;
    for (int t = 0; t < 2; ++t) {
      if (p.H[t] == 0) continue;
      if (reinterpret_cast<uintptr_t>(p.x[t]) % bytes || reinterpret_cast<uintptr_t>(p.y[t]) % bytes)
        return false;
      for (int i = 0; i < 3; ++i)
        if (p.xs[t][i] % w || p.ys[t][i] % w) return false;
    }
    return true;
  };
  while (v > 1 && !fits(v)) v /= 2;
  if (p.bf16) return p.interleaved ? launch_v<__nv_bfloat16, true>(p, v, stream)
                                   : launch_v<__nv_bfloat16, false>(p, v, stream);
  return p.interleaved ? launch_v<float, true>(p, v, stream) : launch_v<float, false>(p, v, stream);
}

}  // namespace spa
