// append.cu -- the new keys and values of a ragged batch into the projected
// key cache: row pos[b] + t of sequence b receives K~ = k P_h in fp16 with its
// power-of-two multiplier, and the value row as it is.
//
// Per key head the rows of all sequences are one matrix [B*T][d] times P_h, so
// a decode step (T = 1) fills the 16-row tiles of the tensor cores with the
// sequences of the batch.  Rows are independent: a row's bits depend on the
// row alone.
//
// The row multiplier 2^e puts the row's largest magnitude in [2^13, 2^14).
// Where the fp32 maximum is within 2^-12 of a power of two, which side it is
// on is decided on 64-bit sums of the columns that are as near, so that the
// multiplier is the exact one unless the row's sums cancel to below 2^-6 of their
// terms: 256 features are 16 products of 16 features one after the other, each
// off by 2^-22 of the terms at most, 2^-18 in all.  Beyond that it may belong to
// the neighbouring power, which fp16 holds as well.
//
// Bound by memory for long prompts: keys and values are read once and K~ and
// values written once.  4 x up to 4095 rows of 8 heads (d = d_v = 128, m = 32; 82
// MB, 12.1 us at the measured 6.8 TB/s): 22.7 us a call in a stream of calls, 3.6
// TB/s.  The 64-bit sums are dealt out over a warp's lanes, feature by feature, for the
// columns that need them alone; with a column per lane and all features one after the
// other a row took longer than the rest of its warp's work, and the calls 30 to 39 us.
// 64 sequences' one row each: the kernel 5.7 us, two round trips to memory behind the
// launch (14.5 us a call, the host's time).  A warp holds 16 rows' keys in registers as the A fragments, so a row
// needs one load and no staging; value rows are copied by CTAs of their own, whose
// loads wait for nothing else.  With P_h staged element by element and the values
// behind the keys in the same warps the prompts took 33 us.
#include <math.h>

#include "decode_shared.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace spa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr uint32_t kNear = 2048;  // 2^-12 in fp32 steps above a power of two; half as far in steps below it

__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// e with top * 2^-e in [2^13, 2^14); 0 for a row without a finite magnitude
__device__ __forceinline__ int row_exponent(double top) {
  if (!(top > 0.0) || !isfinite(top)) return 0;
  int E;
  frexp(top, &E);
  return max(-125, min(125, E - 14));
}

__device__ __forceinline__ uint32_t pair_at(const __nv_bfloat16* x, int k, int d) {
  const uint32_t lo = k < d ? __bfloat16_as_ushort(x[k]) : 0u;
  const uint32_t hi = k + 1 < d ? __bfloat16_as_ushort(x[k + 1]) : 0u;
  return lo | (hi << 16);
}

// P_h as mma B fragments in shared memory: fragment (step, tile) holds for
// lane l the pairs of rows k0..k0+3 (see below) of column n(l, tile).
//   features: the sum over k may run in any order, so lane quarter q of a group
//   of 32 features takes features 8q .. 8q+7, which it reads with one 16-byte
//   load: step s of the group uses 8q + 4s + {0,1} and 8q + 4s + {2,3}.
//   columns: tile j, quarter q, holds columns q*(M/4) + 2j + {0,1} of a row, so
//   a lane ends up with M/4 adjacent columns of the result.
template <int M>
__device__ __forceinline__ void stage_projection(uint2* frag, const __nv_bfloat16* P, int d,
                                                 int groups, int tid) {
  uint16_t* f = reinterpret_cast<uint16_t*>(frag);
  const int vectors = groups * 32 * (M / 8);  // 8 columns of one feature each
  constexpr int E = 8;                        // loads in flight
  for (int i0 = tid; i0 < vectors; i0 += E * kThreads) {
    uint4 x[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i = i0 + e * kThreads, k = i / (M / 8);
      x[e] = i < vectors && k < d ? __ldg(reinterpret_cast<const uint4*>(P) + i) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i = i0 + e * kThreads;
      if (i >= vectors) break;
      const int k = i / (M / 8), n0 = 8 * (i % (M / 8));
      const int g = k >> 5, q = (k >> 3) & 3, r = k & 7;
      const int step = 2 * g + (r >> 2), pos = r & 3;  // pos 0,1: first register, 2,3: second
      const uint32_t w[4] = {x[e].x, x[e].y, x[e].z, x[e].w};
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        // column n = qn*(M/4) + 2j + o is fragment column 2*qn + o of tile j
        const int n = n0 + u, qn = n / (M / 4), j = (n % (M / 4)) >> 1, o = n & 1;
        const int lane = (2 * qn + o) * 4 + q;  // B fragment: lane = column * 4 + quarter
        f[((step * (M / 8) + j) * 32 + lane) * 4 + pos] = static_cast<uint16_t>(w[u >> 1] >> (16 * (u & 1)));
      }
    }
  }
}

// CTAs per SM, half of them for the keys and half for the value rows: as many as the
// registers of 128 features in flight allow, and all of a call's CTAs resident at once,
// so that P_h is staged once.  (m = 32, the prompts above in a graph, with the slower
// sums: 25 us; 8 or 10 per SM in more than one wave 31 and 37; keys and values in the
// same warps, 5 per SM 27, 4 per SM in two waves 31.)
template <int M>
constexpr int kCtas = M <= 32 ? 6 : M == 64 ? 4 : 3;

template <int M>
__global__ void __launch_bounds__(kThreads, kCtas<M>) append_kernel(const AppendParams p, int tiles) {
  extern __shared__ uint2 frag[];
  const int h = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q = lane & 3, r0 = lane >> 2;
  const long long R = static_cast<long long>(p.B) * p.T;
  // where row r comes from (a row of k and v) and goes to; false: nowhere
  auto place = [&](long long r, long long* from, long long* dst, int* b, int* t) {
    if (r >= R) return false;
    *b = static_cast<int>(r / p.T);
    *t = static_cast<int>(r - static_cast<long long>(*b) * p.T);
    const long long at = static_cast<long long>(p.pos[*b]) + *t;
    if ((p.count && *t >= p.count[*b]) || at < 0 || at >= p.cap) return false;
    *from = (static_cast<long long>(*b) * p.H + h) * p.T + *t;
    *dst = (static_cast<long long>(*b) * p.H + h) * p.cap + at;
    return true;
  };
  if (blockIdx.z == 1) {
    // value rows, 16 per warp and turn: a lane a piece of 16 bytes of two or four rows at
    // a time, all of the tile in flight; the lanes 0-15 (and 16-31) know a row each
    constexpr int kPieces = 8;
    const int pieces = p.dv / 8;  // per row: 8 or 16
    for (int tile = blockIdx.x * kWarps + warp; tile < tiles; tile += gridDim.x * kWarps) {
      long long from = 0, dst = -1;
      int b, t;
      place(static_cast<long long>(tile) * 16 + (lane & 15), &from, &dst, &b, &t);
      uint4 v[kPieces];
#pragma unroll
      for (int e = 0; e < kPieces; ++e) {
        const int at = 32 * e + lane, row = at / pieces;
        const long long s = __shfl_sync(0xffffffffu, from, row & 15), d = __shfl_sync(0xffffffffu, dst, row & 15);
        if (row < 16 && d >= 0) v[e] = __ldg(reinterpret_cast<const uint4*>(p.v + s * p.dv) + at % pieces);
      }
#pragma unroll
      for (int e = 0; e < kPieces; ++e) {
        const int at = 32 * e + lane, row = at / pieces;
        const long long d = __shfl_sync(0xffffffffu, dst, row & 15);
        if (row < 16 && d >= 0) *(reinterpret_cast<uint4*>(p.vc + d * p.dv) + at % pieces) = v[e];
      }
    }
    return;
  }
  const int groups = (p.d + 31) / 32;
  const __nv_bfloat16* P = p.P + static_cast<size_t>(h) * p.d * M;
  stage_projection<M>(frag, P, p.d, groups, tid);
  __syncthreads();
  const bool wide = p.d % 8 == 0;
  for (int tile = blockIdx.x * kWarps + warp; tile < tiles; tile += gridDim.x * kWarps) {
    long long from[2], dst[2];  // this lane's two rows
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      from[i] = 0;
      dst[i] = -1;
      int b, t;
      if (place(static_cast<long long>(tile) * 16 + r0 + 8 * i, &from[i], &dst[i], &b, &t) && q == 0) {
        if (p.acc) p.acc[dst[i]] = 0.f;
        if (p.row_pos) p.row_pos[dst[i]] = (p.token ? p.token[b] : p.pos[b]) + t;
      }
    }
    if (!__any_sync(0xffffffffu, dst[0] >= 0 || dst[1] >= 0)) continue;
    const __nv_bfloat16* x[2] = {p.k + from[0] * p.d, p.k + from[1] * p.d};
    float c[M / 8][4];
#pragma unroll
    for (int j = 0; j < M / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) c[j][e] = 0.f;
    for (int g0 = 0; g0 < groups; g0 += 4) {  // 128 features in flight
      uint4 w[4][2];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int k = 32 * (g0 + g) + 8 * q;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          w[g][i] = make_uint4(0u, 0u, 0u, 0u);
          if (dst[i] < 0 || k >= p.d) continue;
          if (wide) {
            w[g][i] = __ldg(reinterpret_cast<const uint4*>(x[i] + k));
          } else {
            w[g][i] = make_uint4(pair_at(x[i], k, p.d), pair_at(x[i], k + 2, p.d), pair_at(x[i], k + 4, p.d),
                                 pair_at(x[i], k + 6, p.d));
          }
        }
      }
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        if (g0 + g >= groups) break;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const uint32_t a[4] = {s ? w[g][0].z : w[g][0].x, s ? w[g][1].z : w[g][1].x,
                                 s ? w[g][0].w : w[g][0].y, s ? w[g][1].w : w[g][1].y};
          const uint2* f = frag + ((2 * (g0 + g) + s) * (M / 8)) * 32 + lane;
#pragma unroll
          for (int j = 0; j < M / 8; ++j) {
            const uint2 b = f[j * 32];
            ptx::mma_bf16(c[j], a, b.x, b.y);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < M / 8; ++j) top = fmaxf(top, fmaxf(fabsf(c[j][2 * i]), fabsf(c[j][2 * i + 1])));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      int e = row_exponent(top);
      // rows whose maximum is next to a power of two: exact sums decide (below 2^-110 all
      // have the smallest multiplier)
      const uint32_t mant = __float_as_uint(top) & 0x7fffffu;
      const bool near = dst[i] >= 0 && top > 0x1p-110f && isfinite(top) &&
                        (mant < kNear || mant > 0x7fffffu - 2 * kNear);
      uint32_t todo = __ballot_sync(0xffffffffu, near && q == 0), cols = 0;  // this lane's columns as near
      if (near) {
        float edge = __uint_as_float(__float_as_uint(top) & 0x7f800000u);
        if (mant >= kNear) edge *= 2.f;
#pragma unroll
        for (int j = 0; j < M / 4; ++j)
          if (fabsf(fabsf(c[j / 2][2 * i + j % 2]) - edge) <= edge * 0x1.1p-12f) cols |= 1u << j;
      }
      while (todo) {
        const int from = __ffs(todo) - 1;
        todo &= todo - 1;
        const __nv_bfloat16* xr = reinterpret_cast<const __nv_bfloat16*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(x[i]), from));
        double best = 0.0;
#pragma unroll 1
        for (int g = 0; g < 4; ++g) {
          uint32_t left = __shfl_sync(0xffffffffu, cols, from + g);
#pragma unroll 1
          for (; left; left &= left - 1) {
            const __nv_bfloat16* Pn = P + g * (M / 4) + __ffs(left) - 1;
            double s = 0.0;
#pragma unroll 1
            for (int k = lane; k < p.d; k += 32)
              s += static_cast<double>(__bfloat162float(xr[k])) * static_cast<double>(__bfloat162float(Pn[k * M]));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            best = fmax(best, fabs(s));
          }
        }
        if ((lane >> 2) == (from >> 2)) e = row_exponent(best);
      }
      if (dst[i] < 0) continue;
      const float down = pow2i(-e);
      // this lane's M/4 adjacent columns
      uint32_t hw[M / 8];
#pragma unroll
      for (int j = 0; j < M / 8; ++j) {
        const __half2 v = __floats2half2_rn(c[j][2 * i] * down, c[j][2 * i + 1] * down);
        hw[j] = *reinterpret_cast<const uint32_t*>(&v);
      }
      uint16_t* o = p.kc + dst[i] * M + q * (M / 4);
      if constexpr (M == 16) {
        *reinterpret_cast<uint2*>(o) = make_uint2(hw[0], hw[1]);
      } else {
#pragma unroll
        for (int j = 0; j < M / 8; j += 4)
          *reinterpret_cast<uint4*>(o + 2 * j) = make_uint4(hw[j], hw[j + 1], hw[j + 2], hw[j + 3]);
      }
      if (q == 0) p.kc_mul[dst[i]] = pow2i(e);
    }
  }
}

template <int M>
cudaError_t launch(const AppendParams& p, cudaStream_t stream) {
  const long long R = static_cast<long long>(p.B) * p.T;
  const long long tiles = (R + 15) / 16;
  if (tiles > 0x7fffffffLL) return cudaErrorInvalidValue;
  const int smem = (p.d + 31) / 32 * 32 * M * 2;
  // the limit of the widest row, for every call: host threads with other widths may
  // launch at the same time
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = ds::allow_smem(append_kernel<M>, 256 * M * 2, done);
  if (e != cudaSuccess) return e;
  long long blocks = (tiles + kWarps - 1) / kWarps;
  const long long most = (152LL * kCtas<M> / 2 + p.H - 1) / p.H;
  if (blocks > most) blocks = most;
  append_kernel<M><<<dim3(static_cast<unsigned>(blocks), p.H, 2), kThreads, smem, stream>>>(
      p, static_cast<int>(tiles));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append_ragged(const AppendParams& p, cudaStream_t stream) {
  switch (p.m) {
    case 16: return launch<16>(p, stream);
    case 32: return launch<32>(p, stream);
    case 64: return launch<64>(p, stream);
    case 128: return launch<128>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace spa
