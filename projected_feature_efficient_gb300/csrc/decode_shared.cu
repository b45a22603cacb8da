// decode_shared.cu -- one query per (sequence, head) against a prefix that the
// whole batch shares and the sequence's own cache rows, joined in one softmax:
//   s_j = <q P_h, K~_j> / sqrt(m),  O = sum_j softmax(s)_j V_j
// over rows 0 .. plen-1 of the prefix cache and 0 .. lens[b]-1 of the
// sequence's; query heads h*G .. h*G+G-1 share key head h.
//
//   chunk kernel    one (sequence, head) and one chunk of its keys: scores,
//                   chunk maximum and sum, unnormalised P V
//   combine kernel  the log-sum-exp merge of a row's chunks, and its own log-sum-exp
//   weights kernel  acc_out = acc + sum over the group's heads of p_j
#include <math.h>

#include "kernels.cuh"

namespace spa {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 1024;

struct Plan {
  int chunks;
  size_t part, lse, scores, total;
};

Plan plan_of(const DecodeSharedParams& p) {
  Plan L;
  const size_t rows = static_cast<size_t>(p.B) * p.H;
  L.chunks = static_cast<int>((static_cast<long long>(p.plen) + p.cap + kChunk - 1) / kChunk);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = (o + bytes + 255) & ~static_cast<size_t>(255);
    return at;
  };
  L.part = take(rows * L.chunks * (2 + p.dv) * sizeof(float));
  L.lse = take(rows * sizeof(float));
  L.scores = take(p.acc_out ? rows * p.cap * sizeof(float) : 0);
  L.total = o;
  return L;
}

__global__ void __launch_bounds__(kThreads) chunk_kernel(const DecodeSharedParams p, float* part,
                                                         float* scores, int chunks) {
  __shared__ float qs[128], sc[kChunk], red[kThreads / 32], oacc[kThreads];
  const int row = blockIdx.y, chunk = blockIdx.x, tid = threadIdx.x;
  const int b = row / p.H, h = row % p.H, hk = h / p.G;
  const int own = min(max(p.lens[b], 0), p.cap);
  const long long total = static_cast<long long>(p.plen) + own;
  const long long k0 = static_cast<long long>(chunk) * kChunk;
  const int n = static_cast<int>(min(total - k0, static_cast<long long>(kChunk)));
  float* mine = part + (static_cast<size_t>(row) * chunks + chunk) * (2 + p.dv);
  if (n <= 0) {
    if (tid == 0) {
      mine[0] = -INFINITY;
      mine[1] = 0.f;
    }
    return;
  }
  if (tid < p.m) {
    float s = 0.f;
    for (int l = 0; l < p.d; ++l)
      s = fmaf(__bfloat162float(p.q[static_cast<size_t>(row) * p.d + l]),
               __bfloat162float(p.P[(static_cast<size_t>(hk) * p.d + l) * p.m + tid]), s);
    qs[tid] = s * p.qscale;
  }
  __syncthreads();
  const size_t at = (static_cast<size_t>(b) * p.Hk + hk) * p.cap;
  float top = -INFINITY;
  for (int j = tid; j < n; j += kThreads) {
    const long long g = k0 + j;
    const bool shared = g < p.plen;
    const size_t r = shared ? static_cast<size_t>(hk) * p.pcap + g : at + (g - p.plen);
    const __half* k = reinterpret_cast<const __half*>(shared ? p.pkc : p.kc) + r * p.m;
    float s = 0.f;
    for (int c = 0; c < p.m; ++c) s = fmaf(__half2float(k[c]), qs[c], s);
    s *= shared ? p.pkc_mul[r] : p.kc_mul[r];
    if (scores && !shared) scores[static_cast<size_t>(row) * p.cap + (g - p.plen)] = s;
    sc[j] = s;
    top = fmaxf(top, s);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((tid & 31) == 0) red[tid >> 5] = top;
  __syncthreads();
  top = red[0];
  for (int w = 1; w < kThreads / 32; ++w) top = fmaxf(top, red[w]);
  __syncthreads();
  float sum = 0.f;
  for (int j = tid; j < n; j += kThreads) {
    const float e = exp2f(sc[j] - top);
    sc[j] = e;
    sum += e;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((tid & 31) == 0) red[tid >> 5] = sum;
  __syncthreads();
  const int c = tid % p.dv, part_of = tid / p.dv, parts = kThreads / p.dv;
  float o = 0.f;
  for (int j = part_of; j < n; j += parts) {
    const long long g = k0 + j;
    const bool shared = g < p.plen;
    const __nv_bfloat16* v = shared ? p.pv + (static_cast<size_t>(hk) * p.pcap + g) * p.dv
                                    : p.v + (at + (g - p.plen)) * p.dv;
    o = fmaf(sc[j], __bfloat162float(v[c]), o);
  }
  oacc[tid] = o;
  __syncthreads();
  if (tid < p.dv) {
    float s = 0.f;
    for (int i = 0; i < parts; ++i) s += oacc[i * p.dv + tid];
    mine[2 + tid] = s;
  }
  if (tid == 0) {
    float l = 0.f;
    for (int w = 0; w < kThreads / 32; ++w) l += red[w];
    mine[0] = top;
    mine[1] = l;
  }
}

// grid B*H, dv threads
__global__ void combine_kernel(const DecodeSharedParams p, const float* part, float* lse, int chunks) {
  const int row = blockIdx.x, c = threadIdx.x;
  const float* mine = part + static_cast<size_t>(row) * chunks * (2 + p.dv);
  float top = -INFINITY;
  for (int i = 0; i < chunks; ++i) top = fmaxf(top, mine[static_cast<size_t>(i) * (2 + p.dv)]);
  float l = 0.f, o = 0.f;
  if (top > -INFINITY) {
    for (int i = 0; i < chunks; ++i) {
      const float* x = mine + static_cast<size_t>(i) * (2 + p.dv);
      if (x[1] == 0.f) continue;  // a chunk without keys: its sums are not written
      const float w = exp2f(x[0] - top);
      l = fmaf(w, x[1], l);
      o = fmaf(w, x[2 + c], o);
    }
  }
  p.out[static_cast<size_t>(row) * p.dv + c] = __float2bfloat16_rn(l > 0.f ? o / l : 0.f);
  if (c == 0) lse[row] = l > 0.f ? top + log2f(l) : -INFINITY;
}

__global__ void weights_kernel(const DecodeSharedParams p, const float* scores, const float* lse) {
  const int bh = blockIdx.y, b = bh / p.Hk, hk = bh % p.Hk;
  const int n = min(max(p.lens[b], 0), p.cap);
  for (int j = blockIdx.x * blockDim.x + threadIdx.x; j < n; j += gridDim.x * blockDim.x) {
    float w = 0.f;
    for (int g = 0; g < p.G; ++g) {
      const size_t row = static_cast<size_t>(b) * p.H + hk * p.G + g;
      w += exp2f(scores[row * p.cap + j] - lse[row]);
    }
    const size_t at = static_cast<size_t>(bh) * p.cap + j;
    p.acc_out[at] = p.acc[at] + w;
  }
}

}  // namespace

size_t decode_shared_workspace(const DecodeSharedParams& p) { return plan_of(p).total; }

cudaError_t launch_decode_shared(const DecodeSharedParams& p, cudaStream_t stream) {
  const Plan L = plan_of(p);
  float* part = reinterpret_cast<float*>(p.ws + L.part);
  float* lse = reinterpret_cast<float*>(p.ws + L.lse);
  float* scores = p.acc_out ? reinterpret_cast<float*>(p.ws + L.scores) : nullptr;
  const int rows = p.B * p.H;
  cudaError_t e;
  if (L.chunks > 0) {
    chunk_kernel<<<dim3(L.chunks, rows), kThreads, 0, stream>>>(p, part, scores, L.chunks);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  combine_kernel<<<rows, p.dv, 0, stream>>>(p, part, lse, L.chunks);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (p.acc_out && p.cap > 0)
    weights_kernel<<<dim3((p.cap + 1023) / 1024, p.B * p.Hk), kThreads, 0, stream>>>(p, scores, lse);
  return cudaGetLastError();
}

}  // namespace spa
