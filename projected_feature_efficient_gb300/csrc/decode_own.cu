// decode_own.cu -- the shared-prefix decode beside the prefix: the queries'
// projection, the sequences' own rows, and the joining of a row's parts.
#include <math.h>

#include "decode_shared.cuh"
#include "ptx.cuh"
#include "waits.cuh"

namespace spa {
namespace ds {
namespace {

using namespace ptx;

// ------------------------------------------------------------------ queries
// q~ = q P_h * log2(e)/sqrt(m) in fp32, then per row a power of two that puts its
// largest magnitude in [2^13, 2^14) and two fp16 parts (22 bits).  A CTA takes 16
// rows of a row tile: thread = (column, run of features), P_h read once per CTA.
// The last CTA counts the own tiles in front of every sequence.
// Bound by latency: 5 us for 1024 rows (d = 128, m = 32), 8 us for 4096 (m = 64).
constexpr int kQueryThreads = 256, kQueryRows = 16;

__device__ void count_tiles(const Params& a, int* red) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = a.p.B, per = (B + kQueryThreads - 1) / kQueryThreads;
  const int b0 = min(tid * per, B), b1 = min(b0 + per, B), unit = a.g.ounit;
  int sum = 0;
#pragma unroll 4
  for (int b = b0; b < b1; ++b) sum += (length_of(a, b) + unit - 1) / unit;
  int s = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += t;
  }
  if (lane == 31) red[warp] = s;
  __syncthreads();
  int at = s - sum;
  for (int w = 0; w < warp; ++w) at += red[w];
  for (int b = b0; b < b1; ++b) {
    a.w.off[b] = at;
    at += (length_of(a, b) + unit - 1) / unit;
  }
  if (tid == kQueryThreads - 1) a.w.off[B] = at;
}

template <int M>
__global__ void __launch_bounds__(kQueryThreads) decode_query_kernel(const __grid_constant__ Params a) {
  __shared__ union {
    float q[256][kQueryRows];  // transposed: the rows of a feature side by side
    float part[kQueryThreads / M][kQueryRows][M];
  } sh;
  __shared__ int red[kQueryThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, d = a.p.d;
  let_next_start();
  if (blockIdx.x == gridDim.x - 1) {
    if (a.p.cap > 0) count_tiles(a, red);
    else for (int b = tid; b <= a.p.B; b += kQueryThreads) a.w.off[b] = 0;
    return;
  }
  const int slices = (a.g.rows + kQueryRows - 1) / kQueryRows;
  const int tile = blockIdx.x / slices, r0 = (blockIdx.x - tile * slices) * kQueryRows;
  const int hk = a.g.dRT(tile), rt = tile - hk * a.g.RT;
  // row r of the tile: sequence and group member
  auto query_row = [&](int r) -> const __nv_bfloat16* {
    int b, g;
    if (a.g.parts > 1) {
      b = a.g.dparts(rt);
      g = (rt - b * a.g.parts) * kTile + r;
    } else {
      const int i = a.g.dG(r);
      b = i < a.g.spt ? rt * a.g.spt + i : a.p.B;
      g = r - i * a.p.G;
    }
    if (b >= a.p.B || g >= a.p.G) return nullptr;
    return a.p.q + (static_cast<size_t>(b) * a.p.H + hk * a.p.G + g) * d;
  };
  constexpr int kRuns = kQueryThreads / M, kAhead = 16;
  const int n = tid % M, run = tid / M, len = (d + kRuns - 1) / kRuns;
  const int k0 = min(run * len, d), k1 = min(k0 + len, d);
  const __nv_bfloat16* P = a.p.P + static_cast<size_t>(hk) * d * M + n;
  __nv_bfloat16 p[kAhead];  // in flight together with the queries
#pragma unroll
  for (int u = 0; u < kAhead; ++u)
    p[u] = k0 + u < k1 ? P[(k0 + u) * M] : __float2bfloat16_rn(0.f);
  {
    // thread = (row, every 16th feature): neighbours write neighbouring rows
    const int i = tid % kQueryRows;
    const __nv_bfloat16* q = query_row(r0 + i);
#pragma unroll 8
    for (int k = tid / kQueryRows; k < d; k += kQueryThreads / kQueryRows)
      sh.q[k][i] = q ? __bfloat162float(q[k]) : 0.f;
  }
  __syncthreads();
  float acc[kQueryRows];
#pragma unroll
  for (int r = 0; r < kQueryRows; ++r) acc[r] = 0.f;
#pragma unroll 1
  for (int kb = k0; kb < k1; kb += kAhead) {
    float f[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) f[u] = __bfloat162float(p[u]);
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      p[u] = kb + kAhead + u < k1 ? P[(kb + kAhead + u) * M] : __float2bfloat16_rn(0.f);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (kb + u >= k1) break;
      const float4* q = reinterpret_cast<const float4*>(sh.q[kb + u]);
#pragma unroll
      for (int r = 0; r < kQueryRows / 4; ++r) {
        const float4 x = q[r];
        acc[4 * r] = fmaf(x.x, f[u], acc[4 * r]);
        acc[4 * r + 1] = fmaf(x.y, f[u], acc[4 * r + 1]);
        acc[4 * r + 2] = fmaf(x.z, f[u], acc[4 * r + 2]);
        acc[4 * r + 3] = fmaf(x.w, f[u], acc[4 * r + 3]);
      }
    }
  }
  __syncthreads();  // the runs' sums lie where the queries were
#pragma unroll
  for (int r = 0; r < kQueryRows; ++r) sh.part[run][r][n] = acc[r];
  __syncthreads();
  uint16_t* out = a.w.qt + static_cast<size_t>(tile) * kTile * 2 * M;
#pragma unroll
  for (int i = warp; i < kQueryRows; i += kQueryThreads / 32) {
    constexpr int C = M / 32 > 0 ? M / 32 : 1;
    float x[C], top = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      x[c] = 0.f;
      if (lane + 32 * c < M)
        for (int u = 0; u < kRuns; ++u) x[c] += sh.part[u][i][lane + 32 * c];
      x[c] *= a.p.qscale;
      top = fmaxf(top, fabsf(x[c]));
    }
    top = warp_max(top);
    int e = 0;
    if (top > 0.f && isfinite(top)) {
      frexpf(top, &e);
      e = max(-125, min(125, e - 14));
    }
    const float down = __int_as_float((127 - e) << 23);
    const int r = r0 + i;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int k = lane + 32 * c;
      if (k >= M) break;
      const float v = x[c] * down;
      const __half hi = __float2half_rn(v), lo = __float2half_rn(v - __half2float(hi));
      const int at = (r >> 3) * 64 + (r & 7) * 8 + (k & 7);
      out[(k >> 3) * 1024 + at] = __half_as_ushort(hi);
      out[((M + k) >> 3) * 1024 + at] = __half_as_ushort(lo);
    }
    if (lane == 0) a.w.qmul[static_cast<size_t>(tile) * kTile + r] = __int_as_float((127 + e) << 23);
  }
}

// ------------------------------------------------------------------ own rows
// A warp takes a run of 16-key steps over the (sequence, key head) pairs and works
// for itself: K~ and V by TMA (16-row boxes, swizzled for ldmatrix) and the
// multipliers by 4-byte copies into a ring of its own, S = q~ K~^T and O += P V by
// mma.sync with the group's heads as the 16 rows (a group of more than 16: two
// parts), softmax in registers as in the prefix kernel.  Probabilities enter the value
// product in two bf16 parts, 16 bits: an output is off by its own rounding alone, as in
// the decode of one length (one part: 33.9 us for 35.1, on the 16 sequences below with
// their weights).  The rows that 16 heads cannot fill cost nothing here: reading the
// cache bounds the kernel, and the products are a fifth of the time that the bytes take.  (The same rows on
// tcgen05, 128 rows for a group of 4, took 4 times as long: each short segment
// drains the scores, the sums and their output in turn.)
// 128 sequences of 0 to 2047 rows, 8 key heads (m = 64, d_v = 128): 78 us, 412 MB read
// at 5.3 TB/s; 16 sequences of 17 to 8191 rows, 4 key heads (m = 32): 18 us for 85 MB;
// one sequence of 131072 rows, 8 key heads (m = 32): 80 us for the call, 340 MB.
// Behind a prefix kernel it waits for that one's end (moving in as its CTAs left took 47
// us for 50 with 32768 shared keys and 255 for 262 with 65536, but read the queries and
// offsets without the wait that makes another kernel's results visible).  With SMs of
// its own beside the prefix kernel and runs taken as warps came, the calls took longer
// than that (49 and 283).
template <int M, int DV>
struct OwnPlan {
  static constexpr int kV = kStep * DV * 2, kK = kStep * M * 2;
  static constexpr int kStage = (kV + kK + 1023) / 1024 * 1024;
  static constexpr int kFit = (208 * 1024) / (kOwnWarps * kStage);
  static constexpr int kStages = kFit > 6 ? 6 : kFit;
  static constexpr int kBytes = kOwnWarps * kStages * kStage + 1024;
  static_assert(kStages >= 3, "ring");
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two values as bf16 pairs of high and low parts, which add up to them within 2^-16.
__device__ __forceinline__ void split_bf16x2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(x, y);
  lo = pack_bf16x2(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u));
}

// A place in the order (key head, sequence, part, key) of the own rows.
struct Place {
  int hk, b, part, key, len;
  __device__ __forceinline__ void next(const Params& a) {
    key += kStep;
    if (key < len) return;
    key = 0;
    if (++part < a.g.oparts) return;
    part = 0;
    do {
      if (++b == a.p.B) {
        b = 0;
        ++hk;
      }
      len = length_of(a, b);
    } while (len == 0);
  }
};

template <int M, int DV>
__device__ __forceinline__ void run_own(const Params& a, const Maps& maps, uint8_t* smem_raw, uint64_t* full,
                                        float (*mul)[kStep]) {
  using P = OwnPlan<M, DV>;
  constexpr int ST = P::kStages;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = ((smem_u32(smem_raw) + 1023u) & ~1023u) + warp * (ST * P::kStage);
  const int worker = blockIdx.x * kOwnWarps + warp;
  const int all = a.w.off[a.p.B], head = all * a.g.oparts;
  const Deal deal(head * a.p.Hk, a.g);
  const int s0 = deal.start(worker), steps = deal.start(worker + 1) - s0;
  if (steps <= 0) return;
  Place at;
  {
    at.hk = s0 / head;
    int left = s0 - at.hk * head;
    // tiles of `oparts` parts in a row per sequence
    at.b = find_sequence(a, a.g.doparts(left));
    left -= a.w.off[at.b] * a.g.oparts;
    at.len = length_of(a, at.b);
    const int n = (at.len + kStep - 1) / kStep;
    at.part = left / n;
    at.key = (left - at.part * n) * kStep;
  }
  Place ahead = at;  // the next step to load
  int loaded = 0;
  bool ok = true;
  auto load = [&]() {
    const int slot = loaded % ST;
    const uint32_t to = base + slot * P::kStage;
    uint64_t* bar = &full[slot];
    const int plane = ahead.b * a.p.Hk + ahead.hk;
    if (lane < kStep && ahead.key + lane < ahead.len)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(&mul[slot][lane])),
                   "l"(a.p.kc_mul + static_cast<size_t>(plane) * a.p.cap + ahead.key + lane)
                   : "memory");
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
    if (elect_one_sync()) mbar_arrive_expect_tx(bar, P::kV + P::kK);
    // a failure-detection test leaves the first copies of the first warp unissued
    if (!(a.inject_stall && worker == 0 && loaded == 0) && elect_one_sync()) {
      uint8_t* p = smem_raw + (to - smem_u32(smem_raw));
#pragma unroll
      for (int h = 0; h < DV / 64; ++h) tma_load_3d(p + h * 2048, &maps.v[1][1], h * 64, ahead.key, plane, bar);
#pragma unroll
      for (int h = 0; h < (M + 63) / 64; ++h)
        tma_load_3d(p + P::kV + h * 2048, &maps.k[1][1], h * 64, ahead.key, plane, bar);
    }
    __syncwarp();
    if (++loaded < steps) ahead.next(a);
  };
  for (int i = 0; i < ST - 1 && i < steps; ++i) load();

  const int r = lane >> 2, q = lane & 3;  // rows r, r + 8 of the products; columns 2q, 2q + 1 of 8
  int row0 = 0;                           // this segment's first partial row
  float o[DV / 8][4], m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f, qm0 = 0.f, qm1 = 0.f;
  uint32_t qf[2 * M / 16][4];
  float *s_lo = nullptr, *s_hi = nullptr;
  int rows = 0;
  for (int i = 0; i < steps; ++i) {
    if (i == 0 || at.key == 0) {  // a new segment
      const int m0_ = at.part * kStep;
      rows = min(kStep, a.p.G - m0_);
      int tr;
      const int rt = row_tile(a.g, a.p.G, at.b, m0_, &tr);
      const size_t tile = static_cast<size_t>(at.hk) * a.g.RT + rt;
      const uint16_t* qt = a.w.qt + tile * kTile * 2 * M;
      const int ra = tr + r, rb = ra + 8;
      const bool in0 = r < rows, in1 = r + 8 < rows;
#pragma unroll
      for (int k = 0; k < 2 * M / 16; ++k) {
        const uint16_t* x = qt + 2 * k * 1024 + 2 * q;
        const int oa = (ra >> 3) * 64 + (ra & 7) * 8, ob = (rb >> 3) * 64 + (rb & 7) * 8;
        qf[k][0] = in0 ? *reinterpret_cast<const uint32_t*>(x + oa) : 0u;
        qf[k][1] = in1 ? *reinterpret_cast<const uint32_t*>(x + ob) : 0u;
        qf[k][2] = in0 ? *reinterpret_cast<const uint32_t*>(x + 1024 + oa) : 0u;
        qf[k][3] = in1 ? *reinterpret_cast<const uint32_t*>(x + 1024 + ob) : 0u;
      }
      qm0 = in0 ? a.w.qmul[tile * kTile + ra] : 0.f;
      qm1 = in1 ? a.w.qmul[tile * kTile + rb] : 0.f;
#pragma unroll
      for (int c = 0; c < DV / 8; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[c][e] = 0.f;
      m0 = m1 = -INFINITY;
      l0 = l1 = 0.f;
      row0 = (((at.hk * a.p.B + at.b) * a.g.oparts) + at.part + worker) * a.g.orows;
      if (a.w.scores) {
        float* s = a.w.scores + (static_cast<size_t>(at.b) * a.p.H + at.hk * a.p.G + m0_) * a.g.capr;
        s_lo = in0 ? s + static_cast<size_t>(r) * a.g.capr : nullptr;
        s_hi = in1 ? s + static_cast<size_t>(r + 8) * a.g.capr : nullptr;
      }
    }
    if (loaded < steps) load();  // into the slot that the last step left
    const int slot = i % ST, n = min(kStep, at.len - at.key);
    if (!__all_sync(0xffffffffu, mbar_wait(&full[slot], (i / ST) & 1, a.limit_ns))) {
      if (lane == 0) atomicExch(a.err, 1);
      ok = false;
      break;
    }
    const uint32_t vs = base + slot * P::kStage, ks = vs + P::kV;
    if (n < kStep) {  // value rows behind the length: zero
      for (int c = lane; c < (kStep - n) * (DV / 8); c += 32) {
        const int row = n + c / (DV / 8), part = c % (DV / 8);
        st_shared_v4(vs + (part >> 3) * 2048 + row * 128 + (part & 7) * 16, 0u, 0u, 0u, 0u);
      }
      __syncwarp();
    }
    // scores of keys 0-7 and 8-15.  The low parts of q~ come first, while the sums are
    // small: the sums that are rounded at the scores' size are the high parts' alone
    uint32_t kf[M / 16][4];
    float s[2][4] = {};
#pragma unroll
    for (int k = 0; k < M / 16; ++k) {
      const int key = (lane & 7) + ((lane >> 4) << 3), piece = 2 * k + ((lane >> 3) & 1);
      uint32_t addr;
      if constexpr (M >= 64)
        addr = ks + (piece >> 3) * 2048 + key * 128 + (((piece & 7) ^ (key & 7)) << 4);
      else if constexpr (M == 32)
        addr = ks + key * 64 + ((piece ^ ((key >> 1) & 3)) << 4);
      else
        addr = ks + key * 32 + ((piece ^ ((key >> 2) & 1)) << 4);
      ldsm4(kf[k], addr);
      mma_f16(s[0], qf[M / 16 + k], kf[k][0], kf[k][1]);
      mma_f16(s[1], qf[M / 16 + k], kf[k][2], kf[k][3]);
    }
#pragma unroll
    for (int k = 0; k < M / 16; ++k) {
      mma_f16(s[0], qf[k], kf[k][0], kf[k][1]);
      mma_f16(s[1], qf[k], kf[k][2], kf[k][3]);
    }
    float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float2 km = *reinterpret_cast<const float2*>(&mul[slot][8 * h + 2 * q]);
      const bool v0 = 8 * h + 2 * q < n, v1 = 8 * h + 2 * q + 1 < n;
      s[h][0] = v0 ? s[h][0] * (km.x * qm0) : -INFINITY;
      s[h][1] = v1 ? s[h][1] * (km.y * qm0) : -INFINITY;
      s[h][2] = v0 ? s[h][2] * (km.x * qm1) : -INFINITY;
      s[h][3] = v1 ? s[h][3] * (km.y * qm1) : -INFINITY;
      t0 = fmaxf(t0, fmaxf(s[h][0], s[h][1]));
      t1 = fmaxf(t1, fmaxf(s[h][2], s[h][3]));
      const int key = at.key + 8 * h + 2 * q;  // the score rows are padded to 128 keys
      if (s_lo) *reinterpret_cast<float2*>(s_lo + key) = make_float2(s[h][0], s[h][1]);
      if (s_hi) *reinterpret_cast<float2*>(s_hi + key) = make_float2(s[h][2], s[h][3]);
    }
    t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 1));
    t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 1));
    t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 2));
    t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 2));
    const bool g0 = t0 > m0 + kGrow, g1 = t1 > m1 + kGrow;
    if (__any_sync(0xffffffffu, g0 || g1)) {
      const float a0 = g0 ? ex2(m0 - t0) : 1.f, a1 = g1 ? ex2(m1 - t1) : 1.f;  // 0 at first
      if (g0) m0 = t0;
      if (g1) m1 = t1;
      l0 *= a0;
      l1 *= a1;
#pragma unroll
      for (int c = 0; c < DV / 8; ++c) {
        o[c][0] *= a0;
        o[c][1] *= a0;
        o[c][2] *= a1;
        o[c][3] *= a1;
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      s[h][0] = ex2(s[h][0] - m0);
      s[h][1] = ex2(s[h][1] - m0);
      s[h][2] = ex2(s[h][2] - m1);
      s[h][3] = ex2(s[h][3] - m1);
      l0 += s[h][0] + s[h][1];
      l1 += s[h][2] + s[h][3];
    }
    uint32_t p[4], pl[4];  // probabilities in two parts
#pragma unroll
    for (int e = 0; e < 4; ++e) split_bf16x2(s[e >> 1][2 * (e & 1)], s[e >> 1][2 * (e & 1) + 1], p[e], pl[e]);
#pragma unroll
    for (int c = 0; c < DV / 16; ++c) {
      const int key = lane & 15, piece = 2 * c + (lane >> 4);
      uint32_t b[4];
      ldsm4t(b, vs + (piece >> 3) * 2048 + key * 128 + (((piece & 7) ^ (key & 7)) << 4));
      mma_bf16(o[2 * c], p, b[0], b[1]);
      mma_bf16(o[2 * c + 1], p, b[2], b[3]);
      mma_bf16(o[2 * c], pl, b[0], b[1]);
      mma_bf16(o[2 * c + 1], pl, b[2], b[3]);
    }
    if (n < kStep) fence_proxy_async_smem();  // zeroed rows, which a copy overwrites next
    __syncwarp();  // every lane has read the slot
    const bool last = i + 1 == steps || at.key + kStep >= at.len;
    if (last) {  // the segment's sums
      l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
      l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = r + 8 * e;
        if (row < rows) {
          float* x = a.w.oo + static_cast<size_t>(row0 + row) * DV + 2 * q;
#pragma unroll
          for (int c = 0; c < DV / 8; ++c)
            *reinterpret_cast<float2*>(x + 8 * c) = make_float2(o[c][2 * e], o[c][2 * e + 1]);
          if (q == 0)
            *reinterpret_cast<float2*>(a.w.oml + static_cast<size_t>(row0 + row) * 2) =
                make_float2(e ? m1 : m0, e ? l1 : l0);
        }
      }
    }
    if (i + 1 < steps) at.next(a);
  }
  // after a wait that ran out: the copies in flight land before the memory is given up
  if (!ok)
    for (int k = max(0, loaded - ST); k < loaded; ++k) mbar_wait(&full[k % ST], (k / ST) & 1, a.limit_ns);
}

template <int M, int DV>
__global__ void __launch_bounds__(32 * kOwnWarps, 1)
    decode_own_kernel(const __grid_constant__ Params a, const __grid_constant__ Maps maps) {
  using P = OwnPlan<M, DV>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[kOwnWarps][P::kStages];
  __shared__ alignas(8) float mul[kOwnWarps][P::kStages][kStep];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane < P::kStages) mbar_init(&full[warp][lane], 1 + 32);  // the bytes, and every lane's multipliers
  fence_mbar_init();
  __syncwarp();
  // The query kernel's results are seen after this wait alone, also behind a prefix
  // kernel that has waited for them itself.
  wait_for_previous();
  let_next_start();
  run_own<M, DV>(a, maps, smem_raw, full[warp], mul[warp]);
}

// ------------------------------------------------------------------- combine
constexpr int kCombineThreads = 256;

// The partial results of row (b, h): np prefix segments, then own segments; rows
// of the partial buffers.
struct Parts {
  int np, n;
  int prow, orow;
};

__device__ __forceinline__ Parts parts_of(const Params& a, int b, int h) {
  const Geo& g = a.g;
  const int hk = g.dG(h), m = h - hk * a.p.G;
  int row;
  const int rt = row_tile(g, a.p.G, b, m, &row);
  Parts x;
  x.np = g.S;
  x.prow = (hk * g.RT + rt) * g.S * g.rows + row;
  x.n = x.np;
  x.orow = 0;
  const int off = a.w.off[b], n = a.w.off[b + 1] - off, all = a.w.off[a.p.B];
  if (n > 0) {
    const Deal deal(all * g.oparts * a.p.Hk, g);
    const int part = m / g.orows;
    const int t0 = hk * (all * g.oparts) + off * g.oparts + part * n;
    const int c0 = deal.owner(t0);  // the workers with the first and the last tile
    x.orow = ((hk * a.p.B + b) * g.oparts + part + c0) * g.orows + m - part * g.orows;
    x.n += deal.owner(t0 + n - 1) - c0 + 1;
  }
  return x;
}

__device__ __forceinline__ float2 stats_of(const Params& a, const Parts& x, int i) {
  const float* p = i < x.np ? a.w.pml + static_cast<size_t>(x.prow + i * a.g.rows) * 2
                            : a.w.oml + static_cast<size_t>(x.orow + (i - x.np) * a.g.orows) * 2;
  return *reinterpret_cast<const float2*>(p);
}

// Bound by the latency of a row's chain (lengths, statistics, sums) where there are few
// rows, and by issued instructions with weights: 7 us for 1024 rows of 19 + 1 parts, 23
// us for 4096 rows and 4.2 million weights (45 MB read).  One, two or eight warps per
// row: 13, 7 and 8 us, and 23, 26 and 32 us.
// Four warps per row of the output (the first `oblocks` blocks), each a quarter
// of its partial results, a lane per DV/32 of its columns.  The other blocks:
// the weights of 1024 keys of a (sequence, key head).
constexpr int kRowWarps = 4, kBlockRows = kCombineThreads / 32 / kRowWarps;
template <int DV>
__global__ void __launch_bounds__(kCombineThreads)
    decode_combine_kernel(const __grid_constant__ Params a, int oblocks, FastDiv dk, int kblocks) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  wait_for_previous();
  if (static_cast<int>(blockIdx.x) < oblocks) {
    constexpr int C = DV / 32;
    __shared__ float part[kBlockRows][kRowWarps][DV], pm[kBlockRows][kRowWarps], pl[kBlockRows][kRowWarps];
    const int at = warp / kRowWarps, quarter = warp % kRowWarps;
    const int row = blockIdx.x * kBlockRows + at;
    float top = -INFINITY, sum = 0.f, o[C];
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] = 0.f;
    if (row < a.p.B * a.p.H) {
      const int b = a.g.dH(row);
      const Parts x = parts_of(a, b, row - b * a.p.H);
      const int per = (x.n + kRowWarps - 1) / kRowWarps, first = quarter * per, end = min(x.n, first + per);
#pragma unroll 1
      for (int i0 = first; i0 < end; i0 += 32) {
        const float2 st = i0 + lane < end ? stats_of(a, x, i0 + lane) : make_float2(-INFINITY, 0.f);
        const float now = fmaxf(top, warp_max(st.x));
        const float old = ex2(top - now);  // 0 at first
        const float w = st.y > 0.f ? ex2(st.x - now) : 0.f;
        top = now;
        sum = sum * old + warp_sum(w * st.y);
#pragma unroll
        for (int c = 0; c < C; ++c) o[c] *= old;
        const int n = min(32, end - i0);
#pragma unroll 4
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
    }
#pragma unroll
    for (int c = 0; c < C; ++c) part[at][quarter][C * lane + c] = o[c];
    if (lane == 0) {
      pm[at][quarter] = top;
      pl[at][quarter] = sum;
    }
    __syncthreads();
    // thread = a pair of columns of one of the block's rows
    const int orow = tid / (DV / 2), c = 2 * (tid % (DV / 2));
    if (orow >= kBlockRows || blockIdx.x * kBlockRows + orow >= a.p.B * a.p.H) return;
    float m = pm[orow][0];
#pragma unroll
    for (int w = 1; w < kRowWarps; ++w) m = fmaxf(m, pm[orow][w]);
    float l = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) {
      const float f = pl[orow][w] > 0.f ? ex2(pm[orow][w] - m) : 0.f;
      l = fmaf(f, pl[orow][w], l);
      o0 = fmaf(f, part[orow][w][c], o0);
      o1 = fmaf(f, part[orow][w][c + 1], o1);
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;  // a row without keys: 0
    *reinterpret_cast<uint32_t*>(a.p.out + static_cast<size_t>(blockIdx.x * kBlockRows + orow) * DV + c) =
        pack_bf16x2(o0 * inv, o1 * inv);
    return;
  }
  const int w = blockIdx.x - oblocks, bh = dk(w), b = a.g.dHk(bh), hk = bh - b * a.p.Hk;
  const int n = length_of(a, b), k0 = (w - bh * kblocks) * 1024;
  if (k0 >= n) return;
  __shared__ float2 stat[128];  // maximum, one over the sum
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
        const float2 st = i0 + lane < x.n ? stats_of(a, x, i0 + lane) : make_float2(-INFINITY, 0.f);
        const float now = fmaxf(top, warp_max(st.x));
        sum = sum * ex2(top - now) + warp_sum(st.y > 0.f ? ex2(st.x - now) * st.y : 0.f);
        top = now;
      }
      if (lane == 0) stat[g] = make_float2(top, 1.f / sum);
    }
    __syncthreads();
    const float* s = a.w.scores + (static_cast<size_t>(b) * a.p.H + hk * a.p.G + g0) * a.g.capr + k0 + tid;
#pragma unroll 2
    for (int g = 0; g < gn; ++g, s += a.g.capr) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (k0 + tid + e * kCombineThreads < n) acc[e] = fmaf(ex2(s[e * kCombineThreads] - stat[g].x), stat[g].y, acc[e]);
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

template <int M, int DV>
cudaError_t launch_own_t(const Params& a, const Maps& maps, cudaStream_t stream) {
  using P = OwnPlan<M, DV>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(decode_own_kernel<M, DV>, P::kBytes, done);
  if (e != cudaSuccess) return e;
  return launch_after(decode_own_kernel<M, DV>, a.g.workers / kOwnWarps, 32 * kOwnWarps, P::kBytes, stream, a, maps);
}
template <int DV>
cudaError_t launch_own_m(const Params& a, const Maps& maps, cudaStream_t stream) {
  switch (a.p.m) {
    case 16: return launch_own_t<16, DV>(a, maps, stream);
    case 32: return launch_own_t<32, DV>(a, maps, stream);
    case 64: return launch_own_t<64, DV>(a, maps, stream);
    case 128: return launch_own_t<128, DV>(a, maps, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

// A plain launch, behind everything in the stream: the kernels that follow load the
// caches and write the workspace without waiting for more than this one.
cudaError_t launch_query(const Params& a, cudaStream_t stream) {
  const int slices = (a.g.rows + kQueryRows - 1) / kQueryRows;
  const unsigned grid = static_cast<unsigned>(a.p.Hk) * a.g.RT * slices + 1;
  switch (a.p.m) {
    case 16: decode_query_kernel<16><<<grid, kQueryThreads, 0, stream>>>(a); break;
    case 32: decode_query_kernel<32><<<grid, kQueryThreads, 0, stream>>>(a); break;
    case 64: decode_query_kernel<64><<<grid, kQueryThreads, 0, stream>>>(a); break;
    case 128: decode_query_kernel<128><<<grid, kQueryThreads, 0, stream>>>(a); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

cudaError_t launch_own(const Params& a, const Maps& maps, cudaStream_t stream) {
  return a.p.dv == 64 ? launch_own_m<64>(a, maps, stream) : launch_own_m<128>(a, maps, stream);
}

cudaError_t launch_combine(const Params& a, cudaStream_t stream) {
  const int kblocks = a.p.acc_out ? (a.p.cap + 1023) / 1024 : 0;
  const int oblocks = (a.p.B * a.p.H + kBlockRows - 1) / kBlockRows;
  const long long blocks = oblocks + static_cast<long long>(a.p.B) * a.p.Hk * kblocks;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  FastDiv dk;
  dk.set(kblocks > 0 ? kblocks : 1);
  const unsigned grid = static_cast<unsigned>(blocks);
  return a.p.dv == 64
             ? launch_after(decode_combine_kernel<64>, grid, kCombineThreads, 0, stream, a, oblocks, dk, kblocks)
             : launch_after(decode_combine_kernel<128>, grid, kCombineThreads, 0, stream, a, oblocks, dk, kblocks);
}

}  // namespace ds
}  // namespace spa
