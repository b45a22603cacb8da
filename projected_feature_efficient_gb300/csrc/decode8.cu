// decode8.cu -- one query per (sequence, head) against a projected cache of 8-bit pages and
// the 16-bit rows behind them, in one softmax.
//
// A sequence has n = 64 blocks + lens tokens: `blocks` pages, found through its row of the
// table, then `lens` open rows.  The query sees key j if j >= n - window or j < sink
// (window 0: every key):
//   out = softmax(q~ K~^T / sqrt(m)) V,   q~ = q P_h,   K~ = ks * codes, V = vs * codes
//
//   decode8_query_kernel    q~ log2(e)/sqrt(m) of every row in two fp16 parts (22 bits)
//   decode8_kernel          the keys: a warp takes a run of units (a page of 64 keys, or 16
//                           open rows) of (sequence, key head, part of the group) in order
//   decode8_combine_kernel  the parts of a row joined
//
// e4m3 values are exact in fp16, so both products run on them unscaled in fp16 with fp32
// sums, the scales taken outside, in fp32: the key scale multiplies the scores, the value
// scale a page's sums.  A page's weights are held against the page's own maximum, 2^kTop at
// the largest, and rounded to fp16: 2^-12 of a weight for all down to 2^-(kTop + 14) of it,
// 2^-(kTop + 25) of the largest below that.  The page's sums of weights and of weighted values
// then join the running ones in fp32 by one factor.  (Against the running maximum, weights
// 2^14 below it lost bits and 2^25 below it all, but not in the sum of weights: a first key of
// value zero 20 nats above 8192 others left more than ten times the error that fp16 weights
// account for.  Two fp16 parts, 22 bits: 16 sequences with 16 heads per key head 40 us for 35,
// one of 32768 keys 26 for 22, the error against 64 bits, 1.6e-3 of the output's own rounding,
// the same to two digits.)
//
// Keys and value columns are the rows of the products, 16 at a time, and the heads of a
// group their 8 columns (two products for 9 to 16 heads): no row of a product is empty, and
// scores^T leave it in the layout that the value product takes but for a transposition of
// 8 x 8 blocks within the registers.  (With heads as rows, high and low parts of q~ and of
// the probabilities filling up the 16: 630 instructions per page for 450, and 42 us for 33
// with 16 heads per key head.)
//
// Bound by memory: m + d_v bytes per key and key head.  A warp copies a unit ahead into its
// own ring of shared memory with asynchronous copies, waits for nobody and synchronises
// with no other warp.  The order of a column's 64 tokens in a page lets a lane load its
// operands of four value products with one 16-byte load.
//
// 64 sequences of up to 8191 keys, 32 heads on 8 key heads, m = 32, d_v = 128 (340 MB,
// 51 us at the rate of a copy): 68 us for the call, 5.0 TB/s; without the products 65 us, so
// they hide behind the copies.  The first page is there after 8 us (queries, lengths, table
// and page follow on one another), the middle warp ends at 53 us and the last at 62, because
// memory does not serve all SMs alike.  Giving out three sixteenths of each segment's units
// late, in chunks to warps that are done, brought the ends together but cost as much in
// chunks' first loads and sums (74 us).  Looking for a row's parts before the wait for the
// keys' kernel instead of after it: 72 -> 67 us at the time.
#include <cuda_fp16.h>
#include <math.h>

#include "decode_shared.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace spa {
namespace {

using namespace ptx;

constexpr int kOpen = 16;      // open rows of a unit
constexpr int kJoinThreads = 256;
constexpr float kGrow = 8.f;   // log2 units that a running maximum may lag behind
constexpr float kTop = 12.f;   // log2 of a page's largest weight: fp16 ends at 2^16, four units are left for the
                               // rounding of scores (of 2^24 and more) that it is taken from
constexpr int kMaxCtas = 152;  // grid limit (sizes the workspace)
constexpr int kMaxWarps = 8;   // of a CTA

// Shared memory of a unit: K~, V, then the page's scales or the open rows' multipliers.
// NT: products side by side, of 8 heads each.
template <int M, int DV, int NT>
struct Plan {
  static constexpr int kKRow = 2 * M + 16, kVRow = 2 * DV + 16;  // open rows, padded
  static constexpr int kVAt = 64 * M;                            // V of a page
  static constexpr int kVOpen = kOpen * kKRow;                   // V of open rows
  static constexpr int kOpenBytes = kVOpen + kOpen * kVRow, kPageBytes = kPageRows * (M + DV);
  static constexpr int kMeta = kOpenBytes > kPageBytes ? kOpenBytes : kPageBytes;
  static constexpr int kStage = kMeta + kOpen * 4;
  static constexpr int kRoom = 222 * 1024;
  // as many warps as have room for two units each (12 and 16 warps are slower, whose
  // registers no longer hold the operands of more than one step)
  static constexpr int kFitWarps = kRoom / (2 * kStage);
  static constexpr int kWarps = kMaxWarps < kFitWarps ? kMaxWarps : kFitWarps;
  static constexpr int kFit = kRoom / (kWarps * kStage);
  static constexpr int kStages = kFit > 4 ? 4 : kFit;
  static constexpr int kBytes = kWarps * kStages * kStage;
  static_assert(kStages >= 2 && kStage % 16 == 0, "ring");
};

struct Work {
  int parts, rows;   // parts of a group, heads of a part (8 or 16)
  int workers;       // warps that share the units
  __half* q;         // [B*H][2][m] high and low parts
  float* qmul;       // [B*H] power of two
  long long* off;    // [B + 1] units of one (key head, part) in front of each sequence (many sequences)
  float2* ml;        // [slots][rows] maximum and sum
  float* o;          // [slots][rows][dv]
};

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// The parts of the workspace and its size.
size_t lay_out(const Decode8Params& p, int workers, Work* w) {
  w->rows = p.G > 8 ? 16 : 8;
  w->parts = (p.G + w->rows - 1) / w->rows;
  w->workers = workers;
  const size_t bh = static_cast<size_t>(p.B) * p.H;
  // a worker's run cuts at most one segment in front of each end
  const size_t slots = static_cast<size_t>(p.B) * p.Hk * w->parts + workers;
  char* at = p.ws;
  size_t used = 0;
  auto take = [&](size_t bytes) {
    char* x = at ? at + used : nullptr;
    used += up256(bytes);
    return x;
  };
  w->q = reinterpret_cast<__half*>(take(bh * 2 * p.m * sizeof(__half)));
  w->qmul = reinterpret_cast<float*>(take(bh * sizeof(float)));
  w->off = reinterpret_cast<long long*>(take((static_cast<size_t>(p.B) + 1) * sizeof(long long)));
  w->ml = reinterpret_cast<float2*>(take(slots * w->rows * sizeof(float2)));
  w->o = reinterpret_cast<float*>(take(slots * w->rows * p.dv * sizeof(float)));
  return used;
}

// ------------------------------------------------------------------ queries
// 8 rows (b, head of one key head) per CTA; thread = (column, run of features).
constexpr int kQueryThreads = 256, kQueryRows = 8;

template <int M>
__global__ void __launch_bounds__(kQueryThreads) decode8_query_kernel(const Decode8Params p, const Work w) {
  constexpr int kRuns = kQueryThreads / M;
  __shared__ union alignas(16) {
    float q[256][kQueryRows];
    float part[kRuns][kQueryRows][M];
  } sh;
  ds::let_next_start();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, d = p.d;
  const int hk = blockIdx.y, first = blockIdx.x * kQueryRows, all = p.B * p.G;
  // row i of the CTA: sequence b, head g of the group
  auto row_of = [&](int i) { return static_cast<size_t>((first + i) / p.G) * p.H + hk * p.G + (first + i) % p.G; };
  const int n = tid % M, run = tid / M, len = (d + kRuns - 1) / kRuns;
  const int k0 = min(run * len, d), k1 = min(k0 + len, d);
  const __nv_bfloat16* P = p.P + static_cast<size_t>(hk) * d * M + n;
  constexpr int kAhead = 16;
  __nv_bfloat16 f[kAhead];  // in flight together with the queries
#pragma unroll
  for (int u = 0; u < kAhead; ++u) f[u] = k0 + u < k1 ? P[(k0 + u) * M] : __float2bfloat16_rn(0.f);
  if (first + warp < all) {  // a warp per row
    const __nv_bfloat16* q = p.q + row_of(warp) * d;
    for (int k = lane; k < d; k += 32) sh.q[k][warp] = __bfloat162float(q[k]);
  } else {
    for (int k = lane; k < d; k += 32) sh.q[k][warp] = 0.f;
  }
  __syncthreads();
  float acc[kQueryRows] = {};
#pragma unroll 1
  for (int kb = k0; kb < k1; kb += kAhead) {
    float g[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) g[u] = __bfloat162float(f[u]);
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      f[u] = kb + kAhead + u < k1 ? P[(kb + kAhead + u) * M] : __float2bfloat16_rn(0.f);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (kb + u >= k1) break;
      const float4 a = *reinterpret_cast<const float4*>(&sh.q[kb + u][0]);
      const float4 b = *reinterpret_cast<const float4*>(&sh.q[kb + u][4]);
      acc[0] = fmaf(a.x, g[u], acc[0]);
      acc[1] = fmaf(a.y, g[u], acc[1]);
      acc[2] = fmaf(a.z, g[u], acc[2]);
      acc[3] = fmaf(a.w, g[u], acc[3]);
      acc[4] = fmaf(b.x, g[u], acc[4]);
      acc[5] = fmaf(b.y, g[u], acc[5]);
      acc[6] = fmaf(b.z, g[u], acc[6]);
      acc[7] = fmaf(b.w, g[u], acc[7]);
    }
  }
  __syncthreads();  // the runs' sums lie where the queries were
#pragma unroll
  for (int r = 0; r < kQueryRows; ++r) sh.part[run][r][n] = acc[r];
  __syncthreads();
  if (first + warp >= all) return;
  constexpr int C = M / 32 > 0 ? M / 32 : 1;
  float x[C], top = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    x[c] = 0.f;
    if (lane + 32 * c < M)
      for (int u = 0; u < kRuns; ++u) x[c] += sh.part[u][warp][lane + 32 * c];
    x[c] *= p.qscale;
    top = fmaxf(top, fabsf(x[c]));
  }
  top = ds::warp_max(top);
  int e = 0;
  if (top > 0.f && isfinite(top)) {
    frexpf(top, &e);
    e = max(-125, min(125, e - 14));
  }
  const float down = __int_as_float((127 - e) << 23);
  const size_t row = row_of(warp);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int k = lane + 32 * c;
    if (k >= M) break;
    const float v = x[c] * down;
    const __half hi = __float2half_rn(v), lo = __float2half_rn(v - __half2float(hi));
    w.q[row * 2 * M + k] = hi;
    w.q[row * 2 * M + M + k] = lo;
  }
  if (lane == 0) w.qmul[row] = __int_as_float((127 + e) << 23);
}

// ------------------------------------------------------------------ what a sequence sees
struct Seq {
  int blocks, open;   // pages, open rows
  int lo;             // first key of the window
  int sb, wb;         // pages [0, sb) hold first keys that stay visible, [wb, blocks) the window
  int units;          // pages, then open rows, 16 to a unit
};
__device__ __forceinline__ Seq seq_of(const Decode8Params& p, int b) {
  Seq s;
  s.blocks = p.pg.table ? min(max(p.blocks[b], 0), p.pg.width) : 0;
  s.open = p.cap > 0 ? min(max(p.lens[b], 0), p.cap) : 0;
  const int n = s.blocks * kPageRows + s.open;  // the host keeps it within 31 bits
  s.lo = p.window > 0 ? max(n - p.window, 0) : 0;
  if (s.lo <= p.sink) s.lo = 0;
  s.sb = s.lo ? min((p.sink + kPageRows - 1) / kPageRows, s.blocks) : 0;
  s.wb = min(max(s.lo / kPageRows, s.sb), s.blocks);
  s.units = s.sb + (s.blocks - s.wb) + (s.open + kOpen - 1) / kOpen;
  return s;
}

// A place in the order (sequence, key head, part of the group, unit).
struct Place {
  int b, hk, part, u;
  Seq s;
  __device__ __forceinline__ int pages() const { return s.sb + s.blocks - s.wb; }
  __device__ __forceinline__ int block() const { return u < s.sb ? u : s.wb + u - s.sb; }
  __device__ __forceinline__ void next(const Decode8Params& p, int parts) {
    if (++u < s.units) return;
    u = 0;
    if (++part < parts) return;
    part = 0;
    if (++hk < p.Hk) return;
    hk = 0;
    while (b + 1 < p.B) {
      s = seq_of(p, ++b);
      if (s.units > 0) return;
    }
  }
};

// Of W workers (no more than there are units, so that each has one) w takes the units
// [floor(w all / W), floor((w + 1) all / W)); unit x is worker floor(((x + 1) W - 1) / all)'s.
__device__ __forceinline__ int at_work(long long all, int workers) {
  return static_cast<int>(all < workers ? all : workers);
}
__device__ __forceinline__ long long run_start(int w, long long all, int workers) { return w * all / workers; }
__device__ __forceinline__ int owner(long long x, long long all, int workers) {
  return static_cast<int>(((x + 1) * workers - 1) / all);
}

// The sequences are dealt to the T threads of a block in runs of equal length.  Returns the
// units of one (key head, part) in front of the thread's, and all; `sums`: one per warp.
template <int T>
__device__ __forceinline__ int seqs_of_thread(const Decode8Params& p) { return (p.B + T - 1) / T; }
template <int T>
__device__ __forceinline__ long long units_in_front(const Decode8Params& p, long long* sums, long long& total) {
  const int tid = threadIdx.x, lane = tid & 31, per = seqs_of_thread<T>(p);
  const long long first = static_cast<long long>(tid) * per;
  long long mine = 0;
  for (int i = 0; i < per && first + i < p.B; ++i) mine += seq_of(p, static_cast<int>(first) + i).units;
  long long scan = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += t;
  }
  if (lane == 31) sums[tid >> 5] = scan;
  __syncthreads();
  scan -= mine;
  total = 0;
#pragma unroll
  for (int i = 0; i < T / 32; ++i) {
    if (i < tid >> 5) scan += sums[i];
    total += sums[i];
  }
  return scan;
}

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Four e4m3 values as two fp16 pairs, exactly.
__device__ __forceinline__ void half_pairs(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}
__device__ __forceinline__ uint32_t half_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// An 8 x 8 block of 16-bit values, a row per four lanes and two columns per lane.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// c += a b in fp16 with fp32 sums (mma_f16, but free to be moved among its neighbours).
__device__ __forceinline__ void product(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint64_t both(float x) { return pack_f32x2(x, x); }

// ------------------------------------------------------------------ keys
// The 8 x 8 blocks of scores, rows keys and columns heads: a lane has row r = lane / 4 and
// columns 2q, 2q + 1 (q = lane % 4).  The state of a segment (the keys of one sequence, key
// head and part of the group that a worker takes): heads 2q and 2q + 1 of each product, the
// same in the eight lanes with one q but for `sum`, which is the lane's own keys'.
template <int DV, int NT>
struct State {
  float o[NT][DV / 16][4];  // value columns 16 c + r (0, 1) and 16 c + r + 8 (2, 3)
  float top[NT][2], sum[NT][2], qm[NT][2];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int c = 0; c < DV / 16; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][c][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        top[t][e] = -INFINITY;
        sum[t][e] = 0.f;
      }
    }
  }
  // x, a lane's largest scores, becomes the unit's; what was summed so far goes along with the maximum
  __device__ __forceinline__ void raise(float (&x)[NT][2]) {
    bool grow = false;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int o_ = 4; o_ < 32; o_ <<= 1) x[t][e] = fmaxf(x[t][e], __shfl_xor_sync(0xffffffffu, x[t][e], o_));
        grow |= x[t][e] > top[t][e] + kGrow;
      }
    if (!__any_sync(0xffffffffu, grow)) return;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float f[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        f[e] = 1.f;
        if (x[t][e] > top[t][e] + kGrow) {
          f[e] = ex2(top[t][e] - x[t][e]);  // 0 at first
          top[t][e] = x[t][e];
        }
        sum[t][e] *= f[e];
      }
#pragma unroll
      for (int c = 0; c < DV / 16; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][c][e] *= f[e & 1];
    }
  }
  // what a score is held against: keys that are all masked leave no maximum
  __device__ __forceinline__ float base(int t, int e) const { return top[t][e] == -INFINITY ? 0.f : top[t][e]; }
};

// The projected queries as the scores' second operand: head r of each product, four
// features per step and lane.
template <int M, int NT>
struct Query {
  uint32_t hi[NT][M / 16][2], lo[NT][M / 16][2];
};

// Feature 4 k + c of lane q's share is feature share(q, 4k) + c of the row.
template <int M>
__device__ __forceinline__ int share(int q, int i) {
  return M == 128 ? 64 * (i >> 4) + 16 * q + (i & 15) : M / 4 * q + i;
}

template <int M, int DV, int NT>
__device__ __forceinline__ void load_query(const Decode8Params& p, const Work& w, const Place& at, int r, int q,
                                           Query<M, NT>& qf, State<DV, NT>& st) {
  const size_t row0 = static_cast<size_t>(at.b) * p.H + at.hk * p.G + at.part * w.rows;
  const int heads = min(w.rows, p.G - at.part * w.rows);
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const bool in = 8 * t + r < heads;
    const __half* x = w.q + (row0 + (in ? 8 * t + r : 0)) * 2 * M;
#pragma unroll
    for (int k = 0; k < M / 16; ++k) {
      const int from = share<M>(q, 4 * k);
      uint2 hi = *reinterpret_cast<const uint2*>(x + from), lo = *reinterpret_cast<const uint2*>(x + M + from);
      if (!in) hi = lo = make_uint2(0u, 0u);
      qf.hi[t][k][0] = hi.x;
      qf.hi[t][k][1] = hi.y;
      qf.lo[t][k][0] = lo.x;
      qf.lo[t][k][1] = lo.y;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) st.qm[t][e] = 8 * t + 2 * q + e < heads ? w.qmul[row0 + 8 * t + 2 * q + e] : 0.f;
  }
}

// Scores of T tiles of 16 keys, without scales: operands(j, a) loads the rows of tile j.
// The low parts of q~ come first, while the sums are small.  s[t][j][i]: key 16 j + r (+ 8
// for i >= 2), head 8 t + 2 q (+ 1 for odd i).
template <int M, int NT, int T, class F>
__device__ __forceinline__ void scores(const Query<M, NT>& qf, float (&s)[NT][T][4], F operands) {
#pragma unroll
  for (int j = 0; j < T; ++j) {
    uint32_t a[M / 16][4];
    operands(j, a);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[t][j][e] = 0.f;
#pragma unroll
      for (int k = 0; k < M / 16; ++k) product(s[t][j], a[k], qf.lo[t][k][0], qf.lo[t][k][1]);
#pragma unroll
      for (int k = 0; k < M / 16; ++k) product(s[t][j], a[k], qf.hi[t][k][0], qf.hi[t][k][1]);
    }
  }
}

// A page of 64 keys.
template <int M, int DV, int NT>
__device__ __forceinline__ void page_unit(const Decode8Params& p, const Place& at, const uint8_t* st, int r, int q,
                                          const Query<M, NT>& qf, State<DV, NT>& x) {
  using P = Plan<M, DV, NT>;
  const float2 scale = *reinterpret_cast<const float2*>(st + P::kMeta);
  if (scale.x < 0.f) return;  // a block without a page
  float s[NT][4][4];
  scores<M, NT, 4>(qf, s, [&](int j, uint32_t (&a)[M / 16][4]) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {  // keys r and r + 8
      const uint8_t* row = st + (16 * j + 8 * e + r) * M;
      if constexpr (M == 16) {
        half_pairs(*reinterpret_cast<const uint32_t*>(row + 4 * q), a[0][e], a[0][2 + e]);
      } else if constexpr (M == 32) {
        const uint2 v = *reinterpret_cast<const uint2*>(row + 8 * q);
        half_pairs(v.x, a[0][e], a[0][2 + e]);
        half_pairs(v.y, a[1][e], a[1][2 + e]);
      } else {
#pragma unroll
        for (int c = 0; c < M / 64; ++c) {
          const uint4 v = *reinterpret_cast<const uint4*>(row + 64 * c + 16 * q);
          half_pairs(v.x, a[4 * c][e], a[4 * c][2 + e]);
          half_pairs(v.y, a[4 * c + 1][e], a[4 * c + 1][2 + e]);
          half_pairs(v.z, a[4 * c + 2][e], a[4 * c + 2][2 + e]);
          half_pairs(v.w, a[4 * c + 3][e], a[4 * c + 3][2 + e]);
        }
      }
    }
  });
  float f[NT][2];  // of a score
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) f[t][e] = scale.x * x.qm[t][e];
  const int key0 = at.block() * kPageRows;
  if (key0 < at.s.lo && key0 + kPageRows > p.sink) {  // a page that the window's or the first keys' border cuts
    // scaled before they are masked: a factor may be 0, which would make a NaN of the masked score
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int key = key0 + 16 * j + 8 * e + r;
        const bool seen = key >= at.s.lo || key < p.sink;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i) s[t][j][2 * e + i] = seen ? s[t][j][2 * e + i] * f[t][i] : -INFINITY;
      }
#pragma unroll
    for (int t = 0; t < NT; ++t) f[t][0] = f[t][1] = 1.f;
  }
  float top[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float most = s[t][0][e];
#pragma unroll
      for (int j = 0; j < 4; ++j) most = max3(most, s[t][j][e], s[t][j][2 + e]);
      top[t][e] = most * f[t][e];  // f is positive, or 0 where there is no head
    }
  x.raise(top);
  // weights against the page's own maximum (a page whose keys are all masked: the running one), in fp16, transposed:
  // keys 2q, 2q + 1 of head r.  g takes the page's sums of values to the running ones.
  uint32_t b[NT][4][2];
  uint64_t g[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float of[2], to[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float base = x.base(t, e), own = top[t][e] == -INFINITY ? base : top[t][e];
      of[e] = kTop - own;
      to[e] = ex2(-of[e] - base);  // what of rounds off, to puts back
    }
    const uint64_t f2 = pack_f32x2(f[t][0], f[t][1]), of2 = pack_f32x2(of[0], of[1]);
    uint64_t sum2 = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float e0, e1;
        unpack_f32x2(fma_f32x2(pack_f32x2(s[t][j][2 * e], s[t][j][2 * e + 1]), f2, of2), e0, e1);
        e0 = ex2(e0);
        e1 = ex2(e1);
        sum2 = add_f32x2(sum2, pack_f32x2(e0, e1));
        b[t][j][e] = transposed(half_pair(e0, e1));
      }
    g[t] = pack_f32x2(to[0], to[1]);
    unpack_f32x2(fma_f32x2(sum2, g[t], pack_f32x2(x.sum[t][0], x.sum[t][1])), x.sum[t][0], x.sum[t][1]);
    g[t] = mul_f32x2(g[t], both(scale.y));
  }
#pragma unroll
  for (int c = 0; c < DV / 16; ++c) {
    const uint4 v0 = *reinterpret_cast<const uint4*>(st + P::kVAt + (16 * c + r) * kPageRows + 16 * q);
    const uint4 v1 = *reinterpret_cast<const uint4*>(st + P::kVAt + (16 * c + 8 + r) * kPageRows + 16 * q);
    const uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w};
    float o[NT][4] = {};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t a[4];
      half_pairs(w0[j], a[0], a[2]);
      half_pairs(w1[j], a[1], a[3]);
#pragma unroll
      for (int t = 0; t < NT; ++t) product(o[t], a, b[t][j][0], b[t][j][1]);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; e += 2)
        unpack_f32x2(fma_f32x2(pack_f32x2(o[t][e], o[t][e + 1]), g[t], pack_f32x2(x.o[t][c][e], x.o[t][c][e + 1])),
                     x.o[t][c][e], x.o[t][c][e + 1]);
  }
}

// Up to 16 open rows, fp16 K~ with a multiplier each and bf16 V.
template <int M, int DV, int NT>
__device__ __forceinline__ void open_unit(const Decode8Params& p, const Place& at, const uint8_t* st, int lane, int r,
                                          int q, const Query<M, NT>& qf, State<DV, NT>& x) {
  using P = Plan<M, DV, NT>;
  float s[NT][1][4];
  scores<M, NT, 1>(qf, s, [&](int, uint32_t (&a)[M / 16][4]) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint8_t* row = st + (8 * e + r) * P::kKRow;
#pragma unroll
      for (int k = 0; k < M / 16; ++k) {
        const uint2 v = *reinterpret_cast<const uint2*>(row + 2 * share<M>(q, 4 * k));
        a[k][e] = v.x;
        a[k][2 + e] = v.y;
      }
    }
  });
  const int row0 = (at.u - at.pages()) * kOpen, key0 = at.s.blocks * kPageRows + row0, n = at.s.open - row0;
  float top[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) top[t][0] = top[t][1] = -INFINITY;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int c = 8 * e + r;
    const bool seen = c < n && (key0 + c >= at.s.lo || key0 + c < p.sink);
    const float mul = *reinterpret_cast<const float*>(st + P::kMeta + 4 * c);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        s[t][0][2 * e + i] = seen ? s[t][0][2 * e + i] * (mul * x.qm[t][i]) : -INFINITY;
        top[t][i] = fmaxf(top[t][i], s[t][0][2 * e + i]);
      }
  }
  x.raise(top);
  uint32_t b[NT][2], low[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float e0 = ex2(s[t][0][2 * e] - x.base(t, 0)), e1 = ex2(s[t][0][2 * e + 1] - x.base(t, 1));
      x.sum[t][0] += e0;
      x.sum[t][1] += e1;
      split_bf16x2(e0, e1, b[t][e], low[t][e]);  // bf16 values: two parts, 16 bits
      b[t][e] = transposed(b[t][e]);
      low[t][e] = transposed(low[t][e]);
    }
  const uint32_t v = smem_u32(st + P::kVOpen) + ((lane & 7) + 8 * (lane >> 4)) * P::kVRow + 16 * (lane >> 3 & 1);
#pragma unroll
  for (int c = 0; c < DV / 16; ++c) {
    uint32_t a[4];
    ldsm4t(a, v + 32 * c);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      mma_bf16(x.o[t][c], a, b[t][0], b[t][1]);
      mma_bf16(x.o[t][c], a, low[t][0], low[t][1]);
    }
  }
}

template <int M, int DV, int NT>
__global__ void __launch_bounds__(32 * kMaxWarps, 1) decode8_kernel(const Decode8Params p, const Work w) {
  using P = Plan<M, DV, NT>;
  constexpr int W = P::kWarps, T = 32 * W, ST = P::kStages;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ long long sums[W], starts_at[T];
  ds::let_next_start();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, q = lane & 3;
  const int per_seq = p.Hk * w.parts;  // segments of a sequence
  long long total;
  long long in_front = units_in_front<T>(p, sums, total);
  starts_at[tid] = per_seq * in_front;
  if (p.B > kJoinThreads && blockIdx.x == 0) {  // for the joining
    const long long b0 = static_cast<long long>(tid) * seqs_of_thread<T>(p);
    for (int i = 0; i < seqs_of_thread<T>(p) && b0 + i < p.B; ++i) {
      w.off[b0 + i] = in_front;
      in_front += seq_of(p, static_cast<int>(b0) + i).units;
    }
    if (tid == 0) w.off[p.B] = total;
  }
  __syncthreads();
  const long long all = total * per_seq;
  const int busy = at_work(all, w.workers), worker = warp * gridDim.x + blockIdx.x;  // neighbours on different SMs
  if (worker >= busy) {
    // without it a call on nothing but empty sequences could end before its first kernel does
    ds::wait_for_previous();
    return;
  }
  const long long from = run_start(worker, all, busy);
  const int units = static_cast<int>(run_start(worker + 1, all, busy) - from);

  Place at;
  {
    int t = -1;  // the last thread whose sequences start at or in front of the run
#pragma unroll
    for (int i = 0; i < W; ++i) t += __popc(__ballot_sync(0xffffffffu, starts_at[32 * i + lane] <= from));
    long long x = from - starts_at[t];
    for (at.b = t * seqs_of_thread<T>(p);; ++at.b) {
      at.s = seq_of(p, at.b);
      const long long n = static_cast<long long>(at.s.units) * per_seq;
      if (x < n || at.b + 1 >= p.B) break;
      x -= n;
    }
    const int rest = static_cast<int>(x / at.s.units);
    at.u = static_cast<int>(x - static_cast<long long>(rest) * at.s.units);
    at.hk = rest / w.parts;
    at.part = rest - at.hk * w.parts;
  }
  Place ahead = at;  // the next unit to copy
  const uint32_t ring = smem_u32(smem_raw) + warp * (ST * P::kStage);
  int copied = 0, page = 0, page_b = -1, page_u = 0;  // lane's page of unit page_u + lane of sequence page_b
  auto copy = [&]() {
    const uint32_t st = ring + (copied % ST) * P::kStage;
    const int pages = ahead.pages();
    if (ahead.u < pages) {
      if (ahead.b != page_b || ahead.u < page_u || ahead.u >= page_u + 32) {
        page_b = ahead.b;
        page_u = ahead.u;
        const int u = page_u + lane;
        page = u < pages ? p.pg.table[static_cast<size_t>(page_b) * p.pg.width + (u < ahead.s.sb ? u : ahead.s.wb + u - ahead.s.sb)]
                         : -1;
      }
      const int id = __shfl_sync(0xffffffffu, page, ahead.u - page_u);
      if (static_cast<unsigned>(id) < static_cast<unsigned>(p.pg.pages)) {
        const size_t plane = static_cast<size_t>(id) * p.Hk + ahead.hk;
        const uint8_t* k = p.pg.k + plane * (kPageRows * M) + 16 * lane;
        const uint8_t* v = p.pg.v + plane * (kPageRows * DV) + 16 * lane;
#pragma unroll
        for (int i = 0; i < M / 8; ++i) copy16(st + 16 * lane + 512 * i, k + 512 * i);
#pragma unroll
        for (int i = 0; i < DV / 8; ++i) copy16(st + P::kVAt + 16 * lane + 512 * i, v + 512 * i);
        if (lane < 2) copy4(st + P::kMeta + 4 * lane, (lane ? p.pg.vs : p.pg.ks) + plane);
      } else if (lane == 0) {
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(st + P::kMeta), "f"(-1.f) : "memory");
      }
    } else {
      const int row0 = (ahead.u - pages) * kOpen, n = min(kOpen, ahead.s.open - row0);
      const int key0 = ahead.s.blocks * kPageRows + row0;
      const size_t first = (static_cast<size_t>(ahead.b) * p.Hk + ahead.hk) * p.cap + row0;
      const uint16_t* k = p.kc + first * M;
      const __nv_bfloat16* v = p.vc + first * DV;
#pragma unroll
      for (int i = lane; i < kOpen * (M / 8); i += 32) {
        const int row = i / (M / 8), c = i % (M / 8);
        if (row < n) copy16(st + row * P::kKRow + 16 * c, k + static_cast<size_t>(row) * M + 8 * c);
      }
#pragma unroll
      for (int i = lane; i < kOpen * (DV / 8); i += 32) {
        const int row = i / (DV / 8), c = i % (DV / 8);
        const uint32_t to = st + P::kVOpen + row * P::kVRow + 16 * c;
        // a masked row may hold anything: its weight is 0, and so are its values here
        if (row < n && (key0 + row >= ahead.s.lo || key0 + row < p.sink))
          copy16(to, v + static_cast<size_t>(row) * DV + 8 * c);
        else
          st_shared_v4(to, 0u, 0u, 0u, 0u);
      }
      if (lane < n) copy4(st + P::kMeta + 4 * lane, p.kc_mul + first + lane);
    }
    if (++copied < units) ahead.next(p, w.parts);
  };
#pragma unroll 1
  for (int i = 0; i < ST - 1; ++i) {
    if (copied < units) copy();
    copies_commit();
  }
  ds::wait_for_previous();  // the queries

  Query<M, NT> qf;
  State<DV, NT> x;
  for (int i = 0; i < units; ++i) {
    if (copied < units) copy();  // into the slot that the unit before has left
    copies_commit();
    if (i == 0 || at.u == 0) {
      load_query<M, DV, NT>(p, w, at, r, q, qf, x);
      x.clear();
    }
    copies_wait<ST - 1>();
    __syncwarp();
    const uint8_t* st = smem_raw + (warp * ST + i % ST) * P::kStage;
    if (at.u < at.pages()) page_unit<M, DV, NT>(p, at, st, r, q, qf, x);
    else open_unit<M, DV, NT>(p, at, st, lane, r, q, qf, x);
    __syncwarp();  // every lane has read the slot
    if (i + 1 == units || at.u + 1 == at.s.units) {  // the segment's sums
      const size_t slot = (static_cast<size_t>(at.b) * p.Hk + at.hk) * w.parts + at.part + worker;
      const int heads = min(w.rows, p.G - at.part * w.rows);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float sum = x.sum[t][e];
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          const int row = 8 * t + 2 * q + e;
          if (row < heads) {
            float* o = w.o + (slot * w.rows + row) * DV + r;
#pragma unroll
            for (int c = 0; c < DV / 16; ++c) {
              o[16 * c] = x.o[t][c][e];
              o[16 * c + 8] = x.o[t][c][2 + e];
            }
            if (r == 0) w.ml[slot * w.rows + row] = make_float2(x.top[t][e], sum);
          }
        }
    }
    if (i + 1 < units) at.next(p, w.parts);
  }
  copies_wait<0>();
}

// ------------------------------------------------------------------ joining
// `warps` warps per row, each every warps-th part of it; a lane per DV / 32 columns.
template <int DV>
__global__ void __launch_bounds__(kJoinThreads) decode8_combine_kernel(const Decode8Params p, const Work w, int warps) {
  constexpr int C = DV / 32, kRows = kJoinThreads / 32;
  __shared__ float part[kRows][DV], tops[kRows], totals[kRows];
  __shared__ long long starts_at[kJoinThreads], sums[kRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x * (kRows / warps) + warp / warps, mine = warp % warps;
  float top = -INFINITY, sum = 0.f, o[C] = {};
  const bool live = row < p.B * p.H;
  // Which workers had a part of the row: found from the lengths while the keys' kernel ends,
  // or with more sequences than threads, of which every block would walk all, from its sums
  // (4096 sequences of 100 to 600 keys: 190 us for 136).
  const int per_seq = p.Hk * w.parts, b = live ? row / p.H : 0, h = row - b * p.H, hk = h / p.G, g = h - hk * p.G;
  const int in_seq = hk * w.parts + g / w.rows;
  long long off, n, total;
  const bool few = p.B <= kJoinThreads;
  if (few) {
    starts_at[threadIdx.x] = units_in_front<kJoinThreads>(p, sums, total);
    __syncthreads();
    off = starts_at[b];
    n = seq_of(p, b).units;
  } else {
    ds::wait_for_previous();
    off = w.off[b];
    n = w.off[b + 1] - off;
    total = w.off[p.B];
  }
  int w0 = 0, w1 = -1;
  if (live && n > 0) {
    const long long x0 = off * per_seq + in_seq * n, all = total * per_seq;
    const int busy = at_work(all, w.workers);
    w0 = owner(x0, all, busy);
    w1 = owner(x0 + n - 1, all, busy);
  }
  const size_t first = (static_cast<size_t>(b) * per_seq + in_seq) * w.rows + g % w.rows;
  if (few) ds::wait_for_previous();
#pragma unroll 4
  for (int i = w0 + mine; i <= w1; i += warps) {
    const size_t at = first + static_cast<size_t>(i) * w.rows;
    const float2 ml = w.ml[at];
    float v[C];
    if constexpr (C == 4) {
      const float4 f = *reinterpret_cast<const float4*>(w.o + at * DV + 4 * lane);
      v[0] = f.x;
      v[1] = f.y;
      v[2] = f.z;
      v[3] = f.w;
    } else {
      const float2 f = *reinterpret_cast<const float2*>(w.o + at * DV + 2 * lane);
      v[0] = f.x;
      v[1] = f.y;
    }
    const float now = fmaxf(top, ml.x), base = now == -INFINITY ? 0.f : now;
    const float a = ex2(top - base), c = ex2(ml.x - base);
    top = now;
    sum = sum * a + ml.y * c;
#pragma unroll
    for (int k = 0; k < C; ++k) o[k] = o[k] * a + v[k] * c;
  }
  if (warps > 1) {
#pragma unroll
    for (int k = 0; k < C; ++k) part[warp][C * lane + k] = o[k];
    if (lane == 0) {
      tops[warp] = top;
      totals[warp] = sum;
    }
    __syncthreads();
    if (mine || !live) return;
    for (int i = 0; i < warps; ++i) top = fmaxf(top, tops[warp + i]);
    const float base = top == -INFINITY ? 0.f : top;
    sum = 0.f;
#pragma unroll
    for (int k = 0; k < C; ++k) o[k] = 0.f;
    for (int i = 0; i < warps; ++i) {
      const float f = ex2(tops[warp + i] - base);
      sum += totals[warp + i] * f;
#pragma unroll
      for (int k = 0; k < C; ++k) o[k] = fmaf(part[warp + i][C * lane + k], f, o[k]);
    }
  } else if (!live) {
    return;
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;  // a row without keys: 0
  uint32_t* out = reinterpret_cast<uint32_t*>(p.out + static_cast<size_t>(row) * DV) + C / 2 * lane;
#pragma unroll
  for (int k = 0; k < C; k += 2) out[k / 2] = pack_bf16x2(o[k] * inv, o[k + 1] * inv);
}

template <int M, int DV, int NT>
cudaError_t launch_keys(const Decode8Params& p, const Work& w, int ctas, cudaStream_t stream) {
  using P = Plan<M, DV, NT>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = ds::allow_smem(decode8_kernel<M, DV, NT>, P::kBytes, done);
  if (e != cudaSuccess) return e;
  return ds::launch_after(decode8_kernel<M, DV, NT>, ctas, 32 * P::kWarps, P::kBytes, stream, p, w);
}

template <int M>
int warps_for(const Decode8Params& p) {
  if (p.dv == 64) return p.G > 8 ? Plan<M, 64, 2>::kWarps : Plan<M, 64, 1>::kWarps;
  return p.G > 8 ? Plan<M, 128, 2>::kWarps : Plan<M, 128, 1>::kWarps;
}
// Workers of a CTA.
int warps_for(const Decode8Params& p) {
  switch (p.m) {
    case 16: return warps_for<16>(p);
    case 32: return warps_for<32>(p);
    case 64: return warps_for<64>(p);
    default: return warps_for<128>(p);
  }
}

template <int M>
cudaError_t launch_t(const Decode8Params& p, const Work& w, int ctas, cudaStream_t stream) {
  // a plain launch, behind everything in the stream: the kernels after it copy the cache and
  // write the workspace without waiting for more than this one
  decode8_query_kernel<M><<<dim3((p.B * p.G + kQueryRows - 1) / kQueryRows, p.Hk), kQueryThreads, 0, stream>>>(p, w);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (p.dv == 64)
    return w.rows == 8 ? launch_keys<M, 64, 1>(p, w, ctas, stream) : launch_keys<M, 64, 2>(p, w, ctas, stream);
  return w.rows == 8 ? launch_keys<M, 128, 1>(p, w, ctas, stream) : launch_keys<M, 128, 2>(p, w, ctas, stream);
}

}  // namespace

size_t decode8_workspace(const Decode8Params& p) {
  Work w;
  return lay_out(p, kMaxCtas * warps_for(p), &w);
}

cudaError_t launch_decode8(const Decode8Params& p, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  const int ctas = sms < kMaxCtas ? sms : kMaxCtas, per = warps_for(p);
  Work w;
  lay_out(p, ctas * per, &w);
  switch (p.m) {
    case 16: e = launch_t<16>(p, w, ctas, stream); break;
    case 32: e = launch_t<32>(p, w, ctas, stream); break;
    case 64: e = launch_t<64>(p, w, ctas, stream); break;
    case 128: e = launch_t<128>(p, w, ctas, stream); break;
    default: return cudaErrorInvalidValue;
  }
  if (e != cudaSuccess) return e;
  // parts of a row on average, if every worker has units: a warp for each four of them
  const long long parts = w.workers / (static_cast<long long>(p.B) * p.Hk * w.parts) + 1;
  int warps = 1;
  while (warps < 8 && 4 * warps < parts) warps *= 2;
  const int rows = kJoinThreads / 32 / warps;
  const unsigned grid = (p.B * p.H + rows - 1) / rows;
  return p.dv == 64 ? ds::launch_after(decode8_combine_kernel<64>, grid, kJoinThreads, 0, stream, p, w, warps)
                    : ds::launch_after(decode8_combine_kernel<128>, grid, kJoinThreads, 0, stream, p, w, warps);
}

}  // namespace spa
