// spa_api.cu -- the C ABI of libspa.so (declared in include/spa.h): argument
// validation, workspace layout, tensor-map encoding, launches and status codes.
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include "../../include/spa.h"
#include "kernels.cuh"

namespace {

using spa::ProjOut;

// Device word set by a kernel that gave up on a bounded wait.
__device__ int g_spa_device_error;

constexpr int kMaxDevices = 64;
int* g_err_ptr[kMaxDevices] = {};
std::mutex g_err_mu;

int device_error_ptr(int** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return SPA_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_err_mu);
  if (!g_err_ptr[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_spa_device_error) != cudaSuccess) return SPA_ERR_CUDA;
    g_err_ptr[dev] = static_cast<int*>(p);
  }
  *out = g_err_ptr[dev];
  return SPA_OK;
}

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

int get_encode(PFN_cuTensorMapEncodeTiled_v12000* fn) {
  std::call_once(g_encode_once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  *fn = g_encode;
  return g_encode ? SPA_OK : SPA_ERR_CUDA;
}

constexpr int kEmpty = -1;  // internal: nothing to do

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Shape / dtype checks shared by every forward entry point.
int check_shape(int B, int H, int N, int d, int m, int dv, int dtype) {
  if (B < 0 || H < 0 || N < 0 || d < 0 || m < 0 || dv < 0) return SPA_ERR_SHAPE;
  if (dtype != SPA_F32 && dtype != SPA_BF16) return SPA_ERR_DTYPE;
  if (static_cast<long long>(B) * H * N == 0) return kEmpty;
  if (static_cast<long long>(B) * H > 65535) return SPA_ERR_SHAPE;
  if (d < 1 || d > 256 || m < 1 || m > 128 || dv < 1 || dv > 256) return SPA_ERR_UNSUPPORTED;
  if (dtype == SPA_BF16) {
    if (m != 16 && m != 32 && m != 64 && m != 128) return SPA_ERR_UNSUPPORTED;
    if (dv != 64 && dv != 128) return SPA_ERR_UNSUPPORTED;
  }
  return SPA_OK;
}

struct Layout {
  int NT = 0, KD = 0;
  ProjOut mode = ProjOut::F32;
  size_t qs = 0, ks = 0, qmul = 0, kmul = 0;  // bf16 path
  size_t qp = 0, kp = 0;                      // fp32 path
  size_t total = 0;
};

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

Layout make_layout(int B, int H, int N, int m, int dtype) {
  Layout L;
  const size_t BH = static_cast<size_t>(B) * H;
  if (dtype == SPA_BF16) {
    L.NT = (N + spa::kTileRows - 1) / spa::kTileRows;
    L.mode = m == 16 ? ProjOut::BF16X3 : ProjOut::F16X1;
    L.KD = spa::score_depth(m, L.mode);
    const size_t tiles = BH * L.NT * spa::kTileRows * L.KD * 2;
    L.qs = 0;
    L.ks = align256(L.qs + tiles);
    L.qmul = align256(L.ks + tiles);
    L.kmul = align256(L.qmul + BH * L.NT * spa::kTileRows * sizeof(float));
    L.total = align256(L.kmul + BH * L.NT * sizeof(float));
  } else {
    const size_t proj = BH * N * m * sizeof(float);
    L.qp = 0;
    L.kp = align256(proj);
    L.total = align256(L.kp + proj);
  }
  return L;
}

int cuda_status(cudaError_t e) { return e == cudaSuccess ? SPA_OK : SPA_ERR_CUDA; }

spa::ProjParams proj_params(const void* q, const void* k, const void* P, int B, int H, int N,
                            int d, int m, int dtype, const Layout& L, char* w) {
  spa::ProjParams pp{};
  pp.x[0] = q;
  pp.x[1] = k;
  pp.P = P;
  pp.nx = 2;
  pp.BH = B * H;
  pp.H = H;
  pp.N = N;
  pp.d = d;
  pp.m = m;
  pp.bf16_in = dtype == SPA_BF16;
  pp.NT = (N + spa::kTileRows - 1) / spa::kTileRows;
  if (dtype == SPA_F32) {
    pp.mode = ProjOut::F32;
    pp.out[0] = w + L.qp;
    pp.out[1] = w + L.kp;
  } else {
    pp.mode = L.mode;
    pp.out[0] = w + L.qs;
    pp.out[1] = w + L.ks;
    pp.mul[0] = reinterpret_cast<float*>(w + L.qmul);
    pp.mul[1] = reinterpret_cast<float*>(w + L.kmul);
    // scores come out in base-2 logits: fold log2(e) / sqrt(m) into Q
    pp.qscale = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(m)));
  }
  return pp;
}

// Row-major [BH][N][inner] tensor as a 3-D tensor map with 128-byte swizzle and
// 128-row boxes whose inner extent is 128 bytes (64 bf16 or 32 fp32 values).
int encode_rows_map(CUtensorMap* map, const void* base, int inner, int N, int BH,
                    CUtensorMapDataType type, int elem_bytes) {
  PFN_cuTensorMapEncodeTiled_v12000 encode;
  int st = get_encode(&encode);
  if (st) return st;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(N),
                        static_cast<cuuint64_t>(BH)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(inner) * elem_bytes,
                           static_cast<cuuint64_t>(N) * inner * elem_bytes};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / elem_bytes),
                       static_cast<cuuint32_t>(spa::kTileRows), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  if (encode(map, type, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return SPA_ERR_CUDA;
  return SPA_OK;
}
int encode_bf16_rows(CUtensorMap* map, const void* base, int inner, int N, int BH) {
  return encode_rows_map(map, base, inner, N, BH, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2);
}

// Stage 1: projection of q and k into the workspace (and, for the backward,
// plain bf16 tiles of Qp and Kp into qb, kb in the same pass).
int run_prepare(const void* q, const void* k, const void* P, int B, int H, int N, int d, int m,
                int dtype, void* ws, cudaStream_t stream, void* qb = nullptr, void* kb = nullptr,
                unsigned long long limit_ns = 0, int inject_stall = 0) {
  const Layout L = make_layout(B, H, N, m, dtype);
  spa::ProjParams pp = proj_params(q, k, P, B, H, N, d, m, dtype, L, static_cast<char*>(ws));
  pp.use_tc = 1;
  pp.out_b16[0] = qb;
  pp.out_b16[1] = kb;
  pp.limit_ns = limit_ns;
  pp.inject_stall = inject_stall;
  if (spa::project_tc_eligible(pp)) {
    int st;
    if ((st = encode_bf16_rows(&pp.xmap[0], q, d, N, B * H))) return st;
    if ((st = encode_bf16_rows(&pp.xmap[1], k, d, N, B * H))) return st;
    if ((st = device_error_ptr(&pp.err))) return st;
  }
  return cuda_status(spa::launch_project(pp, stream));
}

// Stage 2: scores, mask, online softmax and the value product from a prepared workspace.
constexpr unsigned long long kWaitLimitNs = 2000000000ull;  // 2 s per wait

int run_apply(const void* v, float* out, int B, int H, int N, int m, int dv, int causal,
              int dtype, const void* ws, cudaStream_t stream,
              unsigned long long limit_ns = kWaitLimitNs, int inject_stall = 0,
              float* lse = nullptr) {
  const Layout L = make_layout(B, H, N, m, dtype);
  const int BH = B * H;
  const char* w = static_cast<const char*>(ws);
  if (dtype == SPA_F32) {
    spa::AttnF32Params ap{};
    ap.Qp = reinterpret_cast<const float*>(w + L.qp);
    ap.Kp = reinterpret_cast<const float*>(w + L.kp);
    ap.V = static_cast<const float*>(v);
    ap.out = out;
    ap.BH = BH;
    ap.N = N;
    ap.m = m;
    ap.dv = dv;
    ap.causal = causal != 0;
    ap.scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(m)));
    ap.lse = lse;
    return cuda_status(spa::launch_attn_f32(ap, stream));
  }
  int st;
  spa::AttnTcParams ap{};
  if ((st = encode_bf16_rows(&ap.vmap, v, dv, N, BH))) return st;
  if ((st = encode_rows_map(&ap.omap, out, dv, N, BH, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4)))
    return st;
  int* err = nullptr;
  if ((st = device_error_ptr(&err))) return st;
  ap.Qs = reinterpret_cast<const uint16_t*>(w + L.qs);
  ap.Ks = reinterpret_cast<const uint16_t*>(w + L.ks);
  ap.qmul = reinterpret_cast<const float*>(w + L.qmul);
  ap.kmul = reinterpret_cast<const float*>(w + L.kmul);
  ap.out = out;
  ap.err = err;
  ap.BH = BH;
  ap.N = N;
  ap.NT = L.NT;
  ap.KD = L.KD;
  ap.dv = dv;
  ap.causal = causal != 0;
  ap.f16_ops = L.mode == ProjOut::F16X1;
  ap.limit_ns = limit_ns;
  ap.inject_stall = inject_stall;
  ap.lse = lse;
  return cuda_status(spa::launch_attn_ws(ap, stream));
}

int run_forward(const void* q, const void* k, const void* v, const void* P, float* out, int B,
                int H, int N, int d, int m, int dv, int causal, int dtype, void* ws,
                cudaStream_t stream) {
  int st = run_prepare(q, k, P, B, H, N, d, m, dtype, ws, stream);
  if (st) return st;
  return run_apply(v, out, B, H, N, m, dv, causal, dtype, ws, stream);
}

int check_forward_ptrs(const void* q, const void* k, const void* v, const void* P,
                       const void* out) {
  if (!q || !k || !v || !P || !out) return SPA_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(P) || !aligned16(out))
    return SPA_ERR_ALIGN;
  return SPA_OK;
}

}  // namespace

namespace {

// Host-buffer forward, pipelined over chunks of whole heads of one batch
// entry: chunk c is copied in, projected, attended and copied out on stream
// slot c % kHostSlots, so the copy engines bring chunk c+1 in and take chunk
// c-1 out while chunk c computes.  Heads are independent, and a chunk of heads
// [h0, h0+n) of batch entry b is the problem (B=1, H=n) on the matching slices
// of q, k, v, out and P.
constexpr int kHostSlots = 4;

// The host-buffer forward's device staging comes from a pool of the library's
// own, one per device, which keeps what it has reserved between calls (the
// default pool hands memory back to the driver at every synchronisation, and
// reserving a few GB again costs more than the copies it stages).
cudaMemPool_t g_host_pool[kMaxDevices] = {};
std::mutex g_host_pool_mu;

int host_pool(cudaMemPool_t* out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return SPA_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_host_pool_mu);
  if (!g_host_pool[dev]) {
    cudaMemPoolProps props = {};
    props.allocType = cudaMemAllocationTypePinned;
    props.location.type = cudaMemLocationTypeDevice;
    props.location.id = dev;
    cudaMemPool_t pool = nullptr;
    if (cudaMemPoolCreate(&pool, &props) != cudaSuccess) {
      cudaGetLastError();
      return SPA_ERR_CUDA;
    }
    uint64_t keep = UINT64_MAX;
    if (cudaMemPoolSetAttribute(pool, cudaMemPoolAttrReleaseThreshold, &keep) != cudaSuccess) {
      cudaGetLastError();
      cudaMemPoolDestroy(pool);
      return SPA_ERR_CUDA;
    }
    g_host_pool[dev] = pool;
  }
  *out = g_host_pool[dev];
  return SPA_OK;
}
// Stream-ordered workspace from the library's pool: it keeps what it has
// reserved across synchronisations, so calls in a synchronised loop do not
// reserve device memory again (with the default pool, which hands memory back
// at every synchronisation, the allocating forward took 0.64 ms per call on C3
// against 0.36 ms on a caller workspace).  Released with cudaFreeAsync.
int pool_alloc(void** p, size_t bytes, cudaStream_t s) {
  cudaMemPool_t pool = nullptr;
  if (host_pool(&pool) != SPA_OK) return SPA_ERR_CUDA;
  if (cudaMallocFromPoolAsync(p, bytes, pool, s) != cudaSuccess) {
    cudaGetLastError();
    return SPA_ERR_NOMEM;
  }
  return SPA_OK;
}

// The host-buffer forward's internal streams, created once per device and kept
// until the process exits (creating and destroying them took about 0.05 ms of
// every call).  Calls from several threads may share them: each call orders
// its chunks after its own stream with its own events, so sharing only adds
// ordering between calls.
cudaStream_t g_host_streams[kMaxDevices][kHostSlots] = {};

int host_streams(cudaStream_t (&out)[kHostSlots]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return SPA_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_host_pool_mu);
  for (int j = 0; j < kHostSlots; ++j) {
    if (!g_host_streams[dev][j] &&
        cudaStreamCreateWithFlags(&g_host_streams[dev][j], cudaStreamNonBlocking) != cudaSuccess) {
      cudaGetLastError();
      g_host_streams[dev][j] = nullptr;
      return SPA_ERR_CUDA;
    }
    out[j] = g_host_streams[dev][j];
  }
  return SPA_OK;
}
constexpr size_t kHostChunkBytes = size_t(32) << 20;  // aim for at least this per chunk
// at most this many chunks (C4 shape: one head per chunk; measured on GB300,
// four slots and up to 32 chunks 8.81 ms per forward, three slots and 16
// chunks 9.13 ms)
constexpr int kHostMaxChunks = 32;

int host_forward(const char* q, const char* k, const char* v, const char* P, float* out, int B,
                 int H, int N, int d, int m, int dv, int causal, int dtype, cudaStream_t stream) {
  const size_t es = dtype == SPA_BF16 ? 2 : 4;
  const size_t head_in = static_cast<size_t>(N) * (2 * d + dv) * es;
  const size_t head_out = static_cast<size_t>(N) * dv * sizeof(float);
  const size_t total_heads = static_cast<size_t>(B) * H;
  const size_t want = (total_heads * (head_in + head_out)) / kHostChunkBytes;
  const size_t nchunks = want < 1 ? 1 : (want > kHostMaxChunks ? kHostMaxChunks : want);
  size_t per = (total_heads + nchunks - 1) / nchunks;
  const int nh = static_cast<int>(per < 1 ? 1 : (per > static_cast<size_t>(H) ? H : per));

  // one slot: q, k, v, P slices, out slice and the workspace for nh heads
  const size_t nq = static_cast<size_t>(nh) * N * d * es, nv = static_cast<size_t>(nh) * N * dv * es;
  const size_t np = static_cast<size_t>(nh) * d * m * es, no = static_cast<size_t>(nh) * N * dv * 4;
  const size_t oq = 0, ok = align256(oq + nq), ov = align256(ok + nq), op = align256(ov + nv),
               oo = align256(op + np), ow = align256(oo + no);
  const size_t slot_bytes = align256(ow + make_layout(1, nh, N, m, dtype).total);

  cudaStream_t ss[kHostSlots] = {};
  cudaEvent_t ev_begin = nullptr, ev_end[kHostSlots] = {};
  char* dbuf = nullptr;
  int st = SPA_OK;
  auto fail = [&](cudaError_t e) {
    if (e != cudaSuccess && st == SPA_OK) st = SPA_ERR_CUDA;
    return e != cudaSuccess;
  };
  cudaMemPool_t pool = nullptr;
  if (host_pool(&pool) != SPA_OK || host_streams(ss) != SPA_OK) return SPA_ERR_CUDA;
  if (cudaMallocFromPoolAsync(reinterpret_cast<void**>(&dbuf), kHostSlots * slot_bytes, pool,
                              stream) != cudaSuccess) {
    cudaGetLastError();
    return SPA_ERR_NOMEM;
  }
  bool ready = !fail(cudaEventCreateWithFlags(&ev_begin, cudaEventDisableTiming)) &&
               !fail(cudaEventRecord(ev_begin, stream));
  for (int j = 0; ready && j < kHostSlots; ++j)
    ready = !fail(cudaEventCreateWithFlags(&ev_end[j], cudaEventDisableTiming)) &&
            !fail(cudaStreamWaitEvent(ss[j], ev_begin, 0));
  int c = 0;
  for (int b = 0; ready && st == SPA_OK && b < B; ++b) {
    for (int h0 = 0; st == SPA_OK && h0 < H; h0 += nh, ++c) {
      const int n = H - h0 < nh ? H - h0 : nh;
      cudaStream_t sj = ss[c % kHostSlots];
      char* sb = dbuf + (c % kHostSlots) * slot_bytes;
      const size_t head0 = static_cast<size_t>(b) * H + h0;
      const size_t cq = static_cast<size_t>(n) * N * d * es, cv = static_cast<size_t>(n) * N * dv * es;
      if (fail(cudaMemcpyAsync(sb + oq, q + head0 * N * d * es, cq, cudaMemcpyHostToDevice, sj)) ||
          fail(cudaMemcpyAsync(sb + ok, k + head0 * N * d * es, cq, cudaMemcpyHostToDevice, sj)) ||
          fail(cudaMemcpyAsync(sb + ov, v + head0 * N * dv * es, cv, cudaMemcpyHostToDevice, sj)) ||
          fail(cudaMemcpyAsync(sb + op, P + static_cast<size_t>(h0) * d * m * es,
                               static_cast<size_t>(n) * d * m * es, cudaMemcpyHostToDevice, sj)))
        break;
      st = run_forward(sb + oq, sb + ok, sb + ov, sb + op, reinterpret_cast<float*>(sb + oo), 1, n,
                       N, d, m, dv, causal, dtype, sb + ow, sj);
      if (st) break;
      if (fail(cudaMemcpyAsync(out + head0 * N * dv, sb + oo, static_cast<size_t>(n) * N * dv * 4,
                               cudaMemcpyDeviceToHost, sj)))
        break;
    }
  }
  // join every slot back into the caller's stream, release, and wait
  for (int j = 0; j < kHostSlots; ++j)
    if (ss[j] && ev_end[j] && !fail(cudaEventRecord(ev_end[j], ss[j])))
      fail(cudaStreamWaitEvent(stream, ev_end[j], 0));
  fail(cudaFreeAsync(dbuf, stream));
  fail(cudaStreamSynchronize(stream));
  for (int j = 0; j < kHostSlots; ++j)
    if (ev_end[j]) cudaEventDestroy(ev_end[j]);
  if (ev_begin) cudaEventDestroy(ev_begin);
  return st;
}

// ---------------------------------------------------------------- fused backward
// Workspace of the fused backward: the forward's prepared operands (so that
// the recomputed scores are bit-identical to the forward's), bf16 Qp / Kp
// tiles for the gradient products, the row statistics, the fp32 dQp and dKp
// accumulators (tile layout of bwd_common.cuh), and (when the caller has no
// log-sum-exp) lse plus a scratch output.
struct BwdLayout {
  Layout fwd;
  size_t qb = 0, kb = 0, stats = 0, dqacc = 0, dkacc = 0;
  size_t lse = 0, out2 = 0, total = 0;
};

BwdLayout make_bwd_layout(int B, int H, int N, int d, int m, int dv, bool own_lse) {
  BwdLayout L;
  L.fwd = make_layout(B, H, N, m, SPA_BF16);
  const size_t BH = static_cast<size_t>(B) * H, rows = BH * L.fwd.NT * spa::kTileRows;
  size_t o = L.fwd.total;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align256(o + bytes);
    return at;
  };
  L.qb = take(rows * m * 2);
  L.kb = take(rows * m * 2);
  L.stats = take(rows * 4 * sizeof(float));
  L.dqacc = take(rows * m * sizeof(float));
  L.dkacc = take(rows * m * sizeof(float));
  if (own_lse) {
    L.lse = take(BH * N * sizeof(float));
    L.out2 = take(BH * N * dv * sizeof(float));
  }
  L.total = o;
  return L;
}

// The tensor-core backward (fused kernel and one-pass finish); every other
// shape runs on CUDA cores (run_backward_simt).
bool bwd_fused_eligible(int d, int m, int dv, int dtype) {
  return dtype == SPA_BF16 && spa::bwd_tc_supported(m, dv) && spa::bwd_finish_tc_supported(d, m);
}

// Fused backward, stage 1 on a workspace laid out by make_bwd_layout, after
// run_prepare (given the layout's qb / kb) has put the forward's score operands
// and the bf16 Qp / Kp tiles in it: the zeroed dQp accumulator and the row
// statistics.
int bwd_stage_inputs(const float* out, const float* lse, const void* dO, int B, int H, int N,
                     int d, int m, int d_v, char* w, cudaStream_t stream,
                     unsigned long long limit_ns = kWaitLimitNs, int inject_stall = 0) {
  const BwdLayout L = make_bwd_layout(B, H, N, d, m, d_v, false);
  const int BH = B * H, NT = L.fwd.NT;
  int st;
  const float alpha = static_cast<float>(1.0 / std::sqrt(static_cast<double>(m)));
  if ((st = cuda_status(cudaMemsetAsync(w + L.dqacc, 0,
                                        static_cast<size_t>(BH) * NT * spa::kTileRows * m *
                                            sizeof(float),
                                        stream))))
    return st;
  spa::BwdStatsMaps maps{};
  if ((st = encode_bf16_rows(&maps.domap, dO, d_v, N, BH)) ||
      (st = encode_rows_map(&maps.omap, out, d_v, N, BH, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4)) ||
      (st = device_error_ptr(&maps.err)))
    return st;
  maps.limit_ns = limit_ns;
  maps.inject_stall = inject_stall;
  return cuda_status(spa::launch_bwd_stats(
      maps, lse, reinterpret_cast<const float*>(w + L.fwd.qmul),
      reinterpret_cast<float*>(w + L.stats), BH, N, NT, d_v, alpha, stream));
}

// Fused backward, stage 2: the tensor-core kernel (dV, dKp, dQp).
int bwd_stage_kernel(const void* v, const void* dO, float* dv, int B, int H, int N, int d, int m,
                     int d_v, int causal, char* w, cudaStream_t stream,
                     unsigned long long limit_ns = kWaitLimitNs, int inject_stall = 0) {
  const BwdLayout L = make_bwd_layout(B, H, N, d, m, d_v, false);
  const int BH = B * H;
  int st;
  spa::BwdTcParams bp{};
  if ((st = encode_bf16_rows(&bp.vmap, v, d_v, N, BH))) return st;
  if ((st = encode_bf16_rows(&bp.domap, dO, d_v, N, BH))) return st;
  if ((st = device_error_ptr(&bp.err))) return st;
  bp.Qs = reinterpret_cast<const uint16_t*>(w + L.fwd.qs);
  bp.Ks = reinterpret_cast<const uint16_t*>(w + L.fwd.ks);
  bp.kmul = reinterpret_cast<const float*>(w + L.fwd.kmul);
  bp.Qb = reinterpret_cast<const uint16_t*>(w + L.qb);
  bp.Kb = reinterpret_cast<const uint16_t*>(w + L.kb);
  bp.stats = reinterpret_cast<const float*>(w + L.stats);
  bp.dqacc = reinterpret_cast<float*>(w + L.dqacc);
  bp.dkacc = reinterpret_cast<float*>(w + L.dkacc);
  bp.dv_out = dv;
  bp.BH = BH;
  bp.N = N;
  bp.NT = L.fwd.NT;
  bp.KD = L.fwd.KD;
  bp.m = m;
  bp.dv = d_v;
  bp.causal = causal != 0;
  bp.f16_ops = L.fwd.mode == ProjOut::F16X1;
  bp.alpha = static_cast<float>(1.0 / std::sqrt(static_cast<double>(m)));
  bp.limit_ns = limit_ns;
  bp.inject_stall = inject_stall;
  return cuda_status(spa::launch_bwd_tc(bp, stream));
}

// Fused backward, stage 3: dq, dk and dP from dQp and dKp (one tensor-core pass).
int bwd_stage_finish(const void* q, const void* k, const void* P, float* dq, float* dk, float* dP,
                     int B, int H, int N, int d, int m, int d_v, char* w, cudaStream_t stream,
                     unsigned long long limit_ns = kWaitLimitNs, int inject_stall = 0) {
  const BwdLayout L = make_bwd_layout(B, H, N, d, m, d_v, false);
  const int BH = B * H;
  int st;
  spa::BwdFinishParams fp{};
  if ((st = encode_bf16_rows(&fp.qmap, q, d, N, BH)) ||
      (st = encode_bf16_rows(&fp.kmap, k, d, N, BH)) ||
      (st = encode_rows_map(&fp.dqmap, dq, d, N, BH, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4)) ||
      (st = encode_rows_map(&fp.dkmap, dk, d, N, BH, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4)) ||
      (st = device_error_ptr(&fp.err)))
    return st;
  fp.dqacc = reinterpret_cast<const float*>(w + L.dqacc);
  fp.dkacc = reinterpret_cast<const float*>(w + L.dkacc);
  fp.P = static_cast<const __nv_bfloat16*>(P);
  fp.dP = dP;
  fp.B = B;
  fp.H = H;
  fp.N = N;
  fp.NT = L.fwd.NT;
  fp.d = d;
  fp.m = m;
  fp.limit_ns = limit_ns;
  fp.inject_stall = inject_stall;
  return cuda_status(spa::launch_bwd_finish_tc(fp, stream));
}

// The whole fused backward.  lse == NULL: the forward runs once more to
// produce it (into the layout's own lse and scratch output).
int run_backward_fused(const void* q, const void* k, const void* v, const void* P, const float* out,
                       const float* lse, const void* dO, float* dq, float* dk, float* dv,
                       float* dP, int B, int H, int N, int d, int m, int d_v, int causal, char* w,
                       cudaStream_t stream) {
  const BwdLayout L = make_bwd_layout(B, H, N, d, m, d_v, lse == nullptr);
  int st = run_prepare(q, k, P, B, H, N, d, m, SPA_BF16, w, stream, w + L.qb, w + L.kb);
  if (st) return st;
  if (lse == nullptr) {
    float* own = reinterpret_cast<float*>(w + L.lse);
    st = run_apply(v, reinterpret_cast<float*>(w + L.out2), B, H, N, m, d_v, causal, SPA_BF16, w,
                   stream, kWaitLimitNs, 0, own);
    if (st) return st;
    lse = own;
  }
  if ((st = bwd_stage_inputs(out, lse, dO, B, H, N, d, m, d_v, w, stream))) return st;
  if ((st = bwd_stage_kernel(v, dO, dv, B, H, N, d, m, d_v, causal, w, stream))) return st;
  return bwd_stage_finish(q, k, P, dq, dk, dP, B, H, N, d, m, d_v, w, stream);
}

// Checks shared by the staged entry points (fused shapes only).
int check_bwd_staged(int B, int H, int N, int d, int m, int d_v, int dtype, const void* ws,
                     size_t ws_bytes) {
  int st = check_shape(B, H, N, d, m, d_v, dtype);
  if (st) return st;
  if (!bwd_fused_eligible(d, m, d_v, dtype)) return SPA_ERR_UNSUPPORTED;
  if (!ws) return SPA_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(ws) & 255u) return SPA_ERR_ALIGN;
  if (ws_bytes < make_bwd_layout(B, H, N, d, m, d_v, false).total) return SPA_ERR_NOMEM;
  return SPA_OK;
}

// The backward on CUDA cores (fp32 inputs and the shapes the tensor-core
// kernels do not cover): flash-style, nothing N x N stored.  Workspace (from
// the library's pool): Qp, Kp, dQp, dKp in fp32, the row sums <dO_i, O_i>, the
// dP partials, and (without the caller's log-sum-exp) the forward's workspace,
// a scratch output and lse.
int run_backward_simt(const void* q, const void* k, const void* v, const void* P,
                      const float* out, const float* lse, const void* dO, float* dq, float* dk,
                      float* dv, float* dP, int B, int H, int N, int d, int m, int d_v, int causal,
                      int dtype, cudaStream_t s) {
  const size_t BH = static_cast<size_t>(B) * H, rows = BH * N;
  const int chunks = spa::bwd_simt_chunks(B, N);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align256(o + bytes);
    return at;
  };
  const size_t oqp = take(rows * m * 4), okp = take(rows * m * 4), odq = take(rows * m * 4),
               odk = take(rows * m * 4), ods = take(rows * 4),
               opart = take(static_cast<size_t>(H) * chunks * d * m * 4);
  size_t ofw = 0, oout = 0, olse = 0;
  if (!lse) {
    ofw = take(make_layout(B, H, N, m, dtype).total);
    oout = take(rows * d_v * 4);
    olse = take(rows * 4);
  }
  char* w = nullptr;
  if (int e = pool_alloc(reinterpret_cast<void**>(&w), o, s)) return e;
  int st = SPA_OK;
  if (!lse) {  // the forward once more, for its row log-sum-exp
    st = run_prepare(q, k, P, B, H, N, d, m, dtype, w + ofw, s);
    if (!st)
      st = run_apply(v, reinterpret_cast<float*>(w + oout), B, H, N, m, d_v, causal, dtype, w + ofw,
                     s, kWaitLimitNs, 0, reinterpret_cast<float*>(w + olse));
    lse = reinterpret_cast<const float*>(w + olse);
  }
  if (!st) {  // Qp and Kp in fp32
    spa::ProjParams pp{};
    pp.x[0] = q;
    pp.x[1] = k;
    pp.P = P;
    pp.out[0] = w + oqp;
    pp.out[1] = w + okp;
    pp.nx = 2;
    pp.BH = B * H;
    pp.H = H;
    pp.N = N;
    pp.d = d;
    pp.m = m;
    pp.NT = (N + spa::kTileRows - 1) / spa::kTileRows;
    pp.bf16_in = dtype == SPA_BF16;
    pp.mode = ProjOut::F32;
    st = cuda_status(spa::launch_project(pp, s));
  }
  if (!st) {
    spa::BwdSimtParams bp{};
    bp.q = q;
    bp.k = k;
    bp.v = v;
    bp.P = P;
    bp.dO = dO;
    bp.out = out;
    bp.lse = lse;
    bp.dq = dq;
    bp.dk = dk;
    bp.dv_out = dv;
    bp.dP = dP;
    bp.qp = reinterpret_cast<float*>(w + oqp);
    bp.kp = reinterpret_cast<float*>(w + okp);
    bp.dqp = reinterpret_cast<float*>(w + odq);
    bp.dkp = reinterpret_cast<float*>(w + odk);
    bp.dsum = reinterpret_cast<float*>(w + ods);
    bp.part = reinterpret_cast<float*>(w + opart);
    bp.B = B;
    bp.H = H;
    bp.N = N;
    bp.d = d;
    bp.m = m;
    bp.dv = d_v;
    bp.causal = causal != 0;
    bp.bf16 = dtype == SPA_BF16;
    bp.chunks = chunks;
    st = cuda_status(spa::launch_bwd_simt(bp, s));
  }
  const cudaError_t fe = cudaFreeAsync(w, s);
  if (st) return st;
  return cuda_status(fe);
}

// Shared by both backward entry points; lse may be NULL.
int backward_entry(const void* q, const void* k, const void* v, const void* P, const float* out,
                   const float* lse, const void* dO, float* dq, float* dk, float* dv, float* dP,
                   int B, int H, int N, int d, int m, int d_v, int causal, int dtype,
                   void* stream) {
  int st = check_shape(B, H, N, d, m, d_v, dtype);
  if (st == kEmpty) {
    if (!dP) return SPA_ERR_NULL;  // the projection gradient is still defined: zero
    if (H > 0 && d > 0 && m > 0 &&
        cudaMemsetAsync(dP, 0, static_cast<size_t>(H) * d * m * sizeof(float),
                        static_cast<cudaStream_t>(stream)) != cudaSuccess)
      return SPA_ERR_CUDA;
    return SPA_OK;
  }
  if (st) return st;
  if (d > 128) return SPA_ERR_UNSUPPORTED;
  if (!q || !k || !v || !P || !out || !dO || !dq || !dk || !dv || !dP) return SPA_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(P) || !aligned16(dO) ||
      !aligned16(out) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv) || !aligned16(dP))
    return SPA_ERR_ALIGN;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!bwd_fused_eligible(d, m, d_v, dtype))
    return run_backward_simt(q, k, v, P, out, lse, dO, dq, dk, dv, dP, B, H, N, d, m, d_v, causal,
                             dtype, s);
  const size_t bytes = make_bwd_layout(B, H, N, d, m, d_v, lse == nullptr).total;
  void* ws = nullptr;
  if (int e = pool_alloc(&ws, bytes, s)) return e;
  st = run_backward_fused(q, k, v, P, out, lse, dO, dq, dk, dv, dP, B, H, N, d, m, d_v, causal,
                          static_cast<char*>(ws), s);
  const cudaError_t fe = cudaFreeAsync(ws, s);
  if (st) return st;
  return cuda_status(fe);
}

// The Top-k prologue (spa_topk_features), with the wait limit and the
// failure-detection injection of the TMA kernel as parameters.
int topk_features(const void* x, void* y, long long rows, int d, int k, int dtype,
                  cudaStream_t stream, unsigned long long limit_ns = kWaitLimitNs,
                  int inject_stall = 0) {
  if (rows < 0 || d < 0 || k < 0) return SPA_ERR_SHAPE;
  if (dtype != SPA_F32 && dtype != SPA_BF16) return SPA_ERR_DTYPE;
  if (rows == 0) return SPA_OK;
  if (d != 32 && d != 64 && d != 128 && d != 256) return SPA_ERR_UNSUPPORTED;
  if (k < 1 || k > d) return SPA_ERR_SHAPE;
  if (!x || !y) return SPA_ERR_NULL;
  if (!aligned16(x) || !aligned16(y)) return SPA_ERR_ALIGN;
  spa::TopkParams tp{};
  tp.x = x;
  tp.y = y;
  tp.rows = rows;
  tp.d = d;
  tp.k = k;
  tp.bf16 = dtype == SPA_BF16;
  // bf16 rows of 64 or 128 features go through TMA (row coordinates are 32-bit)
  if (tp.bf16 && (d == 64 || d == 128) && rows <= 0x7fffff00LL) {
    int st;
    if ((st = encode_bf16_rows(&tp.xmap, x, d, static_cast<int>(rows), 1)) ||
        (st = encode_bf16_rows(&tp.ymap, y, d, static_cast<int>(rows), 1)) ||
        (st = device_error_ptr(&tp.err)))
      return st;
    tp.use_tma = 1;
    tp.limit_ns = limit_ns;
    tp.inject_stall = inject_stall;
  }
  return cuda_status(spa::launch_topk(tp, stream));
}

// Size checks of the shared-prefix decode.
int check_decode_shared(int B, int H, int Hk, int plen, int d, int m, int d_v, int cap) {
  if (B < 0 || H < 0 || Hk < 0 || plen < 0 || d < 0 || m < 0 || d_v < 0 || cap < 0)
    return SPA_ERR_SHAPE;
  if (static_cast<long long>(B) * H == 0) return kEmpty;
  if (Hk == 0 || H % Hk || static_cast<long long>(B) * H > 65535) return SPA_ERR_SHAPE;
  if (d < 1 || d > 256 || (m != 16 && m != 32 && m != 64 && m != 128) || (d_v != 64 && d_v != 128))
    return SPA_ERR_UNSUPPORTED;
  return SPA_OK;
}

int decode_shared_sizes(spa::DecodeSharedParams& dp, int B, int H, int Hk, int plen, int d, int m,
                        int d_v, int cap) {
  dp.B = B;
  dp.H = H;
  dp.Hk = Hk;
  dp.G = H / Hk;
  dp.plen = plen;
  dp.d = d;
  dp.m = m;
  dp.dv = d_v;
  dp.cap = cap;
  dp.qscale = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(m)));
  return spa::decode_shared_fits(dp) ? SPA_OK : SPA_ERR_SHAPE;
}

// Rows of a cache as a 3-D tensor map with boxes of `rows` rows and at most 64
// 16-bit features, swizzled over the box's row.
int encode_cache_map(CUtensorMap* map, const void* base, int inner, int cap, int heads, int rows,
                     CUtensorMapDataType type) {
  PFN_cuTensorMapEncodeTiled_v12000 encode;
  int st = get_encode(&encode);
  if (st) return st;
  const cuuint32_t width = inner < 64 ? inner : 64;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(cap),
                        static_cast<cuuint64_t>(heads)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(inner) * 2, static_cast<cuuint64_t>(cap) * inner * 2};
  cuuint32_t box[3] = {width, static_cast<cuuint32_t>(rows), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUtensorMapSwizzle swizzle = width == 16   ? CU_TENSOR_MAP_SWIZZLE_32B
                                     : width == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                   : CU_TENSOR_MAP_SWIZZLE_128B;
  if (encode(map, type, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return SPA_ERR_CUDA;
  return SPA_OK;
}

int run_decode_shared(const spa::DecodeSharedParams& dp, cudaStream_t stream,
                      unsigned long long limit_ns = kWaitLimitNs, int inject_stall = 0) {
  spa::DecodeSharedRun run{};
  int st, dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&run.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return SPA_ERR_CUDA;
  if ((st = device_error_ptr(&run.err))) return st;
  for (int own = 0; own < 2; ++own) {
    const int rows = own ? dp.cap : dp.plen, heads = own ? dp.B * dp.Hk : dp.Hk;
    if (rows == 0) continue;  // never loaded from
    for (int small = own && dp.G <= spa::kDecodeOwnGroup; small < 2; ++small)
      if ((st = encode_cache_map(&run.k[own][small], own ? dp.kc : dp.pkc, dp.m,
                                 own ? dp.cap : dp.pcap, heads, small ? 16 : 128,
                                 CU_TENSOR_MAP_DATA_TYPE_FLOAT16)) ||
          (st = encode_cache_map(&run.v[own][small], own ? dp.v : dp.pv, dp.dv,
                                 own ? dp.cap : dp.pcap, heads, small ? 16 : 128,
                                 CU_TENSOR_MAP_DATA_TYPE_BFLOAT16)))
        return st;
  }
  run.limit_ns = limit_ns;
  run.inject_stall = inject_stall;
  return cuda_status(spa::launch_decode_shared(dp, run, stream));
}

// ---------------------------------------------------------------- attention_window
int check_window(int B, int H, int Hk, int N, int d, int m, int dv, int window, int sink, int dtype) {
  if (B < 0 || H < 0 || Hk < 0 || N < 0 || d < 0 || m < 0 || dv < 0 || window < 0 || sink < 0) return SPA_ERR_SHAPE;
  if (dtype != SPA_F32 && dtype != SPA_BF16) return SPA_ERR_DTYPE;
  if (static_cast<long long>(B) * H * N == 0) return kEmpty;
  if (Hk == 0 || H % Hk || static_cast<long long>(B) * H > 65535 || N > (1 << 30)) return SPA_ERR_SHAPE;
  if (dtype != SPA_BF16 || (d != 64 && d != 128) || (m != 16 && m != 32 && m != 64) || (dv != 64 && dv != 128))
    return SPA_ERR_UNSUPPORTED;
  return SPA_OK;
}

struct WindowLayout {
  int NT, KD, BH, BHk, ns, cuts;  // query and key heads of the batch; cut key tiles and their runs
  ProjOut mode;
  size_t qs, ks, qmul, kmul;                               // score operands
  size_t qb, kb, stats, dqacc, dkacc, dvacc, dP;           // backward
  size_t total;
};

WindowLayout window_layout(int B, int H, int Hk, int N, int d, int m, int dv, int window, int sink, bool gradient) {
  WindowLayout L{};
  L.NT = (N + spa::kTileRows - 1) / spa::kTileRows;
  L.mode = m == 16 ? ProjOut::BF16X3 : ProjOut::F16X1;
  L.KD = spa::score_depth(m, L.mode);
  L.BH = B * H;
  L.BHk = B * Hk;
  L.cuts = spa::window_cuts(N, window, sink);
  L.ns = L.cuts > 1 ? spa::window_sink_tiles(N, window, sink) : 0;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align256(o + bytes);
    return at;
  };
  const size_t q = static_cast<size_t>(L.BH) * L.NT, k = static_cast<size_t>(L.BHk) * L.NT, rows = spa::kTileRows;
  L.qs = take(q * rows * L.KD * 2);
  L.ks = take(k * rows * L.KD * 2);
  L.qmul = take(q * rows * sizeof(float));
  L.kmul = take(k * sizeof(float));
  if (gradient) {
    L.qb = take(q * rows * m * 2);
    L.kb = take(k * rows * m * 2);
    L.stats = take(q * rows * 4 * sizeof(float));
    L.dqacc = take(q * rows * m * sizeof(float));
    L.dkacc = take(k * rows * m * sizeof(float));
    L.dvacc = take(static_cast<size_t>(L.BHk) * L.ns * rows * dv * sizeof(float));
    L.dP = take(static_cast<size_t>(Hk) * d * m * sizeof(float));
  }
  L.total = o;
  return L;
}

// Score operands of q and k (with lse: and their bf16 tiles for the backward), in one launch.
int window_project(const void* q, const void* k, const void* P, int B, int H, int Hk, int N, int d, int m,
                   const WindowLayout& L, char* w, const float* lse, cudaStream_t stream) {
  spa::ProjParams pp{};
  pp.x[0] = q;
  pp.x[1] = k;
  pp.P = P;
  pp.N = N;
  pp.d = d;
  pp.m = m;
  pp.NT = L.NT;
  pp.bf16_in = 1;
  pp.mode = L.mode;
  pp.use_tc = 1;
  pp.out[0] = w + L.qs;
  pp.out[1] = w + L.ks;
  pp.mul[0] = reinterpret_cast<float*>(w + L.qmul);
  pp.mul[1] = reinterpret_cast<float*>(w + L.kmul);
  pp.qscale = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(m)));
  if (lse) {
    pp.out_b16[0] = w + L.qb;
    pp.out_b16[1] = w + L.kb;
    pp.row_lse = lse;
    pp.lse_scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(m)));
  }
  int st;
  if ((st = encode_bf16_rows(&pp.xmap[0], q, d, N, L.BH)) || (st = encode_bf16_rows(&pp.xmap[1], k, d, N, L.BHk)) ||
      (st = device_error_ptr(&pp.err)))
    return st;
  pp.nx = 2;
  pp.BH = L.BH;
  pp.H = H;
  pp.group = H / Hk;
  return cuda_status(spa::launch_project(pp, stream));
}

int window_forward(const void* q, const void* k, const void* v, const void* P, void* out, void* out_lo, float* lse, int B, int H,
                   int Hk, int N, int d, int m, int dv, int window, int sink, char* w, cudaStream_t stream,
                   unsigned long long limit_ns = kWaitLimitNs, int inject_stall = 0) {
  const WindowLayout L = window_layout(B, H, Hk, N, d, m, dv, window, sink, false);
  int st = window_project(q, k, P, B, H, Hk, N, d, m, L, w, nullptr, stream);
  if (st) return st;
  spa::AttnTcParams ap{};
  if ((st = encode_bf16_rows(&ap.vmap, v, dv, N, L.BHk)) || (st = encode_bf16_rows(&ap.omap, out, dv, N, L.BH)) ||
      (st = device_error_ptr(&ap.err)))
    return st;
  ap.Qs = reinterpret_cast<const uint16_t*>(w + L.qs);
  ap.Ks = reinterpret_cast<const uint16_t*>(w + L.ks);
  ap.qmul = reinterpret_cast<const float*>(w + L.qmul);
  ap.kmul = reinterpret_cast<const float*>(w + L.kmul);
  ap.BH = L.BH;
  ap.N = N;
  ap.NT = L.NT;
  ap.KD = L.KD;
  ap.dv = dv;
  ap.causal = 1;
  ap.f16_ops = L.mode == ProjOut::F16X1;
  ap.limit_ns = limit_ns;
  ap.inject_stall = inject_stall;
  ap.lse = lse;
  ap.G = H / Hk;
  ap.window = window;
  ap.sink = sink;
  ap.has_lo = out_lo != nullptr;
  if (out_lo && (st = encode_bf16_rows(&ap.lomap, out_lo, dv, N, L.BH))) return st;
  return cuda_status(spa::launch_attn_window(ap, stream));
}

int window_backward(const void* q, const void* k, const void* v, const void* P, const void* out, const void* out_lo, const float* lse,
                    const void* dO, void* dq, void* dk, void* dv_out, void* dP, int B, int H, int Hk, int N, int d,
                    int m, int dv, int window, int sink, char* w, cudaStream_t stream,
                    unsigned long long limit_ns = kWaitLimitNs, int inject_stall = 0) {
  const WindowLayout L = window_layout(B, H, Hk, N, d, m, dv, window, sink, true);
  int st = window_project(q, k, P, B, H, Hk, N, d, m, L, w, lse, stream);
  if (st) return st;
  const float alpha = static_cast<float>(1.0 / std::sqrt(static_cast<double>(m)));
  // the sums that are added to: dQp, dKp and dV of cut key tiles, dP (dqacc .. dP are the last of the workspace)
  const size_t zeros = L.total - L.dqacc;
  int* err = nullptr;
  if ((st = device_error_ptr(&err))) return st;
  if ((st = cuda_status(spa::launch_window_stats(dO, out, out_lo, lse, reinterpret_cast<const float*>(w + L.qmul),
                                                 reinterpret_cast<float*>(w + L.stats), L.BH, N, L.NT, dv, w + L.dqacc, zeros,
                                                 stream))))
    return st;
  spa::BwdTcParams bp{};
  if ((st = encode_bf16_rows(&bp.domap, dO, dv, N, L.BH)) || (st = encode_bf16_rows(&bp.vmap, v, dv, N, L.BHk)))
    return st;
  bp.Qs = reinterpret_cast<const uint16_t*>(w + L.qs);
  bp.Ks = reinterpret_cast<const uint16_t*>(w + L.ks);
  bp.kmul = reinterpret_cast<const float*>(w + L.kmul);
  bp.Qb = reinterpret_cast<const uint16_t*>(w + L.qb);
  bp.Kb = reinterpret_cast<const uint16_t*>(w + L.kb);
  bp.stats = reinterpret_cast<const float*>(w + L.stats);
  bp.dqacc = reinterpret_cast<float*>(w + L.dqacc);
  bp.dkacc = reinterpret_cast<float*>(w + L.dkacc);
  bp.dvacc = reinterpret_cast<float*>(w + L.dvacc);
  bp.dv_b16 = static_cast<__nv_bfloat16*>(dv_out);
  bp.err = err;
  bp.BH = L.BH;
  bp.N = N;
  bp.NT = L.NT;
  bp.KD = L.KD;
  bp.m = m;
  bp.dv = dv;
  bp.causal = 1;
  bp.f16_ops = L.mode == ProjOut::F16X1;
  bp.alpha = alpha;
  bp.limit_ns = limit_ns;
  bp.inject_stall = inject_stall;
  bp.G = H / Hk;
  bp.window = window;
  bp.sink = window ? sink : 0;
  bp.cuts = L.cuts;
  if ((st = cuda_status(spa::launch_bwd_window(bp, stream)))) return st;
  spa::BwdFinishParams fp{};
  if ((st = encode_bf16_rows(&fp.qmap, q, d, N, L.BH)) || (st = encode_bf16_rows(&fp.kmap, k, d, N, L.BHk)) ||
      (st = encode_bf16_rows(&fp.dqmap, dq, d, N, L.BH)) || (st = encode_bf16_rows(&fp.dkmap, dk, d, N, L.BHk)))
    return st;
  fp.dqacc = bp.dqacc;
  fp.dkacc = bp.dkacc;
  fp.P = static_cast<const __nv_bfloat16*>(P);
  fp.dP = reinterpret_cast<float*>(w + L.dP);
  fp.err = err;
  fp.B = B;
  fp.H = Hk;
  fp.N = N;
  fp.NT = L.NT;
  fp.d = d;
  fp.m = m;
  fp.limit_ns = kWaitLimitNs;
  fp.G = H / Hk;
  if ((st = cuda_status(spa::launch_bwd_finish_window(fp, stream)))) return st;
  return cuda_status(spa::launch_window_round(fp.dP, static_cast<__nv_bfloat16*>(dP),
                                              static_cast<long long>(Hk) * d * m, bp.dvacc, bp.dv_b16, L.BHk, L.ns, N,
                                              dv, stream));
}

// Whether the rows of d features of a strided [size0][size1][size2][d] tensor do not
// overlap: from the innermost dimension outwards, every step goes past all that the
// inner ones reach.
bool rows_apart(const long long (&size)[3], const long long (&step)[3], int d) {
  long long reach = d;
  bool used[3] = {size[0] == 1, size[1] == 1, size[2] == 1};
  for (int left = 3 - used[0] - used[1] - used[2]; left > 0; --left) {
    int at = -1;
    for (int i = 0; i < 3; ++i)
      if (!used[i] && (at < 0 || step[i] < step[at])) at = i;
    if (step[at] < reach) return false;
    if (step[at] > (LLONG_MAX - reach) / size[at]) return false;
    reach += step[at] * (size[at] - 1);
    used[at] = true;
  }
  return true;
}

// Sizes and addresses of the norm with rotary positions, forward and gradient: `in` the
// tensors that are read, `out` those that are written, as queries and keys; strides as
// q, k of each.
int norm_rope_params(spa::NormRopeParams& np, const void* const (*in)[2], int ins, void* const (&out)[2],
                     const long long* strides, const void* wq, const void* wk, const int* pos, int pos0,
                     const unsigned long long* table, int B, int H, int Hk, int N, int d, int rot,
                     int interleaved, float eps, int dtype) {
  if (B < 0 || H < 0 || Hk < 0 || N < 0 || d < 0) return SPA_ERR_SHAPE;
  if (dtype != SPA_F32 && dtype != SPA_BF16) return SPA_ERR_DTYPE;
  if (static_cast<long long>(H) + Hk == 0) return kEmpty;
  if (d < 1 || d > 256) return SPA_ERR_UNSUPPORTED;
  if (rot < 0 || rot > d || rot % 2 || !(eps > 0.f) || !std::isfinite(eps)) return SPA_ERR_SHAPE;
  if (static_cast<long long>(H) + Hk > 65535 || static_cast<long long>(B) * N > (1LL << 29))
    return SPA_ERR_SHAPE;
  if (rot > 0 && !pos && static_cast<long long>(pos0) + N - 1 > INT_MAX) return SPA_ERR_SHAPE;
  // rows are counted in 32 bits, with room for a block's round
  if (static_cast<long long>(B) * N * (H > Hk ? H : Hk) > (1LL << 31)) return SPA_ERR_SHAPE;
  np.B = B;
  np.N = N;
  np.d = d;
  if (static_cast<long long>(B) * N == 0) return kEmpty;
  if (rot > 0 && !table) return SPA_ERR_NULL;
  const uintptr_t es = dtype == SPA_BF16 ? 2 : 4;
  const int heads[2] = {H, Hk};
  const void* weights[2] = {wq, wk};
  for (int t = 0; t < 2; ++t) {
    if (heads[t] == 0) continue;
    const long long size[3] = {B, heads[t], N};
    const long long dense[3] = {static_cast<long long>(heads[t]) * N * d, static_cast<long long>(N) * d, d};
    long long step[3][3];  // inputs, then the output
    for (int x = 0; x <= ins; ++x) {
      const void* at = x < ins ? in[x][t] : out[t];
      if (!at) return SPA_ERR_NULL;
      if (reinterpret_cast<uintptr_t>(at) % es) return SPA_ERR_ALIGN;
      for (int i = 0; i < 3; ++i) {
        step[x][i] = strides ? strides[6 * x + 3 * t + i] : dense[i];
        if (size[i] == 1) step[x][i] = 0;  // a dimension of one row is never stepped along
      }
    }
    if (!rows_apart(size, step[ins], d)) return SPA_ERR_SHAPE;
    for (int x = 0; x < ins; ++x)
      if (in[x][t] == out[t])
        for (int i = 0; i < 3; ++i)
          if (step[x][i] != step[ins][i]) return SPA_ERR_SHAPE;
    if (reinterpret_cast<uintptr_t>(weights[t]) % es) return SPA_ERR_ALIGN;
    for (int i = 0; i < 3; ++i) {
      np.xs[t][i] = step[0][i];
      np.gs[t][i] = ins > 1 ? step[1][i] : 0;
      np.ys[t][i] = step[ins][i];
    }
    np.x[t] = in[0][t];
    np.g[t] = ins > 1 ? in[1][t] : nullptr;
    np.y[t] = out[t];
    np.w[t] = weights[t];
    np.H[t] = heads[t];
  }
  if (rot > 0 && ((reinterpret_cast<uintptr_t>(table) & 7u) || !aligned4(pos))) return SPA_ERR_ALIGN;
  np.pos = pos;
  np.table = table;
  np.rot = rot;
  np.pos0 = pos0;
  np.interleaved = interleaved != 0;
  np.bf16 = dtype == SPA_BF16;
  np.eps = eps;
  return SPA_OK;
}

// Sizes that the calls on 8-bit pages share.
int check_cache8(int B, int Hk, int pages, int width, int m, int d_v, int cap) {
  if (B < 0 || Hk < 0 || pages < 0 || width < 0 || m < 0 || d_v < 0 || cap < 0) return SPA_ERR_SHAPE;
  if (B == 0 || Hk == 0) return kEmpty;
  if (static_cast<long long>(B) * Hk > 65535) return SPA_ERR_SHAPE;
  // token numbers are 31-bit
  if (static_cast<long long>(width) * spa::kPageRows + cap > INT_MAX) return SPA_ERR_SHAPE;
  if ((m != 16 && m != 32 && m != 64 && m != 128) || (d_v != 64 && d_v != 128)) return SPA_ERR_UNSUPPORTED;
  return SPA_OK;
}

spa::Pages pages_of(const void* kc8, const float* ks, const void* vc8, const float* vs, const int* table,
                    int pages, int width) {
  return {static_cast<uint8_t*>(const_cast<void*>(kc8)), const_cast<float*>(ks),
          static_cast<uint8_t*>(const_cast<void*>(vc8)), const_cast<float*>(vs), width > 0 ? table : nullptr,
          pages, width};
}

}  // namespace

extern "C" {

const char* spa_status_str(int status) {
  switch (status) {
    case SPA_OK: return "SPA_OK";
    case SPA_ERR_NULL: return "SPA_ERR_NULL: a required pointer is NULL";
    case SPA_ERR_SHAPE: return "SPA_ERR_SHAPE: a size is negative or too large";
    case SPA_ERR_DTYPE: return "SPA_ERR_DTYPE: dtype must be SPA_F32 or SPA_BF16";
    case SPA_ERR_ALIGN: return "SPA_ERR_ALIGN: pointers must be 16-byte aligned";
    case SPA_ERR_UNSUPPORTED: return "SPA_ERR_UNSUPPORTED: shape outside the implemented kernels";
    case SPA_ERR_NOMEM: return "SPA_ERR_NOMEM: workspace allocation failed or too small";
    case SPA_ERR_CUDA: return "SPA_ERR_CUDA: a CUDA call failed";
    case SPA_ERR_TIMEOUT: return "SPA_ERR_TIMEOUT: a kernel gave up on a bounded wait";
    default: return "SPA_ERR_UNKNOWN";
  }
}

int spa_version(void) { return 100; }

int spa_project(const void* x, const void* P, float* x_proj, int B, int H, int N, int d, int m,
                int dtype, void* stream) {
  if (B < 0 || H < 0 || N < 0 || d < 0 || m < 0) return SPA_ERR_SHAPE;
  if (dtype != SPA_F32 && dtype != SPA_BF16) return SPA_ERR_DTYPE;
  if (static_cast<long long>(B) * H * N == 0) return SPA_OK;
  if (static_cast<long long>(B) * H > 65535) return SPA_ERR_SHAPE;
  if (d < 1 || d > 256 || m < 1 || m > 128) return SPA_ERR_UNSUPPORTED;
  if (!x || !P || !x_proj) return SPA_ERR_NULL;
  if (!aligned16(x) || !aligned16(P) || !aligned16(x_proj)) return SPA_ERR_ALIGN;
  spa::ProjParams pp{};
  pp.x[0] = x;
  pp.P = P;
  pp.out[0] = x_proj;
  pp.nx = 1;
  pp.BH = B * H;
  pp.H = H;
  pp.N = N;
  pp.d = d;
  pp.m = m;
  pp.NT = (N + spa::kTileRows - 1) / spa::kTileRows;
  pp.bf16_in = dtype == SPA_BF16;
  pp.mode = ProjOut::F32;
  return cuda_status(spa::launch_project(pp, static_cast<cudaStream_t>(stream)));
}

int spa_attention_workspace_size(int B, int H, int N, int d, int m, int d_v, int dtype,
                                 size_t* bytes) {
  if (!bytes) return SPA_ERR_NULL;
  const int st = check_shape(B, H, N, d, m, d_v, dtype);
  if (st == kEmpty) {
    *bytes = 0;
    return SPA_OK;
  }
  if (st) return st;
  *bytes = make_layout(B, H, N, m, dtype).total;
  return SPA_OK;
}

int spa_attention_fwd_ws(const void* q, const void* k, const void* v, const void* P, float* out,
                         int B, int H, int N, int d, int m, int d_v, int causal, int dtype,
                         void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_shape(B, H, N, d, m, d_v, dtype);
  if (st == kEmpty) return SPA_OK;
  if (st) return st;
  if ((st = check_forward_ptrs(q, k, v, P, out))) return st;
  if (!workspace) return SPA_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return SPA_ERR_ALIGN;
  if (workspace_bytes < make_layout(B, H, N, m, dtype).total) return SPA_ERR_NOMEM;
  return run_forward(q, k, v, P, out, B, H, N, d, m, d_v, causal, dtype, workspace,
                     static_cast<cudaStream_t>(stream));
}

int spa_attention_prepare(const void* q, const void* k, const void* P, int B, int H, int N,
                          int d, int m, int d_v, int dtype, void* workspace,
                          size_t workspace_bytes, void* stream) {
  int st = check_shape(B, H, N, d, m, d_v, dtype);
  if (st == kEmpty) return SPA_OK;
  if (st) return st;
  if (!q || !k || !P || !workspace) return SPA_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(P) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return SPA_ERR_ALIGN;
  if (workspace_bytes < make_layout(B, H, N, m, dtype).total) return SPA_ERR_NOMEM;
  return run_prepare(q, k, P, B, H, N, d, m, dtype, workspace, static_cast<cudaStream_t>(stream));
}

int spa_attention_apply(const void* v, float* out, int B, int H, int N, int d, int m, int d_v,
                        int causal, int dtype, const void* workspace, size_t workspace_bytes,
                        void* stream) {
  int st = check_shape(B, H, N, d, m, d_v, dtype);
  if (st == kEmpty) return SPA_OK;
  if (st) return st;
  if (!v || !out || !workspace) return SPA_ERR_NULL;
  if (!aligned16(v) || !aligned16(out) || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return SPA_ERR_ALIGN;
  if (workspace_bytes < make_layout(B, H, N, m, dtype).total) return SPA_ERR_NOMEM;
  return run_apply(v, out, B, H, N, m, d_v, causal, dtype, workspace,
                   static_cast<cudaStream_t>(stream));
}

int spa_attention_fwd(const void* q, const void* k, const void* v, const void* P, float* out,
                      int B, int H, int N, int d, int m, int d_v, int causal, int dtype,
                      void* stream) {
  int st = check_shape(B, H, N, d, m, d_v, dtype);
  if (st == kEmpty) return SPA_OK;
  if (st) return st;
  if ((st = check_forward_ptrs(q, k, v, P, out))) return st;
  const size_t bytes = make_layout(B, H, N, m, dtype).total;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  void* ws = nullptr;
  if (int e = pool_alloc(&ws, bytes, s)) return e;
  st = run_forward(q, k, v, P, out, B, H, N, d, m, d_v, causal, dtype, ws, s);
  const cudaError_t fe = cudaFreeAsync(ws, s);
  if (st) return st;
  return cuda_status(fe);
}

int spa_attention_fwd_host(const void* q, const void* k, const void* v, const void* P,
                           float* out, int B, int H, int N, int d, int m, int d_v, int causal,
                           int dtype, void* stream) {
  int st = check_shape(B, H, N, d, m, d_v, dtype);
  if (st == kEmpty) return SPA_OK;
  if (st) return st;
  if (!q || !k || !v || !P || !out) return SPA_ERR_NULL;
  return host_forward(static_cast<const char*>(q), static_cast<const char*>(k),
                      static_cast<const char*>(v), static_cast<const char*>(P), out, B, H, N, d, m,
                      d_v, causal, dtype, static_cast<cudaStream_t>(stream));
}

int spa_kcache_append(const void* k, const void* P, void* kc, float* kc_mul, int B, int H, int T,
                      int d, int m, int pos, int cap, int dtype, void* stream) {
  if (B < 0 || H < 0 || T < 0 || d < 0 || m < 0 || pos < 0 || cap < 0) return SPA_ERR_SHAPE;
  if (dtype != SPA_F32 && dtype != SPA_BF16) return SPA_ERR_DTYPE;
  if (static_cast<long long>(pos) + T > cap) return SPA_ERR_SHAPE;
  if (static_cast<long long>(B) * H * T == 0) return SPA_OK;
  if (static_cast<long long>(B) * H > 65535) return SPA_ERR_SHAPE;
  if (dtype != SPA_BF16) return SPA_ERR_UNSUPPORTED;
  if (d < 1 || d > 256 || (m != 16 && m != 32 && m != 64 && m != 128)) return SPA_ERR_UNSUPPORTED;
  if (!k || !P || !kc || !kc_mul) return SPA_ERR_NULL;
  if (!aligned16(k) || !aligned16(P) || !aligned16(kc) || !aligned16(kc_mul)) return SPA_ERR_ALIGN;
  // the projection kernels with a row-major fp16 output: rows pos .. pos+T-1
  spa::ProjParams pp{};
  pp.x[0] = k;
  pp.P = P;
  pp.out[0] = kc;
  pp.mul[0] = kc_mul;
  pp.nx = 1;
  pp.BH = B * H;
  pp.H = H;
  pp.N = T;
  pp.d = d;
  pp.m = m;
  pp.NT = (T + spa::kTileRows - 1) / spa::kTileRows;
  pp.qscale = 1.f;
  pp.bf16_in = 1;
  pp.mode = ProjOut::F16ROWS;
  pp.out_rows = cap;
  pp.out_pos = pos;
  pp.use_tc = 1;
  if (spa::project_tc_eligible(pp)) {
    int st;
    if ((st = encode_bf16_rows(&pp.xmap[0], k, d, T, B * H))) return st;
    if ((st = device_error_ptr(&pp.err))) return st;
  }
  return cuda_status(spa::launch_project(pp, static_cast<cudaStream_t>(stream)));
}

int spa_attention_decode(const void* q, const void* P, const void* kc, const float* kc_mul,
                         const void* v, float* out, int B, int H, int L, int d, int m, int d_v,
                         int cap, int dtype, void* stream) {
  if (B < 0 || H < 0 || L < 0 || d < 0 || m < 0 || d_v < 0 || cap < 0) return SPA_ERR_SHAPE;
  if (dtype != SPA_F32 && dtype != SPA_BF16) return SPA_ERR_DTYPE;
  if (static_cast<long long>(B) * H == 0) return SPA_OK;
  if (L < 1 || L > cap) return SPA_ERR_SHAPE;
  if (static_cast<long long>(B) * H > 65535) return SPA_ERR_SHAPE;
  if (dtype != SPA_BF16) return SPA_ERR_UNSUPPORTED;
  if (d < 1 || d > 256 || (m != 16 && m != 32 && m != 64 && m != 128) ||
      (d_v != 64 && d_v != 128))
    return SPA_ERR_UNSUPPORTED;
  if (!q || !P || !kc || !kc_mul || !v || !out) return SPA_ERR_NULL;
  if (!aligned16(q) || !aligned16(P) || !aligned16(kc) || !aligned16(kc_mul) || !aligned16(v) ||
      !aligned16(out))
    return SPA_ERR_ALIGN;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return SPA_ERR_CUDA;
  spa::DecodeParams dp{};
  dp.q = static_cast<const __nv_bfloat16*>(q);
  dp.P = static_cast<const __nv_bfloat16*>(P);
  dp.kc = static_cast<const uint16_t*>(kc);
  dp.kc_mul = kc_mul;
  dp.v = static_cast<const __nv_bfloat16*>(v);
  dp.out = out;
  dp.BH = B * H;
  dp.H = H;
  dp.L = L;
  dp.d = d;
  dp.m = m;
  dp.dv = d_v;
  dp.cap = cap;
  dp.qscale = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(m)));
  spa::decode_split(dp.BH, L, sms, &dp.nsplit, &dp.chunk);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t part = static_cast<size_t>(dp.BH) * dp.nsplit * (2 + d_v) * sizeof(float);
  // from the library's own pool, which keeps what it has reserved: a decode loop
  // synchronises every step, and the default pool would hand the scratch back
  // to the driver at each synchronisation and reserve it again on the next call
  cudaMemPool_t pool = nullptr;
  if (host_pool(&pool) != SPA_OK) return SPA_ERR_CUDA;
  if (cudaMallocFromPoolAsync(reinterpret_cast<void**>(&dp.part), part, pool, s) != cudaSuccess) {
    cudaGetLastError();
    return SPA_ERR_NOMEM;
  }
  const int st = cuda_status(spa::launch_decode(dp, s));
  const cudaError_t fe = cudaFreeAsync(dp.part, s);
  if (st) return st;
  return fe == cudaSuccess ? SPA_OK : SPA_ERR_CUDA;
}

int spa_rope_frequencies(double* inv_freq, int rot, double base, int scaling, double factor,
                         double trained, double slow, double fast) {
  if (!inv_freq) return SPA_ERR_NULL;
  if (rot < 2 || rot % 2 || !(base > 0.0) || !std::isfinite(base)) return SPA_ERR_SHAPE;
  if (scaling < SPA_ROPE_PLAIN || scaling > SPA_ROPE_RAMP) return SPA_ERR_UNSUPPORTED;
  if (scaling != SPA_ROPE_PLAIN && (!(factor > 0.0) || !std::isfinite(factor))) return SPA_ERR_SHAPE;
  if (scaling == SPA_ROPE_BASE && rot < 4) return SPA_ERR_SHAPE;
  if (scaling == SPA_ROPE_RAMP &&
      (!(trained > 0.0) || !(slow >= 0.0) || !(fast > slow) || !std::isfinite(fast)))
    return SPA_ERR_SHAPE;
  if (scaling == SPA_ROPE_BASE) base *= std::pow(factor, static_cast<double>(rot) / (rot - 2));
  for (int i = 0; i < rot / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / rot);
    inv_freq[i] = f;
    if (scaling == SPA_ROPE_LINEAR) inv_freq[i] = f / factor;
    if (scaling == SPA_ROPE_RAMP) {
      const double turns = trained * f / 6.283185307179586476925;
      const double keep = turns >= fast ? 1.0 : turns <= slow ? 0.0 : (turns - slow) / (fast - slow);
      inv_freq[i] = keep * f + (1.0 - keep) * f / factor;
    }
  }
  return SPA_OK;
}

int spa_rope_table(const double* inv_freq, int rot, unsigned long long* table) {
  if (!inv_freq || !table) return SPA_ERR_NULL;
  if (rot < 2 || rot % 2) return SPA_ERR_SHAPE;
  for (int i = 0; i < rot / 2; ++i)
    if (!std::isfinite(inv_freq[i])) return SPA_ERR_SHAPE;
  for (int i = 0; i < rot / 2; ++i) {
    // whole turns per position drop out; the rest is at most half a turn
    const double turns = inv_freq[i] / 6.283185307179586476925;
    const double part = std::nearbyint((turns - std::nearbyint(turns)) * 18446744073709551616.0);
    table[i] = part >= 9223372036854775808.0
                   ? 0x8000000000000000ull
                   : static_cast<unsigned long long>(static_cast<long long>(part));
  }
  return SPA_OK;
}

int spa_rope(const void* q, const void* k, void* q_out, void* k_out, const long long* strides,
             const int* pos, int pos0, const unsigned long long* table, int B, int H, int Hk, int N,
             int d, int rot, int interleaved, int inverse, float scale, int dtype, void* stream) {
  if (B < 0 || H < 0 || Hk < 0 || N < 0 || d < 0) return SPA_ERR_SHAPE;
  if (dtype != SPA_F32 && dtype != SPA_BF16) return SPA_ERR_DTYPE;
  if (static_cast<long long>(B) * N == 0 || static_cast<long long>(H) + Hk == 0) return SPA_OK;
  if (d < 1 || d > 1024) return SPA_ERR_UNSUPPORTED;
  if (rot < 2 || rot > d || rot % 2) return SPA_ERR_SHAPE;
  if (static_cast<long long>(H) + Hk > 65535) return SPA_ERR_SHAPE;
  if (static_cast<long long>(B) * N > (1LL << 29)) return SPA_ERR_SHAPE;
  if (!pos && static_cast<long long>(pos0) + N - 1 > INT_MAX) return SPA_ERR_SHAPE;
  if (!table || (H > 0 && (!q || !q_out)) || (Hk > 0 && (!k || !k_out))) return SPA_ERR_NULL;
  const uintptr_t es = dtype == SPA_BF16 ? 2 : 4;
  spa::RopeParams rp{};
  const void* in[2] = {q, k};
  void* out[2] = {q_out, k_out};
  const int heads[2] = {H, Hk};
  for (int t = 0; t < 2; ++t) {
    if (heads[t] == 0) continue;
    if (reinterpret_cast<uintptr_t>(in[t]) % es || reinterpret_cast<uintptr_t>(out[t]) % es)
      return SPA_ERR_ALIGN;
    const long long dense[3] = {static_cast<long long>(heads[t]) * N * d,
                                static_cast<long long>(N) * d, d};
    const long long size[3] = {B, heads[t], N};
    for (int i = 0; i < 3; ++i) {
      rp.xs[t][i] = strides ? strides[3 * t + i] : dense[i];
      rp.ys[t][i] = strides ? strides[6 + 3 * t + i] : dense[i];
      // a dimension of one row is never stepped along
      if (size[i] == 1) rp.xs[t][i] = rp.ys[t][i] = 0;
    }
    if (!rows_apart(size, rp.ys[t], d)) return SPA_ERR_SHAPE;
    if (in[t] == out[t])
      for (int i = 0; i < 3; ++i)
        if (rp.xs[t][i] != rp.ys[t][i]) return SPA_ERR_SHAPE;
    rp.x[t] = in[t];
    rp.y[t] = out[t];
    rp.H[t] = heads[t];
  }
  if ((reinterpret_cast<uintptr_t>(table) & 7u) || (reinterpret_cast<uintptr_t>(pos) & 3u))
    return SPA_ERR_ALIGN;
  rp.pos = pos;
  rp.table = table;
  rp.B = B;
  rp.N = N;
  rp.d = d;
  rp.rot = rot;
  rp.pos0 = pos0;
  rp.interleaved = interleaved != 0;
  rp.inverse = inverse != 0;
  rp.bf16 = dtype == SPA_BF16;
  rp.scale = scale;
  return cuda_status(spa::launch_rope(rp, static_cast<cudaStream_t>(stream)));
}

int spa_kcache_append_ragged(const void* k, const void* v, const void* P, void* kc, float* kc_mul,
                             void* vc, const int* pos, const int* count, float* acc, int* row_pos,
                             const int* token, int B, int H, int T, int d, int m, int d_v, int cap,
                             int dtype, void* stream) {
  if (B < 0 || H < 0 || T < 0 || d < 0 || m < 0 || d_v < 0 || cap < 0) return SPA_ERR_SHAPE;
  if (dtype != SPA_F32 && dtype != SPA_BF16) return SPA_ERR_DTYPE;
  if (B == 0 || H == 0 || T == 0 || cap == 0) return SPA_OK;
  if (static_cast<long long>(B) * H > 65535) return SPA_ERR_SHAPE;
  if (dtype != SPA_BF16) return SPA_ERR_UNSUPPORTED;
  if (d < 1 || d > 256 || (m != 16 && m != 32 && m != 64 && m != 128) || (d_v != 64 && d_v != 128))
    return SPA_ERR_UNSUPPORTED;
  if (!k || !v || !P || !kc || !kc_mul || !vc || !pos) return SPA_ERR_NULL;
  if (!aligned16(k) || !aligned16(v) || !aligned16(P) || !aligned16(kc) || !aligned16(vc) ||
      !aligned4(kc_mul) || !aligned4(pos) || !aligned4(count) || !aligned4(acc) ||
      !aligned4(row_pos) || !aligned4(token))
    return SPA_ERR_ALIGN;
  spa::AppendParams ap{};
  ap.k = static_cast<const __nv_bfloat16*>(k);
  ap.v = static_cast<const __nv_bfloat16*>(v);
  ap.P = static_cast<const __nv_bfloat16*>(P);
  ap.kc = static_cast<uint16_t*>(kc);
  ap.kc_mul = kc_mul;
  ap.vc = static_cast<__nv_bfloat16*>(vc);
  ap.pos = pos;
  ap.count = count;
  ap.acc = acc;
  ap.row_pos = row_pos;
  ap.token = token;
  ap.B = B;
  ap.H = H;
  ap.T = T;
  ap.d = d;
  ap.m = m;
  ap.dv = d_v;
  ap.cap = cap;
  return cuda_status(spa::launch_append_ragged(ap, static_cast<cudaStream_t>(stream)));
}

int spa_attention_decode_shared_workspace_size(int B, int H, int Hk, int plen, int d, int m,
                                               int d_v, int cap, int weights, size_t* bytes) {
  if (!bytes) return SPA_ERR_NULL;
  const int st = check_decode_shared(B, H, Hk, plen, d, m, d_v, cap);
  *bytes = 0;
  if (st == kEmpty) return SPA_OK;
  if (st) return st;
  spa::DecodeSharedParams dp{};
  if (int e = decode_shared_sizes(dp, B, H, Hk, plen, d, m, d_v, cap)) return e;
  float mark = 0.f;
  dp.acc_out = weights ? &mark : nullptr;
  *bytes = spa::decode_shared_workspace(dp);
  return SPA_OK;
}

int spa_attention_decode_shared(const void* q, const void* P, const void* kc, const float* kc_mul,
                                const void* v, const int* lens, const void* pkc,
                                const float* pkc_mul, const void* pv, void* out, const float* acc,
                                float* acc_out, int B, int H, int Hk, int plen, int pcap, int d,
                                int m, int d_v, int cap, int dtype, void* workspace,
                                size_t workspace_bytes, void* stream) {
  if (dtype != SPA_F32 && dtype != SPA_BF16) return SPA_ERR_DTYPE;
  int st = check_decode_shared(B, H, Hk, plen, d, m, d_v, cap);
  if (st == kEmpty) return SPA_OK;
  if (st) return st;
  if (dtype != SPA_BF16) return SPA_ERR_UNSUPPORTED;
  if (pcap < plen) return SPA_ERR_SHAPE;
  if (!q || !P || !out) return SPA_ERR_NULL;
  if (cap > 0 && (!kc || !kc_mul || !v || !lens)) return SPA_ERR_NULL;
  if (plen > 0 && (!pkc || !pkc_mul || !pv)) return SPA_ERR_NULL;
  if ((acc == nullptr) != (acc_out == nullptr)) return SPA_ERR_NULL;
  if (!aligned16(q) || !aligned16(P) || !aligned16(kc) || !aligned16(v) || !aligned16(pkc) ||
      !aligned16(pv) || !aligned16(out) || !aligned4(kc_mul) || !aligned4(lens) ||
      !aligned4(pkc_mul) || !aligned4(acc) || !aligned4(acc_out) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return SPA_ERR_ALIGN;
  spa::DecodeSharedParams dp{};
  if ((st = decode_shared_sizes(dp, B, H, Hk, plen, d, m, d_v, cap))) return st;
  dp.q = static_cast<const __nv_bfloat16*>(q);
  dp.P = static_cast<const __nv_bfloat16*>(P);
  dp.kc = static_cast<const uint16_t*>(kc);
  dp.kc_mul = kc_mul;
  dp.v = static_cast<const __nv_bfloat16*>(v);
  dp.lens = lens;
  dp.pkc = static_cast<const uint16_t*>(pkc);
  dp.pkc_mul = pkc_mul;
  dp.pv = static_cast<const __nv_bfloat16*>(pv);
  dp.out = static_cast<__nv_bfloat16*>(out);
  dp.acc = acc;
  dp.acc_out = cap > 0 ? acc_out : nullptr;
  dp.pcap = pcap;
  const size_t need = spa::decode_shared_workspace(dp);
  if (workspace && workspace_bytes < need) return SPA_ERR_NOMEM;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  void* own = nullptr;
  if (!workspace)
    if (int e = pool_alloc(&own, need, s)) return e;
  dp.ws = static_cast<char*>(workspace ? workspace : own);
  st = run_decode_shared(dp, s);
  const cudaError_t fe = own ? cudaFreeAsync(own, s) : cudaSuccess;
  if (st) return st;
  return cuda_status(fe);
}

int spa_kcache_evict_workspace_size(int B, int H, int cap, int budget, size_t* bytes) {
  if (!bytes) return SPA_ERR_NULL;
  *bytes = 0;
  if (B < 0 || H < 0 || cap < 0) return SPA_ERR_SHAPE;
  if (B == 0 || H == 0 || cap == 0) return SPA_OK;
  if (static_cast<long long>(B) * H > 65535 || budget < 1 || budget > cap) return SPA_ERR_SHAPE;
  *bytes = align256(static_cast<size_t>(B) * H * spa::evict_stride(cap, budget) * sizeof(int));
  return SPA_OK;
}

int spa_kcache_evict(void* kc, float* kc_mul, void* v, const float* acc, const int* row_pos,
                     const int* lens, float* acc_out, int* row_pos_out, int* lens_out, int* src,
                     int B, int H, int m, int d_v, int cap, int budget, int sink, int recent,
                     void* workspace, size_t workspace_bytes, void* stream) {
  size_t need = 0;
  int st = spa_kcache_evict_workspace_size(B, H, cap, budget, &need);
  if (st) return st;
  if (need == 0) return SPA_OK;
  if (sink < 0 || recent < 0 || static_cast<long long>(sink) + recent > budget) return SPA_ERR_SHAPE;
  if (cap > spa::kEvictMaxRows) return SPA_ERR_UNSUPPORTED;
  if ((m != 16 && m != 32 && m != 64 && m != 128) || (d_v != 64 && d_v != 128))
    return SPA_ERR_UNSUPPORTED;
  if (!kc || !kc_mul || !v || !acc || !row_pos || !lens || !acc_out || !row_pos_out || !lens_out ||
      !src)
    return SPA_ERR_NULL;
  if (!aligned16(kc) || !aligned16(v) || !aligned4(kc_mul) || !aligned4(acc) ||
      !aligned4(row_pos) || !aligned4(lens) || !aligned4(acc_out) || !aligned4(row_pos_out) ||
      !aligned4(lens_out) || !aligned4(src) || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return SPA_ERR_ALIGN;
  if (workspace && workspace_bytes < need) return SPA_ERR_NOMEM;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  void* own = nullptr;
  if (!workspace)
    if (int e = pool_alloc(&own, need, s)) return e;
  spa::EvictParams ep{};
  ep.kc = static_cast<uint16_t*>(kc);
  ep.kc_mul = kc_mul;
  ep.v = static_cast<__nv_bfloat16*>(v);
  ep.acc = acc;
  ep.row_pos = row_pos;
  ep.lens = lens;
  ep.acc_out = acc_out;
  ep.row_pos_out = row_pos_out;
  ep.lens_out = lens_out;
  ep.src = src;
  ep.ws = static_cast<int*>(workspace ? workspace : own);
  ep.B = B;
  ep.H = H;
  ep.m = m;
  ep.dv = d_v;
  ep.cap = cap;
  ep.budget = budget;
  ep.sink = sink;
  ep.recent = recent;
  st = cuda_status(spa::launch_evict(ep, s));
  const cudaError_t fe = own ? cudaFreeAsync(own, s) : cudaSuccess;
  if (st) return st;
  return cuda_status(fe);
}

int spa_attention_window_workspace_size(int B, int H, int Hk, int N, int d, int m, int d_v, int window,
                                        int sink, int gradient, size_t* bytes) {
  if (!bytes) return SPA_ERR_NULL;
  *bytes = 0;
  const int st = check_window(B, H, Hk, N, d, m, d_v, window, sink, SPA_BF16);
  if (st) return st == kEmpty ? SPA_OK : st;
  if (window >= N) window = 0;
  if (sink > N) sink = N;
  *bytes = window_layout(B, H, Hk, N, d, m, d_v, window, sink, gradient != 0).total;
  return SPA_OK;
}

int spa_attention_window_fwd(const void* q, const void* k, const void* v, const void* P, void* out,
                             void* out_lo, float* lse, int B, int H, int Hk, int N, int d, int m, int d_v,
                             int window, int sink, int dtype, void* workspace,
                             size_t workspace_bytes, void* stream) {
  int st = check_window(B, H, Hk, N, d, m, d_v, window, sink, dtype);
  if (st) return st == kEmpty ? SPA_OK : st;
  if ((st = check_forward_ptrs(q, k, v, P, out))) return st;
  if ((out_lo == nullptr) != (lse == nullptr)) return SPA_ERR_NULL;
  if (!aligned16(out_lo) || !aligned4(lse) || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return SPA_ERR_ALIGN;
  if (window >= N) window = 0;
  if (sink > N) sink = N;
  const size_t need = window_layout(B, H, Hk, N, d, m, d_v, window, sink, false).total;
  if (workspace && workspace_bytes < need) return SPA_ERR_NOMEM;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  void* own = nullptr;
  if (!workspace)
    if (int e = pool_alloc(&own, need, s)) return e;
  st = window_forward(q, k, v, P, out, out_lo, lse, B, H, Hk, N, d, m, d_v, window, sink,
                      static_cast<char*>(workspace ? workspace : own), s);
  const cudaError_t fe = own ? cudaFreeAsync(own, s) : cudaSuccess;
  if (st) return st;
  return cuda_status(fe);
}

int spa_attention_window_bwd(const void* q, const void* k, const void* v, const void* P,
                             const void* out, const void* out_lo, const float* lse, const void* dO,
                             void* dq, void* dk, void* dv, void* dP, int B, int H, int Hk, int N, int d, int m, int d_v,
                             int window, int sink, int dtype, void* workspace,
                             size_t workspace_bytes, void* stream) {
  int st = check_window(B, H, Hk, N, d, m, d_v, window, sink, dtype);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (st == kEmpty) {  // sums over no queries; H = 0 leaves keys
    const size_t keys = static_cast<size_t>(B) * Hk * N, n = static_cast<size_t>(Hk) * d * m;
    if ((keys * d && !dk) || (keys * d_v && !dv)) return SPA_ERR_NULL;
    if (dP && n && (st = cuda_status(cudaMemsetAsync(dP, 0, n * 2, s))) != SPA_OK) return st;
    if (keys * d && (st = cuda_status(cudaMemsetAsync(dk, 0, keys * d * 2, s))) != SPA_OK) return st;
    if (keys * d_v && (st = cuda_status(cudaMemsetAsync(dv, 0, keys * d_v * 2, s))) != SPA_OK) return st;
    return SPA_OK;
  }
  if (st) return st;
  if ((st = check_forward_ptrs(q, k, v, P, out))) return st;
  if (!out_lo || !lse || !dO || !dq || !dk || !dv || !dP) return SPA_ERR_NULL;
  if (!aligned16(out_lo) || !aligned16(dO) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv) || !aligned16(dP) || !aligned4(lse) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return SPA_ERR_ALIGN;
  if (window >= N) window = 0;
  if (sink > N) sink = N;
  const size_t need = window_layout(B, H, Hk, N, d, m, d_v, window, sink, true).total;
  if (workspace && workspace_bytes < need) return SPA_ERR_NOMEM;
  void* own = nullptr;
  if (!workspace)
    if (int e = pool_alloc(&own, need, s)) return e;
  st = window_backward(q, k, v, P, out, out_lo, lse, dO, dq, dk, dv, dP, B, H, Hk, N, d, m, d_v, window, sink,
                       static_cast<char*>(workspace ? workspace : own), s);
  const cudaError_t fe = own ? cudaFreeAsync(own, s) : cudaSuccess;
  if (st) return st;
  return cuda_status(fe);
}

int spa_norm_rope(const void* q, const void* k, const void* wq, const void* wk, void* q_out,
                  void* k_out, const long long* strides, const int* pos, int pos0,
                  const unsigned long long* table, int B, int H, int Hk, int N, int d, int rot,
                  int interleaved, float eps, int dtype, void* stream) {
  spa::NormRopeParams np{};
  const void* const in[1][2] = {{q, k}};
  void* const out[2] = {q_out, k_out};
  const int st = norm_rope_params(np, in, 1, out, strides, wq, wk, pos, pos0, table, B, H, Hk, N, d, rot,
                                  interleaved, eps, dtype);
  if (st) return st == kEmpty ? SPA_OK : st;
  return cuda_status(spa::launch_norm_rope(np, static_cast<cudaStream_t>(stream)));
}

int spa_norm_rope_bwd_workspace_size(int d, size_t* bytes) {
  if (!bytes) return SPA_ERR_NULL;
  *bytes = 0;
  if (d < 0) return SPA_ERR_SHAPE;
  if (d > 256) return SPA_ERR_UNSUPPORTED;
  *bytes = align256(static_cast<size_t>(spa::kNormRopeBlocks + 1) * d * sizeof(float));
  return SPA_OK;
}

int spa_norm_rope_bwd(const void* q, const void* k, const void* wq, const void* wk,
                      const void* dq_out, const void* dk_out, void* dq, void* dk, float* dwq,
                      float* dwk, const long long* strides, const int* pos, int pos0,
                      const unsigned long long* table, int B, int H, int Hk, int N, int d, int rot,
                      int interleaved, float eps, int dtype, void* workspace,
                      size_t workspace_bytes, void* stream) {
  spa::NormRopeParams np{};
  const void* const in[2][2] = {{q, k}, {dq_out, dk_out}};
  void* const out[2] = {dq, dk};
  int st = norm_rope_params(np, in, 2, out, strides, wq, wk, pos, pos0, table, B, H, Hk, N, d, rot, interleaved,
                            eps, dtype);
  if (st && st != kEmpty) return st;
  if (!aligned4(dwq) || !aligned4(dwk) || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return SPA_ERR_ALIGN;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  float* const dw[2] = {H > 0 ? dwq : nullptr, Hk > 0 ? dwk : nullptr};
  if (st == kEmpty) {  // sums over no rows
    for (float* x : dw)
      if (x && cudaMemsetAsync(x, 0, static_cast<size_t>(d) * sizeof(float), s) != cudaSuccess) return SPA_ERR_CUDA;
    return SPA_OK;
  }
  size_t need = 0;
  if ((st = spa_norm_rope_bwd_workspace_size(d, &need))) return st;
  const bool sums = dw[0] || dw[1];
  if (workspace && workspace_bytes < need) return SPA_ERR_NOMEM;
  void* own = nullptr;
  if (!workspace && sums)
    if (int e = pool_alloc(&own, need, s)) return e;
  np.part = static_cast<float*>(workspace ? workspace : own);
  np.dw[0] = dw[0];
  np.dw[1] = dw[1];
  st = cuda_status(spa::launch_norm_rope(np, s));
  const cudaError_t fe = own ? cudaFreeAsync(own, s) : cudaSuccess;
  if (st) return st;
  return cuda_status(fe);
}

int spa_kcache8_pack_workspace_size(int B, size_t* bytes) {
  if (!bytes) return SPA_ERR_NULL;
  *bytes = 0;
  if (B < 0) return SPA_ERR_SHAPE;
  *bytes = align256(static_cast<size_t>(B) * 2 * sizeof(int));
  return SPA_OK;
}

int spa_kcache8_pack(void* kc, float* kc_mul, void* v, const int* lens, void* kc8, float* ks,
                     void* vc8, float* vs, const int* table, const int* blocks, int* lens_out,
                     int* blocks_out, int B, int Hk, int pages, int width, int m, int d_v, int cap,
                     void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_cache8(B, Hk, pages, width, m, d_v, cap);
  if (st) return st == kEmpty ? SPA_OK : st;
  if (!lens || !blocks || !lens_out || !blocks_out || (cap > 0 && (!kc || !kc_mul || !v)) ||
      (pages > 0 && (!kc8 || !ks || !vc8 || !vs)) || (width > 0 && !table))
    return SPA_ERR_NULL;
  if (!aligned16(kc) || !aligned16(v) || !aligned16(kc8) || !aligned16(vc8) || !aligned4(kc_mul) ||
      !aligned4(ks) || !aligned4(vs) || !aligned4(table) || !aligned4(blocks) || !aligned4(lens) ||
      !aligned4(lens_out) || !aligned4(blocks_out) || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return SPA_ERR_ALIGN;
  size_t need = 0;
  if ((st = spa_kcache8_pack_workspace_size(B, &need))) return st;
  if (workspace && workspace_bytes < need) return SPA_ERR_NOMEM;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  void* own = nullptr;
  if (!workspace)
    if (int e = pool_alloc(&own, need, s)) return e;
  spa::Pack8Params pp{};
  pp.kc = static_cast<uint16_t*>(kc);
  pp.kc_mul = kc_mul;
  pp.vc = static_cast<__nv_bfloat16*>(v);
  pp.lens = lens;
  pp.blocks = blocks;
  pp.lens_out = lens_out;
  pp.blocks_out = blocks_out;
  pp.pg = pages_of(kc8, ks, vc8, vs, table, pages, width);
  pp.ws = static_cast<int*>(workspace ? workspace : own);
  pp.B = B;
  pp.H = Hk;
  pp.m = m;
  pp.dv = d_v;
  pp.cap = cap;
  st = cuda_status(spa::launch_pack8(pp, s));
  const cudaError_t fe = own ? cudaFreeAsync(own, s) : cudaSuccess;
  if (st) return st;
  return cuda_status(fe);
}

int spa_attention_decode8_workspace_size(int B, int H, int Hk, int d, int m, int d_v, size_t* bytes) {
  if (!bytes) return SPA_ERR_NULL;
  const int st = check_decode_shared(B, H, Hk, 0, d, m, d_v, 0);
  *bytes = 0;
  if (st == kEmpty) return SPA_OK;
  if (st) return st;
  spa::Decode8Params dp{};
  dp.B = B;
  dp.H = H;
  dp.Hk = Hk;
  dp.G = H / Hk;
  dp.m = m;
  dp.dv = d_v;
  *bytes = spa::decode8_workspace(dp);
  return SPA_OK;
}

int spa_attention_decode8(const void* q, const void* P, const void* kc8, const float* ks,
                          const void* vc8, const float* vs, const int* table, const int* blocks,
                          const void* kc, const float* kc_mul, const void* v, const int* lens,
                          void* out, int B, int H, int Hk, int pages, int width, int window,
                          int sink, int d, int m, int d_v, int cap, int dtype, void* workspace,
                          size_t workspace_bytes, void* stream) {
  if (dtype != SPA_F32 && dtype != SPA_BF16) return SPA_ERR_DTYPE;
  int st = check_decode_shared(B, H, Hk, 0, d, m, d_v, cap);
  if (st == kEmpty) return SPA_OK;
  if (st) return st;
  if ((st = check_cache8(B, Hk, pages, width, m, d_v, cap))) return st;
  if (window < 0 || sink < 0) return SPA_ERR_SHAPE;
  if (dtype != SPA_BF16) return SPA_ERR_UNSUPPORTED;
  if (!q || !P || !out || (cap > 0 && (!kc || !kc_mul || !v || !lens)) ||
      (width > 0 && (!table || !blocks)) || (pages > 0 && (!kc8 || !ks || !vc8 || !vs)))
    return SPA_ERR_NULL;
  if (!aligned16(q) || !aligned16(P) || !aligned16(out) || !aligned16(kc) || !aligned16(v) ||
      !aligned16(kc8) || !aligned16(vc8) || !aligned4(kc_mul) || !aligned4(ks) || !aligned4(vs) ||
      !aligned4(table) || !aligned4(blocks) || !aligned4(lens) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return SPA_ERR_ALIGN;
  spa::Decode8Params dp{};
  dp.q = static_cast<const __nv_bfloat16*>(q);
  dp.P = static_cast<const __nv_bfloat16*>(P);
  dp.pg = pages_of(kc8, ks, vc8, vs, table, pages, width);
  dp.blocks = blocks;
  dp.kc = static_cast<const uint16_t*>(kc);
  dp.kc_mul = kc_mul;
  dp.vc = static_cast<const __nv_bfloat16*>(v);
  dp.lens = lens;
  dp.out = static_cast<__nv_bfloat16*>(out);
  dp.B = B;
  dp.H = H;
  dp.Hk = Hk;
  dp.G = H / Hk;
  dp.d = d;
  dp.m = m;
  dp.dv = d_v;
  dp.cap = cap;
  dp.window = window;
  dp.sink = sink;
  dp.qscale = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(m)));
  const size_t need = spa::decode8_workspace(dp);
  if (workspace && workspace_bytes < need) return SPA_ERR_NOMEM;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  void* own = nullptr;
  if (!workspace)
    if (int e = pool_alloc(&own, need, s)) return e;
  dp.ws = static_cast<char*>(workspace ? workspace : own);
  st = cuda_status(spa::launch_decode8(dp, s));
  const cudaError_t fe = own ? cudaFreeAsync(own, s) : cudaSuccess;
  if (st) return st;
  return cuda_status(fe);
}

int spa_topk_features(const void* x, void* y, long long rows, int d, int k, int dtype,
                      void* stream) {
  return topk_features(x, y, rows, d, k, dtype, static_cast<cudaStream_t>(stream));
}

int spa_sfa_attention_fwd(const void* q, const void* k, const void* v, float* out, int B, int H,
                          int N, int d, int d_v, int topk, int causal, int dtype, void* stream) {
  // the forward with P = I_d (m = d): scale 1/sqrt(d) on the sparsified rows
  int st = check_shape(B, H, N, d, d, d_v, dtype);
  if (st == kEmpty) return SPA_OK;
  if (st) return st;
  if (d != 32 && d != 64 && d != 128) return SPA_ERR_UNSUPPORTED;
  if (topk < 1 || topk > d) return SPA_ERR_SHAPE;
  if (!q || !k || !v || !out) return SPA_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out)) return SPA_ERR_ALIGN;
  const size_t es = dtype == SPA_BF16 ? 2 : 4;
  const long long rows = static_cast<long long>(B) * H * N;
  const size_t nq = static_cast<size_t>(rows) * d * es;
  const size_t np = static_cast<size_t>(H) * d * d * es;
  const size_t oq = 0, ok = align256(oq + nq), op = align256(ok + nq), ow = align256(op + np);
  const size_t total = ow + make_layout(B, H, N, d, dtype).total;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* buf = nullptr;
  if (int e = pool_alloc(reinterpret_cast<void**>(&buf), total, s)) return e;
  st = spa_topk_features(q, buf + oq, rows, d, topk, dtype, stream);
  if (!st) st = spa_topk_features(k, buf + ok, rows, d, topk, dtype, stream);
  if (!st) st = cuda_status(spa::launch_identity(buf + op, H, d, dtype == SPA_BF16, s));
  if (!st)
    st = run_forward(buf + oq, buf + ok, v, buf + op, out, B, H, N, d, d, d_v, causal, dtype,
                     buf + ow, s);
  const cudaError_t fe = cudaFreeAsync(buf, s);
  if (st) return st;
  return fe == cudaSuccess ? SPA_OK : SPA_ERR_CUDA;
}

int spa_attention_bwd(const void* q, const void* k, const void* v, const void* P,
                      const float* out, const void* dO, float* dq, float* dk, float* dv,
                      float* dP, int B, int H, int N, int d, int m, int d_v, int causal, int dtype,
                      void* stream) {
  return backward_entry(q, k, v, P, out, nullptr, dO, dq, dk, dv, dP, B, H, N, d, m, d_v, causal,
                        dtype, stream);
}

int spa_attention_bwd_lse(const void* q, const void* k, const void* v, const void* P,
                          const float* out, const float* lse, const void* dO, float* dq, float* dk,
                          float* dv, float* dP, int B, int H, int N, int d, int m, int d_v,
                          int causal, int dtype, void* stream) {
  const int st = check_shape(B, H, N, d, m, d_v, dtype);
  if (st != kEmpty && st) return st;
  if (st != kEmpty && !lse) return SPA_ERR_NULL;
  return backward_entry(q, k, v, P, out, lse, dO, dq, dk, dv, dP, B, H, N, d, m, d_v, causal, dtype,
                        stream);
}

int spa_attention_fwd_lse(const void* q, const void* k, const void* v, const void* P, float* out,
                          float* lse, int B, int H, int N, int d, int m, int d_v, int causal,
                          int dtype, void* stream) {
  int st = check_shape(B, H, N, d, m, d_v, dtype);
  if (st == kEmpty) return SPA_OK;
  if (st) return st;
  if ((st = check_forward_ptrs(q, k, v, P, out))) return st;
  if (!lse) return SPA_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(lse) & 3u) return SPA_ERR_ALIGN;
  const size_t bytes = make_layout(B, H, N, m, dtype).total;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  void* ws = nullptr;
  if (int e = pool_alloc(&ws, bytes, s)) return e;
  st = run_prepare(q, k, P, B, H, N, d, m, dtype, ws, s);
  if (!st) st = run_apply(v, out, B, H, N, m, d_v, causal, dtype, ws, s, kWaitLimitNs, 0, lse);
  const cudaError_t fe = cudaFreeAsync(ws, s);
  if (st) return st;
  return cuda_status(fe);
}

int spa_attention_bwd_workspace_size(int B, int H, int N, int d, int m, int d_v, int dtype,
                                     size_t* bytes) {
  if (!bytes) return SPA_ERR_NULL;
  const int st = check_shape(B, H, N, d, m, d_v, dtype);
  if (st == kEmpty) {
    *bytes = 0;
    return SPA_OK;
  }
  if (st) return st;
  if (!bwd_fused_eligible(d, m, d_v, dtype)) return SPA_ERR_UNSUPPORTED;
  *bytes = make_bwd_layout(B, H, N, d, m, d_v, false).total;
  return SPA_OK;
}

int spa_attention_bwd_prepare(const void* q, const void* k, const void* P, const float* out,
                              const float* lse, const void* dO, int B, int H, int N, int d, int m,
                              int d_v, int dtype, void* workspace, size_t workspace_bytes,
                              void* stream) {
  int st = check_bwd_staged(B, H, N, d, m, d_v, dtype, workspace, workspace_bytes);
  if (st == kEmpty) return SPA_OK;
  if (st) return st;
  if (!q || !k || !P || !out || !lse || !dO) return SPA_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(P) || !aligned16(out) || !aligned16(dO))
    return SPA_ERR_ALIGN;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* w = static_cast<char*>(workspace);
  const BwdLayout L = make_bwd_layout(B, H, N, d, m, d_v, false);
  if ((st = run_prepare(q, k, P, B, H, N, d, m, SPA_BF16, w, s, w + L.qb, w + L.kb))) return st;
  return bwd_stage_inputs(out, lse, dO, B, H, N, d, m, d_v, w, s);
}

int spa_attention_bwd_apply(const void* v, const void* dO, float* dv, int B, int H, int N, int d,
                            int m, int d_v, int causal, int dtype, void* workspace,
                            size_t workspace_bytes, void* stream) {
  int st = check_bwd_staged(B, H, N, d, m, d_v, dtype, workspace, workspace_bytes);
  if (st == kEmpty) return SPA_OK;
  if (st) return st;
  if (!v || !dO || !dv) return SPA_ERR_NULL;
  if (!aligned16(v) || !aligned16(dO) || !aligned16(dv)) return SPA_ERR_ALIGN;
  return bwd_stage_kernel(v, dO, dv, B, H, N, d, m, d_v, causal, static_cast<char*>(workspace),
                          static_cast<cudaStream_t>(stream));
}

int spa_attention_bwd_finish(const void* q, const void* k, const void* P, float* dq, float* dk,
                             float* dP, int B, int H, int N, int d, int m, int d_v, int dtype,
                             void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_bwd_staged(B, H, N, d, m, d_v, dtype, workspace, workspace_bytes);
  if (st == kEmpty) {
    if (!dP) return SPA_ERR_NULL;
    if (H > 0 && d > 0 && m > 0 &&
        cudaMemsetAsync(dP, 0, static_cast<size_t>(H) * d * m * sizeof(float),
                        static_cast<cudaStream_t>(stream)) != cudaSuccess)
      return SPA_ERR_CUDA;
    return SPA_OK;
  }
  if (st) return st;
  if (!q || !k || !P || !dq || !dk || !dP) return SPA_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(P) || !aligned16(dq) || !aligned16(dk) ||
      !aligned16(dP))
    return SPA_ERR_ALIGN;
  return bwd_stage_finish(q, k, P, dq, dk, dP, B, H, N, d, m, d_v, static_cast<char*>(workspace),
                          static_cast<cudaStream_t>(stream));
}

int spa_host_pool_trim(void) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return SPA_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_host_pool_mu);
  if (g_host_pool[dev] && cudaMemPoolTrimTo(g_host_pool[dev], 0) != cudaSuccess) return SPA_ERR_CUDA;
  return SPA_OK;
}

int spa_selftest_wait_timeout(int limit_ms) {
  if (limit_ms <= 0 || limit_ms > 2000) return SPA_ERR_SHAPE;
  constexpr int B = 1, H = 1, N = 256, d = 64, m = 32, dv = 64;
  const size_t nq = static_cast<size_t>(N) * d * 2, nv = static_cast<size_t>(N) * dv * 2;
  const size_t np = static_cast<size_t>(d) * m * 2, no = static_cast<size_t>(N) * dv * 4;
  const size_t oq = 0, ok = align256(oq + nq), ov = align256(ok + nq), op = align256(ov + nv),
               oo = align256(op + np), ow = align256(oo + no);
  const size_t total = ow + make_layout(B, H, N, m, SPA_BF16).total;
  int* err = nullptr;
  int st = device_error_ptr(&err);
  if (st) return st;
  char* buf = nullptr;
  if (cudaMalloc(reinterpret_cast<void**>(&buf), total) != cudaSuccess) {
    cudaGetLastError();
    return SPA_ERR_NOMEM;
  }
  st = cuda_status(cudaMemset(buf, 0, total));  // zero inputs: every score is 0
  if (!st) st = run_prepare(buf + oq, buf + ok, buf + op, B, H, N, d, m, SPA_BF16, buf + ow, nullptr);
  if (!st)
    st = run_apply(buf + ov, reinterpret_cast<float*>(buf + oo), B, H, N, m, dv, 0, SPA_BF16,
                   buf + ow, nullptr, static_cast<unsigned long long>(limit_ms) * 1000000ull, 1);
  if (!st) st = cuda_status(cudaDeviceSynchronize());
  int word = 0;
  if (!st) st = cuda_status(cudaMemcpy(&word, err, sizeof word, cudaMemcpyDeviceToHost));
  const int zero = 0;
  if (!st) st = cuda_status(cudaMemcpy(err, &zero, sizeof zero, cudaMemcpyHostToDevice));
  cudaFree(buf);
  if (st) return st;
  return word ? SPA_ERR_TIMEOUT : SPA_OK;
}

int spa_selftest_proj_wait_timeout(int limit_ms, int m) {
  if (limit_ms <= 0 || limit_ms > 2000) return SPA_ERR_SHAPE;
  if (m != 32 && m != 64) return SPA_ERR_UNSUPPORTED;
  // m = 32 runs the per-CTA projection kernel, m = 64 the warp-specialised
  // one; 512 tiles, so each CTA of either takes one to four of them
  constexpr int B = 1, H = 8, N = 4096, d = 64;
  const size_t nq = static_cast<size_t>(B) * H * N * d * 2, np = static_cast<size_t>(H) * d * m * 2;
  const size_t oq = 0, ok = align256(oq + nq), op = align256(ok + nq), ow = align256(op + np);
  const size_t total = ow + make_layout(B, H, N, m, SPA_BF16).total;
  int* err = nullptr;
  int st = device_error_ptr(&err);
  if (st) return st;
  char* buf = nullptr;
  if (cudaMalloc(reinterpret_cast<void**>(&buf), total) != cudaSuccess) {
    cudaGetLastError();
    return SPA_ERR_NOMEM;
  }
  st = cuda_status(cudaMemset(buf, 0, total));  // zero inputs
  if (!st)
    st = run_prepare(buf + oq, buf + ok, buf + op, B, H, N, d, m, SPA_BF16, buf + ow, nullptr,
                     nullptr, nullptr, static_cast<unsigned long long>(limit_ms) * 1000000ull, 1);
  if (!st) st = cuda_status(cudaDeviceSynchronize());
  int word = 0;
  if (!st) st = cuda_status(cudaMemcpy(&word, err, sizeof word, cudaMemcpyDeviceToHost));
  const int zero = 0;
  if (!st) st = cuda_status(cudaMemcpy(err, &zero, sizeof zero, cudaMemcpyHostToDevice));
  cudaFree(buf);
  if (st) return st;
  return word ? SPA_ERR_TIMEOUT : SPA_OK;
}

int spa_selftest_copy_wait_timeout(int limit_ms, int kernel) {
  if (limit_ms <= 0 || limit_ms > 2000) return SPA_ERR_SHAPE;
  if (kernel < 0 || kernel > 2) return SPA_ERR_UNSUPPORTED;
  // 8 heads of 4096 rows (d = 64, m = 32, d_v = 128): 256 row blocks for the
  // statistics and the Top-k kernels, 512 tiles for the finish
  constexpr int B = 1, H = 8, N = 4096, d = 64, m = 32, dv = 128, topk_d = 128, topk_k = 16;
  const size_t rows = static_cast<size_t>(B) * H * N;
  const BwdLayout L = make_bwd_layout(B, H, N, d, m, dv, false);
  const size_t nx = rows * d * 2, np = static_cast<size_t>(H) * d * m * 2;
  const size_t ndo = rows * dv * 2, nout = rows * dv * 4, nlse = rows * 4, ng = rows * d * 4;
  const size_t ndp = static_cast<size_t>(H) * d * m * 4, nt = rows * topk_d * 2;
  const size_t oq = 0, ok = align256(oq + nx), op = align256(ok + nx), odo = align256(op + np),
               oo = align256(odo + ndo), ol = align256(oo + nout), odq = align256(ol + nlse),
               odk = align256(odq + ng), odp = align256(odk + ng), ox = align256(odp + ndp),
               oy = align256(ox + nt), ow = align256(oy + nt);
  const size_t total = ow + L.total;
  int* err = nullptr;
  int st = device_error_ptr(&err);
  if (st) return st;
  char* buf = nullptr;
  if (cudaMalloc(reinterpret_cast<void**>(&buf), total) != cudaSuccess) {
    cudaGetLastError();
    return SPA_ERR_NOMEM;
  }
  st = cuda_status(cudaMemset(buf, 0, total));  // zero inputs, statistics and accumulators
  const unsigned long long lim = static_cast<unsigned long long>(limit_ms) * 1000000ull;
  char* w = buf + ow;
  if (!st && kernel == 0)
    st = bwd_stage_inputs(reinterpret_cast<const float*>(buf + oo),
                          reinterpret_cast<const float*>(buf + ol), buf + odo, B, H, N, d, m, dv, w,
                          nullptr, lim, 1);
  if (!st && kernel == 1)
    st = bwd_stage_finish(buf + oq, buf + ok, buf + op, reinterpret_cast<float*>(buf + odq),
                          reinterpret_cast<float*>(buf + odk), reinterpret_cast<float*>(buf + odp),
                          B, H, N, d, m, dv, w, nullptr, lim, 1);
  if (!st && kernel == 2)
    st = topk_features(buf + ox, buf + oy, static_cast<long long>(rows), topk_d, topk_k, SPA_BF16,
                       nullptr, lim, 1);
  if (!st) st = cuda_status(cudaDeviceSynchronize());
  int word = 0;
  if (!st) st = cuda_status(cudaMemcpy(&word, err, sizeof word, cudaMemcpyDeviceToHost));
  const int zero = 0;
  if (!st) st = cuda_status(cudaMemcpy(err, &zero, sizeof zero, cudaMemcpyHostToDevice));
  cudaFree(buf);
  if (st) return st;
  return word ? SPA_ERR_TIMEOUT : SPA_OK;
}

int spa_selftest_bwd_wait_timeout(int limit_ms) {
  if (limit_ms <= 0 || limit_ms > 2000) return SPA_ERR_SHAPE;
  constexpr int B = 1, H = 1, N = 256, d = 64, m = 32, dv = 64;
  const size_t nq = static_cast<size_t>(N) * d * 2, nv = static_cast<size_t>(N) * dv * 2;
  const size_t np = static_cast<size_t>(d) * m * 2, no = static_cast<size_t>(N) * dv * 4;
  const size_t nl = static_cast<size_t>(N) * 4;
  const size_t oq = 0, ok = align256(oq + nq), ov = align256(ok + nq), op = align256(ov + nv),
               odo = align256(op + np), oo = align256(odo + nv), ol = align256(oo + no),
               odv = align256(ol + nl), ow = align256(odv + no);
  const BwdLayout L = make_bwd_layout(B, H, N, d, m, dv, false);
  const size_t total = ow + L.total;
  int* err = nullptr;
  int st = device_error_ptr(&err);
  if (st) return st;
  char* buf = nullptr;
  if (cudaMalloc(reinterpret_cast<void**>(&buf), total) != cudaSuccess) {
    cudaGetLastError();
    return SPA_ERR_NOMEM;
  }
  // zero inputs and log-sum-exp: every value the kernel computes is finite
  st = cuda_status(cudaMemset(buf, 0, total));
  char* w = buf + ow;
  if (!st)
    st = run_prepare(buf + oq, buf + ok, buf + op, B, H, N, d, m, SPA_BF16, w, nullptr, w + L.qb,
                     w + L.kb);
  if (!st)
    st = bwd_stage_inputs(reinterpret_cast<const float*>(buf + oo),
                          reinterpret_cast<const float*>(buf + ol), buf + odo, B, H, N, d, m, dv, w,
                          nullptr);
  if (!st)
    st = bwd_stage_kernel(buf + ov, buf + odo, reinterpret_cast<float*>(buf + odv), B, H, N, d, m,
                          dv, 1, w, nullptr, static_cast<unsigned long long>(limit_ms) * 1000000ull,
                          1);
  if (!st) st = cuda_status(cudaDeviceSynchronize());
  int word = 0;
  if (!st) st = cuda_status(cudaMemcpy(&word, err, sizeof word, cudaMemcpyDeviceToHost));
  const int zero = 0;
  if (!st) st = cuda_status(cudaMemcpy(err, &zero, sizeof zero, cudaMemcpyHostToDevice));
  cudaFree(buf);
  if (st) return st;
  return word ? SPA_ERR_TIMEOUT : SPA_OK;
}

int spa_selftest_window_wait_timeout(int limit_ms, int kernel) {
  if (limit_ms <= 0 || limit_ms > 2000) return SPA_ERR_SHAPE;
  if (kernel < 0 || kernel > 1) return SPA_ERR_UNSUPPORTED;
  constexpr int B = 1, H = 2, Hk = 1, N = 512, d = 64, m = 32, dv = 64, window = 200, sink = 4;
  const size_t nq = static_cast<size_t>(H) * N * d * 2, no = static_cast<size_t>(H) * N * dv * 2;
  const size_t np = static_cast<size_t>(d) * m * 2, nl = static_cast<size_t>(H) * N * 4;
  // q, k, v, P, out, out_lo, lse, dO and the four gradients, each at the size of the largest
  const size_t each = align256(std::max(std::max(nq, no), std::max(np, nl)));
  const size_t total = 12 * each + window_layout(B, H, Hk, N, d, m, dv, window, sink, true).total;
  int* err = nullptr;
  int st = device_error_ptr(&err);
  if (st) return st;
  char* buf = nullptr;
  if (cudaMalloc(reinterpret_cast<void**>(&buf), total) != cudaSuccess) {
    cudaGetLastError();
    return SPA_ERR_NOMEM;
  }
  // zero inputs and log-sum-exp: every value the kernels compute is finite
  st = cuda_status(cudaMemset(buf, 0, total));
  char* at[13];
  for (int i = 0; i < 13; ++i) at[i] = buf + i * each;
  const unsigned long long limit_ns = static_cast<unsigned long long>(limit_ms) * 1000000ull;
  if (!st && kernel == 0)
    st = window_forward(at[0], at[1], at[2], at[3], at[4], at[5], reinterpret_cast<float*>(at[6]), B, H, Hk, N, d, m, dv,
                        window, sink, at[12], nullptr, limit_ns, 1);
  if (!st && kernel == 1)
    st = window_backward(at[0], at[1], at[2], at[3], at[4], at[5], reinterpret_cast<const float*>(at[6]), at[7], at[8],
                         at[9], at[10], at[11], B, H, Hk, N, d, m, dv, window, sink, at[12], nullptr, limit_ns, 1);
  if (!st) st = cuda_status(cudaDeviceSynchronize());
  int word = 0;
  if (!st) st = cuda_status(cudaMemcpy(&word, err, sizeof word, cudaMemcpyDeviceToHost));
  const int zero = 0;
  if (!st) st = cuda_status(cudaMemcpy(err, &zero, sizeof zero, cudaMemcpyHostToDevice));
  cudaFree(buf);
  if (st) return st;
  return word ? SPA_ERR_TIMEOUT : SPA_OK;
}

int spa_selftest_decode_wait_timeout(int limit_ms, int kernel) {
  if (limit_ms <= 0 || limit_ms > 2000) return SPA_ERR_SHAPE;
  if (kernel < 0 || kernel > 1) return SPA_ERR_UNSUPPORTED;
  // two sequences, four query heads on one key head; the prefix kernel alone or
  // the kernel of the sequences' own rows alone
  constexpr int B = 2, H = 4, Hk = 1, d = 64, m = 32, dv = 64, rows = 1024;
  const int plen = kernel == 0 ? rows : 0, cap = kernel == 1 ? rows : 0;
  spa::DecodeSharedParams dp{};
  int st = decode_shared_sizes(dp, B, H, Hk, plen, d, m, dv, cap);
  if (st) return st;
  const size_t nq = static_cast<size_t>(B) * H * d * 2, np = static_cast<size_t>(Hk) * d * m * 2;
  const size_t nk = static_cast<size_t>(B) * Hk * rows * m * 2, ne = static_cast<size_t>(B) * Hk * rows * 4;
  const size_t nv = static_cast<size_t>(B) * Hk * rows * dv * 2, no = static_cast<size_t>(B) * H * dv * 2;
  const size_t oq = 0, op = align256(oq + nq), ok = align256(op + np), oe = align256(ok + nk),
               ov = align256(oe + ne), ol = align256(ov + nv), oo = align256(ol + B * sizeof(int)),
               ow = align256(oo + no);
  const size_t total = ow + spa::decode_shared_workspace(dp);
  int* err = nullptr;
  if ((st = device_error_ptr(&err))) return st;
  char* buf = nullptr;
  if (cudaMalloc(reinterpret_cast<void**>(&buf), total) != cudaSuccess) {
    cudaGetLastError();
    return SPA_ERR_NOMEM;
  }
  st = cuda_status(cudaMemset(buf, 0, total));  // zero inputs
  if (!st) st = cuda_status(cudaMemset(buf + ol, 1, B * sizeof(int)));  // lengths beyond the capacity: all rows
  dp.q = reinterpret_cast<const __nv_bfloat16*>(buf + oq);
  dp.P = reinterpret_cast<const __nv_bfloat16*>(buf + op);
  dp.kc = dp.pkc = reinterpret_cast<const uint16_t*>(buf + ok);
  dp.kc_mul = dp.pkc_mul = reinterpret_cast<const float*>(buf + oe);
  dp.v = dp.pv = reinterpret_cast<const __nv_bfloat16*>(buf + ov);
  dp.lens = reinterpret_cast<const int*>(buf + ol);
  dp.out = reinterpret_cast<__nv_bfloat16*>(buf + oo);
  dp.pcap = plen;
  dp.ws = buf + ow;
  if (!st) st = run_decode_shared(dp, nullptr, static_cast<unsigned long long>(limit_ms) * 1000000ull, 1);
  if (!st) st = cuda_status(cudaDeviceSynchronize());
  int word = 0;
  if (!st) st = cuda_status(cudaMemcpy(&word, err, sizeof word, cudaMemcpyDeviceToHost));
  const int zero = 0;
  if (!st) st = cuda_status(cudaMemcpy(err, &zero, sizeof zero, cudaMemcpyHostToDevice));
  cudaFree(buf);
  if (st) return st;
  return word ? SPA_ERR_TIMEOUT : SPA_OK;
}

int spa_device_error(int* code) {
  if (!code) return SPA_ERR_NULL;
  int* p = nullptr;
  int st = device_error_ptr(&p);
  if (st) return st;
  if (cudaDeviceSynchronize() != cudaSuccess) return SPA_ERR_CUDA;
  int v = 0;
  if (cudaMemcpy(&v, p, sizeof v, cudaMemcpyDeviceToHost) != cudaSuccess) return SPA_ERR_CUDA;
  const int zero = 0;
  if (cudaMemcpy(p, &zero, sizeof zero, cudaMemcpyHostToDevice) != cudaSuccess) return SPA_ERR_CUDA;
  *code = v ? SPA_ERR_TIMEOUT : SPA_OK;
  return SPA_OK;
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Allocation-free forward.  Some callers cannot allocate device memory while
// they run: code that executes inside a framework that owns all device memory
// and forbids cudaMalloc (or is itself inside an allocator callback), real-time
// loops that must not touch the driver's allocator, or processes whose memory
// budget is fixed up front.  For them the forward can use a scratch buffer that
// the library carries as a file-scope device array, sized once at compile time.
// ---------------------------------------------------------------------------
namespace {

constexpr size_t kNoAllocScratchBytes = size_t(64) << 20;  // 64 MiB per device

// Scratch for the score-operand tiles / projections of spa_attention_fwd_noalloc.
// In host code this symbol is only a stand-in: its device address comes from
// cudaGetSymbolAddress, taken per device below.
static __device__ __align__(256) unsigned char g_noalloc_scratch[kNoAllocScratchBytes];

void* g_noalloc_ptr[kMaxDevices] = {};
std::mutex g_noalloc_mu;

// Once per device, with that device current: the device address of the array.
int noalloc_scratch(void** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return SPA_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_noalloc_mu);
  if (!g_noalloc_ptr[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_noalloc_scratch) != cudaSuccess || !p) return SPA_ERR_CUDA;
    g_noalloc_ptr[dev] = p;
  }
  *out = g_noalloc_ptr[dev];
  return SPA_OK;
}

}  // namespace

extern "C" int spa_attention_fwd_noalloc(const void* q, const void* k, const void* v,
                                         const void* P, float* out, int B, int H, int N, int d,
                                         int m, int d_v, int causal, int dtype, void* stream) {
  int st = check_shape(B, H, N, d, m, d_v, dtype);
  if (st == kEmpty) return SPA_OK;
  if (st) return st;
  if ((st = check_forward_ptrs(q, k, v, P, out))) return st;
  if (make_layout(B, H, N, m, dtype).total > kNoAllocScratchBytes) return SPA_ERR_NOMEM;
  void* scratch = nullptr;
  if ((st = noalloc_scratch(&scratch))) return st;
  // Every scratch byte the attention stage reads is written first by this
  // call's projection stage, so nothing has to be cleared between calls.
  return run_forward(q, k, v, P, out, B, H, N, d, m, d_v, causal, dtype, scratch,
                     static_cast<cudaStream_t>(stream));
}
