// C ABI of the operators (see include/gdit.h): argument checks and launches.
#include <cfloat>
#include <cmath>
#include <mutex>
#include <new>
#include <utility>

#include "ops_attention.cuh"
#include "ops_linear.cuh"
#include "ops_norm.cuh"

using namespace gdit;

namespace {

template <typename F>
int guarded_op(F&& fn) {
  try {
    g_create_error.clear();
    fn();
    return GDIT_OK;
  } catch (const GditError& e) {
    try {
      g_create_error = e.what();
    } catch (...) {
    }
    return e.code;
  } catch (const std::bad_alloc&) {
    return GDIT_ENOMEM;
  } catch (...) {
    return GDIT_ECUDA;
  }
}

// The current device, checked once: its SMs.
int current_sms() {
  static std::mutex mu;
  static int sms[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    throw GditError(GDIT_ENODEV, "no CUDA device");
  }
  if (dev < 0 || dev >= kMaxDevices) throw GditError(GDIT_ENODEV, fmt("device ordinal %d out of range", dev));
  std::lock_guard<std::mutex> lock(mu);
  if (sms[dev] == 0) {
    int major = 0, n = 0;
    CUDA_TRY(cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev));
    CUDA_TRY(cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev));
    if (major != 10) throw GditError(GDIT_ENODEV, fmt("device %d is not an sm_100 device", dev));
    sms[dev] = n;
  }
  return sms[dev];
}

// A device made current, and the one before again at the end.
struct DeviceGuard {
  int before = 0;
  explicit DeviceGuard(int device) {
    CUDA_TRY(cudaGetDevice(&before));
    CUDA_TRY(cudaSetDevice(device));
  }
  ~DeviceGuard() { cudaSetDevice(before); }
};

bool is_dtype(int t) { return t == GDIT_F32 || t == GDIT_BF16; }
int size_of(int t) { return t == GDIT_F32 ? 4 : 2; }
bool aligned_to(const void* p, int bytes) { return ((uintptr_t)p % (uintptr_t)bytes) == 0; }

// Strides times sizes stay far inside 64 bits.
constexpr int64_t kMaxStride = (int64_t)1 << 40;
// Rows, columns and keys: the last tile's end still fits 32 bits.
constexpr int64_t kMaxRows = (int64_t)INT32_MAX - 1024;

// Checks the arguments of a product; false where there is nothing to do.
bool linear_args(const gdit_linear_args* p, LinearArgs& a) {
  REQUIRE(p != nullptr, "NULL arguments");
  REQUIRE(p->m >= 0 && p->m <= kMaxRows, "m %lld out of range", (long long)p->m);
  REQUIRE(p->n >= 1 && p->k >= 8 && p->k % 8 == 0, "need n >= 1 and k >= 8, a multiple of 8 (n %d, k %d)", p->n, p->k);
  REQUIRE(p->n <= kMaxRows && p->k <= kMaxRows, "n %d or k %d out of range", p->n, p->k);
  REQUIRE(is_dtype(p->out_dtype), "out_dtype %d", p->out_dtype);
  REQUIRE(p->activation >= GDIT_ACT_NONE && p->activation <= GDIT_ACT_SILU, "activation %d", p->activation);
  if (p->m == 0) return false;
  REQUIRE(p->x && p->w && p->out, "NULL matrix");
  const int es = size_of(p->out_dtype);
  REQUIRE(p->ldx >= p->k && p->ldx % 8 == 0 && p->ldx <= kMaxStride, "ldx %lld: at least k and a multiple of 8", (long long)p->ldx);
  REQUIRE(p->ldw >= p->k && p->ldw % 8 == 0 && p->ldw <= kMaxStride, "ldw %lld: at least k and a multiple of 8", (long long)p->ldw);
  REQUIRE(p->ldo >= p->n && p->ldo <= kMaxStride, "ldo %lld below n", (long long)p->ldo);
  REQUIRE(p->residual == nullptr || (p->ldr >= p->n && p->ldr <= kMaxStride), "ldr %lld below n", (long long)p->ldr);
  REQUIRE(aligned_to(p->x, 16) && aligned_to(p->w, 16), "x and w must be 16-byte aligned");
  REQUIRE(aligned_to(p->out, es) && aligned_to(p->residual, es) && aligned_to(p->bias, 4),
          "bias, residual or out not aligned to its element");
  a.x = static_cast<const __nv_bfloat16*>(p->x);
  a.w = static_cast<const __nv_bfloat16*>(p->w);
  a.bias = p->bias;
  a.residual = p->residual;
  a.out = p->out;
  a.m = p->m, a.ldx = p->ldx, a.ldw = p->ldw, a.ldr = p->ldr, a.ldo = p->ldo;
  a.n = p->n, a.k = p->k;
  a.out_f32 = p->out_dtype == GDIT_F32;
  a.act = p->activation;
  return true;
}

__global__ void clear_status_kernel(unsigned bits) { atomicAnd(&g_op_status, ~bits); }

// Two warps and the operators' three waits on a barrier that nothing arrives at: the
// first runs out, the others end with it.
__global__ void op_wait_expiry_kernel(unsigned long long limit_ns) {
  __shared__ __align__(8) uint64_t bar;
  __shared__ volatile int s_abort;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    fence_mbar_init();
    s_abort = 0;
  }
  __syncthreads();
  if (threadIdx.x == 0) op_wait(&bar, 0, &s_abort, limit_ns);
  __syncwarp();
  op_wait_through(&bar, 0, &s_abort);
  op_wait_warp_cluster(&bar, 0, &s_abort);
  __syncthreads();
  if (threadIdx.x == 0) op_leave(&s_abort);
}

}  // namespace

extern "C" {

int gdit_linear(const gdit_linear_args* p, void* cuda_stream) {
  return guarded_op([&] {
    LinearArgs a;
    if (!linear_args(p, a)) return;
    launch_linear(a, current_sms(), (cudaStream_t)cuda_stream);
  });
}

int gdit_debug_linear_plan(const gdit_linear_args* p, int num_sms, int* pair, int* bn, int* splits) {
  return guarded_op([&] {
    LinearArgs a;
    REQUIRE(pair && bn && splits, "NULL output");
    REQUIRE(num_sms == 0 || num_sms >= 8, "num_sms %d: 0, or at least 8", num_sms);   // (a cluster of 8)
    REQUIRE(linear_args(p, a), "no rows");
    SplitSlots slots = {{0}};
    for (int n = 1; n <= 8; ++n) slots.of[n] = num_sms / n * n;
    const int sms = num_sms > 0 ? num_sms : current_sms();
    const LinearPlan plan = plan_linear(a, sms, num_sms > 0 ? slots : split_slots(sms));
    *pair = plan.pair_bn > 0;
    *bn = plan.pair_bn > 0 ? plan.pair_bn : plan.split.bn;
    *splits = plan.pair_bn > 0 ? 1 : plan.split.splits;
  });
}

int gdit_norm_residual(const gdit_norm_args* p, void* cuda_stream) {
  return guarded_op([&] {
    REQUIRE(p != nullptr, "NULL arguments");
    REQUIRE(p->rows >= 0 && p->rows <= ((int64_t)1 << 40), "rows %lld out of range", (long long)p->rows);
    REQUIRE(p->dim >= 1 && p->dim <= 16384, "dim %d: 1 to 16384", p->dim);
    REQUIRE(is_dtype(p->h_dtype) && is_dtype(p->y_dtype) && is_dtype(p->u_dtype), "dtype codes %d %d %d", p->h_dtype,
            p->y_dtype, p->u_dtype);
    for (int k : {p->post, p->pre}) REQUIRE(k >= GDIT_NORM_NONE && k <= GDIT_NORM_RMS, "norm kind %d", k);
    REQUIRE(p->gate_groups >= 1 && p->mod_groups >= 1, "group counts must be at least 1");
    REQUIRE((p->gate_groups == 1 && p->mod_groups == 1) || p->row_group != nullptr || p->rows == 0,
            "several groups need row_group");
    REQUIRE(std::isfinite(p->eps) && p->eps >= 0.f, "eps must be finite and not negative");
    REQUIRE(std::isfinite(p->residual_scale), "residual_scale must be finite");
    REQUIRE(p->y != nullptr || (p->post == GDIT_NORM_NONE && p->gate == nullptr), "post and gate need y");
    if (p->rows == 0) return;
    REQUIRE(p->h != nullptr, "NULL h");
    REQUIRE(p->out_h != nullptr || p->out_u != nullptr, "out_h and out_u are both NULL");
    const int hs = size_of(p->h_dtype), ys = size_of(p->y_dtype), us = size_of(p->u_dtype);
    auto ld_ok = [&](int64_t ld) { return ld >= p->dim && ld <= kMaxStride; };
    REQUIRE(ld_ok(p->ldh), "ldh %lld below dim", (long long)p->ldh);
    REQUIRE(p->y == nullptr || ld_ok(p->ldy), "ldy %lld below dim", (long long)p->ldy);
    REQUIRE(p->out_h == nullptr || ld_ok(p->ldoh), "ldoh %lld below dim", (long long)p->ldoh);
    REQUIRE(p->out_u == nullptr || ld_ok(p->ldou), "ldou %lld below dim", (long long)p->ldou);
    REQUIRE(aligned_to(p->h, hs) && aligned_to(p->y, ys) && aligned_to(p->out_h, hs) && aligned_to(p->out_u, us),
            "a matrix is not aligned to its element");
    for (const void* v : {(const void*)p->post_gain, (const void*)p->post_bias, (const void*)p->gate,
                          (const void*)p->pre_gain, (const void*)p->pre_bias, (const void*)p->scale,
                          (const void*)p->shift, (const void*)p->row_group})
      REQUIRE(aligned_to(v, 4), "a vector is not aligned to its element");
    const int sms = current_sms();
    NormArgs a;
    a.h = p->h, a.y = p->y, a.out_h = p->out_h, a.out_u = p->out_u;
    a.post_gain = p->post_gain, a.post_bias = p->post_bias, a.gate = p->gate;
    a.pre_gain = p->pre_gain, a.pre_bias = p->pre_bias, a.scale = p->scale, a.shift = p->shift;
    a.row_group = p->row_group;
    a.rows = p->rows, a.ldh = p->ldh, a.ldy = p->ldy, a.ldoh = p->ldoh, a.ldou = p->ldou;
    a.dim = p->dim;
    a.h_f32 = p->h_dtype == GDIT_F32, a.y_f32 = p->y_dtype == GDIT_F32, a.u_f32 = p->u_dtype == GDIT_F32;
    a.post = p->post, a.pre = p->pre;
    a.gate_groups = p->gate != nullptr ? p->gate_groups : 1;
    a.mod_groups = p->scale != nullptr || p->shift != nullptr ? p->mod_groups : 1;
    a.residual_scale = p->residual_scale, a.eps = p->eps;
    launch_norm(a, sms, (cudaStream_t)cuda_stream);
  });
}

int gdit_attention(const gdit_attention_args* p, void* cuda_stream) {
  return guarded_op([&] {
    REQUIRE(p != nullptr, "NULL arguments");
    REQUIRE(p->batch >= 0 && p->batch <= 65535, "batch %d: 0 to 65535", p->batch);
    REQUIRE(p->kv_heads >= 1 && p->heads >= p->kv_heads && p->heads % p->kv_heads == 0 && p->heads <= 65535,
            "heads %d must be a multiple of kv_heads %d", p->heads, p->kv_heads);
    REQUIRE(p->heads / p->kv_heads <= 128, "heads / kv_heads %d above 128", p->heads / p->kv_heads);
    REQUIRE(p->head_dim >= 8 && p->head_dim <= 128 && p->head_dim % 8 == 0, "head_dim %d: a multiple of 8 up to 128",
            p->head_dim);
    REQUIRE(p->total_q >= 0 && p->total_q <= kMaxRows && p->total_k >= 0 && p->total_k <= kMaxRows,
            "total_q %lld or total_k %lld out of range", (long long)p->total_q, (long long)p->total_k);
    REQUIRE(p->total_q * (p->heads / p->kv_heads) <= kMaxRows - 256, "total_q * heads / kv_heads out of range");
    REQUIRE(p->max_q >= 0 && p->max_k >= 0, "max_q %d, max_k %d", p->max_q, p->max_k);
    const float scale_log2 = p->scale * 1.4426950408889634f;
    REQUIRE(std::isfinite(p->scale), "scale must be finite");
    REQUIRE(std::isfinite(scale_log2), "scale %g out of range", p->scale);
    if (p->batch == 0 || p->total_q == 0) return;
    REQUIRE(p->q && p->out && p->cu_q && p->cu_k, "NULL q, out, cu_q or cu_k");
    REQUIRE(p->total_k == 0 || (p->k && p->v), "NULL k or v");
    for (const void* t : {p->q, p->k, p->v}) REQUIRE(aligned_to(t, 16), "q, k and v must be 16-byte aligned");
    for (int64_t s : {p->q_token_stride, p->q_head_stride, p->k_token_stride, p->k_head_stride, p->v_token_stride,
                      p->v_head_stride})
      REQUIRE(s > 0 && s % 8 == 0 && s <= kMaxStride / 4, "stride %lld: positive and a multiple of 8", (long long)s);
    for (int64_t s : {p->out_token_stride, p->out_head_stride})
      REQUIRE(s > 0 && s <= kMaxStride / 4, "out stride %lld", (long long)s);
    REQUIRE(aligned_to(p->out, 2) && aligned_to(p->lse, 4) && aligned_to(p->cu_q, 4) && aligned_to(p->cu_k, 4) &&
                aligned_to(p->k_len, 4),
            "out, lse or the offsets not aligned to their elements");
    const int sms = current_sms();
    AttnArgs a;
    a.q = static_cast<const __nv_bfloat16*>(p->q);
    a.k = static_cast<const __nv_bfloat16*>(p->k);
    a.v = static_cast<const __nv_bfloat16*>(p->v);
    a.out = static_cast<__nv_bfloat16*>(p->out);
    a.lse = p->lse;
    a.cu_q = p->cu_q, a.cu_k = p->cu_k, a.k_len = p->k_len;
    a.total_q = p->total_q, a.total_k = p->total_k;
    a.q_t = p->q_token_stride, a.q_h = p->q_head_stride, a.k_t = p->k_token_stride, a.k_h = p->k_head_stride;
    a.v_t = p->v_token_stride, a.v_h = p->v_head_stride, a.o_t = p->out_token_stride, a.o_h = p->out_head_stride;
    a.batch = p->batch, a.heads = p->heads, a.kv_heads = p->kv_heads, a.dim = p->head_dim;
    a.max_q = p->max_q, a.max_k = p->max_k, a.causal = p->causal != 0;
    // a score of -infinity (a masked one) times 0 would be NaN; the smallest scale leaves all but the largest others at 0
    a.scale_log2 = std::fabs(scale_log2) < FLT_MIN ? FLT_MIN : scale_log2;
    launch_attention(a, sms, (cudaStream_t)cuda_stream);
  });
}

int gdit_op_status(int device, void* cuda_stream) {
  unsigned bits = 0;
  const int rc = guarded_op([&] {
    int n = 0;
    if (cudaGetDeviceCount(&n) != cudaSuccess || n == 0) {
      cudaGetLastError();
      throw GditError(GDIT_ENODEV, "no CUDA device");
    }
    REQUIRE(device >= 0 && device < n, "device %d out of range", device);
    const DeviceGuard guard(device);
    cudaStream_t s = (cudaStream_t)cuda_stream;
    CUDA_TRY(cudaMemcpyFromSymbolAsync(&bits, g_op_status, sizeof(bits), 0, cudaMemcpyDeviceToHost, s));
    CUDA_TRY(cudaStreamSynchronize(s));
    if (bits != 0) {   // only what has been read, so that a bit set meanwhile is kept
      clear_status_kernel<<<1, 1, 0, s>>>(bits);
      CUDA_TRY(cudaGetLastError());
      CUDA_TRY(cudaStreamSynchronize(s));
    }
    if (bits & DEV_ERR_TIMEOUT) throw GditError(GDIT_ETIMEOUT, "a device-side wait timed out");
    if (bits & OP_ERR_GROUP)
      throw GditError(GDIT_EDEVICE, "norm_residual: row_group out of range (those rows are NaN)");
    if (bits & OP_ERR_OFFSETS)
      throw GditError(GDIT_EDEVICE, "attention: sequence offsets or lengths out of range (those sequences are skipped)");
  });
  return rc;
}

int gdit_debug_op_wait_expiry(int device, unsigned long long limit_ns) {
  const int rc = guarded_op([&] {
    REQUIRE(limit_ns >= 1000ull && limit_ns <= 1000000000ull, "limit_ns %llu outside [1 us, 1 s]", limit_ns);
    int n = 0;
    if (cudaGetDeviceCount(&n) != cudaSuccess || n == 0) {
      cudaGetLastError();
      throw GditError(GDIT_ENODEV, "no CUDA device");
    }
    REQUIRE(device >= 0 && device < n, "device %d of %d", device, n);
    const DeviceGuard guard(device);
    op_wait_expiry_kernel<<<1, 64>>>(limit_ns);
    CUDA_TRY(cudaGetLastError());
  });
  return rc != GDIT_OK ? rc : gdit_op_status(device, nullptr);
}

}  // extern "C"
