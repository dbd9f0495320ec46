// C ABI of libfp8lin: argument checks on the host, then kernel launches on the
// caller's stream.  No allocation, no host synchronisation, no state beyond a
// per-device "is this gfx950" flag and the per-device address of the static
// scratch that fp8_scaled_gemm_noalloc uses.
#include <atomic>
#include <cmath>
#include <cstring>

#include "internal.h"
#include "seq_attn.h"

namespace {

constexpr int kMaxDevices = 64;
constexpr int64_t kMaxTokens = ((int64_t)1 << 31) - (1 << 16);  // of the embedding's gradient
constexpr int64_t kMaxRowStride = 1 << 24;  // of attention over packed sequences
// 0 = not checked yet, 1 = gfx950, 2 = something else.
std::atomic<int> g_arch_ok[kMaxDevices];

// The split workspace of fp8_scaled_gemm_noalloc, for callers that cannot
// allocate: one copy per device, held until the process ends.  Host code never
// passes `scratch` itself (on the host it names a stand-in, not device memory):
// it passes the device address hipGetSymbolAddress returns for the current
// device, looked up on the first call on that device and kept in g_scratch.
static __device__ __align__(256) __attribute__((used)) uint8_t scratch[FP8_NOALLOC_SCRATCH_BYTES];
std::atomic<void*> g_scratch[kMaxDevices];

bool misaligned(const void* p) { return ((uintptr_t)p & 15u) != 0; }
// amax and bias words: their natural 4-byte alignment (atomics need it)
bool misaligned_word(const void* p) { return ((uintptr_t)p & 3u) != 0; }
// E3M4 has no MFMA operand type: quantisation only.
bool bad_format(int f) { return f != FP8_E4M3 && f != FP8_E5M2 && f != FP8_E3M4; }
bool bad_operand_format(int f) { return f != FP8_E4M3 && f != FP8_E5M2; }
bool bad_dtype(int d) { return d != FP8_IN_BF16 && d != FP8_IN_FP32; }
bool bad_dim(int64_t v) { return v < 0 || v > (int64_t)0x7FFFFFFF; }

// The current device must be a gfx950.  Checked once per device.
int device_ok() {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return FP8_ERR_DEVICE;
  if (dev >= kMaxDevices) return FP8_ERR_DEVICE;
  int state = g_arch_ok[dev].load(std::memory_order_acquire);
  if (state == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return FP8_ERR_DEVICE;
    state = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
    g_arch_ok[dev].store(state, std::memory_order_release);
  }
  return state == 1 ? FP8_OK : FP8_ERR_DEVICE;
}

int hip_status(hipError_t e) { return e == hipSuccess ? FP8_OK : FP8_ERR_HIP; }

// The current device's copy of `scratch` (device_ok() has already checked the
// device index).  Several threads may look it up at once: each gets the same
// address.
int scratch_of_current_device(void** ptr) {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return FP8_ERR_DEVICE;
  void* p = g_scratch[dev].load(std::memory_order_acquire);
  if (!p) {
    if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p) return FP8_ERR_HIP;
    g_scratch[dev].store(p, std::memory_order_release);
  }
  *ptr = p;
  return FP8_OK;
}

// The operands are a_rows x a_cols and b_rows x b_cols, each of those one of
// M, N, K: the products are formed only after the range check.
int gemm_checks(const uint8_t* a, int fa, const int32_t* ba, const uint8_t* b, int fb,
                const int32_t* bb, int64_t M, int64_t N, int64_t K, const float* out,
                int64_t a_rows, int64_t a_cols, int64_t b_rows, int64_t b_cols) {
  if (bad_dim(M) || bad_dim(N) || bad_dim(K)) return FP8_ERR_SIZE;
  const int64_t a_elems = a_rows * a_cols, b_elems = b_rows * b_cols;
  // the launch grid (at most one block per 128 x 128 output tile) is 32-bit
  if (((M + 127) / 128) * ((N + 127) / 128) > (int64_t)0x7FFFFFFF) return FP8_ERR_SIZE;
  if (bad_operand_format(fa) || bad_operand_format(fb)) return FP8_ERR_FORMAT;
  if (M == 0 || N == 0) return FP8_OK;
  if (!out || !ba || !bb) return FP8_ERR_NULL;
  if ((a_elems > 0 && !a) || (b_elems > 0 && !b)) return FP8_ERR_NULL;
  if (misaligned(out) || (a && misaligned(a)) || (b && misaligned(b))) return FP8_ERR_ALIGN;
  if (misaligned_word(ba) || misaligned_word(bb)) return FP8_ERR_ALIGN;
  return FP8_OK;
}

// fp8_quantize's argument checks (no device call).
int quantize_checks(const void* x, int dtype, int64_t n, int fmt, int32_t margin, const uint8_t* y,
                    const float* amax, const int32_t* bias) {
  if (n < 0) return FP8_ERR_SIZE;
  if (bad_dtype(dtype)) return FP8_ERR_DTYPE;
  if (bad_format(fmt)) return FP8_ERR_FORMAT;
  if (margin > FP8_MAX_MARGIN || margin < -FP8_MAX_MARGIN) return FP8_ERR_MARGIN;
  if (!amax || !bias || (n > 0 && (!x || !y))) return FP8_ERR_NULL;
  if (misaligned_word(amax) || misaligned_word(bias)) return FP8_ERR_ALIGN;
  if (n > 0 && (misaligned(x) || misaligned(y))) return FP8_ERR_ALIGN;
  return FP8_OK;
}

// The checks that the norm's forward entry points share.
int norm_checks(const void* x, int x_dtype, const void* r, int r_dtype, const void* w, int w_dtype, int64_t rows,
                int64_t d, const void* h, const float* rstd, const void* y) {
  if (rows < 0 || rows > (int64_t)0x7FFFFFFF || d < 1) return FP8_ERR_SIZE;
  if (d > (d % 4 == 0 ? fp8lin::kNormMaxD : fp8lin::kNormMaxOddD)) return FP8_ERR_SIZE;
  if (bad_dtype(x_dtype) || bad_dtype(w_dtype) || (r && bad_dtype(r_dtype))) return FP8_ERR_DTYPE;
  if (rows > 0 && (!x || !w || !y || (r && !h))) return FP8_ERR_NULL;
  if (rows > 0 && (misaligned(x) || misaligned(w) || misaligned(y))) return FP8_ERR_ALIGN;
  if (rows > 0 && r && (misaligned(r) || misaligned(h))) return FP8_ERR_ALIGN;
  if (misaligned_word(rstd)) return FP8_ERR_ALIGN;
  return FP8_OK;
}

// A cache's and a batch's host-side fields (no device call).
int kv_checks(const fp8_kv_cache_t* c, const fp8_kv_batch_t* b) {
  if (!c || !b) return FP8_ERR_NULL;
  if (c->num_blocks < 1 || c->heads < 1) return FP8_ERR_SIZE;
  if (c->block_size != 16 && c->block_size != 32 && c->block_size != 64 && c->block_size != 128) return FP8_ERR_SIZE;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return FP8_ERR_SIZE;
  if (bad_operand_format(c->fmt)) return FP8_ERR_FORMAT;
  if (b->batch < 0 || b->table_width < 0 || b->tokens < 0 || b->max_new < 0 || b->max_len < 0) return FP8_ERR_SIZE;
  if (b->max_len > (1 << 30) || b->max_len > (int64_t)b->table_width * c->block_size) return FP8_ERR_SIZE;
  if (b->batch == 0 || b->tokens == 0 || b->max_new == 0) return FP8_OK;  // nothing to do
  if (!c->k || !c->v || !c->k_bias || !c->v_bias || !b->cu_tokens || !b->lens || (b->table_width > 0 && !b->block_table))
    return FP8_ERR_NULL;
  if (misaligned(c->k) || misaligned(c->v)) return FP8_ERR_ALIGN;
  if (misaligned_word(c->k_bias) || misaligned_word(c->v_bias) || misaligned_word(b->cu_tokens) ||
      misaligned_word(b->lens) || misaligned_word(b->block_table))
    return FP8_ERR_ALIGN;
  return FP8_OK;
}

// Rows of packed heads, `stride` elements of `bytes` each apart.
int rows_checks(const void* p, int64_t stride, int64_t heads, int64_t head_dim, int bytes) {
  if (!p) return FP8_ERR_NULL;
  if (stride < heads * head_dim || stride > (int64_t)0x7FFFFFFF) return FP8_ERR_SIZE;
  if (misaligned(p) || (stride * bytes) % 16 != 0) return FP8_ERR_ALIGN;
  return FP8_OK;
}

// The batch with max_new held to what tokens and max_len allow: grids, splits
// and workspaces go by it, and a caller's bound may be loose.
fp8_kv_batch_t bounded(const fp8_kv_batch_t* b) {
  fp8_kv_batch_t r = *b;
  if (r.max_new > r.tokens) r.max_new = r.tokens;
  if (r.max_new > r.max_len) r.max_new = r.max_len;
  return r;
}

bool kv_empty(const fp8_kv_batch_t& b) { return b.batch == 0 || b.tokens == 0 || b.max_new == 0; }

// Packed sequences and the heads over them (no device call).
int seqs_checks(const fp8_seqs_t* s, int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
  if (!s) return FP8_ERR_NULL;
  if (s->batch < 0 || s->tokens < 0 || s->max_len < 0 || s->max_len > (1 << 30)) return FP8_ERR_SIZE;
  if (q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0) return FP8_ERR_SIZE;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return FP8_ERR_SIZE;
  if ((int64_t)q_heads * head_dim > kMaxRowStride) return FP8_ERR_SIZE;
  // workgroups are counted in 32 bits: three kinds of them in the backward pass
  // (cut walks and their joins are of shapes with few)
  const int64_t longest = s->max_len < s->tokens ? s->max_len : s->tokens;
  if ((longest + 127) / 128 * s->batch > (int64_t)0x7FFFFFFF / (3 * (int64_t)q_heads) ||
      s->tokens > (int64_t)0x7FFFFFFF / q_heads)
    return FP8_ERR_SIZE;
  if (s->batch == 0 || s->tokens == 0 || s->max_len == 0) return FP8_OK;  // nothing to do
  if (!s->cu_tokens) return FP8_ERR_NULL;
  if (misaligned_word(s->cu_tokens)) return FP8_ERR_ALIGN;
  return FP8_OK;
}
// The kernels take it times log2(e), which has to be finite too.
constexpr float kLog2e = 1.44269504088896340736f;
bool bad_scale(float scale) { return !std::isfinite(scale * kLog2e); }
bool seqs_empty(const fp8_seqs_t& s) { return s.batch == 0 || s.tokens == 0 || s.max_len == 0; }
fp8lin::SeqAttnArgs seq_args(const fp8_seqs_t& s, int32_t q_heads, int32_t kv_heads, float scale, int32_t causal,
                             int32_t window) {
  fp8lin::SeqAttnArgs a{};
  a.cu = s.cu_tokens;
  a.batch = s.batch;
  a.tokens = s.tokens;
  a.max_len = s.max_len < s.tokens ? s.max_len : s.tokens;  // a caller's bound may be loose
  a.q_heads = q_heads;
  a.heads = kv_heads;
  a.group = q_heads / kv_heads;
  a.scale = scale;
  a.scale_log2 = scale * kLog2e;
  a.causal = causal != 0;
  a.window = window;
  return a;
}
// Ids and sizes of the embedding (no device call).
int embedding_checks(const void* ids, int32_t id_bits, int64_t tokens, int64_t vocab, int64_t d) {
  if (id_bits != 32 && id_bits != 64) return FP8_ERR_DTYPE;
  if (tokens < 0 || tokens > kMaxTokens || vocab < 0 || vocab > (int64_t)0x7FFFFFFF || d < 1 || d > (1 << 24))
    return FP8_ERR_SIZE;
  // workgroups of 1024 elements are counted in 32 bits
  if (tokens * ((d + 1023) / 1024) > (int64_t)0x7FFFFFFF) return FP8_ERR_SIZE;
  if (tokens > 0 && !ids) return FP8_ERR_NULL;
  if (((uintptr_t)ids & (id_bits / 8 - 1)) != 0) return FP8_ERR_ALIGN;
  return FP8_OK;
}

// The fused rows of queries, keys and values, their norms and their rotation.
int qk_checks(const fp8lin::QkProblem& p) {
  if (p.tokens < 0 || p.tokens > (int64_t)0x7FFFFFFF || p.q_heads < 1 || p.kv_heads < 1) return FP8_ERR_SIZE;
  if (p.head_dim != 64 && p.head_dim != 128 && p.head_dim != 256) return FP8_ERR_SIZE;
  const int64_t heads = (int64_t)p.q_heads + 2 * (int64_t)p.kv_heads;
  if (heads * p.head_dim > kMaxRowStride) return FP8_ERR_SIZE;
  if (!(p.eps >= 0)) return FP8_ERR_SIZE;
  if (bad_dtype(p.x_dtype) || (p.wq && bad_dtype(p.w_dtype))) return FP8_ERR_DTYPE;
  if (!p.wq != !p.wk || !p.cos != !p.sin) return FP8_ERR_NULL;
  if (p.cos && (p.rope_rows < 1 || (!p.positions && p.rope_rows < p.tokens))) return FP8_ERR_SIZE;
  if (misaligned(p.wq) || misaligned(p.wk) || misaligned(p.cos) || misaligned(p.sin) || misaligned_word(p.positions))
    return FP8_ERR_ALIGN;
  if (p.tokens == 0) return FP8_OK;
  return rows_checks(p.x, p.x_stride, heads, p.head_dim, p.x_dtype == FP8_IN_FP32 ? 4 : 2);
}

// Rows whose 32-bit offsets within a tile the kernels form.
int seq_rows_checks(const void* p, int64_t stride, int64_t heads, int64_t head_dim) {
  if (stride > kMaxRowStride) return FP8_ERR_SIZE;
  return rows_checks(p, stride, heads, head_dim, 2);
}

}  // namespace

extern "C" {

const char* fp8_status_string(int status) {
  switch (status) {
    case FP8_OK: return "ok";
    case FP8_ERR_NULL: return "a required pointer is NULL";
    case FP8_ERR_SIZE: return "a size is negative or too large";
    case FP8_ERR_FORMAT: return "unknown FP8 format";
    case FP8_ERR_DTYPE: return "unknown input dtype";
    case FP8_ERR_ALIGN: return "a pointer is misaligned (16 bytes for tensors, 4 for amax outputs)";
    case FP8_ERR_MARGIN: return "margin out of range";
    case FP8_ERR_DEVICE: return "no gfx950 HIP device is current";
    case FP8_ERR_HIP: return "a HIP launch failed";
    case FP8_ERR_OP: return "unknown product or math selector";
    default: return "unknown status";
  }
}

int fp8_amax(const void* x, fp8_dtype_t dtype, int64_t n, float* amax, void* stream) {
  if (n < 0) return FP8_ERR_SIZE;
  if (bad_dtype(dtype)) return FP8_ERR_DTYPE;
  if (!amax || (n > 0 && !x)) return FP8_ERR_NULL;
  if ((n > 0 && misaligned(x)) || misaligned_word(amax)) return FP8_ERR_ALIGN;
  if (int s = device_ok()) return s;
  return hip_status(fp8lin::launch_amax(x, dtype, n, amax, (hipStream_t)stream));
}

int fp8_compute_bias(const float* amax, fp8_format_t fmt, int32_t margin, int32_t* bias,
                     void* stream) {
  if (bad_format(fmt)) return FP8_ERR_FORMAT;
  if (margin > FP8_MAX_MARGIN || margin < -FP8_MAX_MARGIN) return FP8_ERR_MARGIN;
  if (!amax || !bias) return FP8_ERR_NULL;
  if (misaligned_word(amax) || misaligned_word(bias)) return FP8_ERR_ALIGN;
  if (int s = device_ok()) return s;
  return hip_status(fp8lin::launch_bias(amax, fmt, margin, bias, (hipStream_t)stream));
}

int fp8_scale_cast(const void* x, fp8_dtype_t dtype, int64_t n, const int32_t* bias,
                   fp8_format_t fmt, uint8_t* y, void* stream) {
  if (n < 0) return FP8_ERR_SIZE;
  if (bad_dtype(dtype)) return FP8_ERR_DTYPE;
  if (bad_format(fmt)) return FP8_ERR_FORMAT;
  if (n == 0) return FP8_OK;
  if (!x || !y || !bias) return FP8_ERR_NULL;
  if (misaligned(x) || misaligned(y) || misaligned_word(bias)) return FP8_ERR_ALIGN;
  if (int s = device_ok()) return s;
  return hip_status(fp8lin::launch_cast(x, dtype, n, bias, fmt, y, nullptr, (hipStream_t)stream));
}

int fp8_quantize(const void* x, fp8_dtype_t dtype, int64_t n, fp8_format_t fmt, int32_t margin,
                 uint8_t* y, float* amax, int32_t* bias, void* stream) {
  if (int s = quantize_checks(x, dtype, n, fmt, margin, y, amax, bias)) return s;
  if (int s = device_ok()) return s;
  return hip_status(fp8lin::launch_quantize(x, dtype, n, fmt, margin, y, amax, bias,
                                            (hipStream_t)stream));
}

int fp8_quantize_multi(const fp8_quant_desc_t* descs, int32_t count, void* stream) {
  if (count < 0) return FP8_ERR_SIZE;
  if (count == 0) return FP8_OK;
  if (!descs) return FP8_ERR_NULL;
  for (int32_t i = 0; i < count; ++i) {
    const fp8_quant_desc_t& d = descs[i];
    if (int st = quantize_checks(d.x, d.dtype, d.n, d.fmt, d.margin, d.y, d.amax, d.bias)) return st;
  }
  if (int st = device_ok()) return st;
  constexpr int kChunk = 256;  // descriptors converted per host batch
  fp8lin::QuantDesc q[kChunk];
  for (int32_t first = 0; first < count; first += kChunk) {
    const int m = count - first < kChunk ? count - first : kChunk;
    for (int i = 0; i < m; ++i) {
      const fp8_quant_desc_t& d = descs[first + i];
      q[i] = fp8lin::QuantDesc{d.x, d.n, d.dtype, d.fmt, d.margin, d.y, d.amax, d.bias};
    }
    if (int st = hip_status(fp8lin::launch_quantize_multi(q, m, (hipStream_t)stream))) return st;
  }
  return FP8_OK;
}

int fp8_scale_cast_amax(const void* x, fp8_dtype_t dtype, int64_t n, const int32_t* bias,
                        fp8_format_t fmt, uint8_t* y, float* x_amax, void* stream) {
  if (n < 0) return FP8_ERR_SIZE;
  if (bad_dtype(dtype)) return FP8_ERR_DTYPE;
  if (bad_format(fmt)) return FP8_ERR_FORMAT;
  if (!x_amax) return FP8_ERR_NULL;
  if (misaligned_word(x_amax)) return FP8_ERR_ALIGN;
  if (n > 0) {
    if (!x || !y || !bias) return FP8_ERR_NULL;
    if (misaligned(x) || misaligned(y) || misaligned_word(bias)) return FP8_ERR_ALIGN;
  }
  if (int s = device_ok()) return s;
  return hip_status(fp8lin::launch_cast(x, dtype, n, bias, fmt, y,
                                        reinterpret_cast<uint32_t*>(x_amax), (hipStream_t)stream));
}

int fp8_quantize_delayed(const void* x, fp8_dtype_t dtype, int64_t n, fp8_format_t fmt,
                         int32_t margin, uint8_t* y, float* amax, int32_t* bias, void* stream) {
  if (int s = quantize_checks(x, dtype, n, fmt, margin, y, amax, bias)) return s;
  if (int s = device_ok()) return s;
  return hip_status(fp8lin::launch_quantize_delayed(x, dtype, n, fmt, margin, y, amax, bias,
                                                    (hipStream_t)stream));
}

}  // extern "C"

namespace {

// The three products; out_amax (optional) receives max |out|.  Every argument
// is checked before any HIP call; on error nothing is written.
// The product's output as rows x cols with contraction `depth`, for each op.
bool out_shape(fp8_gemm_op_t op, int64_t M, int64_t N, int64_t K, int64_t& rows, int64_t& cols,
               int64_t& depth) {
  switch (op) {
    case FP8_GEMM_FWD: rows = M; cols = N; depth = K; return true;
    case FP8_GEMM_DGRAD: rows = M; cols = K; depth = N; return true;
    case FP8_GEMM_WGRAD: rows = N; cols = K; depth = M; return true;
    default: return false;
  }
}

// Where a split product's workspace comes from: none (never split), the
// caller's (fp8_scaled_gemm_ws: ws / ws_bytes checked here) or the library's
// static scratch (fp8_scaled_gemm_noalloc).
enum WsMode { kNoWorkspace, kCallerWorkspace, kStaticScratch };

// The checks of one product and its problem in kernel terms (rows, columns and
// contraction of the output; each operand's layout); empty: no output.
int make_problem(fp8_gemm_op_t op, int math, const uint8_t* a, fp8_format_t fa, const int32_t* ba,
                 const uint8_t* b, fp8_format_t fb, const int32_t* bb, int64_t M, int64_t N, int64_t K,
                 float* out, fp8lin::GemmProblem& p, bool& empty) {
  if (math != FP8_GEMM_EXACT && math != FP8_GEMM_NATIVE_FP8) return FP8_ERR_OP;
  empty = false;
  switch (op) {
    case FP8_GEMM_FWD:
      // Y[M x N]: X8 and W8 both contraction (K) contiguous.
      if (int s = gemm_checks(a, fa, ba, b, fb, bb, M, N, K, out, M, K, N, K)) return s;
      empty = M == 0 || N == 0;
      p = fp8lin::GemmProblem{a, K, true, fa, ba, b, K, true, fb, bb, out, N,
                              (int)M, (int)N, (int)K, math, nullptr, false};
      break;
    case FP8_GEMM_DGRAD:
      // dX[M x K]: rows of dY8 (contraction N contiguous) times W8 read as
      // [contraction N][K] (the contraction is its slow index).
      if (int s = gemm_checks(a, fa, ba, b, fb, bb, M, K, N, out, M, N, N, K)) return s;
      empty = M == 0 || K == 0;
      p = fp8lin::GemmProblem{a, N, true, fa, ba, b, K, false, fb, bb, out, K,
                              (int)M, (int)K, (int)N, math, nullptr, false};
      break;
    case FP8_GEMM_WGRAD:
      // dW[N x K]: dY8 read as [contraction M][N] times X8 read as [contraction M][K].
      if (int s = gemm_checks(a, fa, ba, b, fb, bb, N, K, M, out, M, N, M, K)) return s;
      empty = N == 0 || K == 0;
      p = fp8lin::GemmProblem{a, N, false, fa, ba, b, K, false, fb, bb, out, K,
                              (int)N, (int)K, (int)M, math, nullptr, false};
      break;
    default:
      return FP8_ERR_OP;
  }
  return FP8_OK;
}

int scaled_gemm(fp8_gemm_op_t op, int math, const uint8_t* a, fp8_format_t fa, const int32_t* ba,
                const uint8_t* b, fp8_format_t fb, const int32_t* bb, int64_t M, int64_t N,
                int64_t K, float* out, float* out_amax, WsMode ws_mode, void* ws, int64_t ws_bytes,
                hipStream_t st, bool accumulate = false) {
  fp8lin::GemmProblem p{};
  bool empty = false;
  if (int s = make_problem(op, math, a, fa, ba, b, fb, bb, M, N, K, out, p, empty)) return s;
  p.accumulate = accumulate;
  bool split = false;
  // the static scratch bounds its plan; a caller's workspace is sized by
  // fp8_scaled_gemm_workspace_bytes (no bound)
  const int64_t max_bytes = ws_mode == kStaticScratch ? (int64_t)FP8_NOALLOC_SCRATCH_BYTES : INT64_MAX;
  if (ws_mode != kNoWorkspace && !empty) {
    const int64_t need = fp8lin::gemm_split_workspace_bytes(p.m, p.n, p.k, max_bytes);
    if (need > 0) {
      if (ws_mode == kStaticScratch) {
        if (need > (int64_t)FP8_NOALLOC_SCRATCH_BYTES) return FP8_ERR_SIZE;
      } else {
        if (!ws) return FP8_ERR_NULL;
        if (misaligned(ws)) return FP8_ERR_ALIGN;
        if (ws_bytes < need) return FP8_ERR_SIZE;
      }
      split = true;
    }
  }
  if (empty && !out_amax) return FP8_OK;
  if (int s = device_ok()) return s;
  if (split && ws_mode == kStaticScratch) {
    if (int s = scratch_of_current_device(&ws)) return s;
  }
  if (out_amax) {
    p.amax = reinterpret_cast<uint32_t*>(out_amax);
    if (int s = hip_status(fp8lin::launch_clear_u32(p.amax, st))) return s;
  }
  if (empty) return FP8_OK;
  if (split) {
    float* w = static_cast<float*>(ws);
    switch (op) {
      case FP8_GEMM_FWD: return hip_status(fp8lin::launch_gemm_fwd_ws(p, w, max_bytes, st));
      case FP8_GEMM_DGRAD: return hip_status(fp8lin::launch_gemm_dgrad_ws(p, w, max_bytes, st));
      default: return hip_status(fp8lin::launch_gemm_wgrad_ws(p, w, max_bytes, st));
    }
  }
  switch (op) {
    case FP8_GEMM_FWD: return hip_status(fp8lin::launch_gemm_fwd(p, st));
    case FP8_GEMM_DGRAD: return hip_status(fp8lin::launch_gemm_dgrad(p, st));
    default: return hip_status(fp8lin::launch_gemm_wgrad(p, st));
  }
}

// The problems of a group call (checked) and their plan; count products at
// most kGroupMaxProducts.  Returns the workspace bytes (>= 0) or a status.
int64_t group_problems(int math, const fp8_gemm_desc_t* d, int32_t count, fp8lin::GemmProblem* ps,
                       fp8lin::GroupSlot* plan, int* live) {
  if (count < 0 || count > fp8lin::kGroupMaxProducts) return FP8_ERR_SIZE;
  if (count > 0 && !d) return FP8_ERR_NULL;
  *live = 0;
  for (int32_t i = 0; i < count; ++i) {
    bool empty = false;
    fp8lin::GemmProblem p{};
    if (int s = make_problem((fp8_gemm_op_t)d[i].op, math, d[i].a, (fp8_format_t)d[i].fa, d[i].ba, d[i].b,
                             (fp8_format_t)d[i].fb, d[i].bb, d[i].M, d[i].N, d[i].K, d[i].out, p, empty))
      return s;
    if (!empty) ps[(*live)++] = p;
  }
  return fp8lin::gemm_group_plan(ps, *live, plan);
}

}  // namespace

extern "C" {

int64_t fp8_scaled_gemm_group_workspace_bytes(int math, const fp8_gemm_desc_t* descs, int32_t count) {
  fp8lin::GemmProblem ps[fp8lin::kGroupMaxProducts];
  fp8lin::GroupSlot plan[fp8lin::kGroupMaxProducts];
  int live = 0;
  return group_problems(math, descs, count, ps, plan, &live);
}

int fp8_scaled_gemm_group(int math, const fp8_gemm_desc_t* descs, int32_t count, void* ws,
                          int64_t ws_bytes, void* stream) {
  fp8lin::GemmProblem ps[fp8lin::kGroupMaxProducts];
  fp8lin::GroupSlot plan[fp8lin::kGroupMaxProducts];
  int live = 0;
  const int64_t need = group_problems(math, descs, count, ps, plan, &live);
  if (need < 0) return (int)need;
  if (ws_bytes < 0) return FP8_ERR_SIZE;
  if (need > 0) {
    if (!ws) return FP8_ERR_NULL;
    if (misaligned(ws)) return FP8_ERR_ALIGN;
    if (ws_bytes < need) return FP8_ERR_SIZE;
  }
  if (live == 0) return FP8_OK;
  if (int s = device_ok()) return s;
  hipStream_t st = (hipStream_t)stream;
  int idx[3][fp8lin::kGroupMaxProducts];
  int n[3] = {0, 0, 0};
  int step[fp8lin::kGroupMaxProducts];
  int nstep = 0;
  for (int i = 0; i < live; ++i) {
    const fp8lin::GemmProblem& p = ps[i];
    const int layout = p.a_kmajor && p.b_kmajor ? 0 : (p.a_kmajor ? 1 : 2);
    if (plan[i].grouped) {
      if (fp8lin::gemm_step_variant(p) >= 0) step[nstep++] = i;
      else idx[layout][n[layout]++] = i;
      continue;
    }
    hipError_t e = layout == 0 ? fp8lin::launch_gemm_fwd(p, st)
                   : layout == 1 ? fp8lin::launch_gemm_dgrad(p, st) : fp8lin::launch_gemm_wgrad(p, st);
    if (e != hipSuccess) return FP8_ERR_HIP;
  }
  uint8_t* w = static_cast<uint8_t*>(ws);
  if (int s = hip_status(fp8lin::launch_gemm_step_group(ps, plan, step, nstep, w, st))) return s;
  if (int s = hip_status(fp8lin::launch_gemm_fwd_group(ps, plan, idx[0], n[0], w, st))) return s;
  if (int s = hip_status(fp8lin::launch_gemm_dgrad_group(ps, plan, idx[1], n[1], w, st))) return s;
  return hip_status(fp8lin::launch_gemm_wgrad_group(ps, plan, idx[2], n[2], w, st));
}

int fp8_scaled_gemm(fp8_gemm_op_t op, int math, const uint8_t* a, fp8_format_t fa,
                    const int32_t* ba, const uint8_t* b, fp8_format_t fb, const int32_t* bb,
                    int64_t M, int64_t N, int64_t K, float* out, void* stream) {
  return scaled_gemm(op, math, a, fa, ba, b, fb, bb, M, N, K, out, nullptr, kNoWorkspace, nullptr,
                     0, (hipStream_t)stream);
}

int64_t fp8_scaled_gemm_workspace_bytes(fp8_gemm_op_t op, int64_t M, int64_t N, int64_t K) {
  if (bad_dim(M) || bad_dim(N) || bad_dim(K)) return FP8_ERR_SIZE;
  int64_t rows, cols, depth;
  if (!out_shape(op, M, N, K, rows, cols, depth)) return FP8_ERR_OP;
  return fp8lin::gemm_split_workspace_bytes(rows, cols, depth, INT64_MAX);
}

int fp8_scaled_gemm_ws(fp8_gemm_op_t op, int math, const uint8_t* a, fp8_format_t fa,
                       const int32_t* ba, const uint8_t* b, fp8_format_t fb, const int32_t* bb,
                       int64_t M, int64_t N, int64_t K, float* out, void* ws, int64_t ws_bytes,
                       void* stream) {
  if (ws_bytes < 0) return FP8_ERR_SIZE;
  return scaled_gemm(op, math, a, fa, ba, b, fb, bb, M, N, K, out, nullptr, kCallerWorkspace, ws,
                     ws_bytes, (hipStream_t)stream);
}

int fp8_scaled_gemm_noalloc(fp8_gemm_op_t op, int math, const uint8_t* a, fp8_format_t fa,
                            const int32_t* ba, const uint8_t* b, fp8_format_t fb,
                            const int32_t* bb, int64_t M, int64_t N, int64_t K, float* out,
                            void* stream) {
  return scaled_gemm(op, math, a, fa, ba, b, fb, bb, M, N, K, out, nullptr, kStaticScratch,
                     nullptr, 0, (hipStream_t)stream);
}

int fp8_scaled_gemm_amax(fp8_gemm_op_t op, int math, const uint8_t* a, fp8_format_t fa,
                         const int32_t* ba, const uint8_t* b, fp8_format_t fb, const int32_t* bb,
                         int64_t M, int64_t N, int64_t K, float* out, float* out_amax,
                         void* stream) {
  if (!out_amax) return FP8_ERR_NULL;
  if (misaligned_word(out_amax)) return FP8_ERR_ALIGN;
  return scaled_gemm(op, math, a, fa, ba, b, fb, bb, M, N, K, out, out_amax, kNoWorkspace, nullptr,
                     0, (hipStream_t)stream);
}

int fp8_scaled_gemm_accumulate(fp8_gemm_op_t op, int math, const uint8_t* a, fp8_format_t fa,
                               const int32_t* ba, const uint8_t* b, fp8_format_t fb,
                               const int32_t* bb, int64_t M, int64_t N, int64_t K, float* out,
                               void* stream) {
  return scaled_gemm(op, math, a, fa, ba, b, fb, bb, M, N, K, out, nullptr, kNoWorkspace, nullptr,
                     0, (hipStream_t)stream, true);
}

int fp8_scaled_gemm_fwd(const uint8_t* x8, fp8_format_t fx, const int32_t* bx,
                        const uint8_t* w8, fp8_format_t fw, const int32_t* bw, int64_t M,
                        int64_t N, int64_t K, float* y, void* stream) {
  return fp8_scaled_gemm(FP8_GEMM_FWD, FP8_GEMM_EXACT, x8, fx, bx, w8, fw, bw, M, N, K, y, stream);
}

int fp8_scaled_gemm_dgrad(const uint8_t* dy8, fp8_format_t fdy, const int32_t* bdy,
                          const uint8_t* w8, fp8_format_t fw, const int32_t* bw, int64_t M,
                          int64_t N, int64_t K, float* dx, void* stream) {
  return fp8_scaled_gemm(FP8_GEMM_DGRAD, FP8_GEMM_EXACT, dy8, fdy, bdy, w8, fw, bw, M, N, K, dx,
                         stream);
}

int fp8_scaled_gemm_wgrad(const uint8_t* dy8, fp8_format_t fdy, const int32_t* bdy,
                          const uint8_t* x8, fp8_format_t fx, const int32_t* bx, int64_t M,
                          int64_t N, int64_t K, float* dw, void* stream) {
  return fp8_scaled_gemm(FP8_GEMM_WGRAD, FP8_GEMM_EXACT, dy8, fdy, bdy, x8, fx, bx, M, N, K, dw,
                         stream);
}

}  // extern "C"

namespace {

int swiglu_checks(const void* h, const void* da, bool need_da, int64_t rows, int64_t f,
                  const void* out, const float* out_amax) {
  if (rows < 0 || f < 0 || rows > (int64_t)0x7FFFFFFF || f > (int64_t)0x3FFFFFFF)
    return FP8_ERR_SIZE;
  if (fp8lin::swiglu_blocks(rows, f) > (int64_t)0x7FFFFFFF) return FP8_ERR_SIZE;
  if (out_amax && misaligned_word(out_amax)) return FP8_ERR_ALIGN;
  if (rows == 0 || f == 0) return FP8_OK;
  if (!h || !out || (need_da && !da)) return FP8_ERR_NULL;
  if (misaligned(h) || misaligned(out) || (need_da && misaligned(da))) return FP8_ERR_ALIGN;
  return FP8_OK;
}

}  // namespace

extern "C" {

int fp8_swiglu_fwd(const float* h, int64_t rows, int64_t f, uint16_t* a, float* out_amax,
                   void* stream) {
  if (int s = swiglu_checks(h, nullptr, false, rows, f, a, out_amax)) return s;
  if ((rows == 0 || f == 0) && !out_amax) return FP8_OK;
  if (int s = device_ok()) return s;
  return hip_status(fp8lin::launch_swiglu_fwd(h, rows, f, a, reinterpret_cast<uint32_t*>(out_amax),
                                              (hipStream_t)stream));
}

int fp8_swiglu_bwd(const float* h, const float* da, int64_t rows, int64_t f, uint16_t* dh,
                   float* out_amax, void* stream) {
  if (int s = swiglu_checks(h, da, true, rows, f, dh, out_amax)) return s;
  if ((rows == 0 || f == 0) && !out_amax) return FP8_OK;
  if (int s = device_ok()) return s;
  return hip_status(fp8lin::launch_swiglu_bwd(h, da, rows, f, dh,
                                              reinterpret_cast<uint32_t*>(out_amax),
                                              (hipStream_t)stream));
}

int fp8_rmsnorm_fwd(const void* x, fp8_dtype_t x_dtype, const void* residual, fp8_dtype_t r_dtype, const void* w,
                    fp8_dtype_t w_dtype, int64_t rows, int64_t d, float eps, void* h, float* rstd, uint16_t* y,
                    float* y_amax, void* stream) {
  int st = norm_checks(x, x_dtype, residual, r_dtype, w, w_dtype, rows, d, h, rstd, y);
  if (st == FP8_OK && misaligned_word(y_amax)) st = FP8_ERR_ALIGN;
  if (st != FP8_OK || (rows == 0 && !y_amax)) return st;
  if ((st = device_ok()) != FP8_OK) return st;
  const fp8lin::NormProblem p{x, (int)x_dtype, residual, (int)r_dtype, w, (int)w_dtype, rows, d, eps, h, rstd};
  return hip_status(fp8lin::launch_norm_fwd(p, y, reinterpret_cast<uint32_t*>(y_amax), (hipStream_t)stream));
}

int fp8_rmsnorm_cast(const void* x, fp8_dtype_t x_dtype, const void* residual, fp8_dtype_t r_dtype, const void* w,
                     fp8_dtype_t w_dtype, int64_t rows, int64_t d, float eps, void* h, float* rstd,
                     const int32_t* bias, fp8_format_t fmt, uint8_t* y, float* y_amax, void* stream) {
  int st = norm_checks(x, x_dtype, residual, r_dtype, w, w_dtype, rows, d, h, rstd, y);
  if (st != FP8_OK) return st;
  if (bad_operand_format(fmt)) return FP8_ERR_FORMAT;
  if (!bias) return FP8_ERR_NULL;
  if (misaligned_word(bias) || misaligned_word(y_amax)) return FP8_ERR_ALIGN;
  if (rows == 0 && !y_amax) return FP8_OK;
  if ((st = device_ok()) != FP8_OK) return st;
  const fp8lin::NormProblem p{x, (int)x_dtype, residual, (int)r_dtype, w, (int)w_dtype, rows, d, eps, h, rstd};
  return hip_status(
      fp8lin::launch_norm_cast(p, bias, fmt, y, reinterpret_cast<uint32_t*>(y_amax), (hipStream_t)stream));
}

int fp8_rmsnorm_quantize(const void* x, fp8_dtype_t x_dtype, const void* residual, fp8_dtype_t r_dtype, const void* w,
                         fp8_dtype_t w_dtype, int64_t rows, int64_t d, float eps, void* h, float* rstd,
                         fp8_format_t fmt, int32_t margin, uint8_t* y, float* row_amax, float* amax, int32_t* bias,
                         void* stream) {
  int st = norm_checks(x, x_dtype, residual, r_dtype, w, w_dtype, rows, d, h, rstd, y);
  if (st != FP8_OK) return st;
  if (bad_operand_format(fmt)) return FP8_ERR_FORMAT;
  if (margin > FP8_MAX_MARGIN || margin < -FP8_MAX_MARGIN) return FP8_ERR_MARGIN;
  if (!amax || !bias || (rows > 0 && (!rstd || !row_amax))) return FP8_ERR_NULL;
  if (misaligned_word(amax) || misaligned_word(bias) || misaligned_word(row_amax)) return FP8_ERR_ALIGN;
  if ((st = device_ok()) != FP8_OK) return st;
  const fp8lin::NormProblem p{x, (int)x_dtype, residual, (int)r_dtype, w, (int)w_dtype, rows, d, eps, h, rstd};
  return hip_status(fp8lin::launch_norm_quantize(p, fmt, margin, y, reinterpret_cast<uint32_t*>(row_amax),
                                                 reinterpret_cast<uint32_t*>(amax), bias, (hipStream_t)stream));
}

int64_t fp8_rmsnorm_bwd_workspace_bytes(int64_t rows, int64_t d) {
  if (rows < 0 || rows > (int64_t)0x7FFFFFFF || d < 1) return FP8_ERR_SIZE;
  if (d > (d % 4 == 0 ? fp8lin::kNormMaxD : fp8lin::kNormMaxOddD)) return FP8_ERR_SIZE;
  return fp8lin::norm_bwd_workspace_bytes(rows, d);
}

int fp8_rmsnorm_bwd(const void* dy, fp8_dtype_t dy_dtype, const void* h, fp8_dtype_t h_dtype, const void* w,
                    fp8_dtype_t w_dtype, const float* rstd, const void* dh, int64_t rows, int64_t d, void* dx,
                    float* dw, float* dx_amax, void* ws, int64_t ws_bytes, void* stream) {
  const int64_t need = fp8_rmsnorm_bwd_workspace_bytes(rows, d);
  if (need < 0) return (int)need;
  if (bad_dtype(dy_dtype) || bad_dtype(h_dtype) || bad_dtype(w_dtype)) return FP8_ERR_DTYPE;
  if (!dw || (rows > 0 && (!dy || !h || !w || !rstd || !dx || !ws))) return FP8_ERR_NULL;
  if (misaligned_word(rstd) || misaligned_word(dx_amax) || misaligned(dw)) return FP8_ERR_ALIGN;
  if (rows > 0 && (misaligned(dy) || misaligned(h) || misaligned(w) || misaligned(dh) || misaligned(dx) ||
                   misaligned(ws)))
    return FP8_ERR_ALIGN;
  if (ws_bytes < need) return FP8_ERR_SIZE;
  const int st = device_ok();
  if (st != FP8_OK) return st;
  return hip_status(fp8lin::launch_norm_bwd(dy, dy_dtype, h, h_dtype, w, w_dtype, rstd, dh, rows, d, dx, dw,
                                            reinterpret_cast<uint32_t*>(dx_amax), static_cast<float*>(ws),
                                            (hipStream_t)stream));
}

int fp8_kv_append(const fp8_kv_cache_t* cache, const fp8_kv_batch_t* batch, const void* k, int64_t k_stride,
                  const void* v, int64_t v_stride, fp8_dtype_t dtype, const void* q, int64_t q_stride,
                  int32_t q_heads, uint16_t* q_out, const float* cos, const float* sin, int32_t rope_rows,
                  int32_t rope_pairs, void* stream) {
  int st = kv_checks(cache, batch);
  if (st != FP8_OK) return st;
  if (bad_dtype(dtype)) return FP8_ERR_DTYPE;
  if (q && q_heads < 1) return FP8_ERR_SIZE;
  if (!cos != !sin) return FP8_ERR_NULL;
  if (cos && rope_rows < batch->max_len) return FP8_ERR_SIZE;
  const fp8_kv_batch_t b = bounded(batch);
  if (kv_empty(b)) return FP8_OK;
  const int bytes = dtype == FP8_IN_FP32 ? 4 : 2;
  if ((st = rows_checks(k, k_stride, cache->heads, cache->head_dim, bytes)) != FP8_OK) return st;
  if ((st = rows_checks(v, v_stride, cache->heads, cache->head_dim, bytes)) != FP8_OK) return st;
  if (q) {
    if ((st = rows_checks(q, q_stride, q_heads, cache->head_dim, bytes)) != FP8_OK) return st;
    if (!q_out) return FP8_ERR_NULL;
    if (misaligned(q_out)) return FP8_ERR_ALIGN;
  }
  if (misaligned(cos) || misaligned(sin)) return FP8_ERR_ALIGN;
  if (fp8lin::kv_append_groups(*cache, b, q != nullptr) > (int64_t)0x7FFFFFFF) return FP8_ERR_SIZE;
  if ((st = device_ok()) != FP8_OK) return st;
  return hip_status(fp8lin::launch_kv_append(*cache, b, k, k_stride, v, v_stride, dtype, q, q_stride, q_heads,
                                             q_out, cos, sin, rope_rows, rope_pairs, (hipStream_t)stream));
}

int fp8_kv_read(const fp8_kv_cache_t* cache, const fp8_kv_batch_t* batch, fp8_dtype_t out_dtype, void* k_out,
                void* v_out, void* stream) {
  int st = kv_checks(cache, batch);
  if (st != FP8_OK) return st;
  if (bad_dtype(out_dtype)) return FP8_ERR_DTYPE;
  if (misaligned(k_out) || misaligned(v_out)) return FP8_ERR_ALIGN;
  const fp8_kv_batch_t b = bounded(batch);
  if (kv_empty(b) || (!k_out && !v_out)) return FP8_OK;
  if (fp8lin::kv_append_groups(*cache, b, false) > (int64_t)0x7FFFFFFF) return FP8_ERR_SIZE;
  if ((st = device_ok()) != FP8_OK) return st;
  return hip_status(fp8lin::launch_kv_read(*cache, b, out_dtype, k_out, v_out, (hipStream_t)stream));
}

int64_t fp8_kv_attention_workspace_bytes(const fp8_kv_cache_t* cache, const fp8_kv_batch_t* batch, int32_t q_heads) {
  const int st = kv_checks(cache, batch);
  if (st != FP8_OK) return st;
  if (q_heads < 1 || q_heads % cache->heads != 0) return FP8_ERR_SIZE;
  const fp8_kv_batch_t b = bounded(batch);
  if (kv_empty(b)) return 0;
  return fp8lin::kv_attention_workspace_bytes(*cache, b, q_heads);
}

int fp8_kv_attention(const fp8_kv_cache_t* cache, const fp8_kv_batch_t* batch, const uint16_t* q, int64_t q_stride,
                     int32_t q_heads, float scale, int32_t causal, int32_t window, uint16_t* out, float* lse, void* ws,
                     int64_t ws_bytes, void* stream) {
  const int64_t need = fp8_kv_attention_workspace_bytes(cache, batch, q_heads);
  if (need < 0) return (int)need;
  if (window < 0 || (window > 0 && !causal) || !std::isfinite(scale)) return FP8_ERR_SIZE;
  const fp8_kv_batch_t b = bounded(batch);
  if (kv_empty(b)) return FP8_OK;
  int st = rows_checks(q, q_stride, q_heads, cache->head_dim, 2);
  if (st != FP8_OK) return st;
  if (!out || (need > 0 && !ws)) return FP8_ERR_NULL;
  if (misaligned(out) || misaligned_word(lse) || misaligned(ws)) return FP8_ERR_ALIGN;
  if (ws_bytes < need) return FP8_ERR_SIZE;
  if ((st = device_ok()) != FP8_OK) return st;
  const fp8lin::AttnProblem p{*cache, b, q, q_stride, q_heads, scale, causal, window, out, lse};
  return hip_status(fp8lin::launch_kv_attention(p, ws, (hipStream_t)stream));
}

int fp8_attention_fwd(const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                      int64_t v_stride, const fp8_seqs_t* seqs, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                      float scale, int32_t causal, int32_t window, uint16_t* out, float* lse, void* stream) {
  int st = seqs_checks(seqs, q_heads, kv_heads, head_dim);
  if (st != FP8_OK) return st;
  if (window < 0 || (window > 0 && !causal) || bad_scale(scale)) return FP8_ERR_SIZE;
  if (seqs_empty(*seqs)) return FP8_OK;
  if ((st = seq_rows_checks(q, q_stride, q_heads, head_dim)) != FP8_OK) return st;
  if ((st = seq_rows_checks(k, k_stride, kv_heads, head_dim)) != FP8_OK) return st;
  if ((st = seq_rows_checks(v, v_stride, kv_heads, head_dim)) != FP8_OK) return st;
  if (!out || !lse) return FP8_ERR_NULL;
  if (misaligned(out) || misaligned_word(lse)) return FP8_ERR_ALIGN;
  if ((st = device_ok()) != FP8_OK) return st;
  fp8lin::SeqAttnArgs a = seq_args(*seqs, q_heads, kv_heads, scale, causal, window);
  a.q = q, a.k = k, a.v = v;
  a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride;
  a.out = out;
  a.lse = lse;
  return hip_status(fp8lin::launch_seq_attn_fwd(a, head_dim, (hipStream_t)stream));
}

int64_t fp8_attention_bwd_workspace_bytes(const fp8_seqs_t* seqs, int32_t q_heads, int32_t kv_heads,
                                          int32_t head_dim) {
  const int st = seqs_checks(seqs, q_heads, kv_heads, head_dim);
  if (st != FP8_OK) return st;
  if (seqs_empty(*seqs)) return 0;
  const fp8lin::SeqAttnArgs a = seq_args(*seqs, q_heads, kv_heads, 1.0f, 0, 0);
  return fp8lin::seq_attn_bwd_workspace_bytes({a.batch, a.tokens, a.max_len, q_heads, kv_heads, head_dim});
}

int fp8_attention_bwd(const uint16_t* dout, int64_t dout_stride, const uint16_t* q, int64_t q_stride,
                      const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride, const uint16_t* out,
                      const float* lse, const fp8_seqs_t* seqs, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                      float scale, int32_t causal, int32_t window, uint16_t* dq, int64_t dq_stride, uint16_t* dk,
                      int64_t dk_stride, uint16_t* dv, int64_t dv_stride, void* ws, int64_t ws_bytes, void* stream) {
  const int64_t need = fp8_attention_bwd_workspace_bytes(seqs, q_heads, kv_heads, head_dim);
  if (need < 0) return (int)need;
  if (window < 0 || (window > 0 && !causal) || bad_scale(scale)) return FP8_ERR_SIZE;
  if (seqs_empty(*seqs)) return FP8_OK;
  int st = FP8_OK;
  const struct { const void* p; int64_t stride; int32_t heads; } rows[] = {
      {dout, dout_stride, q_heads}, {q, q_stride, q_heads}, {k, k_stride, kv_heads}, {v, v_stride, kv_heads},
      {dq, dq_stride, q_heads}, {dk, dk_stride, kv_heads}, {dv, dv_stride, kv_heads}};
  for (const auto& r : rows)
    if ((st = seq_rows_checks(r.p, r.stride, r.heads, head_dim)) != FP8_OK) return st;
  if (!out || !lse || !ws) return FP8_ERR_NULL;
  if (misaligned(out) || misaligned_word(lse) || misaligned(ws)) return FP8_ERR_ALIGN;
  if (ws_bytes < need) return FP8_ERR_SIZE;
  if ((st = device_ok()) != FP8_OK) return st;
  fp8lin::SeqAttnArgs a = seq_args(*seqs, q_heads, kv_heads, scale, causal, window);
  a.q = q, a.k = k, a.v = v, a.dout = dout;
  a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride, a.dout_stride = dout_stride;
  a.out = const_cast<uint16_t*>(out);
  a.lse = const_cast<float*>(lse);
  a.dq = dq, a.dk = dk, a.dv = dv;
  a.dq_stride = dq_stride, a.dk_stride = dk_stride, a.dv_stride = dv_stride;
  return hip_status(fp8lin::launch_seq_attn_bwd(a, head_dim, ws, (hipStream_t)stream));
}

int fp8_embedding_fwd(const void* ids, int32_t id_bits, int64_t tokens, const void* table, fp8_dtype_t table_dtype,
                      int64_t vocab, int64_t d, float scale, void* out, fp8_dtype_t out_dtype, void* stream) {
  int st = embedding_checks(ids, id_bits, tokens, vocab, d);
  if (st != FP8_OK) return st;
  if (bad_dtype(table_dtype) || bad_dtype(out_dtype)) return FP8_ERR_DTYPE;
  if (tokens == 0) return FP8_OK;
  if (!out || (vocab > 0 && !table)) return FP8_ERR_NULL;
  if (misaligned(table) || misaligned(out)) return FP8_ERR_ALIGN;
  if ((st = device_ok()) != FP8_OK) return st;
  return hip_status(fp8lin::launch_embedding_fwd(ids, id_bits == 64, tokens, table, table_dtype, vocab, d, scale, out,
                                                 out_dtype, (hipStream_t)stream));
}

int64_t fp8_embedding_bwd_workspace_bytes(int64_t tokens, int64_t vocab, int64_t d) {
  const int st = embedding_checks(reinterpret_cast<const void*>(16), 32, tokens, vocab, d);
  return st != FP8_OK ? st : fp8lin::embedding_bwd_workspace_bytes(tokens, vocab, d);
}

int fp8_embedding_bwd(const void* dout, fp8_dtype_t dout_dtype, const void* ids, int32_t id_bits, int64_t tokens,
                      int64_t vocab, int64_t d, float scale, int32_t accumulate, float* dtable, void* ws,
                      int64_t ws_bytes, void* stream) {
  int st = embedding_checks(ids, id_bits, tokens, vocab, d);
  if (st != FP8_OK) return st;
  if (bad_dtype(dout_dtype)) return FP8_ERR_DTYPE;
  if (vocab == 0 || (tokens == 0 && accumulate)) return FP8_OK;
  if (!dtable || (tokens > 0 && (!dout || !ws))) return FP8_ERR_NULL;
  if (misaligned(dtable) || misaligned(dout) || misaligned(ws)) return FP8_ERR_ALIGN;
  if (ws_bytes < fp8lin::embedding_bwd_workspace_bytes(tokens, vocab, d)) return FP8_ERR_SIZE;
  if ((st = device_ok()) != FP8_OK) return st;
  const fp8lin::EmbeddingGrad g{dout, dout_dtype, ids, id_bits == 64, tokens, vocab, d, scale, accumulate != 0, dtable};
  return hip_status(fp8lin::launch_embedding_bwd(g, ws, (hipStream_t)stream));
}

int fp8_qk_norm_rope_fwd(const void* x, fp8_dtype_t x_dtype, int64_t x_stride, int64_t tokens, int32_t q_heads,
                         int32_t kv_heads, int32_t head_dim, const void* wq, const void* wk, fp8_dtype_t w_dtype,
                         float eps, const int32_t* positions, const float* cos, const float* sin, int32_t rope_rows,
                         int32_t rope_pairs, uint16_t* y, void* stream) {
  const fp8lin::QkProblem p{x, x_dtype, x_stride, tokens, q_heads, kv_heads, head_dim, wq, wk, w_dtype, eps,
                            positions, cos, sin, rope_rows, rope_pairs};
  int st = qk_checks(p);
  if (st != FP8_OK) return st;
  if (tokens == 0) return FP8_OK;
  if (!y) return FP8_ERR_NULL;
  if (misaligned(y)) return FP8_ERR_ALIGN;
  if ((st = device_ok()) != FP8_OK) return st;
  return hip_status(fp8lin::launch_qk_norm_fwd(p, y, (hipStream_t)stream));
}

int64_t fp8_qk_norm_rope_bwd_workspace_bytes(int64_t tokens, int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
  fp8lin::QkProblem p{};
  p.x = reinterpret_cast<const void*>(16);
  p.x_stride = ((int64_t)q_heads + 2 * (int64_t)kv_heads) * head_dim;
  p.tokens = tokens, p.q_heads = q_heads, p.kv_heads = kv_heads, p.head_dim = head_dim;
  const int st = qk_checks(p);
  return st != FP8_OK ? st : fp8lin::qk_norm_bwd_workspace_bytes(p);
}

int fp8_qk_norm_rope_bwd(const uint16_t* dq, int64_t dq_stride, const uint16_t* dk, int64_t dk_stride,
                         const uint16_t* dv, int64_t dv_stride, const void* x, fp8_dtype_t x_dtype, int64_t x_stride,
                         int64_t tokens, int32_t q_heads, int32_t kv_heads, int32_t head_dim, const void* wq,
                         const void* wk, fp8_dtype_t w_dtype, float eps, const int32_t* positions, const float* cos,
                         const float* sin, int32_t rope_rows, int32_t rope_pairs, void* dx, float* dwq, float* dwk,
                         void* ws, int64_t ws_bytes, void* stream) {
  const fp8lin::QkProblem p{x, x_dtype, x_stride, tokens, q_heads, kv_heads, head_dim, wq, wk, w_dtype, eps,
                            positions, cos, sin, rope_rows, rope_pairs};
  int st = qk_checks(p);
  if (st != FP8_OK) return st;
  if (tokens > 0) {
    if ((st = rows_checks(dq, dq_stride, q_heads, head_dim, 2)) != FP8_OK) return st;
    if ((st = rows_checks(dk, dk_stride, kv_heads, head_dim, 2)) != FP8_OK) return st;
    if ((st = rows_checks(dv, dv_stride, kv_heads, head_dim, 2)) != FP8_OK) return st;
    if (!dx) return FP8_ERR_NULL;
    if (misaligned(dx)) return FP8_ERR_ALIGN;
  }
  if (wq) {
    if (!dwq || !dwk || !ws) return FP8_ERR_NULL;
    if (misaligned_word(dwq) || misaligned_word(dwk) || misaligned(ws)) return FP8_ERR_ALIGN;
    if (ws_bytes < fp8lin::qk_norm_bwd_workspace_bytes(p)) return FP8_ERR_SIZE;
  } else if (tokens == 0) {
    return FP8_OK;
  }
  if ((st = device_ok()) != FP8_OK) return st;
  const fp8lin::QkGrads g{dq, dk, dv, dq_stride, dk_stride, dv_stride, dx, dwq, dwk};
  return hip_status(fp8lin::launch_qk_norm_bwd(p, g, static_cast<float*>(ws), (hipStream_t)stream));
}

}  // extern "C"
