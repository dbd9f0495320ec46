// RMS norm, forward (norm_kernel.h).
#include "norm_kernel.h"

namespace fp8lin {
namespace {

// What the forward kernel writes.
constexpr int kOutBf16 = 0;    // y in bf16
constexpr int kOutCodes = 1;   // codes at *bias
constexpr int kOutStats = 2;   // row_amax only (the codes need every row's), or,
                               // where there is one row, its amax, bias and codes

struct FwdArgs {
  const void* x;
  const void* r;
  const void* w;
  int w_dtype;
  int64_t rows;
  int d;
  float eps;
  void* h;         // written where there is a residual
  float* rstd;     // optional
  void* y;         // bf16 or codes
  int fmt;
  int32_t margin;
  const int32_t* bias_in;  // kOutCodes
  uint32_t* amax;          // optional (folded, cleared before); kOutStats: one row's
  uint32_t* row_amax;      // kOutStats
  int32_t* bias_out;       // kOutStats, one row
};

template <int XT, int RT, int V, int U, int W, int OUT>
__global__ __launch_bounds__(kBlock<W>) void norm_fwd_kernel(FwdArgs a) {
  constexpr int kLanes = 64 * W;                 // lanes per row
  constexpr int kRows = kBlock<W> / kLanes;      // rows per workgroup
  __shared__ float part[2][W];
  const int t = W == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int sub = W == 1 ? threadIdx.x >> 6 : 0;
  const int d = a.d;
  uint32_t top = 0;
  int parity = 0;
  int32_t bias = 0;
  if constexpr (OUT == kOutCodes) bias = *a.bias_in;
  for (int64_t row = (int64_t)blockIdx.x * kRows + sub; row < a.rows; row += (int64_t)gridDim.x * kRows) {
    const int64_t base = row * d;
    float h[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = (u * kLanes + t) * V;
      if (j < d) {
        load_stream<XT, V>(a.x, base + j, h[u]);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) h[u][e] = 0.0f;
      }
    }
    if constexpr (RT != kNone) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = (u * kLanes + t) * V;
        if (j < d) {
          float r[V];
          load_stream<RT, V>(a.r, base + j, r);
#pragma unroll
          for (int e = 0; e < V; ++e) h[u][e] += r[e];
          round_to<RT, V>(h[u]);
          store_as<RT, V>(a.h, base + j, h[u]);
        }
      }
    }
    float ss = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < V; ++e) ss = fmaf(h[u][e], h[u][e], ss);
    // two sets of words: a wave may reach the next row's sum while another
    // still reads this one's
    ss = row_sum<W>(ss, part[parity]);
    parity ^= 1;
    const float rstd = 1.0f / sqrtf(ss / (float)d + a.eps);
    if (a.rstd && t == 0) a.rstd[row] = rstd;
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = (u * kLanes + t) * V;
      if (j < d) {
        float w[V];
        load_cached<V>(a.w, a.w_dtype, j, w);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          h[u][e] = h[u][e] * rstd * w[e];
          if constexpr (OUT == kOutBf16)
            m = max(m, (bf16_bits(h[u][e]) & 0x7FFFu) << 16);
          else
            m = max(m, __float_as_uint(h[u][e]) & 0x7FFFFFFFu);
        }
        if constexpr (OUT == kOutBf16) store_as<FP8_IN_BF16, V>(a.y, base + j, h[u]);
        if constexpr (OUT == kOutCodes) store_codes<V>(static_cast<uint8_t*>(a.y), base + j, h[u], a.fmt, bias);
      }
    }
    if constexpr (OUT == kOutStats) {
      m = row_max<W>(m, reinterpret_cast<uint32_t*>(part[parity]));
      parity ^= 1;
      if (t == 0) a.row_amax[row] = m;
      if (a.rows == 1) {
        const int32_t b = bias_from_amax_bits(m, a.fmt, a.margin);
        if (t == 0) {
          *a.amax = m;
          *a.bias_out = b;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int j = (u * kLanes + t) * V;
          if (j < d) store_codes<V>(static_cast<uint8_t*>(a.y), base + j, h[u], a.fmt, b);
        }
      }
    } else {
      top = max(top, m);
    }
  }
  if constexpr (OUT == kOutBf16 || OUT == kOutCodes)
    if (a.amax) fold_amax_wave(top, a.amax);
}

// The second half of fp8_rmsnorm_quantize: the tensor's amax from every row's,
// the bias from it, and the codes of y formed again from h.  The rows are
// walked from the last one: what the first half wrote last is still cached.
template <int V>
__global__ __launch_bounds__(256) void norm_cast_kernel(const void* h, int h_dtype, const float* rstd,
                                                        const void* w, int w_dtype, int64_t rows, int d,
                                                        const uint32_t* row_amax, int fmt, int32_t margin,
                                                        uint8_t* y, uint32_t* amax, int32_t* bias) {
  __shared__ uint32_t part[4];
  uint32_t m = 0;
  for (int64_t i = threadIdx.x; i < rows; i += 256) m = max(m, row_amax[i]);
  m = row_max<4>(m, part);
  const int32_t b = bias_from_amax_bits(m, fmt, margin);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *amax = m;
    *bias = b;
  }
  for (int64_t k = blockIdx.x; k < rows; k += gridDim.x) {
    const int64_t row = rows - 1 - k;
    const float rs = rstd[row];
#pragma unroll 4
    for (int j = threadIdx.x * V; j < d; j += 256 * V) {
      float v[V], ww[V];
      load_cached<V>(h, h_dtype, row * d + j, v);
      load_cached<V>(w, w_dtype, j, ww);
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = v[e] * rs * ww[e];
      store_codes<V>(y, row * d + j, v, fmt, b);
    }
  }
}

constexpr int64_t kMaxBlocks = 2048;  // eight 256-lane workgroups per CU

template <int OUT>
void launch_fwd(const NormProblem& p, const FwdArgs& a, hipStream_t stream) {
  for_dtype(p.x_dtype, [&](auto xt) {
    if constexpr (xt.value != kNone) {
      for_dtype(p.r ? p.r_dtype : kNone, [&](auto rt) {
        for_shape(a.d, [&](auto v, auto u, auto w) {
          constexpr int W = w.value;
          const int64_t rows_per = kBlock<W> / (64 * W);
          const int64_t blocks = (a.rows + rows_per - 1) / rows_per;
          const int64_t cap = W == 16 ? kMaxBlocks / 4 : kMaxBlocks;
          hipLaunchKernelGGL((norm_fwd_kernel<xt.value, rt.value, v.value, u.value, W, OUT>),
                             dim3((uint32_t)(blocks < cap ? blocks : cap)), dim3(kBlock<W>), 0, stream, a);
        });
      });
    }
  });
}

FwdArgs fwd_args(const NormProblem& p) {
  FwdArgs a{};
  a.x = p.x;
  a.r = p.r;
  a.w = p.w;
  a.w_dtype = p.w_dtype;
  a.rows = p.rows;
  a.d = (int)p.d;
  a.eps = p.eps;
  a.h = p.h;
  a.rstd = p.rstd;
  return a;
}

}  // namespace

hipError_t launch_norm_fwd(const NormProblem& p, uint16_t* y, uint32_t* amax, hipStream_t stream) {
  FwdArgs a = fwd_args(p);
  a.y = y;
  a.amax = amax;
  if (amax) hipLaunchKernelGGL(clear_kernel, dim3(1), dim3(1), 0, stream, amax);
  if (p.rows > 0) launch_fwd<kOutBf16>(p, a, stream);
  return hipGetLastError();
}

hipError_t launch_norm_cast(const NormProblem& p, const int32_t* bias, int fmt, uint8_t* y, uint32_t* amax,
                            hipStream_t stream) {
  FwdArgs a = fwd_args(p);
  a.y = y;
  a.fmt = fmt;
  a.bias_in = bias;
  a.amax = amax;
  if (amax) hipLaunchKernelGGL(clear_kernel, dim3(1), dim3(1), 0, stream, amax);
  if (p.rows > 0) launch_fwd<kOutCodes>(p, a, stream);
  return hipGetLastError();
}

hipError_t launch_norm_quantize(const NormProblem& p, int fmt, int32_t margin, uint8_t* y, uint32_t* row_amax,
                                uint32_t* amax, int32_t* bias, hipStream_t stream) {
  FwdArgs a = fwd_args(p);
  a.y = y;
  a.fmt = fmt;
  a.margin = margin;
  a.row_amax = row_amax;
  a.amax = amax;
  a.bias_out = bias;
  if (p.rows > 0) launch_fwd<kOutStats>(p, a, stream);
  if (p.rows == 1) return hipGetLastError();
  const void* h = p.r ? p.h : p.x;
  const int h_dtype = p.r ? p.r_dtype : p.x_dtype;
  const int64_t blocks = p.rows < kMaxBlocks ? (p.rows > 0 ? p.rows : 1) : kMaxBlocks;
  if (p.d % 4 == 0)
    hipLaunchKernelGGL(norm_cast_kernel<4>, dim3((uint32_t)blocks), dim3(256), 0, stream, h, h_dtype, p.rstd, p.w,
                       p.w_dtype, p.rows, (int)p.d, row_amax, fmt, margin, y, amax, bias);
  else
    hipLaunchKernelGGL(norm_cast_kernel<1>, dim3((uint32_t)blocks), dim3(256), 0, stream, h, h_dtype, p.rstd, p.w,
                       p.w_dtype, p.rows, (int)p.d, row_amax, fmt, margin, y, amax, bias);
  return hipGetLastError();
}

}  // namespace fp8lin
