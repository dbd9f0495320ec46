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

// With current scaling (kOutStats) 8192 rows of 8192, fp32 x and a bf16
// residual, move 537 MB here in 89-91 us: 5.9 TB/s.  Codes at a known bias leave
// this kernel alone: 8000 rows of 4096 in 57 us, 5.2 TB/s.
template <int XT, int RT, bool WHOLE, int U, int W, int OUT>
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
  const Codes codes(a.fmt, bias);
  // the weight stays in registers over the workgroup's rows (where sixteen
  // waves leave enough), its loads in flight with the first row's
  constexpr bool kKeepW = W < 16;
  float w[kKeepW ? U : 1][4];
  if constexpr (kKeepW) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = (u * kLanes + t) * 4;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[u][e] = 0.0f;
      if (j < d) load_weight<WHOLE>(a.w, a.w_dtype, j, d - j, w[u]);
    }
  }
  for (int64_t row = (int64_t)blockIdx.x * kRows + sub; row < a.rows; row += (int64_t)gridDim.x * kRows) {
    const int64_t base = row * d;
    float h[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = (u * kLanes + t) * 4;
      if (j < d) {
        load_stream<XT, WHOLE>(a.x, base + j, d - j, h[u]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) h[u][e] = 0.0f;
      }
    }
    if constexpr (RT != kNone) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = (u * kLanes + t) * 4;
        if (j < d) {
          float r[4];
          load_stream<RT, WHOLE>(a.r, base + j, d - j, r);
#pragma unroll
          for (int e = 0; e < 4; ++e) h[u][e] += r[e];
          round_to<RT>(h[u]);
          store_as<RT, WHOLE>(a.h, base + j, d - j, h[u]);
        }
      }
    }
    float ss = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) ss = fmaf(h[u][e], h[u][e], ss);
    // two sets of words: a wave may reach the next row's sum while another
    // still reads this one's
    ss = row_sum<W>(ss, part[parity]);
    parity ^= 1;
    const float rstd = 1.0f / sqrtf(ss / (float)d + a.eps);
    if (a.rstd && t == 0) a.rstd[row] = rstd;
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = (u * kLanes + t) * 4;
      if (j < d) {
        float* wu = w[kKeepW ? u : 0];
        if constexpr (!kKeepW) load_weight<WHOLE>(a.w, a.w_dtype, j, d - j, w[0]);
#pragma unroll
        for (int e = 0; e < 4; ++e) h[u][e] = h[u][e] * rstd * wu[e];
        if constexpr (OUT == kOutBf16) round_to<FP8_IN_BF16>(h[u]);
        m = unit_max<WHOLE>(m, d - j, h[u]);
        if constexpr (OUT == kOutBf16) store_as<FP8_IN_BF16, WHOLE>(a.y, base + j, d - j, h[u]);
        if constexpr (OUT == kOutCodes) codes.store<WHOLE>(static_cast<uint8_t*>(a.y), base + j, d - j, h[u]);
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
        const Codes c(a.fmt, b);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int j = (u * kLanes + t) * 4;
          if (j < d) c.store<WHOLE>(static_cast<uint8_t*>(a.y), base + j, d - j, h[u]);
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
// the bias from it, and the codes of y formed again from h.  A workgroup takes
// 1024 columns, whose weights its lanes keep, of every `groups`-th row, four
// rows in flight; the first ones' loads stand before the amax.  Rows are walked
// from the last one: what the first half wrote last is still cached.
// 8192 x 8192: 201 MB in 39 us, 5.1 TB/s.
constexpr int kCastRows = 4;
template <int HT, bool WHOLE>
__global__ __launch_bounds__(256) void norm_cast_kernel(const void* h, const float* rstd, const void* w, int w_dtype,
                                                        int64_t rows, int d, int col_blocks, int groups,
                                                        const uint32_t* row_amax, int fmt, int32_t margin, uint8_t* y,
                                                        uint32_t* amax, int32_t* bias) {
  __shared__ uint32_t part[4];
  const int t = threadIdx.x;
  const int j = ((int)(blockIdx.x % col_blocks) * 256 + t) * 4;
  const int64_t group = blockIdx.x / col_blocks;
  const bool live = j < d && rows > 0;  // without rows w need not be there
  float ww[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) ww[e] = 0.0f;
  if (live) load_weight<WHOLE>(w, w_dtype, j, d - j, ww);
  Raw<HT> x[kCastRows];
  float rs[kCastRows];
  auto fetch = [&](int64_t k) {
#pragma unroll
    for (int q = 0; q < kCastRows; ++q) {
      const int64_t at = k + (int64_t)q * groups;
      if (live && at < rows) {
        const int64_t row = rows - 1 - at;
        rs[q] = rstd[row];
        x[q] = load_raw<HT, WHOLE, false>(h, row * d + j, d - j);
      }
    }
  };
  fetch(group);
  uint32_t m = 0;
  int64_t done = 0;
  if (((uintptr_t)row_amax & 15u) == 0) {
    const uint4* v = reinterpret_cast<const uint4*>(row_amax);
#pragma unroll 4
    for (int64_t i = t; i < rows / 4; i += 256) {
      const uint4 q = v[i];
      m = max(max(m, max(q.x, q.y)), max(q.z, q.w));
    }
    done = rows / 4 * 4;
  }
  for (int64_t i = done + t; i < rows; i += 256) m = max(m, row_amax[i]);
  m = row_max<4>(m, part);
  const int32_t b = bias_from_amax_bits(m, fmt, margin);
  if (blockIdx.x == 0 && t == 0) {
    *amax = m;
    *bias = b;
  }
  const Codes codes(fmt, b);
  for (int64_t k = group; k < rows; k += (int64_t)kCastRows * groups) {
#pragma unroll
    for (int q = 0; q < kCastRows; ++q) {
      const int64_t at = k + (int64_t)q * groups;
      if (live && at < rows) {
        float v[4];
        unpack<HT>(x[q], v);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = v[e] * rs[q] * ww[e];
        codes.store<WHOLE>(y, (rows - 1 - at) * d + j, d - j, v);
      }
    }
    fetch(k + (int64_t)kCastRows * groups);
  }
}

// Most workgroups: eight of 256 lanes per CU; three of 512 (8192 x 8192 in 91
// us; 1024 workgroups 111, 2048 94), two of 1024.
constexpr int64_t kMaxBlocks = 2048;
// Of the second half, six per CU: not a power of two, which makes the rows in
// flight meet in few memory channels (8192 x 8192 in 39 us; 1024: 49, 2048: 49).
constexpr int64_t kCastBlocks = 1536;

template <int OUT>
void launch_fwd(const NormProblem& p, const FwdArgs& a, hipStream_t stream) {
  for_dtype(p.x_dtype, [&](auto xt) {
    if constexpr (xt.value != kNone) {
      for_dtype(p.r ? p.r_dtype : kNone, [&](auto rt) {
        for_shape(a.d, [&](auto whole, auto u, auto w) {
          constexpr int W = w.value;
          const int64_t rows_per = kBlock<W> / (64 * W);
          const int64_t blocks = (a.rows + rows_per - 1) / rows_per;
          const int64_t cap = W == 16 ? 512 : W == 8 ? 768 : kMaxBlocks;
          hipLaunchKernelGGL((norm_fwd_kernel<xt.value, rt.value, whole.value, u.value, W, OUT>),
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
  const int col_blocks = (int)((p.d + 1023) / 1024);
  // rows shared out over kCastBlocks workgroups, each with whole batches of
  // kCastRows where there are rows enough
  int64_t groups = (p.rows + kCastRows - 1) / kCastRows;
  const int64_t most = kCastBlocks / col_blocks > 0 ? kCastBlocks / col_blocks : 1;
  groups = groups < most ? groups : most;
  if (groups == 0) groups = 1;
  auto run = [&](auto ht, auto whole) {
    hipLaunchKernelGGL((norm_cast_kernel<ht.value, whole.value>), dim3((uint32_t)(groups * col_blocks)), dim3(256), 0,
                       stream, h, p.rstd, p.w, p.w_dtype, p.rows, (int)p.d, col_blocks, (int)groups, row_amax, fmt,
                       margin, y, amax, bias);
  };
  for_dtype(h_dtype, [&](auto ht) {
    if constexpr (ht.value != kNone) {
      if (p.d % 4 == 0) run(ht, std::bool_constant<true>{});
      else run(ht, std::bool_constant<false>{});
    }
  });
  return hipGetLastError();
}

}  // namespace fp8lin
