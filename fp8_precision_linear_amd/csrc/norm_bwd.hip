// RMS norm, backward (norm_kernel.h).
#include "norm_kernel.h"

namespace fp8lin {
namespace {

struct BwdArgs {
  const void* dy;
  const void* h;
  const void* w;
  int w_dtype;
  const float* rstd;
  const void* dh;  // optional
  int64_t rows;
  int d;
  void* dx;
  float* partial;  // [gridDim.x][d]
  uint32_t* amax;  // optional, cleared before
};

// Each workgroup walks rows blockIdx.x, + gridDim.x, ...; this lane's share of
// dw stays in registers, and the weight where they suffice.  dw leaves as one
// row of `partial` per workgroup, added in a fixed order by norm_dw_kernel.
// 4095 rows of 5120, fp32 dy, bf16 h, dh and dx: 210 MB in 52-53 us (4.0 TB/s:
// eight rows a workgroup, of which the first's loads and the last's sum overlap
// nothing), and 4.7 us for dw.
template <int YT, int HT, bool WHOLE, int U, int W>
__global__ __launch_bounds__(kBlock<W>) void norm_bwd_kernel(BwdArgs a) {
  constexpr int kLanes = 64 * W;
  constexpr int kRows = kBlock<W> / kLanes;
  __shared__ float part[2][W];
  const int t = W == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int sub = W == 1 ? threadIdx.x >> 6 : 0;
  const int d = a.d;
  // sixteen waves leave 128 registers a lane, too few to keep w as well
  constexpr bool kKeepW = W < 16;
  float w[kKeepW ? U : 1][4], dw[U][4];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int j = (u * kLanes + t) * 4;
#pragma unroll
    for (int e = 0; e < 4; ++e) dw[u][e] = 0.0f;
    if constexpr (kKeepW) {
#pragma unroll
      for (int e = 0; e < 4; ++e) w[u][e] = 0.0f;
      if (j < d) load_weight<WHOLE>(a.w, a.w_dtype, j, d - j, w[u]);
    }
  }
  uint32_t top = 0;
  int parity = 0;
  // a row's inputs, loaded one row ahead (the sixteen-wave shape has no
  // registers for that: its loads stand where they are used)
  constexpr bool kAhead = W < 16;
  Raw<YT> ry[U];
  Raw<HT> rh[U], rd[U];
  float rs_next = 0.0f;
  auto fetch = [&](int64_t row) {
    if (row >= a.rows) return;
    const int64_t base = row * d;
    rs_next = a.rstd[row];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = (u * kLanes + t) * 4;
      if (j < d) {
        ry[u] = load_raw<YT, WHOLE, true>(a.dy, base + j, d - j);
        rh[u] = load_raw<HT, WHOLE, true>(a.h, base + j, d - j);
        if (kAhead && a.dh) rd[u] = load_raw<HT, WHOLE, true>(a.dh, base + j, d - j);
      }
    }
  };
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t row = (int64_t)blockIdx.x * kRows + sub;
  if constexpr (kAhead) fetch(row);
  for (; row < a.rows; row += step) {
    if constexpr (!kAhead) fetch(row);
    const int64_t base = row * d;
    const float rs = rs_next;
    float g[U][4], xh[U][4];
    Raw<HT> rd_now[kAhead ? U : 1];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = (u * kLanes + t) * 4;
#pragma unroll
      for (int e = 0; e < 4; ++e) g[u][e] = xh[u][e] = 0.0f;
      if (j < d) {
        unpack<YT>(ry[u], g[u]);
        unpack<HT>(rh[u], xh[u]);
        if constexpr (kAhead) rd_now[u] = rd[u];
      }
    }
    if constexpr (kAhead) fetch(row + step);
    float c = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float* wu = w[kKeepW ? u : 0];
      if constexpr (!kKeepW) {
        int j = (u * kLanes + t) * 4;
        asm volatile("" : "+v"(j));  // or the loads leave the loop, into registers again
        float ww[4] = {};
        if (j < d) load_weight<WHOLE>(a.w, a.w_dtype, j, d - j, ww);
#pragma unroll
        for (int e = 0; e < 4; ++e) wu[e] = ww[e];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        xh[u][e] *= rs;
        dw[u][e] = fmaf(g[u][e], xh[u][e], dw[u][e]);
        g[u][e] *= wu[e];
        c = fmaf(g[u][e], xh[u][e], c);
      }
    }
    c = row_sum<W>(c, part[parity]) / (float)d;
    parity ^= 1;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = (u * kLanes + t) * 4;
      if (j < d) {
        float o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = rs * (g[u][e] - xh[u][e] * c);
        if (a.dh) {
          float past[4];
          if constexpr (kAhead) unpack<HT>(rd_now[u], past);
          else load_stream<HT, WHOLE>(a.dh, base + j, d - j, past);
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] += past[e];
        }
        round_to<HT>(o);
        store_as<HT, WHOLE>(a.dx, base + j, d - j, o);
        top = unit_max<WHOLE>(top, d - j, o);
      }
    }
  }
  if (a.amax) fold_amax_wave(top, a.amax);
  // a workgroup of four one-wave rows adds its waves' shares in wave order
  if constexpr (kRows > 1) {
    __shared__ float acc[kRows - 1][U * 4][64];
    if (sub > 0) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[sub - 1][u * 4 + e][t] = dw[u][e];
    }
    __syncthreads();
    if (sub > 0) return;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int s = 0; s < kRows - 1; ++s) dw[u][e] += acc[s][u * 4 + e][t];
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int j = (u * kLanes + t) * 4;
    if (j < d) store_as<FP8_IN_FP32, WHOLE>(a.partial, (int64_t)blockIdx.x * d + j, d - j, dw[u]);
  }
}

// dw[j] = sum over the `parts` rows of partial, 16 interleaved shares of the
// rows first, then those in order; in 64 bits, since up to 512 parts in a row
// would add more to the error than all that went before (the time is that of the
// loads: 4.7 us for 512 x 5120).
constexpr int kDwCols = 64, kDwShares = 16;
__global__ __launch_bounds__(kDwCols* kDwShares) void norm_dw_kernel(const float* partial, int parts, int d,
                                                                    float* dw) {
  __shared__ double s[kDwShares][kDwCols];
  const int c = threadIdx.x & (kDwCols - 1), q = threadIdx.x / kDwCols;
  const int j = blockIdx.x * kDwCols + c;
  double v = 0.0;
  if (j < d) {
#pragma unroll 8
    for (int p = q; p < parts; p += kDwShares) v += partial[(int64_t)p * d + j];
  }
  s[q][c] = v;
  __syncthreads();
  if (q == 0 && j < d) {
    for (int k = 1; k < kDwShares; ++k) v += s[k][c];
    dw[j] = (float)v;
  }
}

// Workgroups (and rows of partial sums) of the backward pass.
int bwd_parts(int64_t rows, int64_t d) {
  const int64_t rows_per = d <= 1024 ? 4 : 1;
  const int64_t blocks = (rows + rows_per - 1) / rows_per;
  return (int)(blocks < 512 ? blocks : 512);
}

}  // namespace

int64_t norm_bwd_workspace_bytes(int64_t rows, int64_t d) { return (int64_t)bwd_parts(rows, d) * d * 4; }

hipError_t launch_norm_bwd(const void* dy, int dy_dtype, const void* h, int h_dtype, const void* w, int w_dtype,
                           const float* rstd, const void* dh, int64_t rows, int64_t d, void* dx, float* dw,
                           uint32_t* amax, float* ws, hipStream_t stream) {
  if (amax) hipLaunchKernelGGL(clear_kernel, dim3(1), dim3(1), 0, stream, amax);
  const int parts = bwd_parts(rows, d);
  if (rows > 0) {
    const BwdArgs a{dy, h, w, w_dtype, rstd, dh, rows, (int)d, dx, ws, amax};
    for_dtype(dy_dtype, [&](auto yt) {
      for_dtype(h_dtype, [&](auto ht) {
        if constexpr (yt.value != kNone && ht.value != kNone)
          for_shape((int)d, [&](auto whole, auto u, auto w_) {
            hipLaunchKernelGGL((norm_bwd_kernel<yt.value, ht.value, whole.value, u.value, w_.value>),
                               dim3((uint32_t)parts), dim3(kBlock<w_.value>), 0, stream, a);
          });
      });
    });
  }
  hipLaunchKernelGGL(norm_dw_kernel, dim3((uint32_t)((d + kDwCols - 1) / kDwCols)), dim3(kDwCols * kDwShares), 0,
                     stream, ws, parts, (int)d, dw);
  return hipGetLastError();
}

}  // namespace fp8lin
