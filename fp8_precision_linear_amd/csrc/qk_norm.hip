// Norms of queries and keys for each head with the rotary positions, forward
// and backward (include/fp8lin_train.h has the definitions).
//
//   y = R(pos) n,  n_j = x_j rstd w_j          R: rotation by the token's angles
//   dn = R(-pos) dy,  g = dn w,  xhat = x rstd
//   dx_j = rstd (g_j - xhat_j mean(g xhat)),  dw_j = sum dn_j xhat_j
//
// HBM-bound: every element is read once and written once, x of the values by the
// forward alone (8192 tokens of 80 heads of 128: 93 us, 5.4 TB/s; gradients of 4095
// of 120: 122 us, 4.5 TB/s, and 12 for the weights').  A lane holds a unit of eight
// dimensions of a head -- four and the four that they rotate with -- so D / 8 lanes
// hold a head, its sums take log2(D / 8) shuffles, and the rotation none.  A wave
// takes several steps of 64 units of one token: the lane's unit of a head, and with
// it its weights and angles, are the same in all of them.
#include <algorithm>

#include "quotient.h"
#include "rope.h"

namespace fp8lin {
namespace {

struct QkArgs {
  const void* x;
  int64_t x_stride;
  const void* wq;
  const void* wk;
  int w_dtype;
  float eps;
  const int32_t* positions;
  Rope rope;
  int64_t tokens;
  int q_heads, heads;  // heads: of keys, and of values
  int steps;           // of 64 units of a token
  int per;             // steps of an item
  int items;           // of a token
  int64_t all_items;
  uint16_t* y;
  // backward
  const uint16_t *dq, *dk, *dv;
  int64_t dq_stride, dk_stride, dv_stride;
  void* dx;
  float* part;  // [workgroups][2][D]
  int64_t run;  // items of a workgroup
  uint32_t first;
};

// Most steps of an item, whose loads are in flight together.  The backward pass
// holds two tensors and twelve sums beside them: two steps leave four waves a SIMD
// (4095 tokens of 120 heads of 128: four steps 134 us, two 126).
constexpr int kSteps = 4, kBwdSteps = 2;

// The sum over the LANES lanes of a head, in every one of them.
template <int LANES>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int off = 1; off < LANES; off <<= 1) v += __shfl_xor(v, off, 64);
  return v;
}

template <int D>
__device__ __forceinline__ void load_weights(const QkArgs& a, const void* w, int u, float (&v)[8]) {
  if (a.w_dtype == FP8_IN_FP32) {
    load4<FP8_IN_FP32>(w, unit_lo<D>(u), v);
    load4<FP8_IN_FP32>(w, unit_hi<D>(u), v + 4);
  } else {
    load4<FP8_IN_BF16>(w, unit_lo<D>(u), v);
    load4<FP8_IN_BF16>(w, unit_hi<D>(u), v + 4);
  }
}

// A wave's share of one token: units [64 step0, ...) in up to kSteps steps.
struct Item {
  int64_t token;
  int step0, steps;
};
__device__ __forceinline__ Item item_of(const QkArgs& a, int64_t i) {
  Item r;
  r.token = quotient(i, a.items);
  r.step0 = (int)(i - r.token * a.items) * a.per;
  r.steps = min(a.per, a.steps - r.step0);
  return r;
}
__device__ __forceinline__ int position_of(const QkArgs& a, int64_t token) {
  const int64_t p = a.positions ? a.positions[token] : token;
  return (int)max((int64_t)0, min(p, (int64_t)a.rope.rows - 1));
}

template <int DT, int D, int ROPE, bool NORM>
__global__ __launch_bounds__(256) void qk_norm_fwd_kernel(QkArgs a) {
  constexpr int kLanes = D / 8;
  const int lane = threadIdx.x & 63, u = lane % kLanes;
  const int64_t i = (int64_t)(a.first + blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (i >= a.all_items) return;
  const Item it = item_of(a, i);
  const int all = a.q_heads + 2 * a.heads;
  auto head_of = [&](int s) { return (64 * (it.step0 + s) + lane) / kLanes; };
  float v[kSteps][8], angle[8], wq[8], wk[8];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    if (s < it.steps && head_of(s) < all) {
      const int64_t at = it.token * a.x_stride + head_of(s) * D;
      load4<DT>(a.x, at + unit_lo<D>(u), v[s]);
      load4<DT>(a.x, at + unit_hi<D>(u), v[s] + 4);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[s][e] = 0.0f;
    }
  }
  if constexpr (NORM) {
    load_weights<D>(a, a.wq, u, wq);
    load_weights<D>(a, a.wk, u, wk);
  }
  if constexpr (ROPE != kRopeNone) load_angles<D, ROPE>(angle, u, position_of(a, it.token), a.rope);
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    if (s >= it.steps) break;
    const int head = head_of(s);
    float n[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) n[e] = v[s][e];
    if constexpr (NORM) {
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(n[e], n[e], sum);
      const float r = rsqrtf(head_sum<kLanes>(sum) * (1.0f / D) + a.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) n[e] = n[e] * r * (head < a.q_heads ? wq[e] : wk[e]);
    }
    rotate<ROPE>(n, angle);
    if (head >= all) continue;
#pragma unroll
    for (int e = 0; e < 8; ++e) n[e] = head < a.q_heads + a.heads ? n[e] : v[s][e];
    uint16_t* y = a.y + (it.token * all + head) * D;
    *reinterpret_cast<uint2*>(y + unit_lo<D>(u)) = bf16x4(n);
    *reinterpret_cast<uint2*>(y + unit_hi<D>(u)) = bf16x4(n + 4);
  }
}

// dx, and this workgroup's share of dwq and dwk: a lane adds its dimensions of
// the heads that its wave meets, the workgroup adds its lanes in LDS.
template <int DT, int D, int ROPE, bool NORM>
__global__ __launch_bounds__(256) void qk_norm_bwd_kernel(QkArgs a) {
  constexpr int kSteps = kBwdSteps;
  constexpr int kLanes = D / 8, kHeads = 64 / kLanes;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, u = lane % kLanes;
  const int all = a.q_heads + 2 * a.heads;
  float wq[8], wk[8], sum_q[8], sum_k[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sum_q[e] = sum_k[e] = 0.0f;
  if constexpr (NORM) {
    load_weights<D>(a, a.wq, u, wq);
    load_weights<D>(a, a.wk, u, wk);
  }
  // a run of the items, which its waves take in turn
  const int64_t begin = (int64_t)blockIdx.x * a.run, end = min(begin + a.run, a.all_items);
  for (int64_t i = begin + wave; i < end; i += 4) {
    const Item it = item_of(a, i);
    auto head_of = [&](int s) { return (64 * (it.step0 + s) + lane) / kLanes; };
    float v[kSteps][8], g[kSteps][8], angle[8];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int head = head_of(s);
      if (s < it.steps && head < all) {
        const bool is_q = head < a.q_heads, is_v = head >= a.q_heads + a.heads;
        const uint16_t* dy = is_q ? a.dq + it.token * a.dq_stride + head * D
                                  : (is_v ? a.dv + it.token * a.dv_stride + (head - a.q_heads - a.heads) * D
                                          : a.dk + it.token * a.dk_stride + (head - a.q_heads) * D);
        load4<FP8_IN_BF16>(dy, unit_lo<D>(u), g[s]);
        load4<FP8_IN_BF16>(dy, unit_hi<D>(u), g[s] + 4);
        if (NORM && !is_v) {
          const int64_t at = it.token * a.x_stride + head * D;
          load4<DT>(a.x, at + unit_lo<D>(u), v[s]);
          load4<DT>(a.x, at + unit_hi<D>(u), v[s] + 4);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[s][e] = 0.0f;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[s][e] = g[s][e] = 0.0f;
      }
    }
    if constexpr (ROPE != kRopeNone) {
      load_angles<D, ROPE>(angle, u, position_of(a, it.token), a.rope);
#pragma unroll
      for (int e = 4; e < 8; ++e) angle[e] = -angle[e];  // back
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      if (s >= it.steps) break;
      const int head = head_of(s);
      const bool is_q = head < a.q_heads, is_v = head >= a.q_heads + a.heads;
      float n[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) n[e] = g[s][e];
      rotate<ROPE>(n, angle);
      if constexpr (NORM) {
        float xx = 0.0f, gx = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float w = n[e] * (is_q ? wq[e] : wk[e]);
          xx = fmaf(v[s][e], v[s][e], xx);
          gx = fmaf(w, v[s][e], gx);
        }
        const float r = rsqrtf(head_sum<kLanes>(xx) * (1.0f / D) + a.eps);
        const float c = head_sum<kLanes>(gx) * (1.0f / D) * r;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float xhat = v[s][e] * r, dw = n[e] * xhat;
          sum_q[e] += is_q ? dw : 0.0f;
          sum_k[e] += is_q || is_v ? 0.0f : dw;
          n[e] = r * (n[e] * (is_q ? wq[e] : wk[e]) - xhat * c);
        }
      }
      if (head >= all) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) n[e] = is_v ? g[s][e] : n[e];
      const int64_t at = (it.token * all + head) * D;
      if constexpr (DT == FP8_IN_FP32) {
        float* dx = static_cast<float*>(a.dx) + at;
        *reinterpret_cast<float4*>(dx + unit_lo<D>(u)) = make_float4(n[0], n[1], n[2], n[3]);
        *reinterpret_cast<float4*>(dx + unit_hi<D>(u)) = make_float4(n[4], n[5], n[6], n[7]);
      } else {
        uint16_t* dx = static_cast<uint16_t*>(a.dx) + at;
        *reinterpret_cast<uint2*>(dx + unit_lo<D>(u)) = bf16x4(n);
        *reinterpret_cast<uint2*>(dx + unit_hi<D>(u)) = bf16x4(n + 4);
      }
    }
  }
  if constexpr (NORM) {
    __shared__ float sums[2][4 * kHeads][D];
    const int row = wave * kHeads + lane / kLanes;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int d = e < 4 ? unit_lo<D>(u) + e : unit_hi<D>(u) + e - 4;
      sums[0][row][d] = sum_q[e];
      sums[1][row][d] = sum_k[e];
    }
    __syncthreads();
    for (int j = threadIdx.x; j < 2 * D; j += 256) {
      float s = 0.0f;
#pragma unroll
      for (int r = 0; r < 4 * kHeads; ++r) s += sums[j / D][r][j % D];
      a.part[(int64_t)blockIdx.x * 2 * D + j] = s;
    }
  }
}

// dwq and dwk: the workgroups' shares added in 64 bits, in order.  A workgroup
// takes 16 columns: four lanes of four columns, 64 of them down the rows, eight
// rows of each on their way at once.
__global__ __launch_bounds__(256) void qk_norm_dw_kernel(const float* part, int rows, int D, float* dwq, float* dwk) {
  __shared__ double sums[64][17];
  const int quad = threadIdx.x & 3, lane = threadIdx.x >> 2, col = blockIdx.x * 16 + 4 * quad;
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  for (int r0 = lane; r0 < rows; r0 += 64 * 8) {
    float4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = r0 + 64 * i;
      v[i] = r < rows ? *reinterpret_cast<const float4*>(part + (int64_t)r * 2 * D + col) : make_float4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) s[0] += v[i].x, s[1] += v[i].y, s[2] += v[i].z, s[3] += v[i].w;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) sums[lane][4 * quad + e] = s[e];
  __syncthreads();
  // 16 lanes a column, then across them
  const int c = threadIdx.x >> 4, part_of = threadIdx.x & 15;
  double t = (sums[part_of][c] + sums[part_of + 16][c]) + (sums[part_of + 32][c] + sums[part_of + 48][c]);
#pragma unroll
  for (int off = 1; off < 16; off <<= 1) t += __shfl_xor(t, off, 64);
  const int to = blockIdx.x * 16 + c;
  if (part_of == 0) (to < D ? dwq : dwk)[to % D] = (float)t;
}

template <typename F>
void for_kind(const QkProblem& p, F&& f) {
  using std::bool_constant;
  using std::integral_constant;
  auto dtype = [&](auto d, auto rope, auto norm) {
    if (p.x_dtype == FP8_IN_FP32) f(integral_constant<int, FP8_IN_FP32>{}, d, rope, norm);
    else f(integral_constant<int, FP8_IN_BF16>{}, d, rope, norm);
  };
  auto normed = [&](auto d, auto rope) {
    if (p.wq) dtype(d, rope, bool_constant<true>{});
    else dtype(d, rope, bool_constant<false>{});
  };
  auto turned = [&](auto d) {
    if (!p.cos) normed(d, integral_constant<int, kRopeNone>{});
    else if (p.rope_pairs) normed(d, integral_constant<int, kRopePairs>{});
    else normed(d, integral_constant<int, kRopeHalves>{});
  };
  if (p.head_dim == 64) turned(integral_constant<int, 64>{});
  else if (p.head_dim == 128) turned(integral_constant<int, 128>{});
  else turned(integral_constant<int, 256>{});
}

QkArgs args_of(const QkProblem& p, int most_steps) {
  QkArgs a{};
  a.x = p.x, a.x_stride = p.x_stride;
  a.wq = p.wq, a.wk = p.wk, a.w_dtype = p.w_dtype, a.eps = p.eps;
  a.positions = p.positions;
  a.rope = {p.cos, p.sin, p.rope_rows};
  a.tokens = p.tokens, a.q_heads = p.q_heads, a.heads = p.kv_heads;
  a.steps = (int)(((int64_t)(p.q_heads + 2 * p.kv_heads) * (p.head_dim / 8) + 63) / 64);
  a.items = (a.steps + most_steps - 1) / most_steps;
  a.per = (a.steps + a.items - 1) / a.items;
  a.items = (a.steps + a.per - 1) / a.per;
  a.all_items = p.tokens * a.items;
  return a;
}

// Items of a workgroup of the backward kernel, whose share of the weights'
// gradients is joined with the others': few where there are few items, so that
// every CU has work (2048 tokens of 36 heads of 64, 8 and 16 items 25-26 us, 64 38);
// otherwise 32 (4095 tokens of 120 heads of 128: 16 items 135 us, 32 126, and a
// resident grid that strides over them 141), and no more than kMostGroups shares.
constexpr int64_t kLeastRun = 4, kMostRun = 32, kWantGroups = 512, kMostGroups = 16384;
int64_t run_of(const QkArgs& a) {
  const int64_t run = std::max(kLeastRun, std::min(kMostRun, a.all_items / kWantGroups & ~(int64_t)3));
  return std::max(run, (a.all_items + kMostGroups - 1) / kMostGroups);
}
int64_t bwd_groups(const QkArgs& a) { return std::max<int64_t>(1, (a.all_items + run_of(a) - 1) / run_of(a)); }

}  // namespace

hipError_t launch_qk_norm_fwd(const QkProblem& p, uint16_t* y, hipStream_t stream) {
  QkArgs a = args_of(p, kSteps);
  a.y = y;
  in_stretches((a.all_items + 3) / 4, 256, [&](uint32_t first, uint32_t count) {
    a.first = first;
    for_kind(p, [&](auto dt, auto d, auto rope, auto norm) {
      hipLaunchKernelGGL((qk_norm_fwd_kernel<decltype(dt)::value, decltype(d)::value, decltype(rope)::value,
                                             decltype(norm)::value>),
                         dim3(count), dim3(256), 0, stream, a);
    });
  });
  return hipGetLastError();
}

int64_t qk_norm_bwd_workspace_bytes(const QkProblem& p) { return bwd_groups(args_of(p, kBwdSteps)) * 2 * p.head_dim * 4; }

hipError_t launch_qk_norm_bwd(const QkProblem& p, const QkGrads& g, float* ws, hipStream_t stream) {
  QkArgs a = args_of(p, kBwdSteps);
  a.dq = g.dq, a.dk = g.dk, a.dv = g.dv;
  a.dq_stride = g.dq_stride, a.dk_stride = g.dk_stride, a.dv_stride = g.dv_stride;
  a.dx = g.dx;
  a.part = ws;
  a.run = run_of(a);
  const int groups = (int)bwd_groups(a);
  for_kind(p, [&](auto dt, auto d, auto rope, auto norm) {
    hipLaunchKernelGGL((qk_norm_bwd_kernel<decltype(dt)::value, decltype(d)::value, decltype(rope)::value,
                                           decltype(norm)::value>),
                       dim3(groups), dim3(256), 0, stream, a);
  });
  if (p.wq)
    hipLaunchKernelGGL(qk_norm_dw_kernel, dim3(2 * p.head_dim / 16), dim3(256), 0, stream, (const float*)ws, groups,
                       p.head_dim, g.dwq, g.dwk);
  return hipGetLastError();
}

}  // namespace fp8lin
