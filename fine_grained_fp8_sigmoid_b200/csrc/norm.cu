// The pre-norm of the layer and its gradient: s = x + residual,
// y = s / sqrt(mean s^2 + eps) * w, with y in bf16 for the router and in E4M3
// with one FP32 scale per 1x128 tile for the experts.
#include "host.cuh"

namespace moe {
namespace norm {

// Eight consecutive values as FP32: bf16 (one 16-byte access) or FP32 (two).
// Plain loads, not the read-only path: outputs may alias inputs.
__device__ __forceinline__ void load8(const uint16_t* p, float (&f)[8]) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  const float4 b = *reinterpret_cast<const float4*>(p + 4);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  return float_to_bf16_bits(lo) | (static_cast<uint32_t>(float_to_bf16_bits(hi)) << 16);
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&f)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(bf16x2(f[0], f[1]), bf16x2(f[2], f[3]), bf16x2(f[4], f[5]), bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}

// Sums N values over the blockDim.x threads of one row (blockDim.y rows a
// block); every thread of the row gets the sums. red: 32 * N floats a row.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* red) {
#pragma unroll
  for (int k = 0; k < N; ++k)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return;
  if (lane_id() == 0)
#pragma unroll
    for (int k = 0; k < N; ++k) red[k * 32 + (threadIdx.x >> 5)] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    float s = 0.0f;
    for (int i = 0; i < warps; ++i) s += red[k * 32 + i];
    v[k] = s;
  }
}

// One row per blockDim.x threads, VPT runs of 8 channels a thread, held in
// registers between the sum of squares and the outputs.
template <typename S, typename W, int VPT>
__global__ void __launch_bounds__(1024) rmsnorm_quant_kernel(const uint16_t* x, long long ldx, const S* res,
                                                             const W* w, float eps, int rows, int d, S* h,
                                                             uint16_t* y, uint8_t* q, float* scale) {
  __shared__ float red_all[4 * 32];
  const int row = blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = row < rows;
  const int V = d >> 3;
  const size_t base = static_cast<size_t>(live ? row : 0) * d;
  float s[VPT][8];
  float ss[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (live && v < V) {
      load8(x + static_cast<size_t>(row) * ldx + v * 8, s[i]);
      if (res != nullptr) {
        float r[8];
        load8(res + base + v * 8, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[i][j] += r[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss[0] = fmaf(s[i][j], s[i][j], ss[0]);
    }
  }
  row_sum(ss, red_all + threadIdx.y * 32);
  const float rstd = __frsqrt_rn(ss[0] / static_cast<float>(d) + eps);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    const bool on = live && v < V;           // uniform over the 16 lanes of a tile
    float t[8];
    float amax = 0.0f;
    if (on) {
      if (h != nullptr) store8(h + base + v * 8, s[i]);
      load8(w + v * 8, t);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        t[j] *= s[i][j] * rstd;
        amax = fmaxf(amax, fabsf(t[j]));
      }
      if (y != nullptr) store8(y + base + v * 8, t);
    }
    if (q != nullptr) {                      // uniform: every lane takes part in the shuffles
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      if (on) {
        const float sc = tile_scale(amax);
        uint32_t c[2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
          c[k] = e4m3x2(__fdiv_rn(t[4 * k], sc), __fdiv_rn(t[4 * k + 1], sc)) |
                 (e4m3x2(__fdiv_rn(t[4 * k + 2], sc), __fdiv_rn(t[4 * k + 3], sc)) << 16);
        *reinterpret_cast<uint2*>(q + base + v * 8) = make_uint2(c[0], c[1]);
        if ((v & 15) == 0) scale[static_cast<size_t>(row) * (d >> 7) + (v >> 4)] = sc;
      }
    }
  }
}

// Rows blockIdx.x, blockIdx.x + gridDim.x, ..: a thread owns its channels for
// all of them, so dw needs no exchange before the partial row it writes.
template <typename S, typename W, int VPT>
__global__ void __launch_bounds__(512) rmsnorm_backward_kernel(const uint16_t* dy, const S* h, const W* w,
                                                               float eps, const S* dres, int rows, int d, S* dh,
                                                               float* part) {
  __shared__ float red_all[2][2 * 32];
  const int V = d >> 3;
  float dw[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  int flip = 0;
  for (int row = blockIdx.x; row < rows; row += gridDim.x, flip ^= 1) {
    const size_t base = static_cast<size_t>(row) * d;
    float hv[VPT][8], gy[VPT][8];
    float sum[2] = {0.0f, 0.0f};             // sum h^2, sum dy w h
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < V) {
        float wv[8];
        load8(h + base + v * 8, hv[i]);
        load8(dy + base + v * 8, gy[i]);
        load8(w + v * 8, wv);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          sum[0] = fmaf(hv[i][j], hv[i][j], sum[0]);
          sum[1] = fmaf(gy[i][j] * wv[j], hv[i][j], sum[1]);
        }
      }
    }
    row_sum(sum, red_all[flip]);             // two buffers: the next row's sums may start early
    const float r = __frsqrt_rn(sum[0] / static_cast<float>(d) + eps);
    const float c = sum[1] / static_cast<float>(d) * r * r;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < V) {
        float wv[8], o[8];
        load8(w + v * 8, wv);
        if (dres != nullptr) {
          load8(dres + base + v * 8, o);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          dw[i][j] = fmaf(gy[i][j], hv[i][j] * r, dw[i][j]);
          o[j] = fmaf(r, gy[i][j] * wv[j] - hv[i][j] * c, o[j]);
        }
        store8(dh + base + v * 8, o);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v < V) store8(part + static_cast<size_t>(blockIdx.x) * d + v * 8, dw[i]);
  }
}

// dw = sum of the n partial rows, in a fixed order: 32 columns a block, eight
// threads a column.
__global__ void __launch_bounds__(256) column_sum_kernel(const float* __restrict__ part, int n, int d, float* dw) {
  __shared__ float red[8][33];
  const int col = blockIdx.x * 32 + threadIdx.x;
  float s = 0.0f;
  if (col < d)
    for (int i = threadIdx.y; i < n; i += 8) s += part[static_cast<size_t>(i) * d + col];
  red[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && col < d) {
#pragma unroll
    for (int k = 1; k < 8; ++k) s += red[k][threadIdx.x];
    dw[col] = s;
  }
}

constexpr int MAX_D = 1024 * 8 * 4;
constexpr int BWD_MAX_D = 512 * 8 * 4;
constexpr int MAX_PARTS = 592;

inline int vpt_for(int V, int threads) {
  int vpt = 1;
  while ((V + vpt - 1) / vpt > threads) vpt *= 2;
  return vpt;
}

}  // namespace norm
}  // namespace moe

extern "C" int moe_rmsnorm_quant(const uint16_t* x, long long ldx, const void* res, int stream_is_fp32,
                                 const void* w, int w_is_bf16, float eps, int rows, int d, void* h, uint16_t* y,
                                 uint8_t* q, float* scale, void* stream) {
  using namespace moe;
  using namespace moe::norm;
  MOE_CHECK_ARG(rows >= 0 && d >= 0 && eps >= 0.0f && ldx >= d);
  MOE_CHECK_SUPPORTED(d % 8 == 0 && d <= MAX_D && ldx % 8 == 0 && (q == nullptr || d % 128 == 0));
  if (rows == 0 || d == 0) return MOE_OK;
  MOE_CHECK_ARG(x && w && (h || y || q) && (q == nullptr) == (scale == nullptr));
  const uintptr_t all = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(res) |
                        reinterpret_cast<uintptr_t>(w) | reinterpret_cast<uintptr_t>(h) |
                        reinterpret_cast<uintptr_t>(y) | (reinterpret_cast<uintptr_t>(q) << 1);
  MOE_CHECK_ARG(all % 16 == 0 && reinterpret_cast<uintptr_t>(scale) % 4 == 0);
  DeviceInfo di;
  if (int st = device_info(&di)) return st;
  const int V = d / 8;
  const int vpt = vpt_for(V, rows <= di.sm_count || V > 256 * 4 ? 1024 : 256);
  const int nt = ((V + vpt - 1) / vpt + 31) / 32 * 32;
  const int per = nt >= 128 ? 1 : 128 / nt;
  const dim3 block(nt, per);
  const unsigned grid = static_cast<unsigned>((static_cast<long long>(rows) + per - 1) / per);
  auto launch = [&](auto s, auto wt, auto n) {
    using S = decltype(s);
    using W = decltype(wt);
    rmsnorm_quant_kernel<S, W, decltype(n)::value><<<grid, block, 0, as_stream(stream)>>>(
        x, ldx, static_cast<const S*>(res), static_cast<const W*>(w), eps, rows, d, static_cast<S*>(h), y, q, scale);
  };
  auto by_vpt = [&](auto s, auto wt) {
    if (vpt == 1) launch(s, wt, std::integral_constant<int, 1>{});
    else if (vpt == 2) launch(s, wt, std::integral_constant<int, 2>{});
    else launch(s, wt, std::integral_constant<int, 4>{});
  };
  if (stream_is_fp32) { if (w_is_bf16) by_vpt(0.0f, uint16_t(0)); else by_vpt(0.0f, 0.0f); }
  else { if (w_is_bf16) by_vpt(uint16_t(0), uint16_t(0)); else by_vpt(uint16_t(0), 0.0f); }
  return launch_status("rmsnorm launch");
}

extern "C" size_t moe_rmsnorm_backward_workspace(int rows, int d) {
  if (rows <= 0 || d <= 0) return 0;
  const size_t n = rows < moe::norm::MAX_PARTS ? rows : moe::norm::MAX_PARTS;
  return n * d * sizeof(float);
}

extern "C" int moe_rmsnorm_backward(const uint16_t* dy, const void* h, int stream_is_fp32, const void* w,
                                    int w_is_bf16, float eps, const void* dres, int rows, int d, void* dh, float* dw,
                                    void* workspace, size_t ws_bytes, void* stream) {
  using namespace moe;
  using namespace moe::norm;
  MOE_CHECK_ARG(rows >= 0 && d >= 0 && eps >= 0.0f);
  MOE_CHECK_SUPPORTED(d % 8 == 0 && d <= BWD_MAX_D);
  if (d == 0) return MOE_OK;
  MOE_CHECK_ARG(dw);
  cudaStream_t st_ = as_stream(stream);
  if (rows == 0) return cuda_status(cudaMemsetAsync(dw, 0, static_cast<size_t>(d) * 4, st_), "rmsnorm backward: zero dw");
  MOE_CHECK_ARG(dy && h && w && dh && workspace && ws_bytes >= moe_rmsnorm_backward_workspace(rows, d));
  const uintptr_t all = reinterpret_cast<uintptr_t>(dy) | reinterpret_cast<uintptr_t>(h) |
                        reinterpret_cast<uintptr_t>(w) | reinterpret_cast<uintptr_t>(dres) |
                        reinterpret_cast<uintptr_t>(dh) | reinterpret_cast<uintptr_t>(dw) |
                        reinterpret_cast<uintptr_t>(workspace);
  MOE_CHECK_ARG(all % 16 == 0);
  DeviceInfo di;
  if (int st = device_info(&di)) return st;
  const int V = d / 8;
  const int vpt = vpt_for(V, V > 256 * 4 || rows <= di.sm_count ? 512 : 256);
  const int nt = ((V + vpt - 1) / vpt + 31) / 32 * 32;
  int parts = di.sm_count * (nt <= 256 ? 3 : 2);
  if (parts > rows) parts = rows;
  if (parts > MAX_PARTS) parts = MAX_PARTS;
  float* part = parts == 1 ? dw : static_cast<float*>(workspace);
  auto launch = [&](auto s, auto wt, auto n) {
    using S = decltype(s);
    using W = decltype(wt);
    rmsnorm_backward_kernel<S, W, decltype(n)::value><<<parts, nt, 0, st_>>>(
        dy, static_cast<const S*>(h), static_cast<const W*>(w), eps, static_cast<const S*>(dres), rows, d,
        static_cast<S*>(dh), part);
  };
  auto by_vpt = [&](auto s, auto wt) {
    if (vpt == 1) launch(s, wt, std::integral_constant<int, 1>{});
    else if (vpt == 2) launch(s, wt, std::integral_constant<int, 2>{});
    else launch(s, wt, std::integral_constant<int, 4>{});
  };
  if (stream_is_fp32) { if (w_is_bf16) by_vpt(0.0f, uint16_t(0)); else by_vpt(0.0f, 0.0f); }
  else { if (w_is_bf16) by_vpt(uint16_t(0), uint16_t(0)); else by_vpt(uint16_t(0), 0.0f); }
  if (int st = launch_status("rmsnorm backward launch")) return st;
  if (parts > 1) {
    column_sum_kernel<<<(d + 31) / 32, dim3(32, 8), 0, st_>>>(part, parts, d, dw);
    return launch_status("rmsnorm backward: column sums");
  }
  return MOE_OK;
}
