// The pre-norm of the layer and its gradient: s = x + residual,
// y = s / sqrt(mean s^2 + eps) * w, with y in bf16 for the router and in E4M3
// with one FP32 scale per 1x128 tile for the experts.
#include "host.cuh"

namespace moe {
namespace norm {

// Eight consecutive values as FP32: bf16 (one 16-byte access) or FP32 (two).
// Plain loads, not the read-only path: outputs may alias inputs.
template <typename T>
struct Raw8;                                 // as loaded: what is still on its way
template <>
struct Raw8<uint16_t> {
  uint4 v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
};
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&f)[8]) {
  Raw8<T> r;
  r.load(p);
  r.get(f);
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

// Four E4M3 codes of fl32(t / s) from t and inv = fl32(1 / s). fl32(t inv) is
// within 1.5 2^-23 of fl32(t / s), so where both ends of a 2^-21 bracket around
// it round to the same codes those are the codes; false where a rounding border
// lies inside, and the values have to be divided. Dividing every value took 125
// us in place of 115 at T = 8192, d = 7168, before what else was changed.
__device__ __forceinline__ bool codes_by_reciprocal(const float* t, float inv, uint32_t& q) {
  constexpr float LO = 1.0f - 0x1p-21f, HI = 1.0f + 0x1p-21f;
  const float a = t[0] * inv, b = t[1] * inv, c = t[2] * inv, d = t[3] * inv;
  q = e4m3x2(a * LO, b * LO) | (e4m3x2(c * LO, d * LO) << 16);
  return q == (e4m3x2(a * HI, b * HI) | (e4m3x2(c * HI, d * HI) << 16));
}

// Eight values t of a 1x128 tile, held by 16 neighbouring lanes: their codes and
// the tile's scale (moe_quant_1x128's rule). Every lane of the warp calls it;
// `on` is the same for the 16 lanes of a tile.
__device__ __forceinline__ void store_codes(const float (&t)[8], bool on, uint8_t* q, float* scale, bool first) {
  float amax = 0.0f;
  if (on)
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(t[j]));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (!on) return;
  const float sc = tile_scale(amax);
  const float inv = __frcp_rn(sc);
  uint32_t c[2];
  bool sure = sc >= 0x1p-100f;               // 1 / sc and the products are normal numbers
  sure = codes_by_reciprocal(t, inv, c[0]) && sure;
  sure = codes_by_reciprocal(t + 4, inv, c[1]) && sure;
  if (!sure) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
      c[k] = e4m3x2(__fdiv_rn(t[4 * k], sc), __fdiv_rn(t[4 * k + 1], sc)) |
             (e4m3x2(__fdiv_rn(t[4 * k + 2], sc), __fdiv_rn(t[4 * k + 3], sc)) << 16);
  }
  *reinterpret_cast<uint2*>(q) = make_uint2(c[0], c[1]);
  if (first) *scale = sc;
}

// One row per blockDim.x threads, VPT runs of 8 channels a thread, held in
// registers between the sum of squares and the outputs: every input is read
// once and every output written once. Memory bounds it: T = 8192, d = 7168 with
// a bf16 residual moves 530 MB in 88 us, 6.0 of the copy's 6.45 TB/s (events
// around one call behind a read of 256 MB, as all figures here; 86 us from a
// graph of calls, 92 to 95 as calls one after the other through the binding,
// each behind the last one's writes). What carries it is that x and res are all on their way before the first is used
// (100 us with a load per use: stores and loads that may alias keep their
// order) and that many rows share an SM, whose waits overlap: a block per row
// beats blocks that stay and fetch the next row ahead, into registers (108 us
// against 100) or by bulk copies into a ring (106), and w is loaded late, which
// costs a wait and spares the registers of a fourth block (102 us with w loaded
// at once after the sum). With at most a row per SM the row's latency counts,
// and a thread takes one run.
template <typename S, typename W, int VPT>
__global__ void __launch_bounds__(1024) rmsnorm_quant_kernel(const uint16_t* x, long long ldx, const S* res,
                                                             const W* w, float eps, float inv_d, int rows, int d,
                                                             S* h,
                                                             uint16_t* y, uint8_t* q, float* scale) {
  __shared__ float red_all[4 * 32];
  const int row = blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = row < rows;
  const int V = d >> 3;
  const size_t base = static_cast<size_t>(live ? row : 0) * d;
  float s[VPT][8];
  float ss[1] = {0.0f};
  Raw8<uint16_t> xr[VPT];                    // all loads before the first use
  Raw8<S> rr[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (live && v < V) {
      xr[i].load(x + static_cast<size_t>(row) * ldx + v * 8);
      if (res != nullptr) rr[i].load(res + base + v * 8);
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (live && v < V) {
      xr[i].get(s[i]);
      if (res != nullptr) {
        float r[8];
        rr[i].get(r);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[i][j] += r[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss[0] = fmaf(s[i][j], s[i][j], ss[0]);
      if (h != nullptr) store8(h + base + v * 8, s[i]);
    }
  }
  row_sum(ss, red_all + threadIdx.y * 32);
  const float rstd = rsqrtf(fmaf(ss[0], inv_d, eps));
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    const bool on = live && v < V;
    float t[8];
    if (on) {
      load8(w + v * 8, t);
#pragma unroll
      for (int j = 0; j < 8; ++j) t[j] *= s[i][j] * rstd;
      if (y != nullptr) store8(y + base + v * 8, t);
    }
    if (q != nullptr)
      store_codes(t, on, q + base + v * 8, scale + static_cast<size_t>(row) * (d >> 7) + (v >> 4), (v & 15) == 0);
  }
}

// Sums two values over the `warps` (at most 16) first warps of a block; every
// thread gets the sums. The lower half of a warp sums the first value and the
// upper half the second: 11 shuffles in place of 20. red: 32 floats that the
// next call does not use.
__device__ __forceinline__ void block_sum2(float& a, float& b, float* red, int warps) {
  const int warp = threadIdx.x >> 5, lane = lane_id();
  const bool up = lane >= 16;
  float v = (up ? b : a) + __shfl_xor_sync(0xffffffffu, up ? a : b, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (warps > 1) {
    if ((lane & 15) == 0) red[lane + warp] = v;          // the first value's 16 places, then the second's
    named_bar_sync(1, warps * 32);
    v = (lane & 15) < warps ? red[lane] : 0.0f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  }
  a = __shfl_sync(0xffffffffu, v, 0);
  b = __shfl_sync(0xffffffffu, v, 16);
}

__device__ __forceinline__ void bulk_row(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

constexpr int MAX_RING = 8;

// Rows blockIdx.x, blockIdx.x + gridDim.x, ..: a thread owns its channels for
// all of them, so w stays in registers and dw needs no exchange before the
// partial row it writes. The last warp keeps a ring of whole rows (h, dy, dres)
// on their way into shared memory by bulk copies: a row is used twice with a
// sum over the block between, and with plain loads the block stood still for
// their latency twice a row. T = 8192, d = 7168: 79 us with the column sums
// (470 MB, 6.0 TB/s; events around one call, 75 us from a graph, 80 to 84 as
// calls one after the other) against 247 with plain loads; 4096 x 2048 in FP32: 25 us,
// where half of the issue slots are taken and the sums over a row's warps cost
// as much as its arithmetic.
template <typename S, typename W, int VPT>
__global__ void __launch_bounds__(544) rmsnorm_backward_kernel(const uint16_t* dy, const S* h, const W* w, float eps, float inv_d,
                                                               const S* dres, int rows, int d, int ring, S* dh,
                                                               float* part) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint64_t full[MAX_RING], empty[MAX_RING];
  __shared__ float red_all[2][32];
  __shared__ int abort_flag;
  volatile int* abort = &abort_flag;
  const int warps = (blockDim.x >> 5) - 1, warp = threadIdx.x >> 5;
  const uint32_t hb = d * sizeof(S), yb = d * 2, stage = hb + yb + (dres != nullptr ? hb : 0);
  if (threadIdx.x == 0) {
    for (int i = 0; i < ring; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], warps); }
    abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == warps) {
    if (lane_id() == 0) {
      int s = 0, n = 0;
      uint32_t lap = 1;
      bool ok = true;
      // dh may lie over h or dres: a row is written only after its own copies have landed
      for (int row = blockIdx.x; ok && row < rows; row += gridDim.x, ++n) {
        if (!(ok = mbar_wait(&empty[s], lap, abort))) break;
        uint8_t* dst = smem + static_cast<size_t>(s) * stage;
        const size_t base = static_cast<size_t>(row) * d;
        mbar_arrive_expect_tx(&full[s], stage);
        bulk_row(dst, h + base, hb, &full[s]);
        bulk_row(dst + hb, dy + base, yb, &full[s]);
        if (dres != nullptr) bulk_row(dst + hb + yb, dres + base, hb, &full[s]);
        if (++s == ring) { s = 0; lap ^= 1; }
      }
      for (int j = max(0, n - ring); j < n; ++j) mbar_drain(&full[j % ring], (j / ring) & 1);
    }
  } else {
    const int V = d >> 3;
    float dw[VPT][8], wv[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * warps * 32;
#pragma unroll
      for (int j = 0; j < 8; ++j) dw[i][j] = wv[i][j] = 0.0f;
      if (v < V) load8(w + v * 8, wv[i]);
    }
    int s = 0, flip = 0;
    uint32_t lap = 0;
    bool ok = true;
    for (int row = blockIdx.x; row < rows; row += gridDim.x, flip ^= 1) {
      ok = ok && warp_wait(&full[s], lap, abort);
      const uint8_t* src = smem + static_cast<size_t>(s) * stage;
      float hv[VPT][8], gy[VPT][8];
      float hh = 0.0f, gh = 0.0f;            // sum h^2, sum dy w h
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = threadIdx.x + i * warps * 32;
        if (v < V) {
          load8(reinterpret_cast<const S*>(src) + v * 8, hv[i]);
          load8(reinterpret_cast<const uint16_t*>(src + hb) + v * 8, gy[i]);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            hh = fmaf(hv[i][j], hv[i][j], hh);
            gh = fmaf(gy[i][j] * wv[i][j], hv[i][j], gh);
          }
        }
      }
      block_sum2(hh, gh, red_all[flip], warps);
      const float r = rsqrtf(fmaf(hh, inv_d, eps));
      const float c = gh * inv_d * r * r;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = threadIdx.x + i * warps * 32;
        if (v < V) {
          float o[8];
          if constexpr (VPT > 2) {           // too many to keep: read again
            load8(reinterpret_cast<const S*>(src) + v * 8, hv[i]);
            load8(reinterpret_cast<const uint16_t*>(src + hb) + v * 8, gy[i]);
          }
          if (dres != nullptr) {
            load8(reinterpret_cast<const S*>(src + hb + yb) + v * 8, o);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = 0.0f;
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            dw[i][j] = fmaf(gy[i][j], hv[i][j] * r, dw[i][j]);
            o[j] = fmaf(r, gy[i][j] * wv[i][j] - hv[i][j] * c, o[j]);
          }
          if (ok) store8(dh + static_cast<size_t>(row) * d + v * 8, o);
        }
      }
      __syncwarp();
      if (lane_id() == 0) mbar_arrive(&empty[s]);
      if (++s == ring) { s = 0; lap ^= 1; }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * warps * 32;
      if (v < V) store8(part + static_cast<size_t>(blockIdx.x) * d + v * 8, dw[i]);
    }
  }
  __syncthreads();
}

// dw = sum of the n partial rows, in a fixed order: 32 columns a block, 32
// threads a column.
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* part, int n, int d, float* dw) {
  __shared__ float red[32][33];
  const int col = blockIdx.x * 32 + threadIdx.x;
  float s = 0.0f;
  asm volatile("griddepcontrol.wait;" ::: "memory");     // launched before the partial rows are there
  if (col < d)
#pragma unroll 4
    for (int i = threadIdx.y; i < n; i += 32) s += part[static_cast<size_t>(i) * d + col];
  red[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  s = red[threadIdx.x][threadIdx.y];                     // a warp a column
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (threadIdx.x == 0 && blockIdx.x * 32 + threadIdx.y < d) dw[blockIdx.x * 32 + threadIdx.y] = s;
}

constexpr int MAX_D = 1024 * 8 * 4;
constexpr int BWD_MAX_D = 512 * 8 * 4;
constexpr int BWD_MAX_ROWS = 1 << 30;         // a block's row, stepped past the last one, stays in 32 bits
constexpr int MAX_PARTS = 592;
constexpr int BWD_SMEM = 220 * 1024;          // of an SM's 227 KB, for the rings of its blocks

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
        x, ldx, static_cast<const S*>(res), static_cast<const W*>(w), eps, 1.0f / d, rows, d,
        static_cast<S*>(h), y, q, scale);
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
  MOE_CHECK_SUPPORTED(d % 8 == 0 && d <= BWD_MAX_D && rows <= BWD_MAX_ROWS);
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
  // Threads a row, measured at 8192 rows: 256 runs of 8 channels took 36 us with 128 threads and four blocks an SM,
  // 39 with 256 and three; 896 took 82 us with 224 threads and two blocks, 107 with 448 and one (33 and 79
  // of the ones taken since a row's two sums share an exchange).
  const int vpt = vpt_for(V, V <= 256 ? 128 : V <= 1024 ? 256 : 512);
  const int nt = ((V + vpt - 1) / vpt + 31) / 32 * 32 + 32;      // and the copying warp
  const size_t row_bytes = static_cast<size_t>(d) * (2 + (stream_is_fp32 ? 4 : 2) * (dres ? 2 : 1));
  int per_sm = nt <= 160 ? 4 : nt <= 288 && row_bytes <= 36 * 1024 ? 3 : row_bytes <= 54 * 1024 ? 2 : 1;
  if (rows <= di.sm_count) per_sm = 1;
  int ring = static_cast<int>(BWD_SMEM / per_sm / row_bytes);
  if (ring > MAX_RING) ring = MAX_RING;
  if (ring < 1) ring = 1;
  int parts = di.sm_count * per_sm;
  if (parts > rows) parts = rows;
  if (parts > MAX_PARTS) parts = MAX_PARTS;
  const int most = (rows + parts - 1) / parts;                   // rows of a block
  if (ring > most) ring = most;
  const size_t smem = ring * row_bytes;
  float* part = parts == 1 ? dw : static_cast<float*>(workspace);
  int attr = MOE_OK;
  auto launch = [&](auto s, auto wt, auto n) {
    using S = decltype(s);
    using W = decltype(wt);
    auto k = rmsnorm_backward_kernel<S, W, decltype(n)::value>;
    // With the static part more than 48 KB need asking. The limit belongs to the function, not to the launch: one value
    // for every shape, so that a call of another host thread cannot lower it before this launch.
    if (smem > 40 * 1024)
      attr = cuda_status(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, BWD_SMEM),
                         "rmsnorm backward: smem attribute");
    if (attr == MOE_OK)
      k<<<parts, nt, smem, st_>>>(dy, static_cast<const S*>(h), static_cast<const W*>(w), eps, 1.0f / d, static_cast<const S*>(dres),
                                  rows, d, ring, static_cast<S*>(dh), part);
  };
  auto by_vpt = [&](auto s, auto wt) {
    if (vpt == 1) launch(s, wt, std::integral_constant<int, 1>{});
    else if (vpt == 2) launch(s, wt, std::integral_constant<int, 2>{});
    else launch(s, wt, std::integral_constant<int, 4>{});
  };
  if (stream_is_fp32) { if (w_is_bf16) by_vpt(0.0f, uint16_t(0)); else by_vpt(0.0f, 0.0f); }
  else { if (w_is_bf16) by_vpt(uint16_t(0), uint16_t(0)); else by_vpt(uint16_t(0), 0.0f); }
  if (attr != MOE_OK) return attr;
  if (int st = launch_status("rmsnorm backward launch")) return st;
  if (parts > 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((d + 31) / 32);
    cfg.blockDim = dim3(32, 32);
    cfg.stream = st_;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, column_sum_kernel, static_cast<const float*>(part), parts, d, dw),
                       "rmsnorm backward: column sums");
  }
  return MOE_OK;
}
