// The whole layer for at most 16 tokens in one kernel: router, selection,
// selected experts and the shared one, combine.
//
// Every byte of the touched experts' weights is read once and nothing else is
// large, so the kernel is a stream of weights: one CTA per SM (a cooperative
// launch), a producer warp that keeps a ring of bulk copies in flight across
// all phases, and eight warps that multiply. The weights do not depend on the
// exchange between the phases, only on the selection, so the ring fills with
// the shared expert while the router runs and with W_down while the last
// intermediate rows are written.
//
// The products run on the register tensor-core path (m16n8k32, E4M3): 16
// weight rows by 8 tokens. Tokens fill at most two such tiles, the products
// need a small part of its rate, and its 16-row granularity splits the rows of
// W_gate, W_up and W_down evenly over the SMs, which 128-row TMEM tiles cannot
// (one token: 9 experts are 144 tiles in the first phase and 252 in the
// second, for 148 SMs).
#include "host.cuh"

namespace moe {
namespace few {

constexpr int MAX_T = 16;
constexpr int MAX_K = 16;
constexpr int MAX_N = 256;
constexpr int MAX_SLOTS = MAX_N + 1;
constexpr int MAX_ENTRIES = MAX_T * MAX_K + MAX_T;
constexpr int CW = 8;                        // multiplying warps
constexpr int KC = CW * 128;                 // channels of a stage: one 128-block a warp
constexpr int ROWS = 16;                     // weight rows of a stage
constexpr int STAGE = ROWS * KC;
constexpr int MAX_STAGES = 12;
constexpr int MAX_HBUF = 4;
constexpr int MAX_TILES = 4;                 // 16-row tiles of W_down a CTA owns
constexpr int RCOL = 20;                     // padded rows of a reduction column
constexpr int THREADS = (CW + 1 + 3) * 32;   // 12 warps: 168 registers a thread
constexpr int SMEM_MAX = 227 * 1024;

// NT: 8-token tiles. EW: warps that finish units of the first phase.
template <int NT> struct Shape {
  static constexpr int EW = NT == 1 ? 3 : 2;
  static constexpr int RED = CW * NT * 8 * RCOL;      // floats of one unit's partials
};

// Tensor maps of the weights, rows [slot * rows] by 128-byte blocks: a box is
// R rows by KC / 128 blocks, stored [block][row][128] with the 128-byte swizzle.
struct Maps {
  CUtensorMap gate, up;     // R = 8
  CUtensorMap down[5];      // R = 1 << i
};

// Bytes of a row of n bytes such that neighbouring rows start 16 bytes apart
// modulo 128 (n a multiple of 16).
__host__ __device__ constexpr int pitch_of(int n) { return ((n + 111) & ~127) + 16; }

struct Args {
  const uint16_t* u;
  const uint16_t* base;
  const uint16_t* e;
  const float* b;
  const uint8_t* xq;        // the experts' input: the caller's, or the workspace's
  const float* xs;
  uint8_t* xq_ws;           // not NULL: quantise u into the workspace
  float* xs_ws;
  const float *s_gate, *s_up, *s_down;
  uint16_t* out;
  int32_t* topk_idx;
  float* gates;
  int32_t* counts;
  unsigned* grid_ctr;       // two grid barriers, 128 bytes apart
  int* blk_ctr;             // [slot][I/128]: finished 8-row units of a block
  float* scores;            // [T][N_r]
  float* act;               // [T*K + T][I] silu(G) U
  uint8_t* hrec;            // [T*K + T][hrec_bytes]: I codes, then I/128 scales
  int T, d, N_r, K, I;
  int stages, hbufs, xh_bytes, hrec_bytes;
};

// Shared memory behind the dynamic regions.
struct Small {
  uint64_t full[MAX_STAGES], empty[MAX_STAGES];
  uint64_t hfull[MAX_HBUF], hempty[MAX_HBUF];
  uint64_t redfull[4], redempty[4];
  uint64_t sel_ready;
  int abort;
  int n_slots;
  uint32_t mask[MAX_SLOTS];                  // tokens of expert i
  uint16_t slot_expert[MAX_SLOTS];
  uint16_t slot_of[MAX_SLOTS];
  uint16_t slot_start[MAX_SLOTS + 1];
  uint16_t ent_row[MAX_ENTRIES];             // row of act and hrec
  uint8_t ent_tok[MAX_ENTRIES];
  float ent_gate[MAX_ENTRIES];
  double dots[CW][16];
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void box_load(void* dst, const CUtensorMap* m, uint64_t* bar, int row, int block) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(m), "r"(smem_u32(bar)), "r"(0), "r"(row), "r"(block)
      : "memory");
}

__device__ __forceinline__ void mma_e4m3(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void grid_arrive(unsigned* ctr) {
  __threadfence();
  asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(ctr) : "memory");
}

// Waits until all CTAs have arrived; bounded as mbar_wait is.
__device__ __forceinline__ bool grid_wait(const unsigned* ctr, unsigned n, volatile int* abort) {
  uint64_t t0 = 0;
  for (uint32_t i = 0;; ++i) {
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(ctr) : "memory");
    if (v >= n) return true;
    if ((i & 63) == 63) {
      if (*abort) return false;
      const uint64_t t = globaltimer_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > kWaitLimitNs) {
        set_device_error(MOE_ERR_TIMEOUT);
        *abort = 1;
        return false;
      }
    }
  }
}

__device__ __forceinline__ int range_begin(int i, int n, int parts) {
  return static_cast<int>(static_cast<long long>(i) * n / parts);
}

// Partial products of one 128-channel block of a stage: 16 weight rows by
// eight tokens. Lane q of a row's four holds channels 32 q .. 32 q + 31 on both
// sides (the order of channels inside the block is free): two 16-byte words,
// of which a swizzled weight row and an activation row with a pitch of 16
// modulo 128 bytes each serve eight lanes on distinct banks.
struct Frag {
  uint32_t w[8];
};
__device__ __forceinline__ Frag frag_of(const uint4 lo, const uint4 hi) {
  return Frag{{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w}};
}
__device__ __forceinline__ Frag weight_frag(const uint8_t* row, int q4) {    // row: 128 bytes of a swizzled box
  const int x = (smem_u32(row) >> 7) & 7;
  return frag_of(*reinterpret_cast<const uint4*>(row + (((2 * q4) ^ x) << 4)),
                 *reinterpret_cast<const uint4*>(row + (((2 * q4 + 1) ^ x) << 4)));
}
__device__ __forceinline__ Frag token_frag(const uint8_t* p) {
  return frag_of(*reinterpret_cast<const uint4*>(p), *reinterpret_cast<const uint4*>(p + 16));
}
__device__ __forceinline__ void block_product(float (&c)[4], const Frag& r0, const Frag& r8, const Frag& x) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t a[4] = {r0.w[2 * j], r8.w[2 * j], r0.w[2 * j + 1], r8.w[2 * j + 1]};
    mma_e4m3(c, a, x.w[2 * j], x.w[2 * j + 1]);
  }
}

// Row r of a tile of n rows: the rows of the box that holds it (the bits of n,
// largest first), and its offset in the stage.
__device__ __forceinline__ int box_rows(int r, int n) {
  int at = 0;
#pragma unroll
  for (int b = 4; b >= 0; --b) {
    if (!((n >> b) & 1)) continue;
    if (r < at + (1 << b)) return 1 << b;
    at += 1 << b;
  }
  return 1;
}
__device__ __forceinline__ int box_offset(int r, int n) {
  const int R = box_rows(r, n), at = n & ~(2 * R - 1);
  return at * KC + (r - at) * 128;
}

// ---------------------------------------------------------------- router

// Affinities of experts e0 and e1 (e1 < 0: none) with eight tokens from t0.
// The selection is a border, so the logits are summed in FP64 (their products
// are exact) and the affinity is rounded once: keys that differ in FP32 are
// never exchanged by the sum's order. Costs 16 conversions and DFMAs a clock
// and SM while the ring fills.
__device__ __forceinline__ void to_double8(const uint4 v, double (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ void affinities(const Args& a, Small* sm, int e0, int e1, int t0) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  double acc[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.0;
  const int V = a.d >> 3;
  for (int v = tid; v < V; v += CW * 32) {
    double w0[8], w1[8];
    to_double8(__ldg(reinterpret_cast<const uint4*>(a.e + static_cast<size_t>(e0) * a.d) + v), w0);
    to_double8(__ldg(reinterpret_cast<const uint4*>(a.e + static_cast<size_t>(e1 < 0 ? e0 : e1) * a.d) + v), w1);
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      if (t0 + t < a.T) {
        double x[8];
        to_double8(__ldg(reinterpret_cast<const uint4*>(a.u + static_cast<size_t>(t0 + t) * a.d) + v), x);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          acc[t] = fma(x[j], w0[j], acc[t]);
          acc[8 + t] = fma(x[j], w1[j], acc[8 + t]);
        }
      }
    }
  }
  // 16 sums over 32 lanes: each step halves the values a lane still holds
#pragma unroll
  for (int n = 8, o = 16; n >= 1; n >>= 1, o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const double give = up ? acc[i] : acc[i + n];
      const double keep = up ? acc[i + n] : acc[i];
      acc[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], 1);
  // lane bits 4..1 chose the halves: value index = bits 16, 8, 4, 2 of the lane
  if (!(lane & 1)) sm->dots[warp][lane >> 1] = acc[0];
  named_bar_sync(1, CW * 32);
  if (tid < 16) {
    double z = 0.0;
#pragma unroll
    for (int w = 0; w < CW; ++w) z += sm->dots[w][tid];
    const int t = t0 + (tid & 7), ex = tid < 8 ? e0 : e1;
    if (t < a.T && ex >= 0) a.scores[t * a.N_r + ex] = static_cast<float>(1.0 / (1.0 + exp(-z)));
  }
  named_bar_sync(1, CW * 32);
}

// 1x128 tiles of u by moe_quant_1x128's rule, half a warp a tile.
__device__ __forceinline__ void quantise_u(const Args& a) {
  const int half = (blockIdx.x * CW + (threadIdx.x >> 5)) * 2 + ((threadIdx.x >> 4) & 1);
  const int tiles = a.T * (a.d >> 7), sub = threadIdx.x & 15;
  for (int first = half & ~1; first < tiles; first += gridDim.x * CW * 2) {
    const int tile = first + (half & 1);
    const bool live = tile < tiles;
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (live) raw = __ldg(reinterpret_cast<const uint4*>(a.u + static_cast<size_t>(tile) * 128) + sub);
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    float v[8], amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      amax = fmaxf(amax, fmaxf(fabsf(v[2 * i]), fabsf(v[2 * i + 1])));
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float s = tile_scale(amax);
    uint32_t c[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      c[i] = e4m3x2(__fdiv_rn(v[4 * i], s), __fdiv_rn(v[4 * i + 1], s)) |
             (e4m3x2(__fdiv_rn(v[4 * i + 2], s), __fdiv_rn(v[4 * i + 3], s)) << 16);
    if (live) {
      reinterpret_cast<uint2*>(a.xq_ws + static_cast<size_t>(tile) * 128)[sub] = make_uint2(c[0], c[1]);
      if (sub == 0) a.xs_ws[tile] = s;
    }
  }
}

// An FP32 key as an unsigned integer of the same order; NaN below everything.
__device__ __forceinline__ uint32_t ordered(float k) {
  if (!(k == k)) return 1u;
  const uint32_t x = __float_as_uint(k + 0.0f);           // -0 becomes +0
  return (x & 0x80000000u) ? ~x : (x | 0x80000000u);
}

// One warp: the K largest keys of a token, equal ones by the lower index;
// lane k < K ends with the k-th expert and its affinity.
__device__ __forceinline__ void select_token(const Args& a, int t, int& ex, float& s) {
  const int lane = lane_id();
  uint32_t key[MAX_N / 32];
  float sc[MAX_N / 32];
#pragma unroll
  for (int j = 0; j < MAX_N / 32; ++j) {
    const int i = j * 32 + lane;
    sc[j] = i < a.N_r ? __ldcg(a.scores + t * a.N_r + i) : 0.0f;
    key[j] = i < a.N_r ? ordered(sc[j] + __ldg(a.b + i)) : 0u;      // 0: taken or absent
  }
  ex = 0;
  s = 0.0f;
  for (int k = 0; k < a.K; ++k) {
    uint32_t best = 0u;
    int at = MAX_N;
    float bs = 0.0f;
#pragma unroll
    for (int j = 0; j < MAX_N / 32; ++j)
      if (key[j] > best) { best = key[j]; at = j * 32 + lane; bs = sc[j]; }
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    const int win = static_cast<int>(__reduce_min_sync(0xffffffffu, best == top ? static_cast<uint32_t>(at) : MAX_N));
    const float ws = __shfl_sync(0xffffffffu, bs, win & 31);
    if (lane == k) { ex = win; s = ws; }
#pragma unroll
    for (int j = 0; j < MAX_N / 32; ++j)
      if (j * 32 + lane == win) key[j] = 0u;
  }
}

// Every CTA selects for itself: slot 0 is the shared expert with every token,
// then the touched experts in ascending order, their tokens ascending.
__device__ __forceinline__ void select_all(const Args& a, Small* sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int ex[2];
  float g[2];
  for (int r = 0; r < 2; ++r) {
    const int t = warp + r * CW;
    if (t >= a.T) continue;
    float s;
    select_token(a, t, ex[r], s);
    float sum = 0.0f;
    for (int k = 0; k < a.K; ++k) sum += __shfl_sync(0xffffffffu, s, k);
    g[r] = __fdiv_rn(s, sum);
    if (lane < a.K) {
      atomicOr(&sm->mask[ex[r]], 1u << t);
      if (blockIdx.x == 0) {
        a.topk_idx[t * a.K + lane] = ex[r];
        a.gates[t * a.K + lane] = g[r];
      }
    }
  }
  named_bar_sync(1, CW * 32);
  if (warp == 0) {
    int slots = 1, ents = a.T;
    if (lane == 0) { sm->slot_expert[0] = a.N_r; sm->slot_start[0] = 0; }
    for (int i0 = 0; i0 < a.N_r; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t m = i < a.N_r ? sm->mask[i] : 0u;
      const int n = __popc(m);
      const uint32_t on = __ballot_sync(0xffffffffu, n > 0);
      int pre = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, pre, o);
        if (lane >= o) pre += v;
      }
      if (n > 0) {
        const int s = slots + __popc(on & ((1u << lane) - 1u));
        sm->slot_expert[s] = i;
        sm->slot_of[i] = s;
        sm->slot_start[s] = ents + pre - n;
      }
      slots += __popc(on);
      ents += __shfl_sync(0xffffffffu, pre, 31);
      if (blockIdx.x == 0 && a.counts != nullptr && i < a.N_r) a.counts[i] = n;
    }
    if (lane == 0) { sm->slot_start[slots] = ents; sm->n_slots = slots; }
    if (lane < a.T) {
      sm->ent_tok[lane] = lane;
      sm->ent_row[lane] = a.T * a.K + lane;
      sm->ent_gate[lane] = 1.0f;
    }
  }
  named_bar_sync(1, CW * 32);
  for (int r = 0; r < 2; ++r) {
    const int t = warp + r * CW;
    if (t < a.T && lane < a.K) {
      const int p = sm->slot_start[sm->slot_of[ex[r]]] + __popc(sm->mask[ex[r]] & ((1u << t) - 1u));
      sm->ent_tok[p] = t;
      sm->ent_row[p] = t * a.K + lane;
      sm->ent_gate[p] = g[r];
    }
  }
  named_bar_sync(1, CW * 32);
}

// ---------------------------------------------------------------- work lists

// First phase: units of eight gate and the eight matching up rows over all of
// d. A CTA takes its share of the shared expert's units, then its share of the
// routed ones (known after the selection).
struct Units {
  int sh0, sh1, r0, r1;
  __device__ __forceinline__ int count() const { return (sh1 - sh0) + (r1 - r0); }
};
__device__ __forceinline__ void shared_units(const Args& a, Units& u) {
  const int per = a.I >> 3;
  u.sh0 = range_begin(blockIdx.x, per, gridDim.x);
  u.sh1 = range_begin(blockIdx.x + 1, per, gridDim.x);
}
__device__ __forceinline__ void routed_units(const Args& a, int slots, Units& u) {
  const int n = (slots - 1) * (a.I >> 3);
  u.r0 = range_begin(blockIdx.x, n, gridDim.x);
  u.r1 = range_begin(blockIdx.x + 1, n, gridDim.x);
}
__device__ __forceinline__ void unit_at(const Args& a, const Units& u, int i, int& slot, int& row) {
  const int per = a.I >> 3;
  if (i < u.sh1 - u.sh0) {
    slot = 0;
    row = (u.sh0 + i) * 8;
  } else {
    const int k = u.r0 + i - (u.sh1 - u.sh0);
    slot = 1 + k / per;
    row = (k % per) * 8;
  }
}

// ---------------------------------------------------------------- kernel

template <int NT>
__global__ void __launch_bounds__(THREADS, 1) few_tokens_kernel(const __grid_constant__ Maps maps, const Args a) {
  constexpr int EW = Shape<NT>::EW;
  constexpr int RED = Shape<NT>::RED;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ring = smem;
  uint8_t* xh = smem + static_cast<size_t>(a.stages) * STAGE;        // tokens' codes, then the H rows
  float* red = reinterpret_cast<float*>(xh + a.xh_bytes);            // [EW][CW][8 NT][RCOL]
  float* xs = red + EW * RED;                                        // [T][d/128]
  Small* sm = reinterpret_cast<Small*>(xs + ((a.T * (a.d >> 7) + 3) & ~3));

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int xpitch = pitch_of(a.d), hpitch = pitch_of(a.hrec_bytes);
  volatile int* abort = &sm->abort;

  for (int i = threadIdx.x; i < MAX_SLOTS; i += THREADS) sm->mask[i] = 0u;
  if (threadIdx.x == 0) {
    for (int i = 0; i < MAX_STAGES; ++i) { mbar_init(&sm->full[i], 1); mbar_init(&sm->empty[i], CW); }
    for (int i = 0; i < MAX_HBUF; ++i) { mbar_init(&sm->hfull[i], 1); mbar_init(&sm->hempty[i], CW); }
    for (int i = 0; i < 4; ++i) { mbar_init(&sm->redfull[i], CW); mbar_init(&sm->redempty[i], 1); }
    mbar_init(&sm->sel_ready, 1);
    sm->abort = 0;
    fence_mbar_init();
  }
  __syncthreads();

  const int row0 = range_begin(blockIdx.x, a.d, gridDim.x);           // rows of W_down
  const int nrows = range_begin(blockIdx.x + 1, a.d, gridDim.x) - row0;
  const int ntiles = (nrows + ROWS - 1) / ROWS;                       // the last one may be short
  Units un;
  shared_units(a, un);

  if (warp == CW) {
    // ------------------------------------------------------------ producer
    int it = 0;
    bool ok = true;
    auto claim = [&](uint32_t bytes) -> uint8_t* {       // the next stage, expecting so many bytes
      const int s = it % a.stages;
      if (ok && it >= a.stages) ok = warp_wait(&sm->empty[s], ((it / a.stages) - 1) & 1, abort);
      if (ok) {
        ++it;
        if (lane == 0) mbar_arrive_expect_tx(&sm->full[s], bytes);
        __syncwarp();
      }
      return ring + s * STAGE;
    };
    auto gate_up = [&](int i) {
      int slot, row;
      unit_at(a, un, i, slot, row);
      row += (slot == 0 ? a.N_r : sm->slot_expert[slot]) * a.I;
      for (int k = 0; k < a.d; k += KC) {
        uint8_t* dst = claim(STAGE);
        if (ok && lane < 2) box_load(dst + lane * (STAGE / 2), lane == 0 ? &maps.gate : &maps.up, &sm->full[(it - 1) % a.stages], row, k >> 7);
      }
    };
    for (int i = 0; i < un.sh1 - un.sh0; ++i) gate_up(i);
    ok = warp_wait(&sm->sel_ready, 0, abort) && ok;
    if (ok) {
      const int slots = sm->n_slots;
      routed_units(a, slots, un);
      for (int i = un.sh1 - un.sh0; i < un.count(); ++i) gate_up(i);
      for (int si = 0; si < slots; ++si) {
        const int row = sm->slot_expert[si] * a.d + row0;
        for (int t = 0; t < ntiles; ++t) {
          // a short tile is the boxes of its row count's bits, largest first
          const int n = min(ROWS, nrows - t * ROWS);
          const int bit = 4 - lane, above = lane > 0 && lane < 5 ? n & ~((2 << bit) - 1) : 0;
          for (int k = 0; k < a.I; k += KC) {
            uint8_t* dst = claim(n * KC);
            if (ok && lane < 5 && ((n >> bit) & 1))
              box_load(dst + above * KC, &maps.down[bit], &sm->full[(it - 1) % a.stages], row + t * ROWS + above, k >> 7);
          }
        }
      }
    }
    // no copy may be in flight when the CTA ends
    for (int j = max(0, it - a.stages); j < it; ++j) mbar_wait(&sm->full[j % a.stages], (j / a.stages) & 1, &sm->abort);
  } else if (warp > CW && warp <= CW + EW) {
    // ------------------------------------------------------------ finishing warps
    const int e = warp - CW - 1;
    bool ok = warp_wait(&sm->sel_ready, 0, abort);
    const int slots = ok ? sm->n_slots : 0;
    if (ok) {
      routed_units(a, slots, un);
      for (int i = e, n = 0; i < un.count(); i += EW, ++n) {
        if (!(ok = ok && warp_wait(&sm->redfull[e], n & 1, abort))) break;
        int slot, row;
        unit_at(a, un, i, slot, row);
        const int first = sm->slot_start[slot], ntok = sm->slot_start[slot + 1] - first;
        const float* p = red + e * RED;
        float v[(8 * 8 * NT + 31) / 32];
#pragma unroll
        for (int q = 0; q < 2 * NT; ++q) {
          const int o = q * 32 + lane;
          v[q] = 0.0f;
          if (o < 8 * ntok) {
            const float* c = p + (o >> 3) * RCOL + (o & 7);
            float gt = 0.0f, up = 0.0f;
#pragma unroll
            for (int w = 0; w < CW; ++w) {
              gt += c[w * 8 * NT * RCOL];
              up += c[w * 8 * NT * RCOL + 8];
            }
            v[q] = __fdiv_rn(gt, 1.0f + expf(-gt)) * up;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->redempty[e]);
#pragma unroll
        for (int q = 0; q < 2 * NT; ++q) {
          const int o = q * 32 + lane;
          if (o < 8 * ntok) a.act[static_cast<size_t>(sm->ent_row[first + (o >> 3)]) * a.I + row + (o & 7)] = v[q];
        }
        // the warp that finishes a 128-block last quantises it
        __threadfence();
        __syncwarp();
        int last = 0;
        const int blk = row >> 7;
        if (lane == 0) last = atomicAdd(a.blk_ctr + slot * (a.I >> 7) + blk, 1) == 15;
        if (__shfl_sync(0xffffffffu, last, 0)) {
          __threadfence();
          for (int j = 0; j < ntok; ++j) {
            const int r = sm->ent_row[first + j];
            const float4 x = __ldcg(reinterpret_cast<const float4*>(a.act + static_cast<size_t>(r) * a.I + blk * 128) + lane);
            float amax = fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w)));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            const float s = tile_scale(amax);
            uint8_t* rec = a.hrec + static_cast<size_t>(r) * a.hrec_bytes;
            reinterpret_cast<uint32_t*>(rec + blk * 128)[lane] =
                e4m3x2(__fdiv_rn(x.x, s), __fdiv_rn(x.y, s)) | (e4m3x2(__fdiv_rn(x.z, s), __fdiv_rn(x.w, s)) << 16);
            if (lane == 0) reinterpret_cast<float*>(rec + a.I)[blk] = s;
          }
        }
      }
    }
    asm volatile("fence.proxy.async;" ::: "memory");      // the records are read by bulk copies
    __threadfence();
    named_bar_sync(2, EW * 32);
    if (e == 0) {
      // -------------------------------------------------------- loader of H
      int seen = 0;
      if (lane == 0) {
        grid_arrive(a.grid_ctr + 32);
        seen = grid_wait(a.grid_ctr + 32, gridDim.x, abort);
      }
      ok = __shfl_sync(0xffffffffu, seen, 0) != 0 && ok;
      asm volatile("fence.proxy.async;" ::: "memory");
      int si = 0;
      for (; ok && si < slots; ++si) {
        const int bf = si % a.hbufs;
        if (si >= a.hbufs && !(ok = warp_wait(&sm->hempty[bf], ((si / a.hbufs) - 1) & 1, abort))) break;
        const int first = sm->slot_start[si], ntok = sm->slot_start[si + 1] - first;
        if (lane == 0) mbar_arrive_expect_tx(&sm->hfull[bf], ntok * a.hrec_bytes);
        __syncwarp();
        if (lane < ntok)
          bulk_load(xh + (static_cast<size_t>(bf) * a.T + lane) * hpitch,
                    a.hrec + static_cast<size_t>(sm->ent_row[first + lane]) * a.hrec_bytes, a.hrec_bytes, &sm->hfull[bf]);
      }
      for (int j = max(0, si - a.hbufs); j < si; ++j) mbar_wait(&sm->hfull[j % a.hbufs], (j / a.hbufs) & 1, &sm->abort);
    }
  } else if (warp < CW) {
    // ------------------------------------------------------------ multiplying warps
    const int tid = threadIdx.x;
    const int g = lane >> 2, q4 = lane & 3;
    if (a.xq_ws != nullptr) quantise_u(a);
    for (int e0 = blockIdx.x; e0 < a.N_r; e0 += 2 * gridDim.x) {
      const int e1 = e0 + static_cast<int>(gridDim.x) < a.N_r ? e0 + static_cast<int>(gridDim.x) : -1;
      for (int t0 = 0; t0 < a.T; t0 += 8) affinities(a, sm, e0, e1, t0);
    }
    __threadfence();
    named_bar_sync(1, CW * 32);
    if (tid == 0) {
      grid_arrive(a.grid_ctr);
      grid_wait(a.grid_ctr, gridDim.x, abort);
    }
    named_bar_sync(1, CW * 32);
    select_all(a, sm);
    // the tokens' codes and scales
    for (int t = 0; t < a.T; ++t)
      for (int v = tid; v < (a.d >> 4); v += CW * 32)
        *reinterpret_cast<uint4*>(xh + t * xpitch + v * 16) =
            __ldcg(reinterpret_cast<const uint4*>(a.xq + static_cast<size_t>(t) * a.d) + v);
    for (int i = tid; i < a.T * (a.d >> 7); i += CW * 32) xs[i] = __ldcg(a.xs + i);
    named_bar_sync(1, CW * 32);
    if (tid == 0) mbar_arrive(&sm->sel_ready);

    const int slots = sm->n_slots;
    routed_units(a, slots, un);
    const int kb_d = a.d >> 7, kb_i = a.I >> 7;
    int it = 0;
    bool ok = true;
    for (int i = 0; i < un.count(); ++i) {
      int slot, row;
      unit_at(a, un, i, slot, row);
      const int ex = sm->slot_expert[slot];
      const int first = sm->slot_start[slot], ntok = sm->slot_start[slot + 1] - first;
      const float* sg = a.s_gate + (static_cast<size_t>(ex) * kb_i + (row >> 7)) * kb_d;
      const float* su = a.s_up + (static_cast<size_t>(ex) * kb_i + (row >> 7)) * kb_d;
      float acc[NT][4];
      int tok[NT], c0[NT], c1[NT];           // the lane's B column, and its two result columns
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[n][j] = 0.0f;
        tok[n] = sm->ent_tok[first + min(n * 8 + g, ntok - 1)];
        c0[n] = sm->ent_tok[first + min(n * 8 + 2 * q4, ntok - 1)] * kb_d;
        c1[n] = sm->ent_tok[first + min(n * 8 + 2 * q4 + 1, ntok - 1)] * kb_d;
      }
      for (int k0 = 0; k0 < a.d; k0 += KC, ++it) {
        const int s = it % a.stages;
        const int kb = (k0 >> 7) + warp;
        const bool mine = kb < kb_d;
        const float fg = mine ? __ldg(sg + kb) : 0.0f, fu = mine ? __ldg(su + kb) : 0.0f;
        ok = ok && warp_wait(&sm->full[s], (it / a.stages) & 1, abort);
        if (ok && mine) {
          const uint8_t* p = ring + s * STAGE + warp * 1024 + g * 128;
          const Frag r0 = weight_frag(p, q4), r8 = weight_frag(p + STAGE / 2, q4);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (n * 8 < ntok) {
              const Frag x = token_frag(xh + tok[n] * xpitch + kb * 128 + q4 * 32);
              float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
              block_product(c, r0, r8, x);
              const float x0 = xs[c0[n] + kb], x1 = xs[c1[n] + kb];
              acc[n][0] = fmaf(c[0], x0 * fg, acc[n][0]);
              acc[n][1] = fmaf(c[1], x1 * fg, acc[n][1]);
              acc[n][2] = fmaf(c[2], x0 * fu, acc[n][2]);
              acc[n][3] = fmaf(c[3], x1 * fu, acc[n][3]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->empty[s]);
      }
      const int e = i % EW, use = i / EW;
      if (use > 0) ok = ok && warp_wait(&sm->redempty[e], (use - 1) & 1, abort);
      if (ok) {
        float* r = red + e * RED + warp * 8 * NT * RCOL;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float* c = r + (n * 8 + 2 * q4) * RCOL + g;
          c[0] = acc[n][0];
          c[RCOL] = acc[n][1];
          c[8] = acc[n][2];
          c[RCOL + 8] = acc[n][3];
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->redfull[e]);
    }

    // ---------------------------------------------------------- W_down
    float acc[MAX_TILES][NT][4];
#pragma unroll
    for (int t = 0; t < MAX_TILES; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[t][n][j] = 0.0f;
    for (int si = 0; si < slots; ++si) {
      const int bf = si % a.hbufs;
      ok = ok && warp_wait(&sm->hfull[bf], (si / a.hbufs) & 1, abort);
      const int ex = sm->slot_expert[si];
      const int first = sm->slot_start[si];
      const uint32_t mask = si == 0 ? (1u << a.T) - 1u : sm->mask[ex];
      const uint8_t* hb = xh + static_cast<size_t>(bf) * a.T * hpitch;
      const uint8_t* col[NT];                // the lane's B column: its token's row of H, or none
      const float *h0[NT], *h1[NT];          // scales of the two result columns
      float g0[NT], g1[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        auto at = [&](int c) { return (mask >> c) & 1u ? __popc(mask & ((1u << c) - 1u)) : -1; };
        const int jb = at(n * 8 + g), j0 = at(n * 8 + 2 * q4), j1 = at(n * 8 + 2 * q4 + 1);
        col[n] = jb < 0 ? nullptr : hb + jb * hpitch;
        h0[n] = j0 < 0 ? nullptr : reinterpret_cast<const float*>(hb + j0 * hpitch + a.I);
        h1[n] = j1 < 0 ? nullptr : reinterpret_cast<const float*>(hb + j1 * hpitch + a.I);
        g0[n] = j0 < 0 ? 0.0f : sm->ent_gate[first + j0];
        g1[n] = j1 < 0 ? 0.0f : sm->ent_gate[first + j1];
      }
#pragma unroll
      for (int t = 0; t < MAX_TILES; ++t) {
        if (t >= ntiles) continue;
        const int nr = min(ROWS, nrows - t * ROWS);
        const int ra = min(g, nr - 1), rb = min(g + 8, nr - 1);          // rows past a short tile repeat its last
        const int oa = box_offset(ra, nr) + warp * box_rows(ra, nr) * 128, ob = box_offset(rb, nr) + warp * box_rows(rb, nr) * 128;
        const int n0 = (row0 + t * ROWS + ra) >> 7, n8 = (row0 + t * ROWS + rb) >> 7;
        const float* s0 = a.s_down + (static_cast<size_t>(ex) * kb_d + n0) * kb_i;
        const float* s8 = a.s_down + (static_cast<size_t>(ex) * kb_d + n8) * kb_i;
        for (int k0 = 0; k0 < a.I; k0 += KC, ++it) {
          const int s = it % a.stages;
          const int kb = (k0 >> 7) + warp;
          const bool mine = kb < kb_i;
          const float f0 = mine ? __ldg(s0 + kb) : 0.0f, f8 = mine ? __ldg(s8 + kb) : 0.0f;
          ok = ok && warp_wait(&sm->full[s], (it / a.stages) & 1, abort);
          if (ok && mine) {
            const uint8_t* p = ring + s * STAGE;
            const Frag r0 = weight_frag(p + oa, q4), r8 = weight_frag(p + ob, q4);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if ((mask >> (n * 8)) & 0xFFu) {
                Frag x = {{0, 0, 0, 0, 0, 0, 0, 0}};
                if (col[n] != nullptr) x = token_frag(col[n] + kb * 128 + q4 * 32);
                __syncwarp();
                float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                block_product(c, r0, r8, x);
                if (h0[n] != nullptr) {      // a column without a token adds nothing, whatever the weights hold
                  const float x0 = h0[n][kb] * g0[n];
                  acc[t][n][0] = fmaf(c[0], x0 * f0, acc[t][n][0]);
                  acc[t][n][2] = fmaf(c[2], x0 * f8, acc[t][n][2]);
                }
                if (h1[n] != nullptr) {
                  const float x1 = h1[n][kb] * g1[n];
                  acc[t][n][1] = fmaf(c[1], x1 * f0, acc[t][n][1]);
                  acc[t][n][3] = fmaf(c[3], x1 * f8, acc[t][n][3]);
                }
              }
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm->empty[s]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->hempty[bf]);
    }
    // the warps' sums meet in the ring, which is empty now
    named_bar_sync(1, CW * 32);
    float* fin = reinterpret_cast<float*>(ring);             // [CW][8 NT][64]
#pragma unroll
    for (int t = 0; t < MAX_TILES; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float* c = fin + (warp * 8 * NT + n * 8 + 2 * q4) * 64 + t * 16 + g;
        c[0] = acc[t][n][0];
        c[64] = acc[t][n][1];
        c[8] = acc[t][n][2];
        c[72] = acc[t][n][3];
      }
    named_bar_sync(1, CW * 32);
    const uint16_t* base = a.base != nullptr ? a.base : a.u;
    for (int o = tid; o < a.T * 64; o += CW * 32) {
      const int t = o >> 6, r = o & 63;
      if (r >= nrows) continue;
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < CW; ++w) v += fin[(w * 8 * NT + t) * 64 + r];
      const size_t at = static_cast<size_t>(t) * a.d + row0 + r;
      a.out[at] = float_to_bf16_bits(bf16_bits_to_float(base[at]) + v);
    }
  }
  __syncthreads();
}

// ---------------------------------------------------------------- host

inline size_t round_up(size_t n, size_t m) { return (n + m - 1) / m * m; }

struct Layout {
  size_t ctr_bytes, scores, xq, xs, act, hrec, total;
  int hrec_bytes;
};
inline Layout layout(int T, int d, int N_r, int K_r, int I) {
  Layout l;
  const size_t P = static_cast<size_t>(T) * K_r + T;
  const size_t slots = (static_cast<size_t>(T) * K_r < static_cast<size_t>(N_r) ? T * K_r : N_r) + 1;
  l.ctr_bytes = 256 + slots * (I / 128) * 4;
  l.scores = round_up(l.ctr_bytes, 256);
  l.xq = round_up(l.scores + static_cast<size_t>(T) * N_r * 4, 256);
  l.xs = round_up(l.xq + static_cast<size_t>(T) * d, 256);
  l.act = round_up(l.xs + static_cast<size_t>(T) * (d / 128) * 4, 256);
  l.hrec = round_up(l.act + P * I * 4, 256);
  l.hrec_bytes = static_cast<int>(round_up(I + I / 128 * 4, 16));
  l.total = l.hrec + P * l.hrec_bytes;
  return l;
}

inline bool sizes_supported(int T, int d, int N_r, int K_r, int I) {
  return T <= MAX_T && K_r >= 1 && K_r <= MAX_K && K_r <= N_r && N_r <= MAX_N && d % 256 == 0 && d <= 8192 &&
         I % 128 == 0 && I <= 8192;
}

// [rows][cols] codes as (128, rows, cols / 128), boxes of R rows by KC / 128 blocks.
inline int make_map(CUtensorMap* m, const void* base, size_t rows, int cols, int R) {
  auto enc = tensor_map_encoder();
  if (!enc) return record_failure(MOE_ERR_CUDA, "cuTensorMapEncodeTiled", "entry point not found");
  cuuint64_t dims[3] = {128, rows, static_cast<cuuint64_t>(cols / 128)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols), 128};
  cuuint32_t box[3] = {128, static_cast<cuuint32_t>(R), KC / 128}, one[3] = {1, 1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, one,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MOE_OK : record_failure(MOE_ERR_CUDA, "cuTensorMapEncodeTiled", "few tokens: weight map");
}

template <int NT>
int launch(const Maps& maps, Args& a, const DeviceInfo& di, cudaStream_t s) {
  const int xpitch = pitch_of(a.d), hpitch = pitch_of(a.hrec_bytes);
  const int one = a.T * hpitch;
  int xh = a.T * xpitch > 2 * one ? a.T * xpitch : 2 * one;
  a.hbufs = xh / one;
  if (a.hbufs > MAX_HBUF) a.hbufs = MAX_HBUF;
  a.xh_bytes = static_cast<int>(round_up(xh, 16));
  const size_t rest = a.xh_bytes + Shape<NT>::EW * Shape<NT>::RED * 4 + round_up(a.T * (a.d / 128) * 4, 16) + sizeof(Small);
  if (rest + 3 * STAGE > SMEM_MAX)
    return record_failure(MOE_ERR_UNSUPPORTED, "moe_few_tokens", "T * d and T * I do not fit shared memory");
  a.stages = static_cast<int>((SMEM_MAX - rest) / STAGE);
  if (a.stages > MAX_STAGES) a.stages = MAX_STAGES;
  const size_t smem = rest + static_cast<size_t>(a.stages) * STAGE;
  auto k = few_tokens_kernel<NT>;
  if (int st = cuda_status(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)),
                           "few tokens: smem attribute"))
    return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(di.sm_count);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeCooperative;       // every CTA waits for every other twice
  at[0].val.cooperative = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, k, maps, static_cast<const Args>(a)), "few tokens: launch");
}

}  // namespace few
}  // namespace moe

extern "C" size_t moe_few_tokens_workspace(int T, int d, int N_r, int K_r, int I) {
  if (T <= 0 || d <= 0 || N_r <= 0 || K_r <= 0 || I <= 0 || !moe::few::sizes_supported(T, d, N_r, K_r, I)) return 0;
  return moe::few::layout(T, d, N_r, K_r, I).total;
}

extern "C" int moe_few_tokens(const uint16_t* u, const uint8_t* xq, const float* xs, const uint16_t* base,
                              const uint16_t* e, const float* b, int T, int d, int N_r, int K_r,
                              const uint8_t* w_gate, const uint8_t* w_up, const uint8_t* w_down, const float* s_gate,
                              const float* s_up, const float* s_down, int I, uint16_t* out, int32_t* topk_idx,
                              float* gates, int32_t* counts, void* workspace, size_t ws_bytes, void* stream) {
  using namespace moe;
  using namespace moe::few;
  MOE_CHECK_ARG(T >= 0 && d > 0 && N_r > 0 && I > 0);
  MOE_CHECK_SUPPORTED(sizes_supported(T, d, N_r, K_r, I));
  cudaStream_t s = as_stream(stream);
  if (T == 0)
    return counts ? cuda_status(cudaMemsetAsync(counts, 0, N_r * sizeof(int32_t), s), "few tokens: counts") : MOE_OK;
  MOE_CHECK_ARG(u && e && b && w_gate && w_up && w_down && s_gate && s_up && s_down && out && topk_idx && gates);
  MOE_CHECK_ARG((xq == nullptr) == (xs == nullptr));
  const Layout l = layout(T, d, N_r, K_r, I);
  MOE_CHECK_ARG(workspace && ws_bytes >= l.total);
  const uintptr_t all = reinterpret_cast<uintptr_t>(u) | reinterpret_cast<uintptr_t>(e) |
                        reinterpret_cast<uintptr_t>(xq) | reinterpret_cast<uintptr_t>(w_gate) |
                        reinterpret_cast<uintptr_t>(w_up) | reinterpret_cast<uintptr_t>(w_down) |
                        reinterpret_cast<uintptr_t>(workspace);
  MOE_CHECK_ARG(all % 16 == 0);
  DeviceInfo di;
  if (int st = device_info(&di)) return st;
  if (di.sm_count < 1 || (d + di.sm_count - 1) / di.sm_count > MAX_TILES * ROWS)
    return record_failure(MOE_ERR_UNSUPPORTED, "moe_few_tokens", "too few SMs for d");
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  Args a{};
  a.u = u; a.base = base; a.e = e; a.b = b;
  a.xq_ws = xq ? nullptr : ws + l.xq;
  a.xs_ws = xq ? nullptr : reinterpret_cast<float*>(ws + l.xs);
  a.xq = xq ? xq : a.xq_ws;
  a.xs = xq ? xs : a.xs_ws;
  a.s_gate = s_gate; a.s_up = s_up; a.s_down = s_down;
  a.out = out; a.topk_idx = topk_idx; a.gates = gates; a.counts = counts;
  a.grid_ctr = reinterpret_cast<unsigned*>(ws);
  a.blk_ctr = reinterpret_cast<int*>(ws + 256);
  a.scores = reinterpret_cast<float*>(ws + l.scores);
  a.act = reinterpret_cast<float*>(ws + l.act);
  a.hrec = ws + l.hrec;
  a.hrec_bytes = l.hrec_bytes;
  a.T = T; a.d = d; a.N_r = N_r; a.K = K_r; a.I = I;
  Maps maps;
  const size_t G = static_cast<size_t>(N_r) + 1;
  if (int st = make_map(&maps.gate, w_gate, G * I, d, 8)) return st;
  if (int st = make_map(&maps.up, w_up, G * I, d, 8)) return st;
  for (int i = 0; i < 5; ++i)
    if (int st = make_map(&maps.down[i], w_down, G * d, I, 1 << i)) return st;
  if (int st = cuda_status(cudaMemsetAsync(ws, 0, l.ctr_bytes, s), "few tokens: counters")) return st;
  return T <= 8 ? launch<1>(maps, a, di, s) : launch<2>(maps, a, di, s);
}
