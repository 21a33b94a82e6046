// The whole layer for at most 16 tokens in two kernels: the router's affinities
// (and u's quantisation), then selection, selected experts and the shared one,
// combine.
//
// Every byte of the touched experts' weights is read once and nothing else is
// large, so the second kernel is a stream of weights: one CTA per SM (a
// cooperative launch), producers that keep a ring of TMA boxes in flight across
// its phases, and the tensor cores behind it. The weights do not depend on what
// the phases exchange, only on the selection, so the ring fills with the shared
// expert during the selection and with W_down while the last intermediate rows
// are written. The first phase (gate, up, SwiGLU) is dealt in slot order and a
// slot's second phase starts when its own intermediate is quantised, so the
// phases need no barrier over the grid.
//
// Products: weight rows are the MMA's M side, tokens its N side. A stage of the
// ring holds two 128-channel blocks of 64 weight rows, and one MMA takes both:
// its 128 rows are the 64 rows of either block, its columns the R token rows
// (8 or 16) of either block's activations, and of the four quarters of the
// result the two that pair a block with itself are read. That keeps every
// weight row live and halves the number of MMAs, whose issue (70 to 100 cycles
// each at these shapes, measured) otherwise paces the kernel: 8 KB of weights
// arrive in about 340 cycles. For the same reason two warps issue MMAs and two
// issue loads, in turns. 64 rows is a choice of balance: one token has 9
// experts, 576 units of 32 gate and 32 up rows for 148 SMs (0.97 of them busy
// in the last round), and in the second phase a CTA has its own d / SMs rows of
// W_down, at most 64, over all slots.
//
// Measured from a graph of calls over three sets of inputs (d = 7168, I = 2048,
// 8 of 256 experts and the shared one; weights alone take 61 / 216 / 704 us at
// the copy rate of 6.45 TB/s): one token 75 us, of them 4 for the first kernel;
// 4 tokens 230 to 242 us; 16 tokens 713 to 820 us, by the machine and from run
// to run. A call by itself through the binding takes 79 us at one token. DRAM
// bounds them; at one token the starts of the two kernels and the selection
// (about 13 us) come on top. With small experts (d = 2048, I = 1024, 6 of 64)
// one token takes 26 us against 7: the exchange between the phases is six round
// trips through a loaded L2.
#include "host.cuh"

namespace moe {
namespace few {

constexpr int MAX_T = 16;
constexpr int MAX_K = 16;
constexpr int MAX_N = 256;
constexpr int MAX_SLOTS = MAX_N + 1;
constexpr int MAX_ENTRIES = MAX_T * MAX_K + MAX_T;
constexpr int MAX_D = 8192;
constexpr int CW = 8;                        // warps of the selection
constexpr int EW = 3;                        // of them, finishing warps of the first phase
constexpr int PW = 4;                        // of them, warps that add up partials, one per 32 TMEM lanes
constexpr int MI = 2;                        // producers, and MMA issuers: each kind takes turns, and the stages and
                                             // TMEM buffers are multiples of it
constexpr int THREADS = (CW + 2 * MI) * 32;
constexpr int CH = 32;                       // intermediate channels of a unit
constexpr int LIVE = 64;                     // live weight rows of a tile
constexpr int SK = 2;                        // 128-channel blocks of a stage
constexpr int TILE = LIVE * 128;             // bytes of one block of a stage
constexpr int STAGE = SK * TILE;
constexpr int MAX_STAGES = 12;
constexpr int MAX_HBUF = 4;
constexpr int COLS = 16;                     // a row of the scale tables
constexpr int QS = 2;                        // sums of a block's four K = 32 steps: even and odd ones apart
constexpr int BUFS = 8;                      // stages' partials in TMEM
constexpr int MAX_GROUPS = 8;
constexpr int MAX_MEMBERS = 256;             // and CTAs
constexpr int SMEM_MAX = 227 * 1024;

// Tensor maps, all with the 128-byte swizzle. Weights are rows [slot * rows] of codes; boxes are 128 channels by:
struct Maps {
  CUtensorMap gate, up;                      // CH rows, SK blocks: stored [block][row][128]
  CUtensorMap down[2];                       // a CTA's rows of W_down, by the parity of their count
  CUtensorMap x;                             // the tokens' codes: every row, one block
};

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
  unsigned* slot_done;      // [slot] quantised blocks of its H
  int* blk_ctr;             // [slot][I/128]: finished units of a block
  int* join_ctr;            // [member] groups whose sums are written
  float2* scores;           // [T][N_r] key s + b, affinity s
  float* part;              // [group][T][d] sums of a group's slots, with several groups
  float* act;               // [entry][I] silu(G) U; entries are the slots' tokens, slot after slot
  uint8_t* hq;              // its codes, a slot's as [I/128][tokens][128] with the operand tiles' swizzle
  float* hs;                // [entry][hs_pitch] its I/128 scales
  int T, d, N_r, K, I;
  int groups, members;      // second phase: groups of CTAs with a share of the slots each, rows split over a group's members
  int ctr_words;            // slot_done, blk_ctr and join_ctr, zeroed by the first kernel
  int hs_pitch;             // I/128 rounded up to 4
  int stages, hbufs, xh_bytes, hbuf_bytes;
  int reds;                 // buffers of units' sums
};

template <int N>
using Int = std::integral_constant<int, N>;

// R: token rows of an operand tile (T rounded up to 8).
template <int R>
struct Shape {
  static constexpr int N = SK * R;                          // MMA columns: token rows of the stage's two blocks
  static constexpr int BUF_COLS = QS * N;                   // TMEM columns of a stage's partials
  static constexpr int TMEM_COLS = BUFS * BUF_COLS;
  static constexpr int RED = PW * R * CH;                   // floats of one unit's sums, and of the outputs' sums
};

// Shared memory behind the dynamic regions.
struct Small {
  uint64_t full[MAX_STAGES], empty[MAX_STAGES];
  uint64_t hfull[MAX_HBUF], hempty[MAX_HBUF];
  uint64_t tfull[BUFS], tempty[BUFS];
  uint64_t redfull[EW], redempty[EW];
  uint64_t sel_ready, x_ready, x_free, drained;
  uint32_t tmem;
  int abort, last;
  int n_slots;
  uint32_t mask[MAX_N];                      // tokens of expert i
  uint16_t slot_expert[MAX_SLOTS];
  uint16_t slot_of[MAX_N];
  uint16_t slot_start[MAX_SLOTS + 1];
  uint8_t ent_tok[MAX_ENTRIES];
  float ent_gate[MAX_ENTRIES];
  int chunk_slots[CW], chunk_ents[CW];
};

// A position in a ring of barriers: index and the parity of its lap.
struct Cursor {
  int i = 0;
  uint32_t lap = 0;
  __device__ __forceinline__ void next(int n) {
    if (++i == n) {
      i = 0;
      lap ^= 1;
    }
  }
};

__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// One box of [rows][blocks of 128]: coordinates row and block.
__device__ __forceinline__ void box_load(void* dst, const CUtensorMap* m, uint64_t* bar, int row, int block) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(m), "r"(smem_u32(bar)), "r"(0), "r"(row), "r"(block)
      : "memory");
}

// Issues a read of NC consecutive FP32 columns of the thread's TMEM lane.
template <int NC>
__device__ __forceinline__ void tmem_ld_async(uint32_t taddr, uint32_t* r) {
  static_assert(NC == 2 || NC == 4 || NC == 8 || NC == 16, "columns");
  if constexpr (NC == 2) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(taddr));
  } else if constexpr (NC == 4) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr));
  } else {
#pragma unroll
    for (int i = 0; i < NC; i += 8) tmem_ld8_async(taddr + i, r + i);
  }
}

__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

// Counts up after everything the warp wrote before its last __syncwarp.
__device__ __forceinline__ void count_up(unsigned* ctr) {
  asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(ctr) : "memory");
}

// The same, acquiring what the others wrote before theirs; returns the count before.
__device__ __forceinline__ int count_up_seen(int* ctr) {
  int v;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(v) : "l"(ctr) : "memory");
  return v;
}

__device__ __forceinline__ unsigned count_now(const unsigned* ctr) {
  unsigned v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(ctr) : "memory");
  return v;
}

// Waits until a counter has reached n; bounded as mbar_wait is.
__device__ __forceinline__ bool count_wait(const unsigned* ctr, unsigned n, volatile int* abort) {
  uint64_t t0 = 0;
  for (uint32_t i = 0;; ++i) {
    if (count_now(ctr) >= n) return true;
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

__host__ __device__ inline int range_begin(int i, int n, int parts) {
  return static_cast<int>(static_cast<long long>(i) * n / parts);
}

// ---------------------------------------------------------------- router

// Affinities of EB experts with TB tokens, a block of 8 warps. The selection is
// a border, so the logits are summed in FP64 (their products are exact) and the
// affinity is rounded once: keys that differ in FP32 are never exchanged by the
// sum's order. The 2 x 4 sums of a thread leave it the registers to load all
// its runs at once (4 x 8 sums took 16 us at 13 tokens and d = 2048, these 8).
__device__ __forceinline__ void to_double8(const uint4 v, double (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ void quantise_u(const Args& a, int block, int blocks);

constexpr int EB = 2, TB = 4;
__global__ void __launch_bounds__(256) few_route_kernel(const Args a) {
  constexpr int M = EB * TB;                 // sums of a thread
  static_assert(M <= 32 && (M & (M - 1)) == 0, "the sums spread over a warp's lanes");
  __shared__ double dots[8][M];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int block = blockIdx.y * gridDim.x + blockIdx.x, blocks = gridDim.x * gridDim.y;
  const int e0 = blockIdx.x * EB, t0 = blockIdx.y * TB;
  const int V = a.d >> 3;                    // at most four runs of 8 channels a thread
  const uint4 zero = make_uint4(0, 0, 0, 0);
  double acc[M];
#pragma unroll
  for (int i = 0; i < M; ++i) acc[i] = 0.0;
  uint4 we[4][EB], x[4][TB];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int v = tid + i * 256;
#pragma unroll
    for (int k = 0; k < EB; ++k)
      we[i][k] = v < V && e0 + k < a.N_r ? __ldg(reinterpret_cast<const uint4*>(a.e + static_cast<size_t>(e0 + k) * a.d) + v) : zero;
#pragma unroll
    for (int t = 0; t < TB; ++t)
      x[i][t] = v < V && t0 + t < a.T ? __ldg(reinterpret_cast<const uint4*>(a.u + static_cast<size_t>(t0 + t) * a.d) + v) : zero;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    double w[EB][8], f[8];
#pragma unroll
    for (int k = 0; k < EB; ++k) to_double8(we[i][k], w[k]);
#pragma unroll
    for (int t = 0; t < TB; ++t)
      if (t0 + t < a.T) {
        to_double8(x[i][t], f);
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int k = 0; k < EB; ++k) acc[k * TB + t] = fma(f[j], w[k][j], acc[k * TB + t]);
      }
  }
  // M sums over 32 lanes: each step halves the values a lane still holds
  int o = 16;
#pragma unroll
  for (int n = M / 2; n >= 1; n >>= 1, o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const double give = up ? acc[i] : acc[i + n];
      const double keep = up ? acc[i + n] : acc[i];
      acc[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
#pragma unroll
  for (; o >= 1; o >>= 1) acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], o);
  constexpr int SPREAD = 32 / M;             // lanes that hold the same sum
  if (lane % SPREAD == 0) dots[warp][lane / SPREAD] = acc[0];
  __syncthreads();
  if (tid < M) {
    double z = 0.0;
#pragma unroll
    for (int w = 0; w < 8; ++w) z += dots[w][tid];
    const int t = t0 + tid % TB, ex = e0 + tid / TB;
    if (t < a.T && ex < a.N_r) {
      const float s = static_cast<float>(1.0 / (1.0 + exp(-z)));
      a.scores[t * a.N_r + ex] = make_float2(s + __ldg(a.b + ex), s);
    }
  }
  for (int i = block * 256 + tid; i < a.ctr_words; i += blocks * 256) a.slot_done[i] = 0u;
  if (a.xq_ws != nullptr) quantise_u(a, block, blocks);
}

// 1x128 tiles of u by moe_quant_1x128's rule, half a warp a tile.
__device__ __forceinline__ void quantise_u(const Args& a, int block, int blocks) {
  const int half = (block * 8 + (threadIdx.x >> 5)) * 2 + ((threadIdx.x >> 4) & 1);
  const int tiles = a.T * (a.d >> 7), sub = threadIdx.x & 15;
  for (int first = half & ~1; first < tiles; first += blocks * 16) {
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

// ---------------------------------------------------------------- selection

// An FP32 key as an unsigned integer of the same order; NaN below everything.
__device__ __forceinline__ uint32_t ordered(float k) {
  if (!(k == k)) return 1u;
  const uint32_t x = __float_as_uint(k + 0.0f);           // -0 becomes +0
  return (x & 0x80000000u) ? ~x : (x | 0x80000000u);
}

// One warp: the K largest keys of a token, equal ones by the lower index;
// lane k < K ends with the k-th expert and its affinity. score: MAX_N floats of
// the warp's own.
__device__ __forceinline__ void select_token(const Args& a, int t, float* score, int& ex, float& s) {
  const int lane = lane_id();
  __syncwarp();                              // the scratch's last token has been read
  uint32_t key[MAX_N / 32];
#pragma unroll
  for (int j = 0; j < MAX_N / 32; ++j) {
    const int i = j * 32 + lane;
    const float2 v = i < a.N_r ? __ldcg(a.scores + t * a.N_r + i) : make_float2(0.0f, 0.0f);
    score[i] = v.y;
    key[j] = i < a.N_r ? ordered(v.x) : 0u;                          // 0: taken or absent
  }
  ex = 0;
  for (int k = 0; k < a.K; ++k) {
    uint32_t best[4];
    int at[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {            // the lane's best, by a tree; the left side wins ties
      at[j] = key[2 * j + 1] > key[2 * j] ? 2 * j + 1 : 2 * j;
      best[j] = max(key[2 * j], key[2 * j + 1]);
    }
    if (best[1] > best[0]) { best[0] = best[1]; at[0] = at[1]; }
    if (best[3] > best[2]) { best[2] = best[3]; at[2] = at[3]; }
    if (best[2] > best[0]) { best[0] = best[2]; at[0] = at[2]; }
    const uint32_t top = __reduce_max_sync(0xffffffffu, best[0]);
    const int win = static_cast<int>(
        __reduce_min_sync(0xffffffffu, best[0] == top ? static_cast<uint32_t>(at[0] * 32 + lane) : MAX_N));
    if (lane == k) ex = win;
#pragma unroll
    for (int j = 0; j < MAX_N / 32; ++j)
      if (j * 32 + lane == win) key[j] = 0u;
  }
  __syncwarp();
  s = lane < a.K ? score[ex] : 0.0f;
}

// Every CTA selects for itself (scores: CW * MAX_N floats of scratch): slot 0 is the shared expert with every token,
// then the touched experts in ascending order, their tokens ascending.
// A warp selects for R / CW tokens: code runs once and cold here, so there is
// no more of it than the tokens need.
template <int R>
__device__ __forceinline__ void select_all(const Args& a, Small* sm, float* scores) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int PER = R / CW;
  int ex[PER];
  float g[PER];
#pragma unroll
  for (int r = 0; r < PER; ++r) {
    const int t = warp + r * CW;
    ex[r] = 0;
    g[r] = 0.0f;
    if (t >= a.T) continue;
    select_token(a, t, scores + warp * MAX_N, ex[r], g[r]);
    if (lane < a.K) atomicOr(&sm->mask[ex[r]], 1u << t);
    float sum = g[r];                        // MAX_K lanes' affinities, those behind K zero
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    g[r] = __fdiv_rn(g[r], sum);
  }
  named_bar_sync(1, CW * 32);
  const int i = warp * 32 + lane;            // a warp lists 32 experts; the chunks' totals join them
  const int n = i < a.N_r ? __popc(sm->mask[i]) : 0;
  const uint32_t on = __ballot_sync(0xffffffffu, n > 0);
  int pre = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, pre, o);
    if (lane >= o) pre += v;
  }
  if (lane == 31) { sm->chunk_slots[warp] = __popc(on); sm->chunk_ents[warp] = pre; }
  named_bar_sync(1, CW * 32);
  int slots = 1, ents = a.T;
  for (int w = 0; w < warp; ++w) { slots += sm->chunk_slots[w]; ents += sm->chunk_ents[w]; }
  if (n > 0) {
    const int s = slots + __popc(on & ((1u << lane) - 1u));
    sm->slot_expert[s] = i;
    sm->slot_of[i] = s;
    sm->slot_start[s] = ents + pre - n;
  }
  if (warp == CW - 1 && lane == 31) {
    sm->slot_start[slots + __popc(on)] = ents + pre;
    sm->n_slots = slots + __popc(on);
    sm->slot_expert[0] = a.N_r;
    sm->slot_start[0] = 0;
  }
  named_bar_sync(1, CW * 32);
  if (tid == 0) mbar_arrive(&sm->sel_ready); // the producer needs the slots alone
  if (warp == 0 && lane < a.T) {
    sm->ent_tok[lane] = lane;
    sm->ent_gate[lane] = 1.0f;
  }
#pragma unroll
  for (int r = 0; r < PER; ++r) {
    const int t = warp + r * CW;
    if (t < a.T && lane < a.K) {
      const int p = sm->slot_start[sm->slot_of[ex[r]]] + __popc(sm->mask[ex[r]] & ((1u << t) - 1u));
      sm->ent_tok[p] = t;
      sm->ent_gate[p] = g[r];
      if (blockIdx.x == 0) {
        a.topk_idx[t * a.K + lane] = ex[r];
        a.gates[t * a.K + lane] = g[r];
      }
    }
  }
  if (blockIdx.x == 0 && a.counts != nullptr && i < a.N_r) a.counts[i] = n;
}

// ---------------------------------------------------------------- work lists

// First phase: units of CH gate and the matching up rows over all of d, in slot
// order, dealt to the CTAs in turn. The shared expert's come first (they are
// known before the selection), and the slots are finished one after the other,
// so that the second phase can start with the first slots while the last ones
// are still on their way.
__device__ __forceinline__ void unit_at(const Args& a, int unit, int& slot, int& ch) {
  const int per = a.I / CH;
  slot = unit / per;
  ch = (unit - slot * per) * CH;
}

// ---------------------------------------------------------------- kernel

template <int R>
__global__ void __launch_bounds__(THREADS, 1) few_tokens_kernel(const __grid_constant__ Maps maps, const Args a) {
  constexpr int N = Shape<R>::N, BUF_COLS = Shape<R>::BUF_COLS, RED = Shape<R>::RED;
  constexpr int tile_bytes = R * 128;                                // one block of the token operand
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ring = smem;
  uint8_t* xh = smem + static_cast<size_t>(a.stages) * STAGE;        // tokens' codes, then the H tiles
  float* xs = reinterpret_cast<float*>(xh + a.xh_bytes);             // [d/128][16]
  float* red = xs + (a.d >> 7) * COLS;                               // [reds][PW][R][CH]
  float* osum = reinterpret_cast<float*>(xh + a.hbufs * a.hbuf_bytes);   // [PW][R][32], in the second phase
  Small* sm = reinterpret_cast<Small*>(red + a.reds * RED);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kb_d = a.d >> 7, kb_i = a.I >> 7;
  volatile int* abort = &sm->abort;

  for (int i = threadIdx.x; i < MAX_N; i += THREADS) sm->mask[i] = 0u;
  if (threadIdx.x == 0) {
    for (int i = 0; i < MAX_STAGES; ++i) { mbar_init(&sm->full[i], 1); mbar_init(&sm->empty[i], 1); }
    for (int i = 0; i < MAX_HBUF; ++i) { mbar_init(&sm->hfull[i], 1); mbar_init(&sm->hempty[i], MI + PW); }
    for (int i = 0; i < BUFS; ++i) { mbar_init(&sm->tfull[i], 1); mbar_init(&sm->tempty[i], PW); }
    for (int i = 0; i < EW; ++i) { mbar_init(&sm->redfull[i], PW); mbar_init(&sm->redempty[i], 1); }
    mbar_init(&sm->sel_ready, 1);
    mbar_init(&sm->x_ready, MI);
    mbar_init(&sm->x_free, MI);
    mbar_init(&sm->drained, MI);
    sm->abort = 0;
    fence_mbar_init();
  }
  if (warp == CW + MI) {
    tmem_alloc(&sm->tmem, Shape<R>::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm->tmem;

  // second phase: the CTA's rows of W_down, for the slots group, group + groups, ..
  const int group = blockIdx.x / a.members, member = blockIdx.x - group * a.members;
  const int row0 = group < a.groups ? range_begin(member, a.d, a.members) : 0;
  const int nrows = group < a.groups ? range_begin(member + 1, a.d, a.members) - row0 : 0;
  const int per = a.I / CH;

  if (warp >= CW && warp < CW + MI) {
    // ------------------------------------------------------------ producers
    if (lane == 0) {
      Cursor c;
      int turn = warp - CW;                    // stages until this producer's next one
      c.lap = 1;                               // the first lap finds every stage empty
      int issued = 0;
      bool ok = true;
      auto mine = [&] {                        // whether the next stage is; passes it if not
        if (turn-- > 0) {
          ++issued;
          c.next(a.stages);
          return false;
        }
        turn = MI - 1;
        return true;
      };
      auto gate_up = [&](int unit) {
        int slot, ch;
        unit_at(a, unit, slot, ch);
        const int row = (slot == 0 ? a.N_r : sm->slot_expert[slot]) * a.I + ch;
        for (int k = 0; k < kb_d; k += SK) {
          if (!mine()) continue;
          if (!(ok = mbar_wait(&sm->empty[c.i], c.lap, abort))) return;
          uint64_t* bar = &sm->full[c.i];
          uint8_t* dst = ring + c.i * STAGE;
          mbar_arrive_expect_tx(bar, STAGE);   // d is a multiple of SK blocks
          box_load(dst, &maps.gate, bar, row, k);
          box_load(dst + STAGE / 2, &maps.up, bar, row, k);
          ++issued;
          c.next(a.stages);
        }
      };
      int unit = blockIdx.x;
      for (; ok && unit < per; unit += gridDim.x) gate_up(unit);
      ok = ok && mbar_wait(&sm->sel_ready, 0, abort);
      if (ok) {
        const int slots = sm->n_slots;
        for (; ok && unit < slots * per; unit += gridDim.x) gate_up(unit);
        const CUtensorMap* down = &maps.down[nrows & 1];
        for (int si = group; ok && nrows > 0 && si < slots; si += a.groups) {
          const int row = sm->slot_expert[si] * a.d + row0;
          for (int k = 0; k < kb_i; k += SK) {
            if (!mine()) continue;
            if (!(ok = mbar_wait(&sm->empty[c.i], c.lap, abort))) break;
            uint64_t* bar = &sm->full[c.i];
            const int nk = min(SK, kb_i - k);
            mbar_arrive_expect_tx(bar, nk * nrows * 128);
            for (int j = 0; j < nk; ++j) tma_load_2d(ring + c.i * STAGE + j * TILE, down, bar, (k + j) * 128, row);
            ++issued;
            c.next(a.stages);
          }
        }
      }
      // no copy may be in flight when the CTA ends
      for (int j = max(0, issued - a.stages); j < issued; ++j)
        if (j % MI == warp - CW) mbar_drain(&sm->full[j % a.stages], (j / a.stages) & 1);
    }
  } else if (warp >= CW + MI) {
    // ------------------------------------------------------------ MMA issuers (the whole warp keeps step)
    // the tokens' codes as operand tiles [d/128][R][128] (rows behind T stay unset), their scales as [d/128][16]
    if (warp == CW + MI) {
      if (lane == 0) mbar_expect_tx(&sm->x_ready, a.T * a.d);
      __syncwarp();
      for (int k = lane; k < kb_d; k += 32) tma_load_2d(xh + k * tile_bytes, &maps.x, &sm->x_ready, k * 128, 0);
    }
#pragma unroll 4
    for (int i = (warp - CW - MI) * 32 + lane; i < kb_d * COLS; i += MI * 32) {
      const int t = i & (COLS - 1);
      xs[i] = t < a.T ? __ldg(a.xs + t * kb_d + (i >> 4)) : 0.0f;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm->x_ready);
    bool ok = warp_wait(&sm->x_ready, 0, abort) && warp_wait(&sm->sel_ready, 0, abort);
    Cursor c, t;
    t.lap = 1;
    int turn = warp - CW - MI;                  // stages until this warp's next one
    // one stage against the two blocks of the token operand at tok. MMAs into one sum wait for each other:
    // QS sums are interleaved.
    constexpr uint32_t idesc = make_idesc(0, 0, 128, N);
    auto stage = [&](const uint8_t* tok) {
      if (turn-- > 0) {
        c.next(a.stages);
        t.next(BUFS);
        return;
      }
      turn = MI - 1;
      ok = ok && warp_wait(&sm->tempty[t.i], t.lap, abort) && warp_wait(&sm->full[c.i], c.lap, abort);
      if (!ok) return;
      tc_fence_after();
      const uint64_t ad = sw128_kmajor_desc(smem_u32(ring + c.i * STAGE));
      const uint64_t bd = sw128_kmajor_desc(smem_u32(tok));
      const uint32_t dt = tmem + t.i * BUF_COLS;
      if (lane == 0) {
#pragma unroll
        for (int q = 0; q < 4; ++q) umma_f8f6f4(dt + (q % QS) * N, ad + 2 * q, bd + 2 * q, idesc, q >= QS);
        umma_commit(&sm->empty[c.i]);
        umma_commit(&sm->tfull[t.i]);
      }
      __syncwarp();
      c.next(a.stages);
      t.next(BUFS);
    };
    if (ok) {
      const int slots = sm->n_slots;
      for (int unit = blockIdx.x; ok && unit < slots * per; unit += gridDim.x)
        for (int k = 0; ok && k < kb_d; k += SK) stage(xh + k * tile_bytes);
      if (lane == 0) umma_commit(&sm->x_free);
      Cursor h;
      for (int si = group; ok && nrows > 0 && si < slots; si += a.groups) {
        ok = warp_wait(&sm->hfull[h.i], h.lap, abort);
        const uint8_t* hb = xh + h.i * a.hbuf_bytes;
        for (int k = 0; ok && k < kb_i; k += SK) stage(hb + k * tile_bytes);
        if (lane == 0) umma_commit(&sm->hempty[h.i]);
        h.next(a.hbufs);
      }
    }
    if (lane == 0) {
      umma_commit(&sm->drained);                // no MMA may run when the TMEM is freed, and the tokens' codes have landed
      mbar_drain(&sm->drained, 0);
      mbar_drain(&sm->x_ready, 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ selection
    const int tid = threadIdx.x;
    select_all<R>(a, sm, red);
    named_bar_sync(1, CW * 32);
    const int slots = sm->n_slots, units = slots * per;

    if (warp < PW) {
      // ---------------------------------------------------------- sums of the partials: a thread owns a TMEM lane
      // first phase: lanes are 32 gate rows of block 0, of block 1, 32 up rows of block 0, of block 1;
      // second phase: 64 rows of W_down in block 0, then in block 1
      bool ok = warp_wait(&sm->x_ready, 0, abort);              // the scales
      Cursor t, e;
      e.lap = 1;
      int fin = 0;                              // the finishing warp of the unit at hand
      // waits for the stage's partials; NC columns of this warp's quarter from column c0
      const uint32_t taddr = tmem + (static_cast<uint32_t>(warp * 32) << 16);
      auto partials = [&](auto nc, int c0, float* v) {
        constexpr int NC = decltype(nc)::value;
        ok = ok && warp_wait(&sm->tfull[t.i], t.lap, abort);
        if (ok) {
          uint32_t r[QS * NC];
          tc_fence_after();
#pragma unroll
          for (int q = 0; q < QS; ++q) tmem_ld_async<NC>(taddr + t.i * BUF_COLS + q * N + c0, r + q * NC);
          tmem_wait_ld(r);
          tc_fence_before();
#pragma unroll
          for (int c = 0; c < NC; ++c) v[c] = __uint_as_float(r[c]) + __uint_as_float(r[NC + c]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->tempty[t.i]);
        t.next(BUFS);
      };
      {
        const int half = warp & 1;
        const float* s_all = warp < 2 ? a.s_gate : a.s_up;
        // lane i: the weight scale of block 2 i + half of the unit at hand, loaded one unit ahead
        auto scale_of = [&](int unit) {
          int slot, ch;
          unit_at(a, unit, slot, ch);
          const int kb = 2 * lane + half;
          return kb < kb_d ? __ldg(s_all + (static_cast<size_t>(sm->slot_expert[slot]) * kb_i + (ch >> 7)) * kb_d + kb) : 0.0f;
        };
        float next = static_cast<int>(blockIdx.x) < units ? scale_of(blockIdx.x) : 0.0f;
        for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
          const float mine = next;
          if (unit + static_cast<int>(gridDim.x) < units) next = scale_of(unit + gridDim.x);
          float acc[R];
#pragma unroll
          for (int c = 0; c < R; ++c) acc[c] = 0.0f;
          for (int k = 0; k < kb_d; k += SK) {
            float v[R];
            partials(Int<R>{}, half * R, v);
            const float w = __shfl_sync(0xffffffffu, mine, k >> 1);
            const float* x = xs + (k + half) * COLS;
            if (ok) {
#pragma unroll
              for (int c = 0; c < R; c += 4) {
                const float4 f = *reinterpret_cast<const float4*>(x + c);
                acc[c] = fmaf(v[c], f.x * w, acc[c]);
                acc[c + 1] = fmaf(v[c + 1], f.y * w, acc[c + 1]);
                acc[c + 2] = fmaf(v[c + 2], f.z * w, acc[c + 2]);
                acc[c + 3] = fmaf(v[c + 3], f.w * w, acc[c + 3]);
              }
            }
          }
          ok = ok && warp_wait(&sm->redempty[e.i], e.lap, abort);
          if (ok) {
            float* p = red + e.i * RED + warp * R * CH + lane;
#pragma unroll
            for (int c = 0; c < R; ++c) p[c * CH] = acc[c];
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm->redfull[fin]);
          fin = fin + 1 == EW ? 0 : fin + 1;
          e.next(a.reds);
        }
      }

      // W_down: the CTA's rows over every slot, whose tokens are the first columns
      const int kq = warp >> 1;                 // this warp's block of a stage
      const int r = (warp & 1) * 32 + lane;
      const int nb0 = row0 >> 7;                // rows of one or two 128-row blocks
      const bool upper = ((row0 + min(r, max(nrows - 1, 0))) >> 7) != nb0;
      float* sums = osum + warp * R * 32 + lane;
#pragma unroll
      for (int c = 0; c < R; ++c) sums[c * 32] = 0.0f;
      auto scales_of = [&](int si, float& lo, float& hi) {     // lane i: of the warp's block of stage i
        const float* sw = a.s_down + (static_cast<size_t>(sm->slot_expert[si]) * kb_d + nb0) * kb_i;
        const int kb = SK * lane + kq;
        lo = hi = 0.0f;
        if (kb < kb_i) {
          lo = __ldg(sw + kb);
          if (nb0 + 1 < kb_d) hi = __ldg(sw + kb_i + kb);
        }
      };
      Cursor h;
      float next_lo, next_hi;
      scales_of(min(group, slots - 1), next_lo, next_hi);
      for (int si = group; nrows > 0 && si < slots; si += a.groups) {
        const float lo = next_lo, hi = next_hi;
        if (si + a.groups < slots) scales_of(si + a.groups, next_lo, next_hi);
        ok = ok && warp_wait(&sm->hfull[h.i], h.lap, abort);
        const float* hs = reinterpret_cast<const float*>(xh + h.i * a.hbuf_bytes + kb_i * tile_bytes);   // [token][hs_pitch]
        const int first = sm->slot_start[si], ntok = sm->slot_start[si + 1] - first;
        auto rows = [&](auto nc) {
          constexpr int NC = decltype(nc)::value;
          float acc[NC];
#pragma unroll
          for (int c = 0; c < NC; ++c) acc[c] = 0.0f;
          for (int k = 0, n = 0; k < kb_i; k += SK, ++n) {
            float v[NC];
            partials(nc, kq * R, v);
            const float wl = __shfl_sync(0xffffffffu, lo, n), wh = __shfl_sync(0xffffffffu, hi, n);
            const float w = upper ? wh : wl;
            if (ok && k + kq < kb_i) {
#pragma unroll
              for (int c = 0; c < NC; ++c) acc[c] = fmaf(v[c], hs[c * a.hs_pitch + k + kq] * w, acc[c]);
            }
          }
#pragma unroll
          for (int c = 0; c < NC; ++c)
            if (c < ntok) {
              float* p = sums + sm->ent_tok[first + c] * 32;
              *p = fmaf(acc[c], sm->ent_gate[first + c], *p);
            }
        };
        if (ntok <= 2) rows(Int<2>{});
        else if (ntok <= 4) rows(Int<4>{});
        else if (R == 8 || ntok <= 8) rows(Int<8>{});
        else rows(Int<R>{});
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->hempty[h.i]);
        h.next(a.hbufs);
      }
      // both blocks' sums: the outputs with one group, else this group's share of them, and whoever writes a
      // member's last share adds them up in the groups' order
      named_bar_sync(3, PW * 32);
      const uint16_t* base = a.base != nullptr ? a.base : a.u;
      constexpr int W = R * 32;                 // from warp to warp
      if (r < nrows)
        for (int c = kq; c < a.T; c += SK) {
          const size_t at = static_cast<size_t>(c) * a.d + row0 + r;
          const float* p = osum + (warp & 1) * W + c * 32 + lane;
          const float v = p[0] + p[2 * W];
          if (a.groups == 1) a.out[at] = float_to_bf16_bits(bf16_bits_to_float(base[at]) + v);
          else a.part[static_cast<size_t>(group) * a.T * a.d + at] = v;
        }
      if (a.groups > 1 && nrows > 0) {
        named_bar_sync(3, PW * 32);
        if (tid == 0) sm->last = count_up_seen(a.join_ctr + member) == a.groups - 1;
        named_bar_sync(3, PW * 32);
        if (sm->last && r < nrows) {
          for (int c = kq; c < a.T; c += SK) {
            const size_t at = static_cast<size_t>(c) * a.d + row0 + r;
            float v = bf16_bits_to_float(base[at]);
            for (int i = 0; i < a.groups; ++i) v += __ldcg(a.part + static_cast<size_t>(i) * a.T * a.d + at);
            a.out[at] = float_to_bf16_bits(v);
          }
        }
      }
    } else if (warp < PW + EW) {
      // ---------------------------------------------------------- finishing warps: SwiGLU, then the blocks' codes
      const int e = warp - PW;
      uint32_t lap = 0;
      int n = e;                                // the CTA's n-th unit
      for (int unit = blockIdx.x + e * gridDim.x; unit < units; unit += EW * gridDim.x, lap ^= 1, n += EW) {
        if (!warp_wait(&sm->redfull[e], lap, abort)) break;
        const int buf = n % a.reds;
        int slot, ch;
        unit_at(a, unit, slot, ch);
        const int first = sm->slot_start[slot], ntok = sm->slot_start[slot + 1] - first;
        const float* p = red + buf * RED + lane;
        for (int j = 0; j < ntok; ++j) {
          const int t = sm->ent_tok[first + j];
          const float g = p[t * CH] + p[(R + t) * CH], u = p[(2 * R + t) * CH] + p[(3 * R + t) * CH];
          a.act[static_cast<size_t>(first + j) * a.I + ch + lane] = __fdiv_rn(g, 1.0f + expf(-g)) * u;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm->redempty[buf]);
        // the warp that finishes a 128-block last quantises it
        int last = 0;
        const int blk = ch >> 7;
        if (lane == 0) last = count_up_seen(a.blk_ctr + slot * kb_i + blk) == 128 / CH - 1;
        __syncwarp();
        if (__shfl_sync(0xffffffffu, last, 0)) {
          for (int j0 = 0; j0 < ntok; j0 += 4) {         // four rows' loads in flight
            float4 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              x[i] = __ldcg(reinterpret_cast<const float4*>(
                                a.act + static_cast<size_t>(first + min(j0 + i, ntok - 1)) * a.I + blk * 128) + lane);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int j = j0 + i;
              float amax = fmaxf(fmaxf(fabsf(x[i].x), fabsf(x[i].y)), fmaxf(fabsf(x[i].z), fabsf(x[i].w)));
#pragma unroll
              for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
              const float s = tile_scale(amax);
              if (j < ntok) {
                reinterpret_cast<uint32_t*>(a.hq + static_cast<size_t>(first) * a.I + (blk * ntok + j) * 128)[lane ^ ((j & 7) << 2)] =
                    e4m3x2(__fdiv_rn(x[i].x, s), __fdiv_rn(x[i].y, s)) |
                    (e4m3x2(__fdiv_rn(x[i].z, s), __fdiv_rn(x[i].w, s)) << 16);
                if (lane == 0) a.hs[(first + j) * a.hs_pitch + blk] = s;
              }
            }
          }
          fence_proxy_async_all();              // the codes are read by bulk copies
          __syncwarp();
          if (lane == 0) count_up(a.slot_done + slot);
        }
      }
    } else if (warp == PW + EW) {
      // ---------------------------------------------------------- loader of the H tiles, over the tokens' operand
      bool ok = warp_wait(&sm->x_free, 0, abort);
      Cursor h;
      h.lap = 1;
      int n = 0, done = 0;                      // slots taken; those before `done` (in turn) are known to be quantised
      for (int si = group; ok && nrows > 0 && si < slots; si += a.groups, ++n) {
        if (!(ok = warp_wait(&sm->hempty[h.i], h.lap, abort))) break;
        if (n >= done) {                        // look at the next 32 slots at once; wait for the first of them
          int seen = 1;
          if (lane == 0) seen = count_wait(a.slot_done + si, kb_i, abort);
          if (!(ok = __shfl_sync(0xffffffffu, seen, 0) != 0)) break;
          const int at = si + lane * a.groups;
          const bool there = lane == 0 || (at < slots && count_now(a.slot_done + at) >= static_cast<unsigned>(kb_i));
          const uint32_t missing = ~__ballot_sync(0xffffffffu, there);
          done = n + (missing ? __ffs(missing) - 1 : 32);
          __syncwarp();
          fence_proxy_async_all();
        }
        const int first = sm->slot_start[si], ntok = sm->slot_start[si + 1] - first;
        uint8_t* hb = xh + h.i * a.hbuf_bytes;
        if (lane == 0) mbar_arrive_expect_tx(&sm->hfull[h.i], ntok * (a.I + a.hs_pitch * 4));
        __syncwarp();
        for (int k = lane; k < kb_i; k += 32)
          bulk_load(hb + k * tile_bytes, a.hq + static_cast<size_t>(first) * a.I + k * ntok * 128, ntok * 128, &sm->hfull[h.i]);
        if (lane == 31)
          bulk_load(hb + kb_i * tile_bytes, a.hs + first * a.hs_pitch, ntok * a.hs_pitch * 4, &sm->hfull[h.i]);
        h.next(a.hbufs);
      }
      for (int j = max(0, n - a.hbufs); j < n; ++j) mbar_drain(&sm->hfull[j % a.hbufs], (j / a.hbufs) & 1);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == CW + MI) {
    tc_fence_after();
    tmem_dealloc(tmem, Shape<R>::TMEM_COLS);
  }
}

// ---------------------------------------------------------------- host

inline size_t round_up(size_t n, size_t m) { return (n + m - 1) / m * m; }

struct Layout {
  size_t slots, ctr_bytes, scores, xq, xs, part, act, hq, hs, total;
};
inline Layout layout(int T, int d, int N_r, int K_r, int I) {
  Layout l;
  const size_t P = static_cast<size_t>(T) * K_r + T;
  const size_t slots = (T * K_r < N_r ? T * K_r : N_r) + 1;
  l.slots = slots;
  l.ctr_bytes = (slots + slots * (I / 128) + MAX_MEMBERS) * 4;
  l.scores = round_up(l.ctr_bytes, 256);
  l.xq = round_up(l.scores + static_cast<size_t>(T) * N_r * 8, 256);
  l.xs = round_up(l.xq + static_cast<size_t>(T) * d, 256);
  l.part = round_up(l.xs + static_cast<size_t>(T) * (d / 128) * 4, 256);
  l.act = round_up(l.part + static_cast<size_t>(MAX_GROUPS) * T * d * 4, 256);
  l.hq = round_up(l.act + P * I * 4, 256);
  l.hs = round_up(l.hq + P * I, 256);
  l.total = round_up(l.hs + P * round_up(I / 128, 4) * 4, 256);
  return l;
}

// [rows][cols] codes as (128, rows, cols / 128), boxes of CH rows by SK blocks.
inline int make_map(CUtensorMap* m, const void* base, size_t rows, int cols) {
  const cuuint64_t dims[3] = {128, rows, static_cast<cuuint64_t>(cols / 128)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols), 128};
  const cuuint32_t box[3] = {128, CH, SK};
  return encode_tmap(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, base, dims, strides, box);
}

template <int R>
int launch(const Maps& maps, Args& a, int G, cudaStream_t s) {
  // shared memory: the token operand and the H tiles take turns in one
  // region; the ring gets what is left
  const int x_bytes = (a.d / 128) * R * 128;
  const int osum = Shape<R>::RED * 4;            // the outputs' sums, behind the H tiles
  a.hbuf_bytes = static_cast<int>(round_up((a.I / 128) * R * 128 + R * a.hs_pitch * 4, 1024));
  const int want = 4 * a.hbuf_bytes <= 72 * 1024 ? 4 : 2 * a.hbuf_bytes <= 96 * 1024 ? 2 : 1;
  const int h_bytes = want * a.hbuf_bytes + osum;
  a.xh_bytes = x_bytes > h_bytes ? x_bytes : h_bytes;
  a.hbufs = (a.xh_bytes - osum) / a.hbuf_bytes;
  if (a.hbufs > MAX_HBUF) a.hbufs = MAX_HBUF;
  // short units (small d) need several buffers of sums; with long ones one will do, and the others' room
  // goes to the ring
  a.reds = R == 16 && a.d > 4096 ? 1 : EW;
  static_assert((R == 16 ? 1 : EW) * Shape<R>::RED >= CW * MAX_N, "the selection's scratch lies in the units' sums");
  const size_t rest = a.xh_bytes + (a.d / 128) * COLS * 4 + a.reds * Shape<R>::RED * 4 + sizeof(Small);
  a.stages = static_cast<int>((SMEM_MAX - rest) / STAGE);
  if (a.stages > MAX_STAGES) a.stages = MAX_STAGES;
  a.stages -= a.stages % MI;                     // an issuer owns its stages: it never waits for another's lap
  static_assert(MAX_STAGES % MI == 0 && BUFS % MI == 0, "stages and buffers are dealt to the issuers");
  const size_t smem = rest + static_cast<size_t>(a.stages) * STAGE;
  auto k = few_tokens_kernel<R>;
  // the limit belongs to the function, not to the launch: one value for every shape, so that a call of another host
  // thread cannot lower it before this launch
  if (int st = cuda_status(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MAX),
                           "few tokens: smem attribute"))
    return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(G);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeCooperative;       // the CTAs wait for one another
  at[0].val.cooperative = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, k, maps, static_cast<const Args>(a)), "few tokens: launch");
}

inline bool sizes_supported(int T, int d, int N_r, int K_r, int I) {
  return T <= MAX_T && K_r >= 1 && K_r <= MAX_K && K_r <= N_r && N_r <= MAX_N && d % 256 == 0 && d <= MAX_D &&
         I % 128 == 0 && I <= MAX_D;
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
  const int G = di.sm_count < MAX_MEMBERS ? di.sm_count : MAX_MEMBERS;
  if ((d + LIVE - 1) / LIVE > G) return record_failure(MOE_ERR_UNSUPPORTED, "moe_few_tokens", "too few SMs for d");

  uint8_t* ws = static_cast<uint8_t*>(workspace);
  Args a{};
  a.u = u; a.base = base; a.e = e; a.b = b;
  a.xq_ws = xq ? nullptr : ws + l.xq;
  a.xs_ws = xq ? nullptr : reinterpret_cast<float*>(ws + l.xs);
  a.xq = xq ? xq : a.xq_ws;
  a.xs = xq ? xs : a.xs_ws;
  a.s_gate = s_gate; a.s_up = s_up; a.s_down = s_down;
  a.out = out; a.topk_idx = topk_idx; a.gates = gates; a.counts = counts;
  a.slot_done = reinterpret_cast<unsigned*>(ws);
  a.blk_ctr = reinterpret_cast<int*>(ws + l.slots * 4);
  a.ctr_words = static_cast<int>(l.ctr_bytes / 4);
  a.hs_pitch = static_cast<int>(round_up(I / 128, 4));
  a.join_ctr = a.blk_ctr + l.slots * (I / 128);
  a.part = reinterpret_cast<float*>(ws + l.part);
  // With small d a CTA's rows of W_down would be few, and what a slot costs besides its bytes (about 0.7 us)
  // would count: as many groups of CTAs as still leave 64 rows a member then share the slots. At d = 2048,
  // I = 1024, 13 tokens, the second phase takes 48 us with one group.
  a.groups = G / ((d + LIVE - 1) / LIVE);
  if (a.groups > MAX_GROUPS) a.groups = MAX_GROUPS;
  a.members = G / a.groups;
  a.scores = reinterpret_cast<float2*>(ws + l.scores);
  a.act = reinterpret_cast<float*>(ws + l.act);
  a.hq = ws + l.hq;
  a.hs = reinterpret_cast<float*>(ws + l.hs);
  a.T = T; a.d = d; a.N_r = N_r; a.K = K_r; a.I = I;

  Maps maps;
  const auto U8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const uint64_t slots = static_cast<uint64_t>(N_r) + 1;
  if (int st = make_map(&maps.gate, w_gate, slots * I, d)) return st;
  if (int st = make_map(&maps.up, w_up, slots * I, d)) return st;
  if (int st = make_tmap_2d(&maps.x, a.xq, U8, 1, T, d, T, 128)) return st;
  for (int i = 0; i < 2; ++i) {          // members own d / members rows or one more: one count is even, one odd
    const int q = d / a.members, n = q + (q % 2 == i ? 0 : 1);
    if (int st = make_tmap_2d(&maps.down[i], w_down, U8, 1, slots * d, I, n > 0 ? n : 1, 128)) return st;
  }
  few_route_kernel<<<dim3((N_r + EB - 1) / EB, (T + TB - 1) / TB), 256, 0, s>>>(a);
  if (int st = launch_status("few tokens: router launch")) return st;
  return T <= 8 ? launch<8>(maps, a, G, s) : launch<16>(maps, a, G, s);
}
