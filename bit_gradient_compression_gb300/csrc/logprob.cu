// Log probabilities of given tokens with entropies and the most likely alternatives, and the gradient
// of the logits (loco_logprob_forward, loco_logprob_backward).
//
// Forward, one pass over a row: each thread keeps its running maximum M, S = sum 2^t and D = sum 2^t t
// with t = (z - M) scale log2(e), rescaled once a tile when the maximum grows; (M, S, D) of threads,
// warps and CTAs are joined pairwise.  lse = M scale + ln S, entropy = ln S - ln 2 D / S (in deviations
// from M, so that neither loses digits to the size of the logits).
//
// Alternatives: every warp keeps its 32 largest so far, one to a lane, in order of keys (value, then lower column;
// all are different, so the outcome does not depend on the order in which they come).  A value above the warp's
// threshold `thr` is inserted by a ballot and a shift; thr is the warp's own top-th largest, and where a row has
// several warps the least of their each-th largest, each = ceil(top / warps), if that is more.  The first tile's
// thresholds are the same of the lanes' maxima, as there are at least as many values that are not below them.  Columns
// of one warp come in ascending order, so a later value that equals its own threshold loses the tie and `>` is enough;
// against a threshold of other warps a value that equals it is kept.
//
// A row is read by one, two, four or eight warps, more where rows are fewer, or by a cluster of up to eight
// CTAs of eight warps whose results the first joins through distributed shared memory: one launch, no workspace.
// Rows start at any multiple of the element size: the elements before the first 16-byte boundary and
// after the last whole vector are taken one by one.
//
// 4096 x 131072 bf16: 157 us, 6.8 TB/s, without alternatives, a copy's rate; 192 us with eight of them, where the SMs issue
// in 78 % of the cycles, 11.6 instructions an element; candidates are most in a row's first tiles.  8192 x 32000 with
// five: 111 us, 70 % of a copy's rate.  1 x 32000 with twenty: 8.8 us, a launch, a cluster of eight CTAs and their join.
//
// Backward, one read and one write a value: 8192 x 32000 bf16 153 us, 6.9 TB/s, a copy's rate, where rows of logits and of
// the gradient start alike within 16 bytes.  Others go element by element: 333 x 32003 fp32 21 us out of a cold L2, of 12.6.
#include <cooperative_groups.h>

#include "device_common.cuh"
#include "layers_common.cuh"
#include "steps_internal.h"

namespace loco {

namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 8, kThreadsLp = 32 * kWarps;
constexpr int kVectors = 4;                 // 16-byte vectors of a thread in one tile
constexpr float kLowest = -3.402823466e38f; // maximum of nothing; a row's lowest finite value may equal it
constexpr float kLeast = -200.0f;           // 2^t is 0 from here down; keeps t finite under -inf
constexpr float kLn2 = 0.6931471805599453f;
typedef unsigned long long Key;             // value in order, then the complement of the column; 0: none

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Bits that order like the values, both zeros alike.
__device__ __forceinline__ uint32_t in_order(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float out_of_order(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}
__device__ __forceinline__ Key key_of(float v, int64_t column) {
  return Key(in_order(v)) << 32 | (0xFFFFFFFFu - uint32_t(column));
}
__device__ __forceinline__ float key_value(Key k) { return out_of_order(uint32_t(k >> 32)); }
__device__ __forceinline__ int64_t key_column(Key k) { return int64_t(0xFFFFFFFFu - uint32_t(k)); }

// M, S and D of a part of a row.
struct Part {
  float m, s, d;
};
// Both parts under the larger maximum; c = scale log2(e).
__device__ __forceinline__ Part join(Part a, Part b, float c) {
  const float m = max_nan(a.m, b.m);
  const float ta = max_nan((a.m - m) * c, kLeast), tb = max_nan((b.m - m) * c, kLeast);
  const float fa = exp2_f(ta), fb = exp2_f(tb);
  return Part{m, fmaf(fa, a.s, fb * b.s), fmaf(fa, fmaf(a.s, ta, a.d), fb * fmaf(b.s, tb, b.d))};
}

template <bool BF16>
constexpr int kVec = BF16 ? 8 : 4;

// A row of which [head, head + vectors * kVec) is in whole 16-byte vectors.
template <bool BF16>
struct RowShape {
  int64_t head, vectors;
};
template <bool BF16>
__device__ __forceinline__ RowShape<BF16> row_shape(const void* row, int64_t cols) {
  constexpr int kElem = BF16 ? 2 : 4;
  const int64_t lead = int64_t((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / kElem;
  const int64_t head = lead < cols ? lead : cols;
  return RowShape<BF16>{head, (cols - head) / kVec<BF16>};
}

template <bool BF16>
__device__ __forceinline__ float largest(uint4 w) {
  if (BF16) {
    const uint32_t m = max_nan_bf16x2(max_nan_bf16x2(w.x, w.y), max_nan_bf16x2(w.z, w.w));
    return max_nan(bf16lo_to_f32(m), bf16hi_to_f32(m));
  }
  return max_nan(max_nan(__uint_as_float(w.x), __uint_as_float(w.y)), max_nan(__uint_as_float(w.z), __uint_as_float(w.w)));
}
template <bool BF16>
__device__ __forceinline__ void to_pairs(uint4 w, Pair (&v)[kVec<BF16> / 2]) {
  if constexpr (BF16) {
    v[0] = widen(w.x), v[1] = widen(w.y), v[2] = widen(w.z), v[3] = widen(w.w);
  } else {
    v[0] = pair(__uint_as_float(w.x), __uint_as_float(w.y)), v[1] = pair(__uint_as_float(w.z), __uint_as_float(w.w));
  }
}

// The value before the one whose in_order is k: what is above it is not below the value (two steps down from zero,
// whose neighbour is -0).
__device__ __forceinline__ float value_before(uint32_t k) {
  return k <= 0x007FFFFFu ? -INFINITY : out_of_order(k - (k == 0x80000000u ? 2u : 1u));
}

// A warp's largest values.
struct Largest {
  Key key;     // of this lane's: the lane-th largest of the warp, 0 where there are not that many
  float thr;   // what is not above it is not needed
  int top;

  // Inserts the values of a vector that are above the threshold (all lanes of the warp; v: N values, lane 0's from
  // column on, the next lane's behind them).  The threshold of the vector's begin holds for all of it: a lane's last
  // columns are before the next lane's first ones, and win a tie with them.
  template <int N>
  __device__ __forceinline__ void insert(const float (&v)[N], int64_t column, int lane) {
    const float limit = thr;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      uint32_t who = __ballot_sync(0xFFFFFFFFu, v[k] > limit);
      while (who != 0) {
        const int from = __ffs(who) - 1;
        who &= who - 1;
        const Key x = key_of(__shfl_sync(0xFFFFFFFFu, v[k], from), column + from * N + k);
        const int at = __popc(__ballot_sync(0xFFFFFFFFu, key > x));
        const Key before = __shfl_up_sync(0xFFFFFFFFu, key, 1);
        key = lane < at ? key : lane == at ? x : before;
      }
    }
    const uint32_t last = __shfl_sync(0xFFFFFFFFu, uint32_t(key >> 32), top - 1);
    const float t = last != 0 ? out_of_order(last) : -INFINITY;
    if (t > thr) thr = t;
  }
  // What the lanes' maxima of the first tile say: at least `top` of the warp's values are not below the top-th of them.
  // Returns the lane-th largest of them.
  __device__ __forceinline__ uint32_t first(float lane_max, int lane) {
    uint32_t u = in_order(lane_max);
#pragma unroll
    for (int size = 2; size <= 32; size *= 2) {  // descending over the lanes
#pragma unroll
      for (int d = size / 2; d > 0; d /= 2) {
        const uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, u, d);
        u = ((lane & d) == 0) == ((lane & size) == 0) ? max(u, o) : min(u, o);
      }
    }
    const float t = value_before(__shfl_sync(0xFFFFFFFFu, u, top - 1));
    if (t > thr) thr = t;
    return u;
  }
  // The each-th largest of every warp of a row: `top` values of the row are not below the least of them.  (One read
  // early or late is only a lower one: what is left out is never needed.)
  __device__ __forceinline__ void tell(uint32_t* floors, int each, int warp, int lane) const {
    if (lane == each - 1) floors[warp] = max(floors[warp], uint32_t(key >> 32));
  }
  __device__ __forceinline__ void hear(const uint32_t* floors, int warps, int lane) {
    const uint32_t f = *reinterpret_cast<const volatile uint32_t*>(floors + lane % warps);
    const float t = value_before(__reduce_min_sync(0xFFFFFFFFu, f));
    if (t > thr) thr = t;
  }
};

constexpr int kMaxParts = 8;  // CTAs of a cluster
template <bool TOP, int W>
struct Shared {
  Part part[W];
  Part ctas[kMaxParts];
};
template <int W>
struct Shared<true, W> {
  Part part[W];
  Part ctas[kMaxParts];
  Key lists[kMaxParts * LOCO_MAX_TOP];  // the CTAs' largest
  Key chosen[W * LOCO_MAX_TOP];  // of all warps' largest, what can be among the row's
  Key best[LOCO_MAX_TOP];
  int n_chosen;
  uint32_t floors[W], least[W];
};

// N parts, each held by every N-th lane, put together.
template <int N>
__device__ __forceinline__ Part join_lanes(Part x, int lane, float c) {
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) {
    const Part other{__shfl_xor_sync(0xFFFFFFFFu, x.m, o), __shfl_xor_sync(0xFFFFFFFFu, x.s, o),
                     __shfl_xor_sync(0xFFFFFFFFu, x.d, o)};
    x = lane & o ? join(other, x, c) : join(x, other, c);
  }
  return x;
}

// The `top` largest of chosen[0, n), in order, by all threads of the CTA; `best` was 0.
template <int THREADS>
__device__ __forceinline__ void choose(const Key* chosen, int n, int top, Key* best) {
  for (int i = threadIdx.x; i < n; i += THREADS) {
    const Key k = chosen[i];
    int above = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) above += chosen[j] > k;
    if (above < top) best[above] = k;
  }
}

// WPR: warps of a row's part (1: a CTA takes eight rows; 2, 4, 8: one).  CLUSTER: several CTAs to a row.
template <int WPR>
constexpr int kFwdWarps = WPR == 1 ? kWarps : WPR;  // of a CTA
template <bool BF16, int WPR, bool TOP, bool CLUSTER>
__global__ void __launch_bounds__(32 * kFwdWarps<WPR>, 32 / kFwdWarps<WPR>) k_logprob_fwd(const LogprobFwdArgs a) {
  constexpr int W = kFwdWarps<WPR>;
  __shared__ Shared<TOP, W> sh;
  extern __shared__ __align__(128) uint8_t ring[];
  constexpr int kElem = BF16 ? 2 : 4, V = kVec<BF16>, kTeam = 32 * WPR;
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, t = threadIdx.x % kTeam;
  int parts = 1, me = 0;
  if constexpr (CLUSTER) {
    parts = int(cg::this_cluster().num_blocks());
    me = int(cg::this_cluster().block_rank());
    cg::this_cluster().barrier_arrive();  // waited for before the first CTA's memory is written
  }
  const int64_t row = WPR == 1 ? int64_t(blockIdx.x) * W + warp : int64_t(blockIdx.x) / parts;
  if (WPR == 1 && row >= a.rows) return;  // whole warps, and no barrier follows
  const char* z = static_cast<const char*>(a.logits) + row * a.ld * kElem;
  const RowShape<BF16> shape = row_shape<BF16>(z, a.vocab);
  const int64_t v_lo = shape.vectors * me / parts, v_hi = shape.vectors * (me + 1) / parts;
  const uint4* vec = reinterpret_cast<const uint4*>(z + shape.head * kElem);
  const float c = a.scale * kLog2E;
  const Pair c2 = pair(c, c);

  Part mine{kLowest, 0.0f, 0.0f};
  Largest list{0, -INFINITY, a.top};
  if constexpr (TOP && WPR > 1) {
    if (lane == 0) sh.floors[warp] = 0;
    if (threadIdx.x < LOCO_MAX_TOP) sh.best[threadIdx.x] = 0;
    if (threadIdx.x == 0) sh.n_chosen = 0;
    __syncthreads();
  }
  // single elements at the row's ends
  const auto take_one = [&](int64_t from, int n) {
    float v[1] = {t < n ? load_elem(z, from + t, BF16) : -INFINITY};
    const float m = max_nan(mine.m, v[0]);
    const float e = max_nan((v[0] - m) * c, kLeast), s = exp2_f(e);
    mine = join(mine, Part{m, s, s * e}, c);
    if constexpr (TOP) {
      if (__any_sync(0xFFFFFFFFu, v[0] > list.thr)) list.insert(v, from, lane);
    }
  };
  if (me == 0 && shape.head > 0 && t < 32) take_one(0, int(shape.head));

  // Tiles of four vectors a thread; the next one is on its way to shared memory (cp.async by the thread that will read
  // it, so no barrier is needed).
  const uint4 none = BF16 ? make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u)
                          : make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u);
  constexpr uint32_t kPiece = 32 * W * 16, kStage = kVectors * kPiece;
  const uint32_t base = smem_addr(ring) + threadIdx.x * 16;
  uint32_t slot = 0;
  const auto fetch = [&](int64_t from) {
#pragma unroll
    for (int q = 0; q < kVectors; ++q) {
      if (from + q * kTeam < v_hi)
        copy_to_shared16(base + slot + q * kPiece, vec + from + q * kTeam);
      else
        to_shared16(base + slot + q * kPiece, none);
    }
    cp_async_commit();
    slot ^= kStage;
  };
  fetch(v_lo + t);
  bool first = true;
  for (int64_t i = v_lo; i < v_hi; i += kVectors * kTeam) {
    const uint32_t at = base + (slot ^ kStage);
    fetch(i + kVectors * kTeam + t);
    cp_async_wait<1>();
    uint4 w[kVectors];
#pragma unroll
    for (int q = 0; q < kVectors; ++q) w[q] = shared16(at + q * kPiece);
    float tile = largest<BF16>(w[0]);
#pragma unroll
    for (int q = 1; q < kVectors; ++q) tile = max_nan(tile, largest<BF16>(w[q]));
    const float m = max_nan(mine.m, tile);
    const float down = max_nan((mine.m - m) * c, kLeast), f = exp2_f(down);
    Pair s2 = pair(0.0f, 0.0f), d2 = s2;  // of this tile: a long row's sums stay a sum of tiles
    const Pair less = pair(-m, -m);
#pragma unroll
    for (int q = 0; q < kVectors; ++q) {
      Pair v[V / 2];
      to_pairs<BF16>(w[q], v);
#pragma unroll
      for (int k = 0; k < V / 2; ++k) {
        float2 x = halves((v[k] + less) * c2);
        x.x = max_nan(x.x, kLeast), x.y = max_nan(x.y, kLeast);
        const Pair e2 = pair(exp2_f(x.x), exp2_f(x.y));
        s2 = s2 + e2;
        d2 = fma(e2, pair(x.x, x.y), d2);
      }
    }
    const float2 s = halves(s2), d = halves(d2);
    mine = Part{m, fmaf(f, mine.s, s.x + s.y), fmaf(f, fmaf(mine.s, down, mine.d), d.x + d.y)};
    if constexpr (TOP) {
      const int each = (a.top + WPR - 1) / WPR;
      if (first) {
        const uint32_t u = list.first(tile, lane);
        if (WPR > 1) {
          if (lane == each - 1) sh.floors[warp] = u;
          __syncthreads();  // (a row's warps take the same number of tiles)
        }
      }
      if (__any_sync(0xFFFFFFFFu, tile > list.thr)) {
        if (WPR > 1) list.hear(sh.floors, WPR, lane);
#pragma unroll
        for (int q = 0; q < kVectors; ++q) {
          const uint4 again = shared16(at + q * kPiece);  // (not kept in registers for this)
          if (!__any_sync(0xFFFFFFFFu, largest<BF16>(again) > list.thr)) continue;
          Pair v[V / 2];
          to_pairs<BF16>(again, v);
          float x[V];
#pragma unroll
          for (int k = 0; k < V / 2; ++k) {
            const float2 h = halves(v[k]);
            x[2 * k] = h.x, x[2 * k + 1] = h.y;
          }
          list.insert(x, shape.head + (i + q * kTeam + (t - lane)) * V, lane);
        }
        if (WPR > 1) list.tell(sh.floors, each, warp, lane);
      }
      first = false;
    }
  }
  const int64_t tail = shape.head + shape.vectors * V;
  if (me == parts - 1 && tail < a.vocab && t < 32) take_one(tail, int(a.vocab - tail));

  // the warp's part
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Part other{__shfl_xor_sync(0xFFFFFFFFu, mine.m, o), __shfl_xor_sync(0xFFFFFFFFu, mine.s, o),
                     __shfl_xor_sync(0xFFFFFFFFu, mine.d, o)};
    // the same order of operands in both lanes: the same result
    mine = lane & o ? join(other, mine, c) : join(mine, other, c);
  }
  Part all = mine;
  if constexpr (WPR > 1) {
    if (lane == 0) sh.part[warp] = mine;
    if constexpr (TOP) {
      if (lane == 0) sh.least[warp] = in_order(list.thr);
    }
    __syncthreads();
    all = join_lanes<WPR>(sh.part[lane % WPR], lane, c);
    if constexpr (TOP) {
      // no value below the highest of the warps' thresholds can be among the largest
      const uint32_t least = __reduce_max_sync(0xFFFFFFFFu, sh.least[lane % WPR]);
      if (lane < a.top && uint32_t(list.key >> 32) >= least) sh.chosen[atomicAdd(&sh.n_chosen, 1)] = list.key;
      __syncthreads();
      choose<32 * W>(sh.chosen, sh.n_chosen, a.top, sh.best);
    }
    if constexpr (CLUSTER) {
      // everything goes to the first CTA
      const auto cluster = cg::this_cluster();
      cluster.barrier_wait();
      Shared<TOP, W>* to = cluster.map_shared_rank(&sh, 0);
      if (threadIdx.x == 0) to->ctas[me] = all;
      if constexpr (TOP) {
        __syncthreads();
        if (threadIdx.x < a.top) to->lists[me * a.top + threadIdx.x] = sh.best[threadIdx.x];
      }
      cluster.sync();
      if (me != 0) return;
      all = join_lanes<kMaxParts>(lane % kMaxParts < parts ? sh.ctas[lane % kMaxParts] : Part{kLowest, 0.0f, 0.0f}, lane, c);
      if constexpr (TOP) {
        if (threadIdx.x < LOCO_MAX_TOP) sh.best[threadIdx.x] = 0;
        __syncthreads();
        choose<32 * W>(sh.lists, parts * a.top, a.top, sh.best);
      }
    }
    if constexpr (TOP) __syncthreads();
  }

  const bool nan = all.s != all.s, empty = all.s == 0.0f;
  const float ls = empty ? 0.0f : logf(all.s);
  if (t == 0) {
    if (a.lse != nullptr) a.lse[row] = empty ? -INFINITY : fmaf(all.m, a.scale, ls);
    if (a.entropy != nullptr) a.entropy[row] = empty ? 0.0f : ls - kLn2 * (all.d / all.s);
    if (a.logp != nullptr) {
      const int64_t y = a.targets[row];
      float v = 0.0f;
      if (y >= a.vocab)
        v = __uint_as_float(0x7FC00000u);
      else if (y >= 0)
        v = empty ? -INFINITY : (load_elem(z, y, BF16) - all.m) * a.scale - ls;
      a.logp[row] = nan && y >= 0 ? all.s : v;
    }
  }
  if constexpr (TOP) {
    if (t < a.top) {
      const Key k = WPR > 1 ? sh.best[t] : list.key;
      const bool some = k != 0 && !nan;
      if (a.top_ids != nullptr) a.top_ids[row * a.top + t] = some ? key_column(k) : -1;
      if (a.top_logp != nullptr)
        a.top_logp[row * a.top + t] = nan ? all.s : some ? (key_value(k) - all.m) * a.scale - ls : -INFINITY;
    }
  }
}

template <bool BF16, int WPR, bool TOP, bool CLUSTER>
cudaError_t run_fwd(const LogprobFwdArgs& a, int parts, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  cfg.gridDim = dim3(unsigned(WPR == 1 ? (a.rows + kWarps - 1) / kWarps : a.rows * parts));
  constexpr int kThreads = 32 * kFwdWarps<WPR>;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = 2 * kVectors * kThreads * 16;
  cfg.stream = s;
  static LayerGrid grid;  // (asked for the memory that a CTA takes)
  int cap = 0;
  const cudaError_t e = layer_grid(grid, reinterpret_cast<const void*>(&k_logprob_fwd<BF16, WPR, TOP, CLUSTER>), kThreads,
                                   cfg.dynamicSmemBytes, cfg.dynamicSmemBytes + sizeof(Shared<TOP, kFwdWarps<WPR>>), &cap);
  if (e != cudaSuccess) return e;
  if (CLUSTER) {
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = unsigned(parts), attr.val.clusterDim.y = 1, attr.val.clusterDim.z = 1;
    cfg.attrs = &attr, cfg.numAttrs = 1;
  }
  return cudaLaunchKernelEx(&cfg, k_logprob_fwd<BF16, WPR, TOP, CLUSTER>, a);
}
template <bool BF16, bool TOP>
cudaError_t run_fwd_shape(const LogprobFwdArgs& a, int sms, cudaStream_t s) {
  // As few warps to a row as still fill the SMs: a row's beginning and end cost the same for each of its warps.  (us with
  // one, two, four and eight warps, bf16 and five alternatives: 1216 x 2000 8.1, 7.3, 9.4, 16.3; 8192 x 2000 21, 26, 43, 82;
  // 600 x 16000 20, 14, 12, 13; 4096 x 16000 44, 43, 52, 66; 600 x 131072 77, 47, 40, 39; 1216 x 131072 80, 66, 65, 70;
  // 4096 x 131072 203, 187, 194, 212.)
  const int64_t bytes = a.vocab * (BF16 ? 2 : 4), fill = int64_t(sms) * (bytes <= 4096 ? 8 : bytes <= 32768 ? 16 : 32);
  if (a.vocab <= 1024 || a.rows >= fill) return run_fwd<BF16, 1, TOP, false>(a, 1, s);
  if (a.rows * 2 >= fill) return run_fwd<BF16, 2, TOP, false>(a, 1, s);
  if (a.rows * 4 >= fill) return run_fwd<BF16, 4, TOP, false>(a, 1, s);
  // several CTAs to a row while the grid leaves SMs without work and a part still fills a CTA's threads once
  int parts = 1;
  while (parts < 8 && a.rows * parts * 2 <= 2 * sms && a.vocab >= int64_t(parts) * 2 * kThreadsLp * kVec<BF16>) parts *= 2;
  return parts == 1 ? run_fwd<BF16, 8, TOP, false>(a, 1, s) : run_fwd<BF16, 8, TOP, true>(a, parts, s);
}

// ---------------------------------------------------------------------------------------- backward

// dlogits_j = p_j (A + B t_j) (+ C at the given token), t_j = (z_j scale - lse) log2(e), p_j = 2^t_j.  The difference is
// rounded once, before it is taken to base 2: two products would each be rounded at the size of the logits.
struct Slope {
  float scale, lse, a, b, at;
  int64_t target;  // -1: none
};
__device__ __forceinline__ float slope_at(float z, const Slope& k) {
  const float t = max_nan(fmaf(z, k.scale, -k.lse) * kLog2E, kLeast);
  return exp2_f(t) * fmaf(k.b, t, k.a);
}

// 24 bits hold a log sum to 2^-24 of itself, by which p is off: 2^-14 here.  Rows farther from 0 (masked by -1e9 or by the
// type's lowest value from end to end, so that lse is that value however many tokens share the probability) and those
// whose log sum is infinite are summed anew, and p taken in deviations from the row's maximum: one more read (8192 x 32000
// bf16, all of them such rows, 196 us instead of 155).
constexpr float kFar = 1024.0f;

// Maximum and sum of 2^((z - maximum) c) of a row, by its team; the same in all its threads.
template <bool BF16, int WPR>
__device__ __forceinline__ Part far_sum(const char* z, const RowShape<BF16>& shape, int64_t cols, float c, int t) {
  constexpr int kElem = BF16 ? 2 : 4, V = kVec<BF16>, kTeam = 32 * WPR;
  const uint32_t none = BF16 ? 0xFF80FF80u : 0xFF800000u;
  const uint4* vec = reinterpret_cast<const uint4*>(z + shape.head * kElem);
  Part mine{kLowest, 0.0f, 0.0f};
  const auto take_one = [&](int64_t i) {
    const float v = load_elem_rw(z, i, BF16), m = max_nan(mine.m, v);
    mine = join(mine, Part{m, exp2_f(max_nan((v - m) * c, kLeast)), 0.0f}, c);
  };
  const int64_t tail = shape.head + shape.vectors * V;
  if (t < shape.head) take_one(t);
  if (t < cols - tail) take_one(tail + t);
  for (int64_t i = t; i < shape.vectors; i += 4 * kTeam) {
    uint4 w[4];
    float m = mine.m, s = 0.0f;
#pragma unroll
    for (int q = 0; q < 4; ++q) w[q] = i + q * kTeam < shape.vectors ? vec[i + q * kTeam] : make_uint4(none, none, none, none);
#pragma unroll
    for (int q = 0; q < 4; ++q) m = max_nan(m, largest<BF16>(w[q]));
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      Pair v[V / 2];
      to_pairs<BF16>(w[q], v);
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        const float2 x = halves((v[j] + pair(-m, -m)) * pair(c, c));
        s += exp2_f(max_nan(x.x, kLeast)) + exp2_f(max_nan(x.y, kLeast));
      }
    }
    mine = Part{m, fmaf(exp2_f(max_nan((mine.m - m) * c, kLeast)), mine.s, s), 0.0f};
  }
  const int lane = threadIdx.x & 31;
  mine = join_lanes<32>(mine, lane, c);
  if constexpr (WPR > 1) {
    __shared__ Part part[WPR];
    if (lane == 0) part[threadIdx.x / 32] = mine;
    __syncthreads();
    mine = join_lanes<WPR>(part[lane % WPR], lane, c);
  }
  return mine;
}

template <bool BF16>
__device__ __forceinline__ void store_one(void* row, int64_t i, float v) {
  store_elem(row, i, BF16, v);
}

template <bool BF16, int WPR>
__global__ void __launch_bounds__(kThreadsLp) k_logprob_bwd(const LogprobBwdArgs a, int parts) {
  constexpr int kElem = BF16 ? 2 : 4, V = kVec<BF16>, kTeam = 32 * WPR;
  const int warp = threadIdx.x / 32, t = threadIdx.x % kTeam;
  const int64_t row = WPR == 1 ? int64_t(blockIdx.x) * kWarps + warp : int64_t(blockIdx.x) / parts;
  const int me = WPR == 1 ? 0 : int(int64_t(blockIdx.x) % parts);
  if (row >= a.rows) return;
  const char* z = static_cast<const char*>(a.logits) + row * a.ld * kElem;
  char* o = static_cast<char*>(a.dlogits) + row * a.ldd * kElem;
  const int64_t y = a.dlogp != nullptr ? __ldg(a.targets + row) : -1;
  const float lse = __ldg(a.lse + row);
  const float d = a.dlogp != nullptr && y >= 0 ? (y < a.vocab ? __ldg(a.dlogp + row) : __uint_as_float(0x7FC00000u)) : 0.0f;
  const float dh = a.dentropy != nullptr ? __ldg(a.dentropy + row) : 0.0f;
  const float h = a.dentropy != nullptr ? __ldg(a.entropy + row) : 0.0f;
  Slope k;
  k.scale = a.scale, k.lse = lse;
  k.a = -a.scale * fmaf(dh, h, d), k.b = -a.scale * dh * kLn2, k.at = a.scale * d;
  k.target = y < a.vocab ? y : -1;
  const RowShape<BF16> shape = row_shape<BF16>(z, a.vocab);
  float base = 0.0f;  // of the logits: lse is that of their deviations from it
  // Nothing is left where lse is -inf, unless the scale took finite logits there, which one up to 1 cannot.
  bool none = lse == -INFINITY && a.scale <= 1.0f;
  if (fabsf(lse) > kFar && !none) {
    // (in place of the logits one CTA has the row: what it reads first, nobody else may have overwritten)
    if (z == o) {
      if (me != 0) return;
      parts = 1;
    }
    const Part sum = far_sum<BF16, WPR>(z, shape, a.vocab, a.scale * kLog2E, t);
    none = sum.s == 0.0f;
    if (!none) base = sum.m, k.lse = logf(sum.s);
  }
  if (none) k.lse = k.a = k.b = k.at = 0.0f;
  const auto value = [&](float v, int64_t col) {
    const float g = slope_at(v - base, k);
    return col == k.target ? g + k.at : g;
  };
  if ((reinterpret_cast<uintptr_t>(z) & 15) == (reinterpret_cast<uintptr_t>(o) & 15)) {
    const int64_t v_lo = shape.vectors * me / parts, v_hi = shape.vectors * (me + 1) / parts;
    const int64_t tail = shape.head + shape.vectors * V;
    if (me == 0 && t < shape.head) store_one<BF16>(o, t, value(load_elem_rw(z, t, BF16), t));
    if (me == parts - 1 && t < a.vocab - tail)
      store_one<BF16>(o, tail + t, value(load_elem_rw(z, tail + t, BF16), tail + t));
    for (int64_t i = v_lo + t; i < v_hi; i += 4 * kTeam) {
      uint4 w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (i + q * kTeam < v_hi) w[q] = __ldcs(reinterpret_cast<const uint4*>(z + shape.head * kElem) + i + q * kTeam);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (i + q * kTeam >= v_hi) continue;
        const int64_t col = shape.head + (i + q * kTeam) * V;
        Pair v[V / 2];
        to_pairs<BF16>(w[q], v);
        float g[V];
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
          const float2 f = halves(v[j]);
          g[2 * j] = value(f.x, col + 2 * j), g[2 * j + 1] = value(f.y, col + 2 * j + 1);
        }
        uint4 r;
        if (BF16)
          r = make_uint4(pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3]), pack_bf16x2(g[V - 4], g[V - 3]),
                         pack_bf16x2(g[V - 2], g[V - 1]));
        else
          r = make_uint4(__float_as_uint(g[0]), __float_as_uint(g[1]), __float_as_uint(g[2]), __float_as_uint(g[3]));
        __stcs(reinterpret_cast<uint4*>(o + shape.head * kElem) + i + q * kTeam, r);
      }
    }
  } else {
    // rows of logits and gradient start at different places within 16 bytes: neighbouring lanes take neighbouring elements
    const int64_t lo = a.vocab * me / parts, hi = a.vocab * (me + 1) / parts;
    for (int64_t i = lo + t; i < hi; i += 8 * kTeam) {
      float v[8], g[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = i + q * kTeam < hi ? load_elem_rw(z, i + q * kTeam, BF16) : 0.0f;
#pragma unroll
      for (int q = 0; q < 8; ++q) g[q] = value(v[q], i + q * kTeam);
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (i + q * kTeam < hi) store_one<BF16>(o, i + q * kTeam, g[q]);
    }
  }
}

template <bool BF16>
cudaError_t run_bwd(const LogprobBwdArgs& a, int sms, cudaStream_t s) {
  if (a.vocab <= 1024) {
    k_logprob_bwd<BF16, 1><<<unsigned((a.rows + kWarps - 1) / kWarps), kThreadsLp, 0, s>>>(a, 1);
  } else {
    int parts = 1;
    while (parts < 64 && a.rows * parts * 2 <= 8 * sms && a.vocab >= int64_t(parts) * 2 * kThreadsLp * kVec<BF16>) parts *= 2;
    k_logprob_bwd<BF16, 8><<<unsigned(a.rows * parts), kThreadsLp, 0, s>>>(a, parts);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_logprob_forward(const LogprobFwdArgs& a, cudaStream_t s) {
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  if (a.top > 0) return a.bf16 ? run_fwd_shape<true, true>(a, sms, s) : run_fwd_shape<false, true>(a, sms, s);
  return a.bf16 ? run_fwd_shape<true, false>(a, sms, s) : run_fwd_shape<false, false>(a, sms, s);
}

cudaError_t launch_logprob_backward(const LogprobBwdArgs& a, cudaStream_t s) {
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  return a.bf16 ? run_bwd<true>(a, sms, s) : run_bwd<false>(a, sms, s);
}

}  // namespace loco
