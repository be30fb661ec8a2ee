// What the forward and the backward kernels of a join share: rows in registers, and sums over a row.
//
// A row belongs to a team: a warp, a CTA of G threads, or a cluster of up to eight such CTAs, each of which
// has the next G * E columns.  A thread holds E columns, vectors t, t + G, ... of eight.
#pragma once

#include <cooperative_groups.h>

#include <cstddef>

#include "device_common.cuh"
#include "layers_common.cuh"
#include "steps_internal.h"
#include "tensor_core.cuh"

namespace loco {

namespace {

template <int G>
constexpr int kTeamCta = G < 128 ? 128 : G;  // threads of a CTA

// The CTA's dynamic shared memory: rows on their way and the threads' own parameters, by byte offsets.  (Read and written
// as plain memory, so that the compiler may order the accesses; the copies into it and their waits are barriers to that.)
__device__ __forceinline__ uint8_t* ring() {
  extern __shared__ __align__(128) uint8_t join_ring[];
  return join_ring;
}
__device__ __forceinline__ uint4 ring16(uint32_t at) { return *reinterpret_cast<const uint4*>(ring() + at); }
__device__ __forceinline__ void to_ring16(uint32_t at, uint4 v) { *reinterpret_cast<uint4*>(ring() + at) = v; }

// Pairs of the values of eight columns from their 16-byte words.
template <bool BF16>
__device__ __forceinline__ void words_to_pairs(const uint4 (&w)[BF16 ? 1 : 2], Pair* v) {
  if constexpr (BF16) {
    v[0] = widen(w[0].x), v[1] = widen(w[0].y), v[2] = widen(w[0].z), v[3] = widen(w[0].w);
  } else {
    v[0] = pair(__uint_as_float(w[0].x), __uint_as_float(w[0].y)), v[1] = pair(__uint_as_float(w[0].z), __uint_as_float(w[0].w));
    v[2] = pair(__uint_as_float(w[1].x), __uint_as_float(w[1].y)), v[3] = pair(__uint_as_float(w[1].z), __uint_as_float(w[1].w));
  }
}

// Where a matrix ends, for rows that lie anywhere: its last row, and the columns from this CTA's first to the row's end.
struct Edges {
  uint32_t last_row;
  int rest;
  bool first;  // this CTA has the rows' first columns
};

// Bytes [from, to) of sixteen, both even, to the sixteen-byte aligned place q.
__device__ __forceinline__ void store_part(char* q, uint4 w, uint32_t from, uint32_t to) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (uint32_t i = 0; i < 4; ++i) {
    if (from <= 4 * i && 4 * i + 4 <= to) {
      *reinterpret_cast<uint32_t*>(q + 4 * i) = u[i];
    } else {
      if (from <= 4 * i && 4 * i + 2 <= to) *reinterpret_cast<uint16_t*>(q + 4 * i) = uint16_t(u[i]);
      if (from <= 4 * i + 2 && 4 * i + 4 <= to) *reinterpret_cast<uint16_t*>(q + 4 * i + 2) = uint16_t(u[i] >> 16);
    }
  }
}

// Columns in vectors of eight.  A row on its way lies in shared memory: a thread copies its own vectors there (cp.async;
// nobody else reads them, so no barrier is needed), and `settle` puts zeros behind the row's end.
// ANY: rows may start at any element.  Then shared memory holds the aligned sixteen bytes as they lie in memory, a
// thread copies those that its vector begins in, and a warp's last lane the ones that the last vector ends in too;
// `settle` shifts a vector out of its own bytes and the next lane's.  A vector is stored as the aligned sixteen bytes
// that it shares with the lane before it, whose last bytes come by a shuffle; only what sticks out at the ends of a
// warp's run is stored in smaller pieces.
template <int G, int E, bool BF16, bool ANY>
struct Vec {
  static constexpr bool kAny = ANY;
  static constexpr int kReachBack = 8, kReach = 24;  // elements (see `load`)
  static constexpr int kRun = 256, kRunApart = G * 8;  // a warp's columns: runs, and how far they are apart
  static constexpr int kElem = BF16 ? 2 : 4, kWhole = BF16 ? 1 : 2;  // pieces of a vector
  static constexpr uint32_t kApart = kTeamCta<G> * 16;               // of a thread's pieces
  static constexpr uint32_t kVector = kWhole * kApart + (ANY ? kTeamCta<G> / 2 : 0), kBytes = E / 8 * kVector;  // of a CTA and row
  uint32_t at;   // its first piece in shared memory
  uint32_t off;  // bytes by which the row's vectors are off a sixteen-byte boundary

  __device__ static __forceinline__ int column(int t, int i) { return (t + G * (i / 8)) * 8 + i % 8; }
  // Piece k of vector e; k = kWhole is the first of the next lane, or, behind the last lane, the warp's own.
  __device__ __forceinline__ uint32_t piece(int e, int k) const {
    if (k < kWhole) return at + e * kVector + k * kApart;
    const bool last = (threadIdx.x & 31) == 31;
    return last ? at - threadIdx.x * 16 + e * kVector + kWhole * kApart + threadIdx.x / 32 * 16 : at + e * kVector + 16;
  }

  // (all lanes of a warp)
  __device__ __forceinline__ void load(const void* p, uint32_t row, int64_t ld, int t, int cols, const Edges& edges) {
    if (ANY) __syncwarp();  // the next lane, into whose first piece this one may write, is done with what was there
    const char* q = static_cast<const char*>(p) + row * ld * kElem;
    off = ANY ? uint32_t(reinterpret_cast<uintptr_t>(q)) & 15u : 0u;
#pragma unroll
    for (int e = 0; e < E / 8; ++e) {
      const int c0 = (t + G * e) * 8;
      if (c0 >= cols + (ANY ? 8 : 0)) continue;  // (with ANY, the lane behind the last has that one's end in its piece)
      const char* v = q + c0 * kElem;
      // Behind a row's end the matrix goes on, with what lies between its rows or with the next rows: only the pieces of
      // the first vector of the first rows and of the last vectors of the last ones may reach out of it.  A piece begins
      // less than eight columns before its vector and ends less than 24 behind the row's end: that is the first row and
      // the last where the rows are so far apart, and as many as make up so many elements where they are not.
      const uint32_t head = !ANY || ld >= kReachBack ? 1 : kReachBack, tail = !ANY || ld >= kReach ? 1 : kReach;
      const bool in = !((off != 0 && row < head && edges.first && c0 == 0) ||
                        (edges.last_row - row < tail && c0 + 8 + (off != 0 ? 16 / kElem : 0) > edges.rest));
      if (in) {
#pragma unroll
        for (int k = 0; k < kWhole; ++k)
          if (k == 0 || c0 < cols) copy_to_shared16(smem_addr(ring()) + piece(e, k), v - off + k * 16);
        if (ANY && off != 0 && (threadIdx.x & 31) == 31 && c0 < cols)
          copy_to_shared16(smem_addr(ring()) + piece(e, kWhole), v - off + kWhole * 16);
      } else {
        // element by element, with what the lane before has in this one's first piece
        const int before = ANY && c0 > 0 ? int(off) / kElem : 0, n = min(cols - c0, 8);
#pragma unroll 1
        for (int k = -before; k < n; ++k) {
          const uint32_t byte = off + k * kElem, place = piece(e, byte / 16) + byte % 16;
          if (BF16)
            *reinterpret_cast<uint16_t*>(ring() + place) = *reinterpret_cast<const uint16_t*>(v + k * 2);
          else
            *reinterpret_cast<uint32_t*>(ring() + place) = *reinterpret_cast<const uint32_t*>(v + k * 4);
        }
      }
    }
  }
  // Puts a row that has arrived in place, and zeros behind its end (all lanes of a warp).
  __device__ __forceinline__ void settle(int t, int cols) const {
    if (ANY) __syncwarp();
#pragma unroll
    for (int e = 0; e < E / 8; ++e) {
      const int left = (cols - (t + G * e) * 8) * kElem;  // bytes of the row from here on
      if (!ANY && left >= 8 * kElem) continue;
      uint4 w[kWhole + 1];
#pragma unroll
      for (int k = 0; k < kWhole + (ANY ? 1 : 0); ++k) w[k] = ring16(piece(e, k));
      if (ANY) {
        __syncwarp();
#pragma unroll
        for (int k = 0; k < kWhole; ++k)
          if (off != 0) w[k] = shifted16(w[k], w[k + 1], off);
      }
#pragma unroll
      for (int k = 0; k < kWhole; ++k) {
        if (left < 8 * kElem) {
          uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int n = left - k * 16 - i * 4;
            u[i] = n >= 4 ? u[i] : n > 0 ? u[i] & 0xFFFFu : 0u;
          }
          w[k] = make_uint4(u[0], u[1], u[2], u[3]);
        }
        to_ring16(piece(e, k), w[k]);
      }
    }
  }
  // Its columns 8 e to 8 e + 7 as four pairs.
  __device__ __forceinline__ void eight(int e, Pair (&v)[4]) const {
    uint4 w[kWhole];
#pragma unroll
    for (int k = 0; k < kWhole; ++k) w[k] = ring16(piece(e, k));
    words_to_pairs<BF16>(w, v);
  }
  // (all lanes of a warp)
  __device__ static __forceinline__ void store(char* row, int e, int t, int cols, const Pair (&v)[4]) {
    const int c0 = (t + G * e) * 8;
    float f[8];
    floats8(v, f);
    const uint32_t out = ANY ? uint32_t(reinterpret_cast<uintptr_t>(row)) & 15u : 0u;
    if (!ANY || out == 0) {
      if (c0 + 8 <= cols) {
        store8(row, c0, BF16, f);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (c0 + k < cols) store_elem(row, c0 + k, BF16, f[k]);
      }
      return;
    }
    const int lane = threadIdx.x & 31;
    uint4 w[kWhole];
    if constexpr (BF16) {
      w[0] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    } else {
      w[0] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
      w[1] = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
    }
    const uint4 last = w[kWhole - 1];
    uint4 before = make_uint4(__shfl_up_sync(0xFFFFFFFFu, last.x, 1), __shfl_up_sync(0xFFFFFFFFu, last.y, 1),
                              __shfl_up_sync(0xFFFFFFFFu, last.z, 1), __shfl_up_sync(0xFFFFFFFFu, last.w, 1));
    if (c0 >= cols) return;
    // bytes of the vector, counted from the boundary before it: [out, end)
    const uint32_t end = out + uint32_t(min(cols - c0, 8) * kElem);
    char* q = row + c0 * kElem - out;
#pragma unroll
    for (int k = 0; k < kWhole; ++k) {
      const uint4 x = shifted16(before, w[k], 16 - out);
      if ((k > 0 || lane > 0) && end >= uint32_t(16 * k + 16))
        *reinterpret_cast<uint4*>(q + k * 16) = x;
      else if (end > uint32_t(16 * k))
        store_part(q + k * 16, x, k == 0 && lane == 0 ? out : 0u, min(end - 16 * k, 16u));
      before = w[k];
    }
    // the last bytes, where no lane behind takes them
    if (end > uint32_t(16 * kWhole) && (lane == 31 || c0 + 8 >= cols))
      store_part(q + 16 * kWhole, shifted16(before, before, 16 - out), 0u, end - 16 * kWhole);
  }
};

// Single columns t, t + G, ... of rows that lie anywhere, in registers.  For 32-bit rows in the forward pass, where the
// shifting of Vec costs more than four times as many loads do (16384 x 4095 with bf16 y, layer norms: 255 us here, 385
// there; with bf16 rows 232 against 184).
template <int G, int E, bool BF16>
struct Cols {
  static constexpr int kRun = 32, kRunApart = G;
  static constexpr uint32_t kBytes = 0;
  uint32_t at;
  float f[E];

  __device__ static __forceinline__ int column(int t, int i) { return t + G * i; }
  __device__ __forceinline__ void load(const void* p, uint32_t row, int64_t ld, int t, int cols, const Edges&) {
    const char* q = static_cast<const char*>(p) + row * ld * (BF16 ? 2 : 4);
#pragma unroll
    for (int i = 0; i < E; ++i) f[i] = t + G * i < cols ? load_elem_rw(q, t + G * i, BF16) : 0.0f;
  }
  __device__ __forceinline__ void settle(int, int) const {}
  __device__ __forceinline__ void eight(int e, Pair (&v)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pair(f[e * 8 + 2 * i], f[e * 8 + 2 * i + 1]);
  }
  __device__ static __forceinline__ void store(char* row, int e, int t, int cols, const Pair (&v)[4]) {
    float x[8];
    floats8(v, x);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (t + G * (e * 8 + i) < cols) store_elem(row, t + G * (e * 8 + i), BF16, x[i]);
  }
};

// A vector of parameters at a thread's columns: `none` where it is not given, `past` behind the row's end.
// wide: it takes 16-byte loads.
template <typename Row, int E>
__device__ __forceinline__ void params(const void* p, int t, int cols, int bf16, bool wide, float none, float past, Pair* out) {
  float v[E];
  if (wide && p != nullptr && Row::column(t, E - 1) < cols) {
#pragma unroll
    for (int e = 0; e < E / 8; ++e) load8(p, Row::column(t, e * 8), bf16, v + e * 8);
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int c = Row::column(t, i);
      v[i] = c < cols ? (p != nullptr ? load_elem(p, c, bf16) : none) : past;
    }
  }
#pragma unroll
  for (int i = 0; i < E / 2; ++i) out[i] = pair(v[2 * i], v[2 * i + 1]);
}

// Values rounded to the type they are stored in.
__device__ __forceinline__ Pair as_stored(Pair v, int bf16) {
  if (!bf16) return v;
  const float2 h = halves(v);
  return widen(pack_bf16x2(h.x, h.y));
}
__device__ __forceinline__ Pair both(float v) { return pair(v, v); }
__device__ __forceinline__ float total(Pair v) {
  const float2 h = halves(v);
  return h.x + h.y;
}

__device__ __forceinline__ float warp_total(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// A thread's own parameters in shared memory, where it alone reads them: the `which`-th vector of E of them, in pieces
// of four, a CTA's threads apart.
template <int E, int THREADS>
__device__ __forceinline__ void keep(uint32_t at, int which, const Pair* v) {
#pragma unroll
  for (int i = 0; i < E / 2; i += 2) {
    const float2 lo = halves(v[i]), hi = halves(v[i + 1]);
    to_ring16(at + (which * (E / 4) + i / 2) * (THREADS * 16),
                make_uint4(__float_as_uint(lo.x), __float_as_uint(lo.y), __float_as_uint(hi.x), __float_as_uint(hi.y)));
  }
}
template <int E, int THREADS>
__device__ __forceinline__ void recall(uint32_t at, int which, int e, Pair (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const uint4 w = ring16(at + (which * (E / 4) + e * 2 + i / 2) * (THREADS * 16));
    v[i] = pair(__uint_as_float(w.x), __uint_as_float(w.y)), v[i + 1] = pair(__uint_as_float(w.z), __uint_as_float(w.w));
  }
}

// What a team's warps tell one another: N values of each.  Consecutive exchanges alternate between two areas, so that
// one barrier each is enough.  In a cluster every warp sends its values into each CTA's memory, where they count at a
// barrier of the area (st.async; a barrier of the whole cluster would wait for every store to global memory before it
// as well: 4096 x 8192 bf16 forward 60 us with one, 2048 x 16384 89 us).
// An area is written again two exchanges later, by a CTA that has what all warps sent in the exchange between, each
// after it had read this one.
constexpr int kMaxCluster = 8, kMaxSums = 4;  // (means and deviations of two rows)
constexpr uint64_t kWaitNs = 2000000000;  // longest wait for the cluster
constexpr uint64_t kLandNs = 10000000;    // more than a store to another CTA takes
__device__ unsigned long long g_join_timeouts;  // waits that ran out

template <int G, bool CL>
struct Board {
  static constexpr int kW = G / 32, kAll = kW * (CL ? kMaxCluster : 1);
  float v[2][kMaxSums][kAll];
  uint64_t bar[CL ? 2 : 1];
};
template <int G, bool CL>
struct Team {
  Board<G, CL>* board;
  int turn, ctas, rank;
  uint32_t peer, parity;  // the board of the cluster's CTA lane % 8; of the areas' barriers, a bit each
  // A wait ran out: what is read from then on is NaN, and nothing is waited for, sent or arrived at.  (A value sent ahead
  // would count at its barrier for one that is missing.)  So the waits of all other warps run out in their turn.
  bool lost;

  __device__ __forceinline__ Team(Board<G, CL>* b) : board(b), turn(0), ctas(1), rank(0), peer(0), parity(0), lost(false) {
    if constexpr (CL) {
      const auto cluster = cooperative_groups::this_cluster();
      ctas = int(cluster.num_blocks()), rank = int(cluster.block_rank());
      const uint32_t to = threadIdx.x % kMaxCluster;
      asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(peer) : "r"(smem_addr(board)), "r"(to < uint32_t(ctas) ? to : 0u));
      if (threadIdx.x == 0) {
        mbar_init(smem_addr(&board->bar[0]), 1), mbar_init(smem_addr(&board->bar[1]), 1);
        mbar_init_fence();
      }
      cluster.sync();  // every CTA's board is there
    }
  }
  // Before the kernel ends: no CTA leaves while another may still send to it, or while what one has sent is under way,
  // which nobody has waited for where a wait ran out.
  __device__ __forceinline__ void part() const {
    if constexpr (CL) {
      cooperative_groups::this_cluster().sync();
      if (lost) {
        const uint64_t start = global_ns();
        while (global_ns() - start < kLandNs);
      }
    }
  }
  __device__ __forceinline__ int warps() const { return G / 32 * ctas; }
  // Value `which` of this warp; lane `lane` of at least eight neighbours tells it to the cluster's CTA of that number.
  __device__ __forceinline__ void write(int which, int lane, float v) {
    const int warp = threadIdx.x / 32 % (G / 32);
    if constexpr (CL) {
      using B = Board<G, CL>;
      const uint32_t at = peer + uint32_t(offsetof(B, v)) + uint32_t(sizeof(B::v[0])) * turn + uint32_t(sizeof(B::v[0][0])) * which +
                          uint32_t(rank * (G / 32) + warp) * 4;
      if (lane < ctas && !lost)
        asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(at),
                     "r"(__float_as_uint(v)), "r"(peer + uint32_t(offsetof(B, bar)) + 8 * turn)
                     : "memory");
    } else {
      if (lane == 0) board->v[turn][which][warp] = v;
    }
  }
  // All `n` values of every warp are there.
  __device__ __forceinline__ void meet(int n) {
    if constexpr (CL) {
      const uint32_t bar = smem_addr(&board->bar[turn]);
      if (threadIdx.x == 0 && !lost) mbar_arrive_expect(bar, uint32_t(n * warps()) * 4);
      if (!lost && !arrived(bar, parity >> turn & 1)) {
        lost = true;
        if ((threadIdx.x & 31) == 0) atomicAdd(&g_join_timeouts, 1ull);
      }
      parity ^= 1u << turn;
    } else {
      __syncthreads();
    }
  }
  __device__ __forceinline__ static bool arrived(uint32_t bar, uint32_t parity) {
    const auto test = [&] {
      uint32_t done;
      asm volatile(
          "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(done)
          : "r"(bar), "r"(parity)
          : "memory");
      return done != 0;
    };
    if (test()) return true;
    const uint64_t start = global_ns();
    while (global_ns() - start < kWaitNs)
      if (test()) return true;
    return false;
  }
  // Sum of the warps' values `which`, in each lane of a half warp.
  __device__ __forceinline__ float read(int which) const {
    constexpr int kW = G / 32;
    const int l = threadIdx.x % 16;
    float v = 0.0f;
    if constexpr (CL) {
      for (int k = l; k < kW * ctas; k += 16) v += board->v[turn][which][k];
      if (lost) v = __uint_as_float(0x7FC00000u);
    } else if constexpr (kW > 16) {
      v = board->v[turn][which][l] + board->v[turn][which][l + 16];
    } else {
      v = board->v[turn][which][l % kW];
    }
#pragma unroll
    for (int o = CL || kW > 16 ? 8 : kW / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
  }
  // Sums over the team of N values, the same in all its threads, with one exchange between its warps.  Of two or three
  // values the first two take a half of a warp each, so that together they take little more than one does.
  template <int N>
  __device__ __forceinline__ void sum(float (&v)[N]) {
    static_assert(N >= 1 && N <= 3, "");
    const int lane = threadIdx.x & 31;
    const bool upper = N > 1 && lane >= 16;
    float x = v[0];
    if constexpr (N == 1)
      x += __shfl_xor_sync(0xFFFFFFFFu, x, 16);
    else
      x = (upper ? v[1] : v[0]) + __shfl_xor_sync(0xFFFFFFFFu, upper ? v[0] : v[1], 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    if constexpr (N == 3) v[2] = warp_total(v[2]);
    if constexpr (G > 32) {
      write(upper, N > 1 ? lane % 16 : lane, x);
      if constexpr (N == 3) write(2, lane, v[2]);
      meet(N);
      x = read(upper);
      if constexpr (N == 3) v[2] = read(2);
      turn ^= 1;
    }
    if constexpr (N == 1) {
      v[0] = x;
    } else {
      v[0] = __shfl_sync(0xFFFFFFFFu, x, 0), v[1] = __shfl_sync(0xFFFFFFFFu, x, 16);
    }
  }
};

// How many columns the warps have.
struct Counts {
  float inv_warp, inv_cols;  // of this thread's warp, and of the row
  float warp[4];             // columns of the team's warps lane, lane + 32, ...
};

// Means and variances of N rows with one exchange between the warps: each warp takes its own mean and then its squared
// deviations from that; together they make the row's mean, and the variance with what the warps' means are off it.
// No difference of large sums: a row far from 0 loses no digits.  The rows are 0 past their end, of which cols columns
// are this CTA's; v(k, i) is pair i of row k.
template <typename Row, int E, int N, int G, bool CL, typename Values>
__device__ __forceinline__ void layer_stats(Team<G, CL>& team, const Values& v, int t, int cols, const Counts& n,
                                            float (&mean)[N], float (&var)[N]) {
  const bool full = Row::column(t, E - 1) < cols;
  float m[N], q[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    Pair s2 = v(k, 0);
#pragma unroll
    for (int i = 1; i < E / 2; ++i) s2 = s2 + v(k, i);
    m[k] = total(s2);
  }
#pragma unroll
  for (int k = 0; k < N; ++k) m[k] = warp_total(m[k]) * n.inv_warp;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const Pair less = both(-m[k]);
    Pair q2 = both(0.0f);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      Pair d = v(k, i) + less;
      if (!full && Row::column(t, 2 * i + 1) >= cols) d = pair(Row::column(t, 2 * i) < cols ? halves(d).x : 0.0f, 0.0f);
      q2 = fma(d, d, q2);
    }
    q[k] = total(q2);
  }
#pragma unroll
  for (int k = 0; k < N; ++k) q[k] = warp_total(q[k]);
  if constexpr (G > 32) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < N; ++k) team.write(2 * k, lane, m[k]), team.write(2 * k + 1, lane, q[k]);
    team.meet(2 * N);
    constexpr int kW = G / 32, kEntries = CL ? kMaxCluster * kW / 32 : 1;
    const Board<G, CL>& board = *team.board;
    const auto across = [](float x) {
#pragma unroll
      for (int o = CL ? 16 : kW / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
      return x;
    };
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float c = team.lost ? __uint_as_float(0x7FC00000u) : board.v[team.turn][2 * k][0];  // the first warp's mean
      float d[kEntries], s = 0.0f;
      q[k] = 0.0f;
#pragma unroll
      for (int e = 0; e < kEntries; ++e) {
        const int at = CL ? lane + 32 * e : lane % kW;
        d[e] = n.warp[e] > 0.0f ? board.v[team.turn][2 * k][at] - c : 0.0f;
        q[k] += n.warp[e] > 0.0f ? board.v[team.turn][2 * k + 1][at] : 0.0f;
        s = fmaf(n.warp[e], d[e], s);
      }
      const float off = across(s) * n.inv_cols;
#pragma unroll
      for (int e = 0; e < kEntries; ++e) q[k] = fmaf(n.warp[e] * (d[e] - off), d[e] - off, q[k]);
      m[k] = c + off, q[k] = across(q[k]);
    }
    team.turn ^= 1;
  }
#pragma unroll
  for (int k = 0; k < N; ++k) mean[k] = m[k], var[k] = q[k] * n.inv_cols;
}

// all: columns of the row, of which this CTA has `cols`.
template <typename Row, int G, int E, bool CL>
__device__ __forceinline__ Counts row_counts(const Team<G, CL>& team, int t, int cols, int64_t all) {
  // of the columns of one CTA, those of its warp: runs of 32 threads' vectors, G threads' apart
  const auto of = [](int warp, int columns) {
    int k = 0;
#pragma unroll
    for (int i = 0; i < E * 32 / Row::kRun; ++i) k += min(max(columns - (warp * Row::kRun + i * Row::kRunApart), 0), Row::kRun);
    return float(k);
  };
  Counts n;
  const float w = of(t / 32, cols);
  n.inv_warp = w > 0.0f ? 1.0f / w : 0.0f;
  n.inv_cols = 1.0f / float(all);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    n.warp[k] = 0.0f;
    const int at = CL ? int(threadIdx.x & 31) + 32 * k : int(threadIdx.x & 31) % (G / 32);
    if (G > 32 && at < team.warps() && (CL || k == 0)) {
      const int64_t left = all - int64_t(at / (G / 32)) * G * E;  // columns of that warp's CTA
      n.warp[k] = of(at % (G / 32), left <= 0 ? 0 : left < G * E ? int(left) : G * E);
    }
  }
  return n;
}

// Columns c0 and on of a matrix or vector that may be missing.
__device__ __forceinline__ const void* from_column(const void* p, int64_t c0, int bf16) {
  return p == nullptr ? nullptr : static_cast<const char*>(p) + c0 * (bf16 ? 2 : 4);
}
__device__ __forceinline__ void* from_column(void* p, int64_t c0, int bf16) {
  return p == nullptr ? nullptr : static_cast<char*>(p) + c0 * (bf16 ? 2 : 4);
}

inline bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
inline bool on16(const void* p, int64_t ld, int64_t rows, int bf16) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows <= 1 || ld % (bf16 ? 8 : 4) == 0));
}

// CTAs of a grid whose teams walk the rows: `teams` of them in a CTA, or one in a cluster of `ctas`; at most
// `cap` CTAs, which the device holds at once.
inline int64_t team_ctas(int64_t rows, int cap, int teams, int ctas) {
  if (ctas > 1) {
    const int64_t most = cap / ctas > 0 ? cap / ctas : 1;
    return (rows < most ? rows : most) * ctas;
  }
  const int64_t want = (rows + teams - 1) / teams;
  return want < cap ? want : cap;
}
template <typename Args>
cudaError_t launch_teams(void (*kernel)(Args, bool), int64_t rows, int cap, int threads, int teams, int ctas, size_t smem,
                         cudaStream_t s, const Args& a, bool pwide) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  cfg.gridDim = dim3(unsigned(team_ctas(rows, cap, teams, ctas)));
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  if (ctas > 1) {
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = unsigned(ctas), attr.val.clusterDim.y = 1, attr.val.clusterDim.z = 1;
    cfg.attrs = &attr, cfg.numAttrs = 1;
  }
  return cudaLaunchKernelEx(&cfg, kernel, a, pwide);
}

}  // namespace

}  // namespace loco
