// Joins a block's output to the residual stream and normalises the sum for the next block
// (loco_join_forward): two reads and two writes a value, one pass.
//
// A row stays in registers from its loads to its last store (join_common.cuh says who holds what); the
// next row is on its way meanwhile.  Each norm costs one round of sums: a RMS norm's squares, or a layer
// norm's mean and squared deviations together.  The second norm is that of the stream as it is stored,
// rounded to its type, which is what the backward pass will read.
// Rows of more than 4096 columns are shared by the CTAs of a cluster; those of more than 32768 go through L2:
// their CTA reads them once for every step.
#include "join_common.cuh"

namespace loco {

namespace {

// Rows on their way: the one at work and the next.  Behind them lie a thread's own parameters: pg and, where there are
// betas, pb (with the gate in them), gamma and beta.
constexpr int kStages = 2;
template <int G, int E, typename RowX, typename RowY>
size_t ring_bytes(bool betas) {
  return size_t(kStages) * (RowX::kBytes + RowY::kBytes) + size_t(kTeamCta<G>) * (betas ? 4 : 2) * E * sizeof(float);
}

template <int G, int E, bool CL, typename RowX, typename RowY>
__global__ void __launch_bounds__(kTeamCta<G>, (E == 16 ? 768 : 1024) / kTeamCta<G>)
    k_join_fwd(const JoinFwdArgs args, bool pwide) {
  __shared__ Board<G, CL> board;
  constexpr int kTeams = kTeamCta<G> / G, kThreadsCta = kTeamCta<G>, C = E / 8;
  JoinFwdArgs a = args;
  const int t = threadIdx.x % G, place = threadIdx.x / G;
  Team<G, CL> team{&board, 0, 1, 0};
  int64_t c0 = 0;
  uint32_t first = blockIdx.x * kTeams + place, step = gridDim.x * kTeams;  // (rows are below 2^31)
  const uint32_t n_rows = uint32_t(a.rows);
  if constexpr (CL) {
    const auto cluster = cooperative_groups::this_cluster();
    team.ctas = int(cluster.num_blocks()), team.rank = int(cluster.block_rank());
    c0 = int64_t(team.rank) * G * E, first = blockIdx.x / team.ctas, step = gridDim.x / team.ctas;
    a.x = from_column(a.x, c0, a.x_bf16), a.y = from_column(a.y, c0, a.y_bf16);
    a.h = from_column(a.h, c0, a.x_bf16), a.u = from_column(a.u, c0, a.y_bf16);
    a.post_gamma = from_column(a.post_gamma, c0, a.param_bf16), a.post_beta = from_column(a.post_beta, c0, a.param_bf16);
    a.gate = from_column(a.gate, c0, a.param_bf16);
    a.gamma = from_column(a.gamma, c0, a.param_bf16), a.beta = from_column(a.beta, c0, a.param_bf16);
    cluster.sync();  // every CTA's board is there
  }
  const int64_t rest = a.cols - c0;
  const int cols = rest <= 0 ? 0 : rest < G * E ? int(rest) : G * E;
  const Edges edges{n_rows - 1, rest < (1 << 30) ? int(rest) : 1 << 30, c0 == 0};
  const Counts n = row_counts<RowX, G, E, CL>(team, t, cols, a.cols);
  const auto stats = [&](const Pair (&v)[E / 2], float* mean, float* rstd) {
    float var;
    if (a.rms) {
      Pair q = v[0] * v[0];
#pragma unroll
      for (int i = 1; i < E / 2; ++i) q = fma(v[i], v[i], q);
      float s[1] = {total(q)};
      team.sum(s);
      *mean = 0.0f, var = s[0] * n.inv_cols;
    } else {
      layer_stats<RowX, E>(team, v, t, cols, n, mean, &var);
    }
    *rstd = rsqrtf(var + a.eps);
  };
  const uint32_t base = threadIdx.x * 16;
  constexpr uint32_t kStage = RowX::kBytes + RowY::kBytes, kOwn = kStages * kStage;
  const bool betas = a.post_beta != nullptr || a.beta != nullptr;
  RowX xn;
  RowY yn;
  float wn = 1.0f;
  uint32_t slot = 0;
  const auto fetch = [&](uint32_t row) {
    xn.at = base + slot * kStage, yn.at = xn.at + RowX::kBytes;
    if (row < n_rows) {
      xn.load(a.x, row, a.ldx, t, cols, edges);
      yn.load(a.y, row, a.ldy, t, cols, edges);
      if (a.row_gate != nullptr) wn = __ldg(a.row_gate + row);
    }
    cp_async_commit();
    slot ^= 1;
  };
  fetch(first);  // on its way while the parameters come
  {
    // h = a x + w (yh pg + pb), pg and pb with the gate in them, 0 past the row's end
    Pair g[E / 2], v[E / 2];
    params<RowX, E>(a.gate, t, cols, a.param_bf16, pwide, 1.0f, 0.0f, g);
    params<RowX, E>(a.post_gamma, t, cols, a.param_bf16, pwide, 1.0f, 0.0f, v);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) v[i] = v[i] * g[i];
    keep<E, kThreadsCta>(base + kOwn, 0, v);
    if (betas) {
      params<RowX, E>(a.post_beta, t, cols, a.param_bf16, pwide, 0.0f, 0.0f, v);
#pragma unroll
      for (int i = 0; i < E / 2; ++i) v[i] = v[i] * g[i];
      keep<E, kThreadsCta>(base + kOwn, 2, v);
      params<RowX, E>(a.beta, t, cols, a.param_bf16, pwide, 0.0f, 0.0f, v);
      keep<E, kThreadsCta>(base + kOwn, 3, v);
    }
    params<RowX, E>(a.gamma, t, cols, a.param_bf16, pwide, 1.0f, 0.0f, v);
    keep<E, kThreadsCta>(base + kOwn, 1, v);
  }
  const Pair a2 = both(a.a);
  for (uint32_t row = first; row - (kTeams > 1 ? place : 0) < n_rows; row += step) {
    const bool live = row < n_rows;  // (where it is not, the values are an earlier row's, and nothing is stored)
    const RowX xc = xn;
    const RowY yc = yn;
    const Pair w = both(a.s * wn);
    fetch(row + step);
    cp_async_wait<1>();
    if (live) xc.settle(t, cols), yc.settle(t, cols);
    Pair h[E / 2];  // y, then the joined stream
#pragma unroll
    for (int e = 0; e < C; ++e) {
      Pair v[4];
      yc.eight(e, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[e * 4 + i] = v[i];
    }
    float m1 = 0.0f, r1 = 1.0f, m2 = 0.0f, r2 = 1.0f;
    if (a.post) stats(h, &m1, &r1);
    const Pair l1 = both(-m1), f1 = both(r1);
    char* out = static_cast<char*>(a.h) + row * a.ldh * (a.x_bf16 ? 2 : 4);
#pragma unroll
    for (int e = 0; e < C; ++e) {
      Pair x[4], pg[4];
      xc.eight(e, x);
      recall<E, kThreadsCta>(base + kOwn, 0, e, pg);
#pragma unroll
      for (int i = 0; i < 4; ++i) pg[i] = (h[e * 4 + i] + l1) * f1 * pg[i];
      if (betas) {
        Pair pb[4];
        recall<E, kThreadsCta>(base + kOwn, 2, e, pb);
#pragma unroll
        for (int i = 0; i < 4; ++i) pg[i] = pg[i] + pb[i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = as_stored(fma(w, pg[i], a2 * x[i]), a.x_bf16), h[e * 4 + i] = x[i];
      if (live) RowX::store(out, e, t, cols, x);
    }
    if (a.u != nullptr) {
      stats(h, &m2, &r2);
      const Pair l2 = both(-m2), f2 = both(r2);
      out = static_cast<char*>(a.u) + row * a.ldu * (a.y_bf16 ? 2 : 4);
#pragma unroll
      for (int e = 0; e < C; ++e) {
        Pair g[4];
        recall<E, kThreadsCta>(base + kOwn, 1, e, g);
#pragma unroll
        for (int i = 0; i < 4; ++i) g[i] = (h[e * 4 + i] + l2) * f2 * g[i];
        if (betas) {
          Pair b[4];
          recall<E, kThreadsCta>(base + kOwn, 3, e, b);
#pragma unroll
          for (int i = 0; i < 4; ++i) g[i] = g[i] + b[i];
        }
        if (live) RowY::store(out, e, t, cols, g);
      }
    }
    if (a.stats != nullptr && t == 0 && live && team.rank == 0) {
      a.stats[row] = m1, a.stats[a.rows + row] = r1;
      a.stats[2 * a.rows + row] = m2, a.stats[3 * a.rows + row] = r2;
    }
  }
}

// Rows of any length: a CTA of 1024 reads its row for each mean, variance and output.
__global__ void __launch_bounds__(1024, 1) k_join_fwd_long(const JoinFwdArgs a) {
  __shared__ Board<1024, false> board;
  Team<1024, false> team{&board, 0, 1, 0};
  const auto sum = [&](float v) {
    float s[1] = {v};
    team.sum(s);
    return s[0];
  };
  const float inv_cols = 1.0f / float(a.cols);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const int64_t x0 = row * a.ldx, y0 = row * a.ldy, h0 = row * a.ldh, u0 = row * a.ldu;
    const auto stats = [&](const void* p, int64_t at, int bf16, float* mean, float* rstd) {
      float m = 0.0f;
      if (!a.rms) {
        float s = 0.0f;
        for (int64_t j = threadIdx.x; j < a.cols; j += 1024) s += load_elem_rw(p, at + j, bf16);
        m = sum(s) * inv_cols;
      }
      float q = 0.0f;
      for (int64_t j = threadIdx.x; j < a.cols; j += 1024) {
        const float d = load_elem_rw(p, at + j, bf16) - m;
        q = fmaf(d, d, q);
      }
      *mean = m, *rstd = rsqrtf(fmaf(sum(q), inv_cols, a.eps));
    };
    float m1 = 0.0f, r1 = 1.0f, m2 = 0.0f, r2 = 1.0f;
    if (a.post) stats(a.y, y0, a.y_bf16, &m1, &r1);
    const float w = a.s * (a.row_gate != nullptr ? a.row_gate[row] : 1.0f);
    // a thread reads back only what it wrote itself
    for (int64_t j = threadIdx.x; j < a.cols; j += 1024) {
      const float pg = a.post_gamma != nullptr ? load_elem(a.post_gamma, j, a.param_bf16) : 1.0f;
      const float pb = a.post_beta != nullptr ? load_elem(a.post_beta, j, a.param_bf16) : 0.0f;
      const float g = a.gate != nullptr ? load_elem(a.gate, j, a.param_bf16) : 1.0f;
      const float v = fmaf((load_elem(a.y, y0 + j, a.y_bf16) - m1) * r1, pg, pb);
      store_elem(a.h, h0 + j, a.x_bf16, fmaf(w * g, v, a.a * load_elem_rw(a.x, x0 + j, a.x_bf16)));
    }
    if (a.u != nullptr) {
      stats(a.h, h0, a.x_bf16, &m2, &r2);
      for (int64_t j = threadIdx.x; j < a.cols; j += 1024) {
        const float g = a.gamma != nullptr ? load_elem(a.gamma, j, a.param_bf16) : 1.0f;
        const float b = a.beta != nullptr ? load_elem(a.beta, j, a.param_bf16) : 0.0f;
        store_elem(a.u, u0 + j, a.y_bf16, fmaf((load_elem_rw(a.h, h0 + j, a.x_bf16) - m2) * r2, g, b));
      }
    }
    if (a.stats != nullptr && threadIdx.x == 0) {
      a.stats[row] = m1, a.stats[a.rows + row] = r1;
      a.stats[2 * a.rows + row] = m2, a.stats[3 * a.rows + row] = r2;
    }
  }
}

template <int G, int E, bool CL, typename RowX, typename RowY>
cudaError_t run(const JoinFwdArgs& a, bool pwide, int ctas, cudaStream_t s) {
  static LayerGrid grid[2];
  int cap = 0;
  const void* kernel = reinterpret_cast<const void*>(&k_join_fwd<G, E, CL, RowX, RowY>);
  const bool betas = a.post_beta != nullptr || a.beta != nullptr;
  const size_t smem = ring_bytes<G, E, RowX, RowY>(betas);
  const cudaError_t e = layer_grid(grid[betas], kernel, kTeamCta<G>, smem, ring_bytes<G, E, RowX, RowY>(true), &cap);
  if (e != cudaSuccess) return e;
  return launch_teams(k_join_fwd<G, E, CL, RowX, RowY>, a.rows, cap, kTeamCta<G>, kTeamCta<G> / G, ctas, smem, s, a, pwide);
}
template <int G, bool CL>
cudaError_t run_f32(const JoinFwdArgs& a, bool pwide, int ctas, cudaStream_t s) {
  return a.y_bf16 ? run<G, 8, CL, Vec<G, 8, false, false>, Vec<G, 8, true, false>>(a, pwide, ctas, s)
                  : run<G, 8, CL, Vec<G, 8, false, false>, Vec<G, 8, false, false>>(a, pwide, ctas, s);
}
// bf16 rows: sixteen columns to a thread, so that half as many warps add up their sums.
template <int G, int E, bool CL>
cudaError_t run_bf16(const JoinFwdArgs& a, bool pwide, int ctas, cudaStream_t s) {
  return run<G, E, CL, Vec<G, E, true, false>, Vec<G, E, true, false>>(a, pwide, ctas, s);
}
template <int G, int E, bool CL>
cudaError_t run_any_bf16(const JoinFwdArgs& a, bool pwide, int ctas, cudaStream_t s) {
  return a.y_bf16 ? run<G, E, CL, Vec<G, E, true, true>, Vec<G, E, true, true>>(a, pwide, ctas, s)
                  : run<G, E, CL, Vec<G, E, true, true>, Vec<G, E, false, true>>(a, pwide, ctas, s);
}
template <int G, bool CL>
cudaError_t run_any_f32(const JoinFwdArgs& a, int ctas, cudaStream_t s) {
  return a.y_bf16 ? run<G, 8, CL, Cols<G, 8, false>, Cols<G, 8, true>>(a, false, ctas, s)
                  : run<G, 8, CL, Cols<G, 8, false>, Cols<G, 8, false>>(a, false, ctas, s);
}

cudaError_t run_long(const JoinFwdArgs& a, cudaStream_t s) {
  static LayerGrid grid;
  int cap = 0;
  const cudaError_t e = layer_grid(grid, reinterpret_cast<const void*>(&k_join_fwd_long), 1024, 0, 0, &cap);
  if (e != cudaSuccess) return e;
  k_join_fwd_long<<<int(a.rows < cap ? a.rows : cap), 1024, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_join_forward(const JoinFwdArgs& a, cudaStream_t s) {
  const bool wide = on16(a.x, a.ldx, a.rows, a.x_bf16) && on16(a.h, a.ldh, a.rows, a.x_bf16) &&
                    on16(a.y, a.ldy, a.rows, a.y_bf16) && on16(a.u, a.ldu, a.rows, a.y_bf16) && !(a.x_bf16 && !a.y_bf16);
  const bool pwide = on16(a.post_gamma) && on16(a.post_beta) && on16(a.gate) && on16(a.gamma) && on16(a.beta);
  const int ctas = int((a.cols + 4095) / 4096);
  if (ctas > kMaxCluster) return run_long(a, s);
  if (wide && a.x_bf16) {
    if (a.cols <= 256) return run_bf16<32, 8, false>(a, pwide, 1, s);
    if (a.cols <= 512) return run_bf16<32, 16, false>(a, pwide, 1, s);
    if (a.cols <= 1024) return run_bf16<128, 8, false>(a, pwide, 1, s);
    if (a.cols <= 2048) return run_bf16<128, 16, false>(a, pwide, 1, s);
    if (a.cols <= 4096) return run_bf16<256, 16, false>(a, pwide, 1, s);
    return run_bf16<256, 16, true>(a, pwide, ctas, s);
  }
  if (wide) {
    if (a.cols <= 256) return run_f32<32, false>(a, pwide, 1, s);
    if (a.cols <= 1024) return run_f32<128, false>(a, pwide, 1, s);
    if (a.cols <= 2048) return run_f32<256, false>(a, pwide, 1, s);
    if (a.cols <= 4096) return run_f32<512, false>(a, pwide, 1, s);
    return run_f32<512, true>(a, pwide, ctas, s);
  }
  if (a.x_bf16) {
    if (a.cols <= 256) return run_any_bf16<32, 8, false>(a, pwide, 1, s);
    if (a.cols <= 1024) return run_any_bf16<128, 8, false>(a, pwide, 1, s);
    if (a.cols <= 2048) return run_any_bf16<128, 16, false>(a, pwide, 1, s);
    if (a.cols <= 4096) return run_any_bf16<256, 16, false>(a, pwide, 1, s);
    return run_any_bf16<256, 16, true>(a, pwide, ctas, s);
  }
  if (a.cols <= 256) return run_any_f32<32, false>(a, 1, s);
  if (a.cols <= 1024) return run_any_f32<128, false>(a, 1, s);
  if (a.cols <= 2048) return run_any_f32<256, false>(a, 1, s);
  if (a.cols <= 4096) return run_any_f32<512, false>(a, 1, s);
  return run_any_f32<512, true>(a, ctas, s);
}

}  // namespace loco
