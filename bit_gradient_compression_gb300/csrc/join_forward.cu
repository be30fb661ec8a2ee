// Joins a block's output to the residual stream and normalises the sum for the next block
// (loco_join_forward): two reads and two writes a value, one pass.
//
// A row stays in registers from its loads to its last store (join_common.cuh says who holds what); the
// next row is on its way meanwhile.  Each norm costs one round of sums: a RMS norm's squares, or a layer
// norm's mean and squared deviations together.  The second norm is that of the stream as it is stored,
// rounded to its type, which is what the backward pass will read.
// Rows of more than 4096 columns are shared by the CTAs of a cluster; those of more than 32768 go through L2:
// their CTA reads them once for every step.
//
// Bound by HBM where rows are bf16 and aligned: 16384 x 4096 with RMS norms 84 us, 6.4 TB/s, 94 % of a copy's rate (as
// many bytes in flight matter as registers allow, so a thread has sixteen columns, three CTAs an SM); with layer norms
// and betas 128 us, whose parameters leave shared memory for two CTAs.  Wider rows wait for the cluster (2048 x 16384
// 76 us of 40), unaligned ones are shifted (16384 x 4095 184 us).  One row of 4096 takes 3.6 us, the launch and three
// trips to memory.
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

// MERGED: the sums of a row's second norm and those of the next row's first are exchanged together, so that the team's
// warps meet once a row.
template <int G, int E, bool CL, bool MERGED, typename RowX, typename RowY>
__global__ void __launch_bounds__(kTeamCta<G>, (E == 16 || (RowX::kBytes == 0 && (CL || G == 32)) ? 768 : 1024) / kTeamCta<G>)
    k_join_fwd(const JoinFwdArgs args, bool pwide) {
  __shared__ Board<G, CL> board;
  constexpr int kTeams = kTeamCta<G> / G, kThreadsCta = kTeamCta<G>, C = E / 8;
  JoinFwdArgs a = args;
  const int t = threadIdx.x % G, place = threadIdx.x / G;
  Team<G, CL> team(&board);
  int64_t c0 = 0;
  uint32_t first = blockIdx.x * kTeams + place, step = gridDim.x * kTeams;  // (rows are below 2^31)
  const uint32_t n_rows = uint32_t(a.rows);
  if constexpr (CL) {
    c0 = int64_t(team.rank) * G * E, first = blockIdx.x / team.ctas, step = gridDim.x / team.ctas;
    a.x = from_column(a.x, c0, a.x_bf16), a.y = from_column(a.y, c0, a.y_bf16);
    a.h = from_column(a.h, c0, a.x_bf16), a.u = from_column(a.u, c0, a.y_bf16);
    a.post_gamma = from_column(a.post_gamma, c0, a.param_bf16), a.post_beta = from_column(a.post_beta, c0, a.param_bf16);
    a.gate = from_column(a.gate, c0, a.param_bf16);
    a.gamma = from_column(a.gamma, c0, a.param_bf16), a.beta = from_column(a.beta, c0, a.param_bf16);
  }
  const int64_t rest = a.cols - c0;
  const int cols = rest <= 0 ? 0 : rest < G * E ? int(rest) : G * E;
  const Edges edges{n_rows - 1, rest < (1 << 30) ? int(rest) : 1 << 30, c0 == 0};
  const Counts n = row_counts<RowX, G, E, CL>(team, t, cols, a.cols);
  // of N rows; v(k, i): pair i of row k
  const auto stats = [&](auto& mean, auto& rstd, const auto& v) {
    constexpr int N = sizeof(mean) / sizeof(float);
    if (a.rms) {
#pragma unroll
      for (int k = 0; k < N; ++k) {
        Pair q = v(k, 0) * v(k, 0);
#pragma unroll
        for (int i = 1; i < E / 2; ++i) q = fma(v(k, i), v(k, i), q);
        rstd[k] = total(q), mean[k] = 0.0f;
      }
      team.sum(rstd);
#pragma unroll
      for (int k = 0; k < N; ++k) rstd[k] = rsqrtf(fmaf(rstd[k], n.inv_cols, a.eps));
    } else {
      layer_stats<RowX, E>(team, v, t, cols, n, mean, rstd);
#pragma unroll
      for (int k = 0; k < N; ++k) rstd[k] = rsqrtf(rstd[k] + a.eps);
    }
  };
  const uint32_t base = threadIdx.x * 16;
  constexpr uint32_t kStage = RowX::kBytes + RowY::kBytes, kOwn = kStages * kStage;
  const bool betas = a.post_beta != nullptr || a.beta != nullptr;
  RowX x, xn;  // of the row at work and of the next
  RowY y, yn;
  float w = 1.0f, wn = 1.0f;
  const auto fetch = [&](RowX& x, RowY& y, float& w, uint32_t slot, uint32_t row) {
    x.at = base + slot * kStage, y.at = x.at + RowX::kBytes;
    if (row < n_rows) {
      x.load(a.x, row, a.ldx, t, cols, edges);
      y.load(a.y, row, a.ldy, t, cols, edges);
      if (a.row_gate != nullptr) w = __ldg(a.row_gate + row);
    }
    cp_async_commit();
  };
  fetch(x, y, w, 0, first);  // on its way while the parameters come
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
  if constexpr (MERGED) {
    fetch(xn, yn, wn, 1, first + step);
    cp_async_wait<1>();
    if (first < n_rows) x.settle(t, cols), y.settle(t, cols);
  }
  const auto whole = [](const RowY& from, Pair (&v)[E / 2]) {
#pragma unroll
    for (int e = 0; e < C; ++e) {
      Pair p[4];
      from.eight(e, p);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[e * 4 + i] = p[i];
    }
  };
  float m1 = 0.0f, r1 = 1.0f;
  const auto first_norm = [&](Pair (&v)[E / 2]) {
    whole(y, v);
    if (!a.post) return;
    float m[1], r[1];
    stats(m, r, [&](int, int i) { return v[i]; });
    m1 = m[0], r1 = r[0];
  };
  Pair h[E / 2];  // the joined stream; before that, where it is read first, y
  if (MERGED) first_norm(h);
  const Pair a2 = both(a.a);
  uint32_t slot = 0;
  for (uint32_t row = first; row - (kTeams > 1 ? place : 0) < n_rows; row += step) {
    // (where a row is not live, the values are an earlier row's, and nothing is stored)
    const bool live = row < n_rows, next = row + step < n_rows;
    if constexpr (!MERGED) {
      slot ^= 1;
      fetch(xn, yn, wn, slot, row + step);
      cp_async_wait<1>();
      if (live) x.settle(t, cols), y.settle(t, cols);
      first_norm(h);
    }
    const Pair l1 = both(-m1), f1 = both(r1), ws = both(a.s * w);
    char* to_h = static_cast<char*>(a.h) + row * a.ldh * (a.x_bf16 ? 2 : 4);
    char* to_u = static_cast<char*>(a.u) + row * a.ldu * (a.y_bf16 ? 2 : 4);
#pragma unroll
    for (int e = 0; e < C; ++e) {
      Pair v[4], n[4], p[4];
      x.eight(e, v);
      if constexpr (MERGED) {
        y.eight(e, n);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) n[i] = h[e * 4 + i];
      }
      recall<E, kThreadsCta>(base + kOwn, 0, e, p);
#pragma unroll
      for (int i = 0; i < 4; ++i) n[i] = (n[i] + l1) * f1 * p[i];
      if (betas) {
        recall<E, kThreadsCta>(base + kOwn, 2, e, p);
#pragma unroll
        for (int i = 0; i < 4; ++i) n[i] = n[i] + p[i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = as_stored(fma(ws, n[i], a2 * v[i]), a.x_bf16), h[e * 4 + i] = v[i];
      if (!MERGED && live) RowX::store(to_h, e, t, cols, v);
    }
    // x and y are used up
    x = xn, y = yn, w = wn;
    const float m0 = m1, r0 = r1;
    if constexpr (MERGED) {
      // their place takes the row after the next
      fetch(xn, yn, wn, slot, row + 2 * step);
      slot ^= 1;
      cp_async_wait<1>();
      if (next) x.settle(t, cols), y.settle(t, cols);
    }
    float m2 = 0.0f, r2 = 1.0f;
    if (MERGED && a.post && next && a.u != nullptr) {
      Pair v[E / 2];
      whole(y, v);
      float m[2], r[2];
      stats(m, r, [&](int k, int i) { return k == 0 ? h[i] : v[i]; });
      m2 = m[0], r2 = r[0], m1 = m[1], r1 = r[1];
    } else if (MERGED && a.post && next) {
      Pair v[E / 2];
      first_norm(v);
    } else if (a.u != nullptr) {
      float m[1], r[1];
      stats(m, r, [&](int, int i) { return h[i]; });
      m2 = m[0], r2 = r[0];
    }
    if (!live) continue;  // whole teams
    const Pair l2 = both(-m2), f2 = both(r2);
#pragma unroll
    for (int e = 0; e < C; ++e) {
      Pair v[4], g[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = h[e * 4 + i];
      if (MERGED) RowX::store(to_h, e, t, cols, v);
      if (a.u != nullptr) {
        recall<E, kThreadsCta>(base + kOwn, 1, e, g);
#pragma unroll
        for (int i = 0; i < 4; ++i) g[i] = (v[i] + l2) * f2 * g[i];
        if (betas) {
          recall<E, kThreadsCta>(base + kOwn, 3, e, v);
#pragma unroll
          for (int i = 0; i < 4; ++i) g[i] = g[i] + v[i];
        }
        RowY::store(to_u, e, t, cols, g);
      }
    }
    if (a.stats != nullptr && t == 0 && team.rank == 0) {
      a.stats[row] = m0, a.stats[a.rows + row] = r0;
      a.stats[2 * a.rows + row] = m2, a.stats[3 * a.rows + row] = r2;
    }
  }
  team.part();
}

// Rows of any length: a CTA of 1024 reads its row for each mean, variance and output.
__global__ void __launch_bounds__(1024, 1) k_join_fwd_long(const JoinFwdArgs a) {
  __shared__ Board<1024, false> board;
  Team<1024, false> team(&board);
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

template <int G, int E, bool CL, bool MERGED, typename RowX, typename RowY>
cudaError_t run_as(const JoinFwdArgs& a, bool pwide, int ctas, cudaStream_t s) {
  static LayerGrid grid[2];
  int cap = 0;
  const void* kernel = reinterpret_cast<const void*>(&k_join_fwd<G, E, CL, MERGED, RowX, RowY>);
  const bool betas = a.post_beta != nullptr || a.beta != nullptr;
  const size_t smem = ring_bytes<G, E, RowX, RowY>(betas);
  const cudaError_t e = layer_grid(grid[betas], kernel, kTeamCta<G>, smem, ring_bytes<G, E, RowX, RowY>(true), &cap);
  if (e != cudaSuccess) return e;
  return launch_teams(k_join_fwd<G, E, CL, MERGED, RowX, RowY>, a.rows, cap, kTeamCta<G>, kTeamCta<G> / G, ctas, smem, s, a, pwide);
}
// Merged exchanges (us: 16384 x 4096 bf16 layer norms 128 instead of 142, 2048 x 16384 bf16 RMS norms 77 instead of 87), but
// for RMS norms within a CTA, where they only put off the stores (84 us become 87), and for rows in registers, of which
// there would be too many (16384 x 4095 fp32 350 instead of 256).
template <int G, int E, bool CL, typename RowX, typename RowY>
cudaError_t run(const JoinFwdArgs& a, bool pwide, int ctas, cudaStream_t s) {
  if constexpr (RowX::kBytes == 0) {
    return run_as<G, E, CL, false, RowX, RowY>(a, pwide, ctas, s);
  } else if constexpr (CL) {
    return run_as<G, E, CL, true, RowX, RowY>(a, pwide, ctas, s);
  } else {
    return a.rms ? run_as<G, E, CL, false, RowX, RowY>(a, pwide, ctas, s) : run_as<G, E, CL, true, RowX, RowY>(a, pwide, ctas, s);
  }
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

cudaError_t read_join_forward_timeouts(int64_t* count) {
  unsigned long long v = 0;
  const cudaError_t e = cudaMemcpyFromSymbol(&v, g_join_timeouts, sizeof v);
  if (e == cudaSuccess) *count = int64_t(v);
  return e;
}

}  // namespace loco
