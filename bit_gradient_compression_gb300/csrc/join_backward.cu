// Gradients of a join (loco_join_backward): four reads and two writes a value, one pass over the rows,
// and a small kernel that adds up the parameters' gradients.
//
// As in the forward pass a row stays in registers and the next one is on its way (join_common.cuh).
// Two rounds of sums a row: through the norm in front of the next block, then through the one behind
// this block, whose gradient the first makes.  Of the parameters' gradients only four sums over rows are
// needed, with c_j = t_j row_gate (no gate, no scale):
//   sum c yh, sum c, sum du hh, sum du
// from which dpost_gamma = s gate sum c yh, dpost_beta = s gate sum c and dgate = s (post_gamma sum c yh +
// post_beta sum c) follow.  A thread keeps those of its own columns in registers over all its rows; one
// partial row per CTA goes to the workspace and a second kernel adds the partial rows in order: no
// atomics, the same result every run.
#include "join_common.cuh"

namespace loco {

namespace {

// SUMS: 4, or 2 where neither sum c nor sum du is wanted (a RMS norm without betas).
template <int G, int E, bool CL, int SUMS, typename RowX, typename RowY>
__global__ void __launch_bounds__(kTeamCta<G>, 1) k_join_bwd(const JoinBwdArgs args, bool pwide) {
  __shared__ Board<G, CL> board;
  constexpr int kTeams = kTeamCta<G> / G;
  JoinBwdArgs a = args;
  const int t = threadIdx.x % G, place = threadIdx.x / G;
  Team<G, CL> team{&board, 0, 1, 0};
  int64_t c0 = 0, first = int64_t(blockIdx.x) * kTeams + place, step = int64_t(gridDim.x) * kTeams;
  if constexpr (CL) {
    const auto cluster = cooperative_groups::this_cluster();
    team.ctas = int(cluster.num_blocks()), team.rank = int(cluster.block_rank());
    c0 = int64_t(team.rank) * G * E, first = blockIdx.x / team.ctas, step = gridDim.x / team.ctas;
    a.dh = from_column(a.dh, c0, a.x_bf16), a.du = from_column(a.du, c0, a.y_bf16);
    a.h = from_column(a.h, c0, a.x_bf16), a.y = from_column(a.y, c0, a.y_bf16);
    a.dx = from_column(a.dx, c0, a.x_bf16), a.dy = from_column(a.dy, c0, a.y_bf16);
    a.post_gamma = from_column(a.post_gamma, c0, a.param_bf16), a.post_beta = from_column(a.post_beta, c0, a.param_bf16);
    a.gate = from_column(a.gate, c0, a.param_bf16), a.gamma = from_column(a.gamma, c0, a.param_bf16);
    cluster.sync();  // every CTA's board is there
  }
  const int64_t rest = a.cols - c0;
  const int cols = rest <= 0 ? 0 : rest < G * E ? int(rest) : G * E;
  const float inv_cols = 1.0f / float(a.cols);
  const bool level = !a.rms;
  float sums[SUMS][E];  // c yh, du hh (, c, du)
#pragma unroll
  for (int k = 0; k < SUMS; ++k) {
#pragma unroll
    for (int i = 0; i < E; ++i) sums[k][i] = 0.0f;
  }
  // q = du gm ; p = t w pg, pg with the gate and the scale in it, 0 past the row's end: whatever else a thread
  // has there (deviations of nothing from a mean) then reaches no sum of the row
  constexpr bool kKeep = RowX::kShort;  // wider elements leave no registers for them: a thread's own places in shared memory
  __shared__ float4 own[kKeep ? 1 : E / 2][kKeep ? 1 : kTeamCta<G>];
  float gm[E], pg[E];
  params<RowX>(a.gate, t, cols, a.param_bf16, pwide, 1.0f, 0.0f, gm);
  params<RowX>(a.post_gamma, t, cols, a.param_bf16, pwide, 1.0f, 0.0f, pg);
#pragma unroll
  for (int i = 0; i < E; ++i) pg[i] *= a.s * gm[i];
  params<RowX>(a.gamma, t, cols, a.param_bf16, pwide, 1.0f, 0.0f, gm);
  const auto recall = [&](int first, float (&v)[E]) {
    if constexpr (!kKeep) {
#pragma unroll
      for (int i = 0; i < E; i += 4) {
        const float4 f = own[first + i / 4][threadIdx.x];
        v[i] = f.x, v[i + 1] = f.y, v[i + 2] = f.z, v[i + 3] = f.w;
      }
    }
  };
  if constexpr (!kKeep) {
#pragma unroll
    for (int i = 0; i < E; i += 4) {
      own[i / 4][threadIdx.x] = make_float4(gm[i], gm[i + 1], gm[i + 2], gm[i + 3]);
      own[(E + i) / 4][threadIdx.x] = make_float4(pg[i], pg[i + 1], pg[i + 2], pg[i + 3]);
    }
  }
  constexpr bool kAhead = RowX::kShort;  // wider elements leave no registers for a row ahead
  RowX dhn, hn;
  RowY dun, yn;
  const auto fetch = [&](int64_t row) {
    if (row >= a.rows) return;
    if (a.dh != nullptr) dhn.load(a.dh, row, a.lddh, t, cols, a.x_bf16);
    if (a.du != nullptr) {
      dun.load(a.du, row, a.lddu, t, cols, a.y_bf16);
      hn.load(a.h, row, a.ldh, t, cols, a.x_bf16);
    }
    if (a.y != nullptr) yn.load(a.y, row, a.ldy, t, cols, a.y_bf16);
  };
  if constexpr (kAhead) fetch(first);
  for (int64_t row = first; row - (kTeams > 1 ? place : 0) < a.rows; row += step) {
    const bool live = row < a.rows;
    if constexpr (!kAhead) fetch(row);
    float dt[E], du[E], h[E], y[E];
#pragma unroll
    for (int i = 0; i < E; ++i) dt[i] = du[i] = h[i] = y[i] = 0.0f;
    if (live) {
      if (a.dh != nullptr) dhn.values(dt);
      if (a.du != nullptr) dun.values(du), hn.values(h);
      if (a.y != nullptr) yn.values(y);
    }
    float m1 = 0.0f, r1 = 1.0f, m2 = 0.0f, r2 = 1.0f, w = 1.0f;
    if (live) {
      if (a.post) m1 = __ldg(a.stats + row), r1 = __ldg(a.stats + a.rows + row);
      if (a.du != nullptr) m2 = __ldg(a.stats + 2 * a.rows + row), r2 = __ldg(a.stats + 3 * a.rows + row);
      if (a.row_gate != nullptr) w = __ldg(a.row_gate + row);
    }
    if constexpr (kAhead) fetch(row + step);
    if (a.du != nullptr) {
      recall(0, gm);
      float s[2] = {0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < E; ++i) {
        h[i] = (h[i] - m2) * r2;
        sums[1][i] = fmaf(du[i], h[i], sums[1][i]);
        if constexpr (SUMS == 4) sums[3][i] += du[i];
        du[i] *= gm[i];
        s[0] += du[i];
        s[1] = fmaf(du[i], h[i], s[1]);
      }
      team.sum(s);
      const float c1 = level ? s[0] * inv_cols : 0.0f, c2 = s[1] * inv_cols;
#pragma unroll
      for (int i = 0; i < E; ++i) dt[i] = fmaf(r2, du[i] - c1 - h[i] * c2, dt[i]);
    }
#pragma unroll
    for (int i = 0; i < E; ++i) du[i] = a.a * dt[i];
    if (live) RowX::store(a.dx, row, a.lddx, t, cols, a.x_bf16, du);
    recall(E / 4, pg);
    float s[3] = {0.0f, 0.0f, 0.0f};  // of p / w, of p yh / w and of t s gate post_beta
#pragma unroll
    for (int i = 0; i < E; ++i) {
      y[i] = (y[i] - m1) * r1;
      if (!live) dt[i] = 0.0f;
      const float c = dt[i] * w;
      sums[0][i] = fmaf(c, y[i], sums[0][i]);
      if constexpr (SUMS == 4) sums[2][i] += c;
      du[i] = dt[i] * pg[i];
      s[0] += du[i];
      s[1] = fmaf(du[i], y[i], s[1]);
    }
    if (a.drow_gate != nullptr) {
      if (a.post_beta != nullptr) {
        float v[E];
        params<RowX>(a.post_beta, t, cols, a.param_bf16, pwide, 0.0f, 0.0f, v);
#pragma unroll
        for (int i = 0; i < E; ++i) dt[i] *= v[i];
        params<RowX>(a.gate, t, cols, a.param_bf16, pwide, 1.0f, 0.0f, v);
#pragma unroll
        for (int i = 0; i < E; ++i) s[2] = fmaf(dt[i], v[i], s[2]);
      }
      team.sum(s);
      if (t == 0 && live && team.rank == 0) a.drow_gate[row] = fmaf(a.s, s[2], s[1]);
    } else if (a.post) {
      float two[2] = {s[0], s[1]};
      team.sum(two);
      s[0] = two[0], s[1] = two[1];
    }
    if (a.post) {
      const float c1 = level ? s[0] * inv_cols : 0.0f, c2 = s[1] * inv_cols;
      const float f = w * r1;
#pragma unroll
      for (int i = 0; i < E; ++i) du[i] = f * (du[i] - c1 - y[i] * c2);
    } else if (a.row_gate != nullptr) {
#pragma unroll
      for (int i = 0; i < E; ++i) du[i] *= w;
    }
    if (live) RowY::store(a.dy, row, a.lddy, t, cols, a.y_bf16, du);
  }
  if (a.partials == nullptr) return;
  // one partial row a team of CTAs; the teams of a CTA are added through shared memory in their order
  float* out = a.partials + (CL ? int64_t(blockIdx.x) / team.ctas : int64_t(blockIdx.x)) * kJoinSums * a.cols + c0;
  constexpr int kOrder[4] = {0, 2, 1, 3};  // of the sums in the workspace: c yh, c, du hh, du
  if constexpr (kTeams == 1) {
#pragma unroll
    for (int k = 0; k < SUMS; ++k) {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int c = RowX::column(t, i);
        if (c < cols) out[kOrder[k] * a.cols + c] = sums[k][i];
      }
    }
  } else {
    __shared__ float rows[kTeams][G * E];
#pragma unroll
    for (int k = 0; k < SUMS; ++k) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < E; ++i) rows[place][RowX::column(t, i)] = sums[k][i];
      __syncthreads();
      for (int c = threadIdx.x; c < cols; c += kTeamCta<G>) {
        float v = rows[0][c];
#pragma unroll
        for (int q = 1; q < kTeams; ++q) v += rows[q][c];
        out[kOrder[k] * a.cols + c] = v;
      }
    }
  }
}

// Rows of any length: a CTA of 1024 reads its row for each sum and output, and its partial sums lie in the workspace.
__global__ void __launch_bounds__(1024) k_join_bwd_long(const JoinBwdArgs a) {
  __shared__ Board<1024, false> board;
  Team<1024, false> team{&board, 0, 1, 0};
  const float inv_cols = 1.0f / float(a.cols);
  const bool level = !a.rms;
  float* out = a.partials == nullptr ? nullptr : a.partials + int64_t(blockIdx.x) * kJoinSums * a.cols;
  const auto par = [&](const void* p, int64_t j, float none) { return p != nullptr ? load_elem(p, j, a.param_bf16) : none; };
  if (out != nullptr) {
    for (int64_t j = threadIdx.x; j < a.cols; j += 1024) {
#pragma unroll
      for (int k = 0; k < kJoinSums; ++k) out[k * a.cols + j] = 0.0f;
    }
  }
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    float m1 = 0.0f, r1 = 1.0f, m2 = 0.0f, r2 = 1.0f;
    if (a.post) m1 = a.stats[row], r1 = a.stats[a.rows + row];
    if (a.du != nullptr) m2 = a.stats[2 * a.rows + row], r2 = a.stats[3 * a.rows + row];
    const float w = a.row_gate != nullptr ? a.row_gate[row] : 1.0f;
    float c1 = 0.0f, c2 = 0.0f;
    if (a.du != nullptr) {
      float s[2] = {0.0f, 0.0f};
      for (int64_t j = threadIdx.x; j < a.cols; j += 1024) {
        const float q = load_elem(a.du, row * a.lddu + j, a.y_bf16) * par(a.gamma, j, 1.0f);
        s[0] += q;
        s[1] = fmaf(q, (load_elem(a.h, row * a.ldh + j, a.x_bf16) - m2) * r2, s[1]);
      }
      team.sum(s);
      c1 = level ? s[0] * inv_cols : 0.0f, c2 = s[1] * inv_cols;
    }
    // t of column j; dh may be dx, which is written last
    const auto through = [&](int64_t j, float* du, float* hh) {
      float v = a.dh != nullptr ? load_elem_rw(a.dh, row * a.lddh + j, a.x_bf16) : 0.0f;
      *du = *hh = 0.0f;
      if (a.du != nullptr) {
        *du = load_elem(a.du, row * a.lddu + j, a.y_bf16);
        *hh = (load_elem(a.h, row * a.ldh + j, a.x_bf16) - m2) * r2;
        v = fmaf(r2, *du * par(a.gamma, j, 1.0f) - c1 - *hh * c2, v);
      }
      return v;
    };
    float s[3] = {0.0f, 0.0f, 0.0f};
    for (int64_t j = threadIdx.x; j < a.cols; j += 1024) {
      float du, hh;
      const float t = through(j, &du, &hh), pg = par(a.post_gamma, j, 1.0f), g = par(a.gate, j, 1.0f);
      const float yh = a.y != nullptr ? (load_elem(a.y, row * a.ldy + j, a.y_bf16) - m1) * r1 : 0.0f;
      const float c = t * w, p = c * (a.s * g * pg);
      s[0] += p, s[1] = fmaf(p, yh, s[1]);
      if (a.drow_gate != nullptr) s[2] = fmaf(a.s * g * t, fmaf(yh, pg, par(a.post_beta, j, 0.0f)), s[2]);
      if (out != nullptr) {
        out[j] = fmaf(c, yh, out[j]);
        out[a.cols + j] += c;
        out[2 * a.cols + j] = fmaf(du, hh, out[2 * a.cols + j]);
        out[3 * a.cols + j] += du;
      }
    }
    team.sum(s);
    if (a.drow_gate != nullptr && threadIdx.x == 0) a.drow_gate[row] = s[2];
    const float d1 = level ? s[0] * inv_cols : 0.0f, d2 = s[1] * inv_cols;
    for (int64_t j = threadIdx.x; j < a.cols; j += 1024) {
      float du, hh;
      const float t = through(j, &du, &hh);
      float p = t * w * (a.s * par(a.gate, j, 1.0f) * par(a.post_gamma, j, 1.0f));
      if (a.post) p = r1 * (p - d1 - (load_elem(a.y, row * a.ldy + j, a.y_bf16) - m1) * r1 * d2);
      store_elem(a.dy, row * a.lddy + j, a.y_bf16, p);
      store_elem(a.dx, row * a.lddx + j, a.x_bf16, a.a * t);
    }
  }
}

// Adds the partial rows of 32 columns: 32 lanes of columns, eight warps of partial rows, joined in order.
__global__ void __launch_bounds__(256) k_join_bwd_params(const JoinBwdArgs a, int partials, int sums) {
  __shared__ float part[8][kJoinSums][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int64_t c = int64_t(blockIdx.x) * 32 + lane;
  float v[kJoinSums] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (c < a.cols) {
    for (int p = warp; p < partials; p += 8) {
      const float* q = a.partials + int64_t(p) * kJoinSums * a.cols + c;
      v[0] += q[0], v[2] += q[2 * a.cols];
      if (sums == 4) v[1] += q[a.cols], v[3] += q[3 * a.cols];
    }
  }
#pragma unroll
  for (int k = 0; k < kJoinSums; ++k) part[warp][k][lane] = v[k];
  __syncthreads();
  if (warp != 0 || c >= a.cols) return;
#pragma unroll
  for (int k = 0; k < kJoinSums; ++k) {
#pragma unroll
    for (int w = 1; w < 8; ++w) v[k] += part[w][k][lane];
  }
  const float g = a.s * (a.gate != nullptr ? load_elem(a.gate, c, a.param_bf16) : 1.0f);
  if (a.dpost_gamma != nullptr) store_elem(a.dpost_gamma, c, a.grad_bf16, g * v[0]);
  if (a.dpost_beta != nullptr) store_elem(a.dpost_beta, c, a.grad_bf16, g * v[1]);
  if (a.dgate != nullptr) {
    const float pg = a.post_gamma != nullptr ? load_elem(a.post_gamma, c, a.param_bf16) : 1.0f;
    const float d = a.post_beta != nullptr ? load_elem(a.post_beta, c, a.param_bf16) * v[1] : 0.0f;
    store_elem(a.dgate, c, a.grad_bf16, a.s * fmaf(pg, v[0], d));
  }
  if (a.dgamma != nullptr) store_elem(a.dgamma, c, a.grad_bf16, v[2]);
  if (a.dbeta != nullptr) store_elem(a.dbeta, c, a.grad_bf16, v[3]);
}

template <int G, int E, bool CL, int SUMS, typename RowX, typename RowY>
cudaError_t run(const JoinBwdArgs& a, bool pwide, int ctas, int* partials, cudaStream_t s) {
  static LayerGrid grid;
  int cap = 0;
  const void* kernel = reinterpret_cast<const void*>(&k_join_bwd<G, E, CL, SUMS, RowX, RowY>);
  const cudaError_t e = layer_grid(grid, kernel, kTeamCta<G>, 0, 0, &cap);
  if (e != cudaSuccess) return e;
  if (a.partials != nullptr && cap > kJoinPartials * ctas) cap = kJoinPartials * ctas;
  constexpr int kTeams = kTeamCta<G> / G;
  *partials = int(team_ctas(a.rows, cap, kTeams, ctas) / ctas);
  return launch_teams(k_join_bwd<G, E, CL, SUMS, RowX, RowY>, a.rows, cap, kTeamCta<G>, kTeams, ctas, s, a, pwide);
}
template <int G, int E, bool CL, typename RowX, typename RowY>
cudaError_t run_sums(const JoinBwdArgs& a, bool pwide, int ctas, int sums, int* partials, cudaStream_t s) {
  return sums == 4 ? run<G, E, CL, 4, RowX, RowY>(a, pwide, ctas, partials, s)
                   : run<G, E, CL, 2, RowX, RowY>(a, pwide, ctas, partials, s);
}
template <int G, int E, bool CL>
cudaError_t run_vec(const JoinBwdArgs& a, bool pwide, int ctas, int sums, int* partials, cudaStream_t s) {
  if (!a.x_bf16) {
    return a.y_bf16 ? run_sums<G, E, CL, Vec<G, E, false>, Vec<G, E, true>>(a, pwide, ctas, sums, partials, s)
                    : run_sums<G, E, CL, Vec<G, E, false>, Vec<G, E, false>>(a, pwide, ctas, sums, partials, s);
  }
  return run_sums<G, E, CL, Vec<G, E, true>, Vec<G, E, true>>(a, pwide, ctas, sums, partials, s);
}
template <int G, int E, bool CL>
cudaError_t run_cols(const JoinBwdArgs& a, int ctas, int* partials, cudaStream_t s) {
  return run<G, E, CL, 4, Cols<G, E>, Cols<G, E>>(a, false, ctas, partials, s);
}
cudaError_t run_long(const JoinBwdArgs& a, int* partials, cudaStream_t s) {
  static LayerGrid grid;
  int cap = 0;
  const cudaError_t e = layer_grid(grid, reinterpret_cast<const void*>(&k_join_bwd_long), 1024, 0, 0, &cap);
  if (e != cudaSuccess) return e;
  *partials = int(a.rows < cap ? a.rows : cap);
  if (a.partials != nullptr && *partials > kJoinPartials) *partials = kJoinPartials;
  k_join_bwd_long<<<*partials, 1024, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t rows_kernel(const JoinBwdArgs& a, int* sums, int* partials, cudaStream_t s) {
  const bool wide = on16(a.dh, a.lddh, a.rows, a.x_bf16) && on16(a.h, a.ldh, a.rows, a.x_bf16) &&
                    on16(a.dx, a.lddx, a.rows, a.x_bf16) && on16(a.y, a.ldy, a.rows, a.y_bf16) &&
                    on16(a.du, a.lddu, a.rows, a.y_bf16) && on16(a.dy, a.lddy, a.rows, a.y_bf16) &&
                    !(a.x_bf16 && !a.y_bf16);
  const bool pwide = on16(a.post_gamma) && on16(a.post_beta) && on16(a.gate) && on16(a.gamma);
  const int ctas = int((a.cols + 4095) / 4096);
  *sums = 4;
  if (ctas > kMaxCluster) return run_long(a, partials, s);
  if (wide) {
    if (a.dbeta == nullptr && a.dpost_beta == nullptr && (a.dgate == nullptr || a.post_beta == nullptr)) *sums = 2;
    if (a.cols <= 256) return run_vec<32, 8, false>(a, pwide, 1, *sums, partials, s);
    if (a.cols <= 1024) return run_vec<128, 8, false>(a, pwide, 1, *sums, partials, s);
    if (a.cols <= 2048) return run_vec<256, 8, false>(a, pwide, 1, *sums, partials, s);
    if (a.cols <= 4096) return run_vec<512, 8, false>(a, pwide, 1, *sums, partials, s);
    return run_vec<512, 8, true>(a, pwide, ctas, *sums, partials, s);
  }
  if (a.cols <= 256) return run_cols<32, 8, false>(a, 1, partials, s);
  if (a.cols <= 1024) return run_cols<128, 8, false>(a, 1, partials, s);
  if (a.cols <= 4096) return run_cols<512, 8, false>(a, 1, partials, s);
  return run_cols<512, 8, true>(a, ctas, partials, s);
}

}  // namespace

cudaError_t launch_join_backward(const JoinBwdArgs& a, cudaStream_t s) {
  int sums = 4, partials = 0;
  if (a.rows > 0) {
    const cudaError_t e = rows_kernel(a, &sums, &partials, s);
    if (e != cudaSuccess) return e;
  }
  if (a.dpost_gamma == nullptr && a.dpost_beta == nullptr && a.dgate == nullptr && a.dgamma == nullptr && a.dbeta == nullptr)
    return cudaSuccess;
  k_join_bwd_params<<<unsigned((a.cols + 31) / 32), 256, 0, s>>>(a, partials, sums);
  return cudaGetLastError();
}

}  // namespace loco
