// Gradients of a join (loco_join_backward): four reads and two writes a value, one pass over the rows,
// and a small kernel that adds up the parameters' gradients.
//
// As in the forward pass a row stays on the SM and the next one is on its way (join_common.cuh).
// Two rounds of sums a row: through the norm in front of the next block, then through the one behind
// this block, whose gradient the first makes.  Of the parameters' gradients only four sums over rows are
// needed, with c_j = t_j row_gate (no gate, no scale):
//   sum c yh, sum c, sum du hh, sum du
// from which dpost_gamma = s gate sum c yh, dpost_beta = s gate sum c and dgate = s (post_gamma sum c yh +
// post_beta sum c) follow.  A thread keeps those of its own columns in registers over all its rows; one
// partial row per CTA goes to the workspace and a second kernel adds the partial rows in order: no
// atomics, the same result every run.
//
// 16384 x 4096 bf16 with RMS norms takes 153 us, 5.3 TB/s, 78 % of a copy's rate: with the sums over rows in registers two
// CTAs of 256 threads fit an SM (24 % of its warps), which issue in 43 % of the cycles and wait for one another at the two
// sums of each row.  (Merging those of a row with the next one's, as the forward pass does, takes 16 registers more and
// 171 us.)  Layer norms with betas 228 us; 2048 x 16384 193 us; 16384 x 4095 311 us; 500 x 2048 fp32 16 us, of which the
// second kernel is a third.
#include "join_common.cuh"

namespace loco {

namespace {

// Rows on their way: the one at work and the next.  Behind them a thread's own parameters (gm and pg below).
constexpr int kStages = 2;
template <int G, int E, typename RowX, typename RowY>
constexpr size_t kRing = size_t(kStages) * 2 * (RowX::kBytes + RowY::kBytes) + size_t(kTeamCta<G>) * 2 * E * sizeof(float);

// SUMS: 4, or 2 where neither sum c nor sum du is wanted (no betas).
// RMS: no mean is taken, and the reciprocal roots stay out of the products.  (It changes how dx and dy round, SUMS does
// not: they do not depend on which parameters' gradients are asked for.)
template <int G, int E, bool CL, int SUMS, bool RMS, typename RowX, typename RowY>
__global__ void __launch_bounds__(kTeamCta<G>, (E == 16 && SUMS == 4 && (CL || G == 32 || RowX::kAny) ? 256 : 512) / kTeamCta<G>)
    k_join_bwd(const JoinBwdArgs args, bool pwide) {
  __shared__ Board<G, CL> board;
  constexpr int kTeams = kTeamCta<G> / G, kThreadsCta = kTeamCta<G>, P = E / 2, C = E / 8;
  JoinBwdArgs a = args;
  const int t = threadIdx.x % G, place = threadIdx.x / G;
  Team<G, CL> team(&board);
  int64_t c0 = 0;
  uint32_t first = blockIdx.x * kTeams + place, step = gridDim.x * kTeams;  // (rows are below 2^31)
  const uint32_t n_rows = uint32_t(a.rows);
  if constexpr (CL) {
    c0 = int64_t(team.rank) * G * E, first = blockIdx.x / team.ctas, step = gridDim.x / team.ctas;
    a.dh = from_column(a.dh, c0, a.x_bf16), a.du = from_column(a.du, c0, a.y_bf16);
    a.h = from_column(a.h, c0, a.x_bf16), a.y = from_column(a.y, c0, a.y_bf16);
    a.dx = from_column(a.dx, c0, a.x_bf16), a.dy = from_column(a.dy, c0, a.y_bf16);
    a.post_gamma = from_column(a.post_gamma, c0, a.param_bf16), a.post_beta = from_column(a.post_beta, c0, a.param_bf16);
    a.gate = from_column(a.gate, c0, a.param_bf16), a.gamma = from_column(a.gamma, c0, a.param_bf16);
  }
  const int64_t rest = a.cols - c0;
  const int cols = rest <= 0 ? 0 : rest < G * E ? int(rest) : G * E;
  const Edges edges{n_rows - 1, rest < (1 << 30) ? int(rest) : 1 << 30, c0 == 0};
  const float inv_cols = 1.0f / float(a.cols);
  const bool level = !a.rms;
  const Pair zero = both(0.0f);
  Pair sums[SUMS][P];  // c yh, du hh (, c, du)
#pragma unroll
  for (int k = 0; k < SUMS; ++k) {
#pragma unroll
    for (int i = 0; i < P; ++i) sums[k][i] = zero;
  }
  const uint32_t base = threadIdx.x * 16;
  constexpr uint32_t kStage = 2 * (RowX::kBytes + RowY::kBytes), kOwn = kStages * kStage;
  RowX dhn, hn;
  RowY dun, yn;
  float m1n = 0.0f, r1n = 1.0f, m2n = 0.0f, r2n = 1.0f, wn = 1.0f;
  uint32_t slot = 0;
  const auto fetch = [&](uint32_t row) {
    dhn.at = base + slot * kStage, hn.at = dhn.at + RowX::kBytes;
    dun.at = hn.at + RowX::kBytes, yn.at = dun.at + RowY::kBytes;
    if (row < n_rows) {
      if (a.dh != nullptr) dhn.load(a.dh, row, a.lddh, t, cols, edges);
      if (a.du != nullptr) {
        dun.load(a.du, row, a.lddu, t, cols, edges);
        hn.load(a.h, row, a.ldh, t, cols, edges);
      }
      if (a.y != nullptr) yn.load(a.y, row, a.ldy, t, cols, edges);
      if (a.post) m1n = __ldg(a.stats + row), r1n = __ldg(a.stats + a.rows + row);
      if (a.du != nullptr) m2n = __ldg(a.stats + 2 * a.rows + row), r2n = __ldg(a.stats + 3 * a.rows + row);
      if (a.row_gate != nullptr) wn = __ldg(a.row_gate + row);
    }
    cp_async_commit();
    slot ^= 1;
  };
  cudaTriggerProgrammaticLaunchCompletion();  // the parameters' kernel may wait on its SMs
  fetch(first);  // on its way while the parameters come
  // q = du gm ; p = t w pg, pg with the gate and the scale in it, 0 past the row's end: whatever else a thread
  // has there (deviations of nothing from a mean) then reaches no sum of the row
  {
    Pair g[P], v[P];
    params<RowX, E>(a.gate, t, cols, a.param_bf16, pwide, 1.0f, 0.0f, g);
    params<RowX, E>(a.post_gamma, t, cols, a.param_bf16, pwide, 1.0f, 0.0f, v);
#pragma unroll
    for (int i = 0; i < P; ++i) v[i] = v[i] * (g[i] * both(a.s));
    keep<E, kThreadsCta>(base + kOwn, 1, v);
    params<RowX, E>(a.gamma, t, cols, a.param_bf16, pwide, 1.0f, 0.0f, v);
    keep<E, kThreadsCta>(base + kOwn, 0, v);
  }
  const Pair a2 = both(a.a);
  for (uint32_t row = first; row - (kTeams > 1 ? place : 0) < n_rows; row += step) {
    const bool live = row < n_rows;
    RowX dhc = dhn, hc = hn;
    RowY duc = dun, yc = yn;
    const float m1 = m1n, r1 = r1n, m2 = m2n, r2 = r2n, w = wn;
    fetch(row + step);
    cp_async_wait<1>();
    if (live) {
      if (a.dh != nullptr) dhc.settle(t, cols);
      if (a.du != nullptr) duc.settle(t, cols), hc.settle(t, cols);
      if (a.y != nullptr) yc.settle(t, cols);
    }
    // What a value takes part in is formed anew from shared memory in each of the three passes over the row's
    // columns: registers hold the sums over rows and t.
    float s[3] = {0.0f, 0.0f, 0.0f};
    if (a.du != nullptr) {
      if (live) {
        const Pair less = both(-m2), f = both(r2);
        Pair s0 = zero, s1 = zero;
#pragma unroll
        for (int e = 0; e < C; ++e) {
          Pair du[4], h[4], g[4];
          duc.eight(e, du), hc.eight(e, h);
          recall<E, kThreadsCta>(base + kOwn, 0, e, g);
          if constexpr (RMS) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              s1 = fma(du[i] * g[i], h[i], s1);  // over r2
              sums[1][e * 4 + i] = fma(du[i], h[i] * f, sums[1][e * 4 + i]);
              if constexpr (SUMS == 4) sums[3][e * 4 + i] = sums[3][e * 4 + i] + du[i];
            }
            continue;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            h[i] = (h[i] + less) * f;
            sums[1][e * 4 + i] = fma(du[i], h[i], sums[1][e * 4 + i]);
            if constexpr (SUMS == 4) sums[3][e * 4 + i] = sums[3][e * 4 + i] + du[i];
            du[i] = du[i] * g[i];
            s0 = s0 + du[i];
            s1 = fma(du[i], h[i], s1);
          }
        }
        s[0] = total(s0), s[1] = total(s1);
      }
      if constexpr (RMS) {
        float one[1] = {s[1]};
        team.sum(one);
        s[1] = -one[0] * inv_cols * r2 * r2;  // of h in (t - dh) / r2
      } else {
        float two[2] = {s[0], s[1]};
        team.sum(two);
        s[0] = level ? -two[0] * inv_cols : 0.0f, s[1] = -two[1] * inv_cols;
      }
    }
    Pair dt[P];
    if (live) {
      const Pair l2 = both(-m2), f2 = both(r2), c1 = both(s[0]), c2 = both(s[1]), l1 = both(-m1), f1 = both(r1), w2 = both(RMS ? w * r1 : w);
      Pair s0 = zero, s1 = zero, s2 = zero;
      char* out = static_cast<char*>(a.dx) + row * a.lddx * (a.x_bf16 ? 2 : 4);
#pragma unroll
      for (int e = 0; e < C; ++e) {
        Pair v[4], g[4], h[4];
        if (a.dh != nullptr) {
          dhc.eight(e, v);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = zero;
        }
        if (a.du != nullptr) {
          Pair du[4];
          duc.eight(e, du), hc.eight(e, h);
          recall<E, kThreadsCta>(base + kOwn, 0, e, g);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (RMS)
              v[i] = fma(f2, fma(h[i], c2, du[i] * g[i]), v[i]);
            else
              v[i] = fma(f2, fma((h[i] + l2) * f2, c2, fma(du[i], g[i], c1)), v[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) dt[e * 4 + i] = v[i], v[i] = a2 * v[i];
        RowX::store(out, e, t, cols, v);
        if (a.y != nullptr) {
          yc.eight(e, h);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) h[i] = zero;
        }
        recall<E, kThreadsCta>(base + kOwn, 1, e, g);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const Pair p = dt[e * 4 + i] * g[i];  // over w
          if constexpr (RMS) {
            sums[0][e * 4 + i] = fma(dt[e * 4 + i], h[i] * w2, sums[0][e * 4 + i]);
            if constexpr (SUMS == 4) sums[2][e * 4 + i] = fma(dt[e * 4 + i], both(w), sums[2][e * 4 + i]);
            s1 = fma(p, h[i], s1);  // over r1
          } else {
            const Pair yh = (h[i] + l1) * f1, c = dt[e * 4 + i] * w2;
            sums[0][e * 4 + i] = fma(c, yh, sums[0][e * 4 + i]);
            if constexpr (SUMS == 4) sums[2][e * 4 + i] = sums[2][e * 4 + i] + c;
            s0 = s0 + p;
            s1 = fma(p, yh, s1);
          }
        }
      }
      if (a.drow_gate != nullptr && a.post_beta != nullptr) {
        // t s gate post_beta, over s
        Pair b[P], v[P];
        params<RowX, E>(a.post_beta, t, cols, a.param_bf16, pwide, 0.0f, 0.0f, b);
#pragma unroll
        for (int i = 0; i < P; ++i) b[i] = dt[i] * b[i];
        params<RowX, E>(a.gate, t, cols, a.param_bf16, pwide, 1.0f, 0.0f, v);
#pragma unroll
        for (int i = 0; i < P; ++i) s2 = fma(b[i], v[i], s2);
      }
      s[0] = total(s0), s[1] = RMS ? total(s1) * r1 : total(s1), s[2] = total(s2);
    } else {
      s[0] = s[1] = s[2] = 0.0f;
    }
    if (a.drow_gate != nullptr) {
      team.sum(s);
      if (t == 0 && live && team.rank == 0) a.drow_gate[row] = fmaf(a.s, s[2], s[1]);
    } else if (a.post) {
      if constexpr (RMS) {
        float one[1] = {s[1]};
        team.sum(one);
        s[1] = one[0];
      } else {
        float two[2] = {s[0], s[1]};
        team.sum(two);
        s[0] = two[0], s[1] = two[1];
      }
    }
    if (!live) continue;  // whole teams
    {
      const Pair c1 = both(a.post && level ? -s[0] * inv_cols : 0.0f), c2 = both(a.post ? -s[1] * inv_cols * (RMS ? r1 : 1.0f) : 0.0f);
      const Pair l1 = both(-m1), f1 = both(r1), f = both(w * r1);
      char* out = static_cast<char*>(a.dy) + row * a.lddy * (a.y_bf16 ? 2 : 4);
#pragma unroll
      for (int e = 0; e < C; ++e) {
        Pair y[4], g[4];
        recall<E, kThreadsCta>(base + kOwn, 1, e, g);
        if (a.post) {
          yc.eight(e, y);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (RMS)
              g[i] = f * fma(y[i], c2, dt[e * 4 + i] * g[i]);
            else
              g[i] = f * fma((y[i] + l1) * f1, c2, fma(dt[e * 4 + i], g[i], c1));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) g[i] = f * (dt[e * 4 + i] * g[i]);
        }
        RowY::store(out, e, t, cols, g);
      }
    }
  }
  team.part();
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
        const float2 v = halves(sums[k][i / 2]);
        if (c < cols) out[kOrder[k] * a.cols + c] = i % 2 ? v.y : v.x;
      }
    }
  } else {
    float(*rows)[G * E] = reinterpret_cast<float(*)[G * E]>(ring() + kOwn);  // (no thread needs its parameters any more)
#pragma unroll
    for (int k = 0; k < SUMS; ++k) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float2 v = halves(sums[k][i / 2]);
        rows[place][RowX::column(t, i)] = i % 2 ? v.y : v.x;
      }
      __syncthreads();
      for (int c = threadIdx.x; c < cols; c += kThreadsCta) {
        float v = rows[0][c];
#pragma unroll
        for (int q = 1; q < kTeams; ++q) v += rows[q][c];
        out[kOrder[k] * a.cols + c] = v;
      }
    }
  }
}

// Rows of any length: a CTA of 1024 reads its row for each sum and output, and its partial sums lie in the workspace.
__global__ void __launch_bounds__(1024, 1) k_join_bwd_long(const JoinBwdArgs a) {
  __shared__ Board<1024, false> board;
  Team<1024, false> team(&board);
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

// Adds the partial rows of 32 columns, of two sums at a time: those behind the block (y) or those of the next norm.
// A warp takes every eighth partial row of one of the two, sixteen rows' loads under way at a time; the eight are
// joined in order.  (512 threads: 16384 x 4096 153 us with the rows, 64 x 4096 10.5; 1024, which fill an SM's registers,
// 155 and 13.1; 256, 161 and 12.0.)
__global__ void __launch_bounds__(512) k_join_bwd_params(const JoinBwdArgs a, int partials, int sums) {
  constexpr int kGroups = 8;
  __shared__ float part[kGroups][2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, k = warp % 2, group = warp / 2, next = blockIdx.y;
  const int64_t c = int64_t(blockIdx.x) * 32 + lane;
  cudaGridDependencySynchronize();  // launched while the rows' kernel runs
  float v = 0.0f;
  if (c < a.cols && (sums == 4 || k == 0)) {
    const int64_t row = kJoinSums * a.cols;
    const float* q = a.partials + (next * 2 + k) * a.cols + c + group * row;
    for (int p = group; p < partials; p += kGroups * 16, q += kGroups * 16 * row) {
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = p + i * kGroups < partials ? __ldcs(q + i * kGroups * row) : 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) v += x[i];
    }
  }
  part[group][k][lane] = v;
  __syncthreads();
  if (warp != 0 || c >= a.cols) return;
  float s[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    s[i] = part[0][i][lane];
#pragma unroll
    for (int w = 1; w < kGroups; ++w) s[i] += part[w][i][lane];
  }
  if (next) {
    if (a.dgamma != nullptr) store_elem(a.dgamma, c, a.grad_bf16, s[0]);
    if (a.dbeta != nullptr) store_elem(a.dbeta, c, a.grad_bf16, s[1]);
    return;
  }
  const float g = a.s * (a.gate != nullptr ? load_elem(a.gate, c, a.param_bf16) : 1.0f);
  if (a.dpost_gamma != nullptr) store_elem(a.dpost_gamma, c, a.grad_bf16, g * s[0]);
  if (a.dpost_beta != nullptr) store_elem(a.dpost_beta, c, a.grad_bf16, g * s[1]);
  if (a.dgate != nullptr) {
    const float pg = a.post_gamma != nullptr ? load_elem(a.post_gamma, c, a.param_bf16) : 1.0f;
    const float d = a.post_beta != nullptr ? load_elem(a.post_beta, c, a.param_bf16) * s[1] : 0.0f;
    store_elem(a.dgate, c, a.grad_bf16, a.s * fmaf(pg, s[0], d));
  }
}

template <int G, int E, bool CL, int SUMS, bool RMS, typename RowX, typename RowY>
cudaError_t run(const JoinBwdArgs& a, bool pwide, int ctas, int* partials, cudaStream_t s) {
  static LayerGrid grid;
  int cap = 0;
  const void* kernel = reinterpret_cast<const void*>(&k_join_bwd<G, E, CL, SUMS, RMS, RowX, RowY>);
  constexpr size_t kSmem = kRing<G, E, RowX, RowY>;
  const cudaError_t e = layer_grid(grid, kernel, kTeamCta<G>, kSmem, kSmem, &cap);
  if (e != cudaSuccess) return e;
  constexpr int kTeams = kTeamCta<G> / G;
  if (a.partials != nullptr) {
    // few rows: one CTA to an SM, or four rows and more to a team, as partial rows cost the second kernel (us at one, two,
    // four and eight rows a team: 64 x 4096 bf16 13.5, 15.0, 19.0, 25.6; 500 x 2048 fp32 22.1, 21.6, 18.0, 24.8)
    int sms = 0;
    const cudaError_t e2 = sm_count(&sms);
    if (e2 != cudaSuccess) return e2;
    const int64_t four = a.rows / (4 * kTeams) * ctas, most = four > sms ? four : sms;
    if (cap > kJoinPartials * ctas) cap = kJoinPartials * ctas;
    if (cap > most) cap = most > ctas ? int(most) : ctas;
  }
  *partials = int(team_ctas(a.rows, cap, kTeams, ctas) / ctas);
  return launch_teams(k_join_bwd<G, E, CL, SUMS, RMS, RowX, RowY>, a.rows, cap, kTeamCta<G>, kTeams, ctas, kSmem, s, a, pwide);
}
template <int G, int E, bool CL, typename RowX, typename RowY>
cudaError_t run_sums(const JoinBwdArgs& a, bool pwide, int ctas, int sums, int* partials, cudaStream_t s) {
  if (!a.rms) return run<G, E, CL, 4, false, RowX, RowY>(a, pwide, ctas, partials, s);
  return sums == 4 ? run<G, E, CL, 4, true, RowX, RowY>(a, pwide, ctas, partials, s)
                   : run<G, E, CL, 2, true, RowX, RowY>(a, pwide, ctas, partials, s);
}
template <int G, bool CL>
cudaError_t run_f32(const JoinBwdArgs& a, bool pwide, int ctas, int sums, int* partials, cudaStream_t s) {
  return a.y_bf16 ? run_sums<G, 8, CL, Vec<G, 8, false, false>, Vec<G, 8, true, false>>(a, pwide, ctas, sums, partials, s)
                  : run_sums<G, 8, CL, Vec<G, 8, false, false>, Vec<G, 8, false, false>>(a, pwide, ctas, sums, partials, s);
}
// bf16 rows: sixteen columns to a thread, so that half as many warps add up their sums.
template <int G, int E, bool CL>
cudaError_t run_bf16(const JoinBwdArgs& a, bool pwide, int ctas, int sums, int* partials, cudaStream_t s) {
  return run_sums<G, E, CL, Vec<G, E, true, false>, Vec<G, E, true, false>>(a, pwide, ctas, sums, partials, s);
}
template <int G, int E, bool CL>
cudaError_t run_any(const JoinBwdArgs& a, bool pwide, int ctas, int* partials, cudaStream_t s) {
  if (a.x_bf16) {
    return a.y_bf16 ? run<G, E, CL, 4, false, Vec<G, E, true, true>, Vec<G, E, true, true>>(a, pwide, ctas, partials, s)
                    : run<G, E, CL, 4, false, Vec<G, E, true, true>, Vec<G, E, false, true>>(a, pwide, ctas, partials, s);
  }
  return a.y_bf16 ? run<G, E, CL, 4, false, Vec<G, E, false, true>, Vec<G, E, true, true>>(a, pwide, ctas, partials, s)
                  : run<G, E, CL, 4, false, Vec<G, E, false, true>, Vec<G, E, false, true>>(a, pwide, ctas, partials, s);
}
template <int G, bool CL>
cudaError_t run_any_rms(const JoinBwdArgs& a, bool pwide, int ctas, int sums, int* partials, cudaStream_t s) {
  using Row = Vec<G, 16, true, true>;
  return sums == 4 ? run<G, 16, CL, 4, true, Row, Row>(a, pwide, ctas, partials, s)
                   : run<G, 16, CL, 2, true, Row, Row>(a, pwide, ctas, partials, s);
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
  const bool needs_betas = a.dbeta != nullptr || a.dpost_beta != nullptr || (a.dgate != nullptr && a.post_beta != nullptr);
  *sums = 4;
  if (ctas > kMaxCluster) return run_long(a, partials, s);
  if (wide) {
    if (a.rms && !needs_betas) *sums = 2;
    if (a.x_bf16) {
      if (a.cols <= 256) return run_bf16<32, 8, false>(a, pwide, 1, *sums, partials, s);
      if (a.cols <= 512) return run_bf16<32, 16, false>(a, pwide, 1, *sums, partials, s);
      if (a.cols <= 1024) return run_bf16<128, 8, false>(a, pwide, 1, *sums, partials, s);
      if (a.cols <= 2048) return run_bf16<128, 16, false>(a, pwide, 1, *sums, partials, s);
      if (a.cols <= 4096) return run_bf16<256, 16, false>(a, pwide, 1, *sums, partials, s);
      return run_bf16<256, 16, true>(a, pwide, ctas, *sums, partials, s);
    }
    if (a.cols <= 256) return run_f32<32, false>(a, pwide, 1, *sums, partials, s);
    if (a.cols <= 1024) return run_f32<128, false>(a, pwide, 1, *sums, partials, s);
    if (a.cols <= 2048) return run_f32<256, false>(a, pwide, 1, *sums, partials, s);
    if (a.cols <= 4096) return run_f32<512, false>(a, pwide, 1, *sums, partials, s);
    return run_f32<512, true>(a, pwide, ctas, *sums, partials, s);
  }
  // RMS norms of bf16 rows that lie anywhere: as of aligned ones (16384 x 4095 314 us, 378 with eight columns a thread and
  // four sums; four sums and sixteen columns take one CTA's registers)
  if (a.x_bf16 && a.y_bf16 && a.rms && a.cols > 1024) {
    if (!needs_betas) *sums = 2;
    if (a.cols <= 2048) return run_any_rms<128, false>(a, pwide, 1, *sums, partials, s);
    if (a.cols <= 4096) return run_any_rms<256, false>(a, pwide, 1, *sums, partials, s);
    return run_any_rms<256, true>(a, pwide, ctas, *sums, partials, s);
  }
  if (a.cols <= 256) return run_any<32, 8, false>(a, pwide, 1, partials, s);
  if (a.cols <= 1024) return run_any<128, 8, false>(a, pwide, 1, partials, s);
  if (a.cols <= 2048) return run_any<256, 8, false>(a, pwide, 1, partials, s);
  if (a.cols <= 4096) return run_any<512, 8, false>(a, pwide, 1, partials, s);
  return run_any<512, 8, true>(a, pwide, ctas, partials, s);
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
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  cfg.gridDim = dim3(unsigned((a.cols + 31) / 32), 2), cfg.blockDim = dim3(512), cfg.stream = s;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr, cfg.numAttrs = a.rows > 0 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, k_join_bwd_params, a, partials, sums);
}

cudaError_t read_join_backward_timeouts(int64_t* count) {
  unsigned long long v = 0;
  const cudaError_t e = cudaMemcpyFromSymbol(&v, g_join_timeouts, sizeof v);
  if (e == cudaSuccess) *count = int64_t(v);
  return e;
}

}  // namespace loco
