// The joint between two blocks: the norm after a block, its gate and residual
// scale, and the norm before the next block, forward and backward.
//
//   p  = o / sqrt(mean(o^2) + eps) * w_post,   h' = alpha h + beta act(g) p,
//   n  = h' / sqrt(mean(h'^2) + eps) * w_pre
//
// With nh = h'/r', u = dn w_pre the backward is
//   t  = dh' + (u - nh mean(u nh)) / r',       dh = alpha t,   dw_pre = sum dn nh,
//   dp = beta act(g) t,  dg = beta act'(g) t p,  dw_post = sum dp ph,
//   do = (v - ph mean(v ph)) / r   with v = dp w_post, ph = o / r.
//
// Both are HBM-bound: the forward reads o and h and writes h' and n, the
// backward reads o, h', dh' and dn and writes dh and do, each once.  A row
// stays in the registers of the threads that share it (up to 1024), its sums
// go through shuffles and one shared-memory exchange, and a group of threads
// works through a contiguous range of rows, so that gains, a gate shared by
// rows and the column sums of the backward stay in registers too.  The sums of
// squares are taken again in the backward from the rows it reads anyway, which
// costs no traffic and saves a buffer.
#include <cmath>

#include "rows.cuh"

namespace poet {
namespace {

constexpr int MAX_D = 16384;

struct JointFwdArgs {
  const void *o, *h, *gate;
  void *h_out, *n;
  int64_t ldo, ldh, ldg, ldho, ldn;
  const float *w_post, *w_pre;
  int64_t T, rows_per_group, gate_rows;
  int d, tpr;
  int post, gate_kind, gate_sigmoid;
  float alpha, beta, eps;
};

__device__ __forceinline__ float act_of(float g, int sig) { return sig ? 1.f / (1.f + expf(-g)) : g; }

// The row groups of a CTA: `tpr` threads (whole warps) each.
struct Group {
  int tid, warp, warps, bar;
  int64_t id;
  __device__ explicit Group(int tpr) {
    const int rg = threadIdx.x / tpr;
    tid = threadIdx.x - rg * tpr;
    warp = tid >> 5;
    warps = tpr >> 5;
    bar = 1 + rg;
    id = int64_t(blockIdx.x) * (blockDim.x / tpr) + rg;
  }
};

template <typename T, int VW, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT) joint_fwd_kernel(const JointFwdArgs a) {
  __shared__ float red[8][2][32];
  const Group g(a.tpr);
  float(*slot)[32] = red[g.bar - 1];
  int flip = 0;
  using V = RowVec<T, VW>;
  const T *o = static_cast<const T *>(a.o), *h = static_cast<const T *>(a.h), *gate = static_cast<const T *>(a.gate);
  T *ho = static_cast<T *>(a.h_out), *n = static_cast<T *>(a.n);
  const int64_t r0 = g.id * a.rows_per_group;
  const int64_t r1 = r0 + a.rows_per_group < a.T ? r0 + a.rows_per_group : a.T;
  if (r0 >= r1) return;
  float wq[NV][VW], wn[NV][VW];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (g.tid + j * a.tpr) * VW;
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      wq[j][e] = a.beta * (a.w_post && c < a.d ? a.w_post[c + e] : 1.f);
      wn[j][e] = a.w_pre && c < a.d ? a.w_pre[c + e] : 1.f;
    }
  }
  V vo[NV], vh[NV], vg[NV];
  auto load = [&](int64_t r) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (g.tid + j * a.tpr) * VW;
      if (c < a.d) {
        if (o) vo[j].load(o + r * a.ldo + c);
        vh[j].load(h + r * a.ldh + c);
      }
    }
  };
  load(r0);
  int64_t grow = r0 / a.gate_rows, gnext = grow * a.gate_rows;  // the gate row in registers is loaded at gnext
  float gval = 1.f;
  const float inv_d = 1.f / float(a.d);
  for (int64_t r = r0; r < r1; ++r) {
    if (a.gate_kind != POET_GATE_NONE && (r == r0 || r == gnext)) {
      if (r == gnext && r != r0) ++grow;
      gnext = (grow + 1) * a.gate_rows;
      if (a.gate_kind == POET_GATE_ROW) {
        gval = act_of(to_float(gate[grow * a.ldg]), a.gate_sigmoid);
      } else {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int c = (g.tid + j * a.tpr) * VW;
          if (c < a.d) vg[j].load(gate + grow * a.ldg + c);
        }
      }
    }
    float x[NV][VW], q[NV][VW];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (g.tid + j * a.tpr) * VW;
      if (c < a.d) {
        vh[j].get(x[j]);
        if (o) vo[j].get(q[j]);
      } else {
#pragma unroll
        for (int e = 0; e < VW; ++e) x[j][e] = q[j][e] = 0.f;
      }
    }
    if (r + 1 < r1) load(r + 1);
    if (o) {
      float ro = gval;
      if (a.post) {
        float s[1] = {0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int e = 0; e < VW; ++e) s[0] = fmaf(q[j][e], q[j][e], s[0]);
        row_sum<1>(s, slot[flip], g.warps, g.warp, g.bar, a.tpr);
        flip ^= 1;
        ro = gval / sqrtf(s[0] * inv_d + a.eps);
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (g.tid + j * a.tpr) * VW;
        float gv[VW];
        if (a.gate_kind == POET_GATE_CHANNEL && c < a.d) {
          vg[j].get(gv);
#pragma unroll
          for (int e = 0; e < VW; ++e) gv[e] = act_of(gv[e], a.gate_sigmoid);
        } else {
#pragma unroll
          for (int e = 0; e < VW; ++e) gv[e] = 1.f;
        }
#pragma unroll
        for (int e = 0; e < VW; ++e) x[j][e] = fmaf(a.alpha, x[j][e], q[j][e] * ro * wq[j][e] * gv[e]);
        if (c < a.d) V::store(ho + r * a.ldho + c, x[j]);
      }
    }
    if (n) {
      float s[1] = {0.f};
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < VW; ++e) s[0] = fmaf(x[j][e], x[j][e], s[0]);
      row_sum<1>(s, slot[flip], g.warps, g.warp, g.bar, a.tpr);
      flip ^= 1;
      const float rn = 1.f / sqrtf(s[0] * inv_d + a.eps);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (g.tid + j * a.tpr) * VW;
#pragma unroll
        for (int e = 0; e < VW; ++e) x[j][e] *= rn * wn[j][e];
        if (c < a.d) V::store(n + r * a.ldn + c, x[j]);
      }
    }
  }
}

struct JointBwdArgs {
  const void *o, *hp, *gate, *dhp, *dn;
  void *dh, *d_o, *dgate;
  int64_t ldo, ldhp, ldg, lddhp, lddn, lddh, lddo, lddg;
  const float *w_post, *w_pre;
  float *part_post, *part_pre;  // [groups][d]
  float *part_gate;             // [groups][d] (or [groups]) when chunks > 1
  int64_t T, gate_rows;
  // The group's rows: `chunks` groups share one segment of seg_rows rows
  // (chunks > 1), or one group takes segs_per_group whole segments.
  int64_t seg_rows, chunks, segs_per_group;
  int d, tpr;
  int post, gate_kind, gate_sigmoid;
  float alpha, beta, eps;
};

template <typename T, int VW, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT) joint_bwd_kernel(const JointBwdArgs a) {
  __shared__ float red[8][2][3][32];
  const Group g(a.tpr);
  float(*slot)[3][32] = red[g.bar - 1];
  using V = RowVec<T, VW>;
  const T *o = static_cast<const T *>(a.o), *hp = static_cast<const T *>(a.hp), *gate = static_cast<const T *>(a.gate);
  const T *dhp = static_cast<const T *>(a.dhp), *dn = static_cast<const T *>(a.dn);
  T *dh = static_cast<T *>(a.dh), *d_o = static_cast<T *>(a.d_o), *dgate = static_cast<T *>(a.dgate);
  int64_t r0, r1;
  if (a.chunks > 1) {
    const int64_t seg = g.id / a.chunks, k = g.id - seg * a.chunks;
    const int64_t s0 = seg * a.seg_rows, s1 = s0 + a.seg_rows < a.T ? s0 + a.seg_rows : a.T;
    if (s0 >= a.T) return;
    r0 = s0 + (s1 - s0) * k / a.chunks;
    r1 = s0 + (s1 - s0) * (k + 1) / a.chunks;
  } else {
    r0 = g.id * a.segs_per_group * a.seg_rows;
    r1 = r0 + a.segs_per_group * a.seg_rows < a.T ? r0 + a.segs_per_group * a.seg_rows : a.T;
    if (r0 >= a.T) return;
  }
  const bool shared_gate = dgate && a.gate_rows > 1;
  float aq[NV][VW], an[NV][VW], ag[NV][VW];
  float ag_row = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < VW; ++e) aq[j][e] = an[j][e] = ag[j][e] = 0.f;
  const float inv_d = 1.f / float(a.d);
  V vo[NV], vh[NV], vd[NV], vn[NV], vg[NV];
  auto load = [&](int64_t r) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (g.tid + j * a.tpr) * VW;
      if (c < a.d) {
        if (o) vo[j].load(o + r * a.ldo + c);
        if (dn) {
          vh[j].load(hp + r * a.ldhp + c);
          vn[j].load(dn + r * a.lddn + c);
        }
        if (dhp) vd[j].load(dhp + r * a.lddhp + c);
      }
    }
  };
  if (r0 < r1) load(r0);
  int64_t grow = r0 / a.gate_rows, gnext = (grow + 1) * a.gate_rows;
  float graw = 0.f;
  auto load_gate = [&]() {
    if (a.gate_kind == POET_GATE_ROW) {
      graw = to_float(gate[grow * a.ldg]);
    } else if (a.gate_kind == POET_GATE_CHANNEL) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (g.tid + j * a.tpr) * VW;
        if (c < a.d) vg[j].load(gate + grow * a.ldg + c);
      }
    }
  };
  // The gradient of the gate row in registers: to the result, or (where several
  // groups share the row) to this group's partial sums.
  auto flush_gate = [&]() {
    if (!shared_gate) return;
    const bool part = a.chunks > 1;
    if (a.gate_kind == POET_GATE_ROW) {
      if (g.tid == 0) {
        if (part) a.part_gate[g.id] = ag_row;
        else dgate[grow * a.lddg] = from_float<T>(ag_row);
      }
      ag_row = 0.f;
      return;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (g.tid + j * a.tpr) * VW;
      if (c < a.d) {
        if (part) {
#pragma unroll
          for (int e = 0; e < VW; ++e) a.part_gate[g.id * a.d + c + e] = ag[j][e];
        } else {
          V::store(dgate + grow * a.lddg + c, ag[j]);
        }
      }
#pragma unroll
      for (int e = 0; e < VW; ++e) ag[j][e] = 0.f;
    }
  };
  if (r0 < r1) load_gate();
  for (int64_t r = r0; r < r1; ++r) {
    if (r == gnext && a.gate_kind != POET_GATE_NONE) {
      flush_gate();
      ++grow;
      gnext += a.gate_rows;
      load_gate();
    }
    // x: h', then t; y: dn; q: o
    float x[NV][VW], y[NV][VW], q[NV][VW], t[NV][VW];
    float s[3] = {0.f, 0.f, 0.f};  // sum h'^2, sum u h', sum o^2
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (g.tid + j * a.tpr) * VW;
#pragma unroll
      for (int e = 0; e < VW; ++e) x[j][e] = y[j][e] = q[j][e] = t[j][e] = 0.f;
      if (c < a.d) {
        if (dn) {
          vh[j].get(x[j]);
          vn[j].get(y[j]);
        }
        if (dhp) vd[j].get(t[j]);
        if (o) vo[j].get(q[j]);
#pragma unroll
        for (int e = 0; e < VW; ++e) {
          s[0] = fmaf(x[j][e], x[j][e], s[0]);
          s[1] = fmaf(a.w_pre ? y[j][e] * a.w_pre[c + e] : y[j][e], x[j][e], s[1]);
          s[2] = fmaf(q[j][e], q[j][e], s[2]);
        }
      }
    }
    if (r + 1 < r1) load(r + 1);
    row_sum<3>(s, slot[0][0], g.warps, g.warp, g.bar, a.tpr);
    const float rn = 1.f / sqrtf(s[0] * inv_d + a.eps);
    const float mn = s[1] * rn * inv_d;  // mean(u nh)
    const float ro = a.post ? 1.f / sqrtf(s[2] * inv_d + a.eps) : 1.f;
    const float grv = a.gate_kind == POET_GATE_ROW ? act_of(graw, a.gate_sigmoid) : 1.f;
    float w[2] = {0.f, 0.f};  // sum v ph, sum of the row gate's gradient
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (g.tid + j * a.tpr) * VW;
      if (c < a.d) {
        float gv[VW];
        if (a.gate_kind == POET_GATE_CHANNEL) vg[j].get(gv);
        float dg[VW], out[VW];
#pragma unroll
        for (int e = 0; e < VW; ++e) {
          if (dn) {
            const float nh = x[j][e] * rn;
            an[j][e] = fmaf(y[j][e], nh, an[j][e]);
            const float u = a.w_pre ? y[j][e] * a.w_pre[c + e] : y[j][e];
            t[j][e] = fmaf(u - nh * mn, rn, t[j][e]);
          }
          out[e] = o ? a.alpha * t[j][e] : t[j][e];
        }
        V::store(dh + r * a.lddh + c, out);
        if (o) {
#pragma unroll
          for (int e = 0; e < VW; ++e) {
            const float ga = a.gate_kind == POET_GATE_CHANNEL ? act_of(gv[e], a.gate_sigmoid) : grv;
            const float da = a.beta * t[j][e];
            const float dp = da * ga;
            const float ph = q[j][e] * ro;
            const float wp = a.w_post ? a.w_post[c + e] : 1.f;
            dg[e] = da * (ph * wp) * (a.gate_sigmoid ? ga * (1.f - ga) : 1.f);
            if (a.post) aq[j][e] = fmaf(dp, ph, aq[j][e]);
            const float v = dp * wp;
            w[0] = fmaf(v, ph, w[0]);
            w[1] += dg[e];
            t[j][e] = v;
            q[j][e] = ph;
          }
          if (dgate && a.gate_kind == POET_GATE_CHANNEL) {
            if (a.gate_rows == 1) {
              V::store(dgate + r * a.lddg + c, dg);
            } else {
#pragma unroll
              for (int e = 0; e < VW; ++e) ag[j][e] += dg[e];
            }
          }
        }
      }
    }
    if (!o) {
      // the buffer of the first sum is written again in the next row: keep the two-barrier order
      if (g.warps > 1) asm volatile("bar.sync %0, %1;" ::"r"(g.bar), "r"(a.tpr) : "memory");
      continue;
    }
    row_sum<2>(w, slot[1][0], g.warps, g.warp, g.bar, a.tpr);
    const float mo = a.post ? w[0] * inv_d : 0.f;  // mean(v ph)
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (g.tid + j * a.tpr) * VW;
      if (c < a.d) {
#pragma unroll
        for (int e = 0; e < VW; ++e) t[j][e] = (t[j][e] - q[j][e] * mo) * ro;
        V::store(d_o + r * a.lddo + c, t[j]);
      }
    }
    if (dgate && a.gate_kind == POET_GATE_ROW) {
      if (a.gate_rows == 1) {
        if (g.tid == 0) dgate[r * a.lddg] = from_float<T>(w[1]);
      } else {
        ag_row += w[1];
      }
    }
  }
  flush_gate();
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (g.tid + j * a.tpr) * VW;
    if (c < a.d) {
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        if (a.part_post) a.part_post[g.id * a.d + c + e] = aq[j][e];
        if (a.part_pre) a.part_pre[g.id * a.d + c + e] = an[j][e];
      }
    }
  }
}

// Column sums of the groups' partial sums, in the groups' order.  Block (x, y):
// 32 columns of item y; 0: dw_post, 1: dw_pre, 2 + s: gate row s.
struct JointSumArgs {
  const float *part_post, *part_pre, *part_gate;
  float *dw_post, *dw_pre;
  void *dgate;
  int64_t lddg, groups, chunks;
  int d, gate_width;
};
constexpr int SUM_LANES = 16;

template <typename T>
__global__ void __launch_bounds__(32 * SUM_LANES) joint_sum_kernel(const JointSumArgs a) {
  __shared__ float acc[SUM_LANES][33];
  const int64_t item = blockIdx.y;
  const float *src;
  int64_t count;
  int width = a.d;
  if (item == 0) { src = a.dw_post ? a.part_post : nullptr; count = a.groups; }
  else if (item == 1) { src = a.dw_pre ? a.part_pre : nullptr; count = a.groups; }
  else {
    width = a.gate_width;
    src = a.part_gate + (item - 2) * a.chunks * width;
    count = a.chunks;
  }
  const int col = blockIdx.x * 32 + threadIdx.x;
  if (!src || int(blockIdx.x) * 32 >= width) return;
  float s = 0.f;
  if (col < width)
    for (int64_t i = threadIdx.y; i < count; i += SUM_LANES) s += src[i * width + col];
  acc[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y != 0 || col >= width) return;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < SUM_LANES; ++i) s += acc[i][threadIdx.x];
  if (item == 0) a.dw_post[col] = s;
  else if (item == 1) a.dw_pre[col] = s;
  else if (width == 1) static_cast<T *>(a.dgate)[(item - 2) * a.lddg] = from_float<T>(s);
  else static_cast<T *>(a.dgate)[(item - 2) * a.lddg + col] = from_float<T>(s);
}

// ------------------------------------------------------------------ launch shapes

bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Threads of a row and how many rows share a CTA: one vector per thread up to
// 1024 threads (several beyond), CTAs of at least 256 threads where rows are short.
struct RowShape {
  int nv, tpr, groups_per_cta, threads;
};
RowShape row_shape(int d, int vw, int nv_first) {
  RowShape s;
  const int nvec = (d + vw - 1) / vw;
  s.nv = nv_first;
  while ((nvec + s.nv - 1) / s.nv > 1024) s.nv *= 2;
  s.tpr = int(round_up((nvec + s.nv - 1) / s.nv, 32));
  s.groups_per_cta = s.tpr >= 256 ? 1 : 256 / s.tpr;
  s.threads = s.tpr * s.groups_per_cta;
  return s;
}

struct BwdPlan {
  int64_t seg_rows, segs, chunks, segs_per_group, groups;
};
// Groups of rows for the backward, at most `most`: every group lies inside one
// gate segment (the rows that share a gate row; all rows where none do), or
// takes whole segments, so a gate row's sum is either one group's or the sum of
// its `chunks` groups.
BwdPlan bwd_plan(const poet_joint *J, int64_t T, int64_t most) {
  BwdPlan p;
  p.seg_rows = J->gate != POET_GATE_NONE && J->gate_rows > 1 && J->gate_rows < T ? J->gate_rows : T;
  p.segs = (T + p.seg_rows - 1) / p.seg_rows;
  if (p.segs <= most) {
    p.chunks = std::min(most / p.segs, p.seg_rows);
    if (p.chunks < 1) p.chunks = 1;
    p.segs_per_group = 1;
    p.groups = p.segs * p.chunks;
  } else {
    p.chunks = 1;
    p.segs_per_group = (p.segs + most - 1) / most;
    p.groups = (p.segs + p.segs_per_group - 1) / p.segs_per_group;
  }
  return p;
}

// Most groups of rows: enough threads to fill every SM once more than over, and at
// least four rows each (a group's partial sums cost as much as a row).
int64_t bwd_most(int64_t T, int tpr) {
  const int64_t fill = std::max<int64_t>(1, int64_t(num_sms()) * std::max(1, 1536 / tpr));
  return std::max<int64_t>(1, std::min(fill, (T + 3) / 4));
}

poet_status check_joint(const poet_joint *J, const char *what) {
  POET_REQUIRE(J != nullptr, "%s: joint is NULL", what);
  POET_REQUIRE(J->d >= 1 && J->d <= MAX_D, "%s: width %d outside 1..%d", what, J->d, MAX_D);
  POET_REQUIRE(J->dtype == POET_F32 || J->dtype == POET_BF16, "%s: bad dtype %d", what, J->dtype);
  POET_REQUIRE(J->post_norm == 0 || J->post_norm == 1, "%s: post_norm %d must be 0 or 1", what, J->post_norm);
  POET_REQUIRE(J->gate >= POET_GATE_NONE && J->gate <= POET_GATE_ROW, "%s: bad gate %d", what, J->gate);
  POET_REQUIRE(J->gate_act == POET_GATE_LINEAR || J->gate_act == POET_GATE_SIGMOID, "%s: bad gate_act %d", what,
               J->gate_act);
  POET_REQUIRE(J->gate_rows >= 1, "%s: gate_rows %lld must be at least 1", what, (long long)J->gate_rows);
  POET_REQUIRE(std::isfinite(J->alpha) && std::isfinite(J->beta), "%s: alpha and beta must be finite", what);
  POET_REQUIRE(std::isfinite(J->eps) && J->eps > 0.f, "%s: eps must be positive", what);
  POET_REQUIRE((reinterpret_cast<uintptr_t>(J->w_post) & 3) == 0 && (reinterpret_cast<uintptr_t>(J->w_pre) & 3) == 0,
               "%s: gains not 4-byte aligned", what);
  POET_REQUIRE(J->post_norm || !J->w_post, "%s: w_post without post_norm", what);
  return POET_OK;
}

// A T x d operand: present, element-aligned, with a row stride of at least d.
poet_status check_rows(const char *what, const char *name, const void *p, int64_t ld, int64_t width, int dtype) {
  POET_REQUIRE(p != nullptr, "%s: %s is NULL", what, name);
  POET_REQUIRE((reinterpret_cast<uintptr_t>(p) & (esize(dtype) - 1)) == 0, "%s: %s not aligned to its elements", what,
               name);
  POET_REQUIRE(ld >= width, "%s: row stride %lld of %s below its width %lld", what, (long long)ld, name,
               (long long)width);
  return POET_OK;
}

// Whether every row of p starts on 16 bytes.
bool rows16(const void *p, int64_t ld, int dtype) { return !p || (al16(p) && ld * int64_t(esize(dtype)) % 16 == 0); }

template <typename T, int VW, int NV>
poet_status launch_fwd(const JointFwdArgs &a, const RowShape &s, int64_t groups, cudaStream_t st) {
  const unsigned grid = unsigned((groups + s.groups_per_cta - 1) / s.groups_per_cta);
  if (s.threads <= 256) joint_fwd_kernel<T, VW, NV, 256><<<grid, s.threads, 0, st>>>(a);
  else if (s.threads <= 512) joint_fwd_kernel<T, VW, NV, 512><<<grid, s.threads, 0, st>>>(a);
  else joint_fwd_kernel<T, VW, NV, 1024><<<grid, s.threads, 0, st>>>(a);
  count_launch();
  return launch_status("joint");
}

template <typename T, int VW, int NV>
poet_status launch_bwd(const JointBwdArgs &a, const RowShape &s, int64_t groups, cudaStream_t st) {
  const unsigned grid = unsigned((groups + s.groups_per_cta - 1) / s.groups_per_cta);
  if (s.threads <= 256) joint_bwd_kernel<T, VW, NV, 256><<<grid, s.threads, 0, st>>>(a);
  else if (s.threads <= 512) joint_bwd_kernel<T, VW, NV, 512><<<grid, s.threads, 0, st>>>(a);
  else joint_bwd_kernel<T, VW, NV, 1024><<<grid, s.threads, 0, st>>>(a);
  count_launch();
  return launch_status("joint_bwd");
}

}  // namespace
}  // namespace poet

using namespace poet;

extern "C" {

poet_status poet_joint_forward(const poet_joint *J, const void *o, int64_t ldo, const void *h, int64_t ldh,
                               const void *gate, int64_t ldg, int64_t T, void *h_out, int64_t ldho, void *n,
                               int64_t ldn, poet_stream stream) {
  CallRange nvtx_range("poet_joint_forward");
  clear_error();
  const char *what = "poet_joint_forward";
  POET_TRY(check_joint(J, what));
  POET_REQUIRE(T >= 0, "%s: T=%lld is negative", what, (long long)T);
  if (T == 0) return POET_OK;
  const int d = J->d, dt = J->dtype;
  POET_TRY(check_rows(what, "h", h, ldh, d, dt));
  if (o) {
    POET_TRY(check_rows(what, "o", o, ldo, d, dt));
    POET_TRY(check_rows(what, "h_out", h_out, ldho, d, dt));
    if (J->gate != POET_GATE_NONE)
      POET_TRY(check_rows(what, "gate", gate, ldg, J->gate == POET_GATE_CHANNEL ? d : 1, dt));
    else
      POET_REQUIRE(!gate, "%s: a gate was passed to a joint without one", what);
  } else {
    POET_REQUIRE(!h_out && !gate && n, "%s: without o there is only n: h_out and gate must be NULL, n must not", what);
  }
  if (n) POET_TRY(check_rows(what, "n", n, ldn, d, dt));
  JointFwdArgs a{};
  a.o = o; a.h = h; a.gate = gate; a.h_out = h_out; a.n = n;
  a.ldo = ldo; a.ldh = ldh; a.ldg = ldg; a.ldho = ldho; a.ldn = ldn;
  a.w_post = J->w_post; a.w_pre = J->w_pre;
  a.T = T; a.gate_rows = J->gate_rows; a.d = d;
  a.post = J->post_norm;
  a.gate_kind = o ? J->gate : int(POET_GATE_NONE);
  a.gate_sigmoid = J->gate_act == POET_GATE_SIGMOID;
  a.alpha = J->alpha; a.beta = J->beta; a.eps = J->eps;
  const int vw = 16 / int(esize(dt));
  const bool vec = d % vw == 0 && rows16(o, ldo, dt) && rows16(h, ldh, dt) && rows16(h_out, ldho, dt) &&
                   rows16(n, ldn, dt) && (a.gate_kind != POET_GATE_CHANNEL || rows16(gate, ldg, dt));
  const RowShape s = row_shape(d, vec ? vw : 1, vec ? 1 : 8);
  a.tpr = s.tpr;
  const int64_t fill = std::max<int64_t>(1, int64_t(num_sms()) * (2048 / s.tpr));
  a.rows_per_group = (T + fill - 1) / fill;
  const int64_t groups = (T + a.rows_per_group - 1) / a.rows_per_group;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int64_t G = (T + J->gate_rows - 1) / J->gate_rows;
  const double gate_elems = a.gate_kind == POET_GATE_CHANNEL ? double(G) * d : a.gate_kind == POET_GATE_ROW ? double(G) : 0.0;
  TraceScope ts("joint", 14.0 * double(T) * d,
                (double(T) * d * ((o ? 3 : 1) + (n ? 1 : 0)) + gate_elems) * double(esize(dt)), st);
  if (dt == POET_BF16) {
    if (vec) return s.nv == 1 ? launch_fwd<bf16, 8, 1>(a, s, groups, st) : launch_fwd<bf16, 8, 2>(a, s, groups, st);
    return s.nv == 8 ? launch_fwd<bf16, 1, 8>(a, s, groups, st) : launch_fwd<bf16, 1, 16>(a, s, groups, st);
  }
  if (vec) {
    if (s.nv == 1) return launch_fwd<float, 4, 1>(a, s, groups, st);
    return s.nv == 2 ? launch_fwd<float, 4, 2>(a, s, groups, st) : launch_fwd<float, 4, 4>(a, s, groups, st);
  }
  return s.nv == 8 ? launch_fwd<float, 1, 8>(a, s, groups, st) : launch_fwd<float, 1, 16>(a, s, groups, st);
}

size_t poet_joint_workspace_bytes(const poet_joint *J, int64_t T) {
  clear_error();
  if (check_joint(J, "poet_joint_workspace_bytes") != POET_OK || T < 0) return 0;
  if (T == 0) return 256;
  // the most groups that any alignment and gate can give: grows with T, so that
  // one workspace serves smaller calls too
  const int vw = 16 / int(esize(J->dtype));
  size_t most = 0;
  for (int k = 0; k < 2; ++k) {
    const RowShape s = row_shape(J->d, k == 0 ? vw : 1, k == 0 ? 1 : 8);
    most = std::max(most, size_t(bwd_most(T, s.tpr)));
  }
  return 3 * align256(most * size_t(J->d) * 4);
}

poet_status poet_joint_backward(const poet_joint *J, const void *o, int64_t ldo, const void *h_out, int64_t ldho,
                                const void *gate, int64_t ldg, const void *dh_out, int64_t lddho, const void *dn,
                                int64_t lddn, int64_t T, void *dh, int64_t lddh, void *d_o, int64_t lddo, void *dgate,
                                int64_t lddg, float *dw_post, float *dw_pre, void *ws, size_t ws_bytes,
                                poet_stream stream) {
  CallRange nvtx_range("poet_joint_backward");
  clear_error();
  const char *what = "poet_joint_backward";
  POET_TRY(check_joint(J, what));
  POET_REQUIRE(T >= 0, "%s: T=%lld is negative", what, (long long)T);
  const int d = J->d, dt = J->dtype;
  POET_REQUIRE((reinterpret_cast<uintptr_t>(dw_post) & 3) == 0 && (reinterpret_cast<uintptr_t>(dw_pre) & 3) == 0,
               "%s: dw_post / dw_pre not 4-byte aligned", what);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) {
    if (dw_post) POET_CUDA_TRY(cudaMemsetAsync(dw_post, 0, size_t(d) * 4, st));
    if (dw_pre) POET_CUDA_TRY(cudaMemsetAsync(dw_pre, 0, size_t(d) * 4, st));
    return POET_OK;
  }
  POET_REQUIRE(dh_out || dn, "%s: dh_out and dn are both NULL", what);
  POET_REQUIRE(!dw_post || (o && J->post_norm), "%s: dw_post without a norm after the block", what);
  POET_REQUIRE(!dw_pre || dn, "%s: dw_pre without dn", what);
  if (dh_out) POET_TRY(check_rows(what, "dh_out", dh_out, lddho, d, dt));
  if (dn) {
    POET_TRY(check_rows(what, "dn", dn, lddn, d, dt));
    POET_TRY(check_rows(what, "h_out", h_out, ldho, d, dt));
  }
  POET_TRY(check_rows(what, "dh", dh, lddh, d, dt));
  const int gate_width = J->gate == POET_GATE_CHANNEL ? d : 1;
  if (o) {
    POET_TRY(check_rows(what, "o", o, ldo, d, dt));
    POET_TRY(check_rows(what, "d_o", d_o, lddo, d, dt));
    if (J->gate != POET_GATE_NONE) {
      POET_TRY(check_rows(what, "gate", gate, ldg, gate_width, dt));
      if (dgate) POET_TRY(check_rows(what, "dgate", dgate, lddg, gate_width, dt));
    } else {
      POET_REQUIRE(!gate && !dgate, "%s: a gate was passed to a joint without one", what);
    }
  } else {
    POET_REQUIRE(!d_o && !gate && !dgate, "%s: without o, d_o, gate and dgate must be NULL", what);
  }
  const size_t need = poet_joint_workspace_bytes(J, T);
  if (!ws || ws_bytes < need || (reinterpret_cast<uintptr_t>(ws) & 255) != 0) {
    set_error("%s: workspace %zu bytes, need %zu (256-byte aligned)", what, ws_bytes, need);
    return POET_ENOMEM_WS;
  }
  JointBwdArgs a{};
  a.o = o; a.hp = h_out; a.gate = gate; a.dhp = dh_out; a.dn = dn;
  a.dh = dh; a.d_o = d_o; a.dgate = dgate;
  a.ldo = ldo; a.ldhp = ldho; a.ldg = ldg; a.lddhp = lddho; a.lddn = lddn; a.lddh = lddh; a.lddo = lddo; a.lddg = lddg;
  a.w_post = J->w_post; a.w_pre = J->w_pre;
  a.T = T; a.gate_rows = J->gate_rows; a.d = d;
  a.post = J->post_norm;
  a.gate_kind = o ? J->gate : int(POET_GATE_NONE);
  a.gate_sigmoid = a.gate_kind != POET_GATE_NONE && J->gate_act == POET_GATE_SIGMOID;
  a.alpha = J->alpha; a.beta = J->beta; a.eps = J->eps;
  const bool channel = a.gate_kind == POET_GATE_CHANNEL;
  const int vw = 16 / int(esize(dt));
  const bool vec = d % vw == 0 && rows16(o, ldo, dt) && rows16(dn ? h_out : nullptr, ldho, dt) &&
                   rows16(dh_out, lddho, dt) && rows16(dn, lddn, dt) && rows16(dh, lddh, dt) && rows16(d_o, lddo, dt) &&
                   (!channel || (rows16(gate, ldg, dt) && rows16(dgate, lddg, dt)));
  const RowShape s = row_shape(d, vec ? vw : 1, vec ? 1 : 8);
  a.tpr = s.tpr;
  const BwdPlan p = bwd_plan(J, T, bwd_most(T, s.tpr));
  a.seg_rows = p.seg_rows; a.chunks = p.chunks; a.segs_per_group = p.segs_per_group;
  const size_t part = align256(size_t(p.groups) * d * 4);
  char *wb = static_cast<char *>(ws);
  a.part_post = dw_post ? reinterpret_cast<float *>(wb) : nullptr;
  a.part_pre = dw_pre ? reinterpret_cast<float *>(wb + part) : nullptr;
  a.part_gate = reinterpret_cast<float *>(wb + 2 * part);
  const int64_t G = (T + J->gate_rows - 1) / J->gate_rows;
  const double gate_elems = channel ? 2.0 * double(G) * d : a.gate_kind == POET_GATE_ROW ? 2.0 * double(G) : 0.0;
  const int passes = 1 + (o ? 2 : 0) + (dn ? 2 : 0) + (dh_out ? 1 : 0);
  TraceScope ts("joint_bwd", 30.0 * double(T) * d, (double(T) * d * passes + gate_elems) * double(esize(dt)), st);
  poet_status rc;
  if (dt == POET_BF16) {
    if (vec) rc = s.nv == 1 ? launch_bwd<bf16, 8, 1>(a, s, p.groups, st) : launch_bwd<bf16, 8, 2>(a, s, p.groups, st);
    else rc = s.nv == 8 ? launch_bwd<bf16, 1, 8>(a, s, p.groups, st) : launch_bwd<bf16, 1, 16>(a, s, p.groups, st);
  } else if (vec) {
    rc = s.nv == 1   ? launch_bwd<float, 4, 1>(a, s, p.groups, st)
         : s.nv == 2 ? launch_bwd<float, 4, 2>(a, s, p.groups, st)
                     : launch_bwd<float, 4, 4>(a, s, p.groups, st);
  } else {
    rc = s.nv == 8 ? launch_bwd<float, 1, 8>(a, s, p.groups, st) : launch_bwd<float, 1, 16>(a, s, p.groups, st);
  }
  POET_TRY(rc);
  const bool sum_gate = dgate && J->gate_rows > 1 && p.chunks > 1;
  if (!dw_post && !dw_pre && !sum_gate) return POET_OK;
  JointSumArgs u{};
  u.part_post = a.part_post; u.part_pre = a.part_pre; u.part_gate = a.part_gate;
  u.dw_post = dw_post; u.dw_pre = dw_pre; u.dgate = dgate; u.lddg = lddg;
  u.groups = p.groups; u.chunks = p.chunks; u.d = d; u.gate_width = gate_width;
  const dim3 grid(unsigned((d + 31) / 32), unsigned(2 + (sum_gate ? p.segs : 0))), block(32, SUM_LANES);
  if (dt == POET_BF16) joint_sum_kernel<bf16><<<grid, block, 0, st>>>(u);
  else joint_sum_kernel<float><<<grid, block, 0, st>>>(u);
  count_launch();
  return launch_status("joint_bwd");
}

}  // extern "C"
