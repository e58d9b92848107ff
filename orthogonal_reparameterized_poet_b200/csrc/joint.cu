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
// The forward reads o and h and writes h' and n, the backward reads o, h', dh'
// and dn and writes dh and do, each once: what it cannot do without is the HBM
// traffic.  A group of threads shares a row (one 16-byte vector of each operand a
// thread) and works through a contiguous range of rows, so that gains, a gate
// that rows share and the column sums of the backward stay with the thread.  The
// rows to come are copied into shared memory ahead (Ring), the arithmetic is two
// floats an instruction, and a row's sums go through one exchange, together with
// the first sums of the next row.  The sums of squares are taken again in the
// backward from the rows it reads anyway, which costs no traffic and saves a
// buffer.
//
// Measured (bf16, on the GPU): forward of 32768 x 2048 92 us, 5.8 TB/s of a copy's
// 6.56; backward 193 us of 805 MB, of 16384 x 2560 with a gate each 145 us of 671
// MB (a call among others 92 to 96 and 145 to 150).  What bounds the backward is
// latency: no unit is saturated (issue slots 60 %, DRAM 47 %), a warp has about 500
// instructions for its 256 elements of a row, and registers and shared memory leave
// room for two rows an SM at once.  Tried and slower: three CTAs an SM (spills, 276
// us), the gains in registers with 320 threads (spills, 324 us against 164).
#include <cmath>

#include "rows.cuh"

namespace poet {
namespace {

constexpr int MAX_D = 16384;

// How the kernels are specialized by the gate: none or one value per row, a
// channel gate of every row's own, a channel gate shared by rows.
enum { GK_ROW = 0, GK_EACH = 1, GK_SHARED = 2 };

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

// The sigmoid is r = 1 / (1 + e) with e = exp(-g), its slope e r^2: r (1 - r)
// would lose its digits as the gate opens (r rounds to 1 from g = 17 on).  The
// reciprocal is the hardware's, off by a unit in the last place.  So is the
// exponential for bf16 operands: its relative error, about 2^-23 (2 + |g|), stays
// below the rounding of a bf16 result, 2^-9, for every gate whose slope is not 0
// in float.  For float operands it is CUDA's function, off by two units at most.
template <typename T>
__device__ __forceinline__ float exp_minus(float g) {
  if constexpr (sizeof(T) == 4) return expf(-g);
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
  return e;
}
__device__ __forceinline__ float sigmoid_of(float e) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return r;
}
template <typename T>
__device__ __forceinline__ float2 exp_minus(float2 g) {
  return make_float2(exp_minus<T>(g.x), exp_minus<T>(g.y));
}
__device__ __forceinline__ float2 sigmoid_of(float2 e) { return make_float2(sigmoid_of(e.x), sigmoid_of(e.y)); }
// e r is 1 - r, between 0 and 1; infinity times 0, of a closed gate, saturates to
// 0 (a NaN's slope is still one: r is).
__device__ __forceinline__ float2 slope_of(float2 e, float2 r) {
  return mul2(make_float2(__saturatef(e.x * r.x), __saturatef(e.y * r.y)), r);
}
template <typename T>
__device__ __forceinline__ float act_of(float g, int sig) {
  return sig ? sigmoid_of(exp_minus<T>(g)) : g;
}

// A thread's own ring of the rows to come.  With S stages every thread copies
// its 16 bytes of each operand of row r + S - 1 into its own place in shared
// memory (cp.async) while it works on row r, and only it reads them: no barrier
// is needed and S - 1 rows are in flight without holding registers.  S = 0:
// rows are read when they are needed, the next one ahead in registers.
template <int S, int NV>
struct Ring {
  uint32_t base;
  int stride, stage;  // bytes from one vector of a thread to its next, of one stage
  __device__ __forceinline__ void init(int operands) {
    extern __shared__ __align__(16) unsigned char joint_smem[];
    base = uint32_t(__cvta_generic_to_shared(joint_smem)) + threadIdx.x * 16;
    stride = blockDim.x * 16;
    stage = stride * NV * operands;
  }
  // The places of a thread beyond the row's end hold zeros.
  __device__ __forceinline__ void zero(int stages) const {
    for (uint32_t p = base; p < base + stages * stage; p += stride)
      asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(p), "r"(0) : "memory");
  }
  __device__ __forceinline__ uint32_t at(int s, int operand, int j) const {
    return base + s * stage + (operand * NV + j) * stride;
  }
  static __device__ __forceinline__ void copy(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  }
  static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  static __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(S >= 2 ? S - 2 : 0) : "memory"); }
  template <typename V>
  static __device__ __forceinline__ void read(V &v, uint32_t src) {
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(src));
    if constexpr (sizeof(V) == 16) v = *reinterpret_cast<const V *>(&r);
  }
};

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

// The elements of a row that a thread holds, as read: NV vectors of VW
// elements, tpr vectors apart, zero beyond the row's end (where nothing is ever
// loaded).  Their values come in pairs: the arithmetic is two floats an
// instruction, because the kernels issue close to one instruction a cycle.
template <typename T, int VW, int NV>
struct Lane {
  static constexpr int N = VW * NV, NP = N / 2;
  RowVec<T, VW> v[NV];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < NV; ++j) v[j] = RowVec<T, VW>{};
  }
  __device__ __forceinline__ void get(float2 (&x)[NP]) const {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float f[VW];
      v[j].get(f);
#pragma unroll
      for (int e = 0; e < VW; ++e) (((j * VW + e) & 1) ? x[(j * VW + e) / 2].y : x[(j * VW + e) / 2].x) = f[e];
    }
  }
  static __device__ __forceinline__ void put(T *row, int tid, int tpr, int d, const float2 (&x)[NP]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (tid + j * tpr) * VW;
      float f[VW];
#pragma unroll
      for (int e = 0; e < VW; ++e) f[e] = ((j * VW + e) & 1) ? x[(j * VW + e) / 2].y : x[(j * VW + e) / 2].x;
      if (c < d) RowVec<T, VW>::store(row + c, f);
    }
  }
};

// The same elements of a float vector of the row's width: gains, column sums.
template <int VW, int NV>
__device__ __forceinline__ void gains(float2 (&w)[VW * NV / 2], const float *p, int tid, int tpr, int d) {
#pragma unroll
  for (int i = 0; i < VW * NV; ++i) {
    const int c = (tid + i / VW * tpr) * VW + i % VW;
    const float f = p && c < d ? p[c] : 1.f;
    ((i & 1) ? w[i / 2].y : w[i / 2].x) = f;
  }
}
// The gains in the backward: of the ring's variants in shared memory, behind the
// ring, every thread's own (no barrier), because the column sums need the
// registers; of the others in registers.
template <int VW, int NV, bool SMEM>
struct Gains {
  static constexpr int NP = VW * NV / 2;
  float2 w[SMEM ? 1 : NP];
  uint32_t at;
  __device__ __forceinline__ void init(const float *p, uint32_t base, int tid, int tpr, int d) {
    if constexpr (SMEM) {
      float2 f[NP];
      gains<VW, NV>(f, p, tid, tpr, d);
      at = base + threadIdx.x * 16;
#pragma unroll
      for (int i = 0; i < NP; i += 2)
        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at + i / 2 * blockDim.x * 16), "f"(f[i].x),
                     "f"(f[i].y), "f"(f[i + 1].x), "f"(f[i + 1].y)
                     : "memory");
    } else {
      gains<VW, NV>(w, p, tid, tpr, d);
    }
  }
  __device__ __forceinline__ void get(float2 (&f)[NP]) const {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      if constexpr (SMEM) {
        if (i % 2 == 0)
          asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(f[i].x), "=f"(f[i].y), "=f"(f[i + 1].x), "=f"(f[i + 1].y)
                       : "r"(at + i / 2 * blockDim.x * 16));
      } else {
        f[i] = w[i];
      }
    }
  }
};
template <int VW, int NV>
__device__ __forceinline__ void put_floats(float *p, int tid, int tpr, int d, const float2 (&x)[VW * NV / 2]) {
#pragma unroll
  for (int i = 0; i < VW * NV; ++i) {
    const int c = (tid + i / VW * tpr) * VW + i % VW;
    if (c < d) p[c] = (i & 1) ? x[i / 2].y : x[i / 2].x;
  }
}

__device__ __forceinline__ void zero_slots(float *p, int n) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) p[i] = 0.f;
  __syncthreads();
}

template <typename T, int VW, int NV, int S, int GK, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) joint_fwd_kernel(const JointFwdArgs a) {
  __shared__ __align__(16) float red[8][2][2 * 32];
  zero_slots(red[0][0], 8 * 2 * 2 * 32);
  const Group g(a.tpr);
  using L = Lane<T, VW, NV>;
  constexpr int NP = L::NP;
  const T *o = static_cast<const T *>(a.o), *h = static_cast<const T *>(a.h), *gate = static_cast<const T *>(a.gate);
  T *ho = static_cast<T *>(a.h_out), *n = static_cast<T *>(a.n);
  const int64_t r0 = g.id * a.rows_per_group;
  const int64_t r1 = r0 + a.rows_per_group < a.T ? r0 + a.rows_per_group : a.T;
  if (r0 >= r1) return;
  constexpr bool EACH = GK == GK_EACH, SHARED = GK == GK_SHARED;
  float *slot = red[g.bar - 1][0], *other = red[g.bar - 1][1];
  L vo, vh, vg;
  vo.clear();
  vh.clear();
  vg.clear();
  Ring<S, NV> ring;
  if (S) {
    ring.init(1 + (o ? 1 : 0) + (EACH ? 1 : 0));
    if (g.tid * VW >= a.d) ring.zero(S);
  }
  // the rows' addresses advance a row at a time: those to load, those to write
  const int c0 = g.tid * VW;
  const T *lh = h + r0 * a.ldh + c0, *lo = o + r0 * a.ldo + c0, *lg = EACH ? gate + r0 * a.ldg + c0 : nullptr;
  T *sh = ho + r0 * a.ldho, *sn = n + r0 * a.ldn;
  auto load = [&](int64_t r, int st) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int step = j * a.tpr * VW;
      if (c0 + step < a.d && r < r1) {
        if constexpr (S > 0) {
          ring.copy(ring.at(st, 0, j), lh + step);
          if (o) ring.copy(ring.at(st, 1, j), lo + step);
          if (EACH) ring.copy(ring.at(st, 2, j), lg + step);
        } else {
          vh.v[j].load(lh + step);
          if (o) vo.v[j].load(lo + step);
          if (EACH) vg.v[j].load(lg + step);
        }
      }
    }
    lh += a.ldh;
    lo += a.ldo;
    if (EACH) lg += a.ldg;
    if constexpr (S > 0) ring.commit();
  };
  int st = 0;
  if constexpr (S > 0) {
#pragma unroll
    for (int k = 0; k < S - 1; ++k) load(r0 + k, k);
  } else {
    load(r0, 0);
  }
  // beta w_post, times a gate that rows share
  float2 wq[NP], wn[NP];
  gains<VW, NV>(wn, a.w_pre, g.tid, a.tpr, a.d);
  auto branch_gains = [&]() {
    gains<VW, NV>(wq, a.w_post, g.tid, a.tpr, a.d);
#pragma unroll
    for (int p = 0; p < NP; ++p) wq[p] = mul2(wq[p], both(a.beta));
  };
  branch_gains();
  int64_t grow = r0 / a.gate_rows, gnext = a.gate_kind != POET_GATE_NONE && !EACH ? r0 : a.T;
  float gval = 1.f;
  const float inv_d = 1.f / float(a.d);
  const float2 alpha = both(a.alpha);
  const bool post = o && a.post;
  auto read = [&](L &v, int stage, int place) {
    if constexpr (S > 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j) ring.read(v.v[j], ring.at(stage, place, j));
    }
  };
  // One exchange a row: the sum over row r's new stream together with the one
  // over row r + 1's branch (both wait for all the row's threads).
  float2 s2 = both(0.f);
  float s[2] = {0.f, 0.f};
  auto branch_sum = [&](int stage) {
    float2 q[NP];
    read(vo, stage, 1);
    vo.get(q);
    s2 = both(0.f);
#pragma unroll
    for (int p = 0; p < NP; ++p) s2 = fma2(q[p], q[p], s2);
    s[0] = s2.x + s2.y;
  };
  auto exchange = [&]() {
    row_sum_2(s, slot, g.warps, g.warp, g.bar, a.tpr);
    float *const was = slot;
    slot = other;
    other = was;
  };
  if constexpr (S > 0) ring.wait();
  if (post) {
    branch_sum(0);
    exchange();
  }
  for (int64_t r = r0; r < r1; ++r) {
    if (r == gnext) {  // the next gate row
      if (r != r0) ++grow;
      gnext = (grow + 1) * a.gate_rows;
      if (!SHARED) {
        gval = act_of<T>(to_float(gate[grow * a.ldg]), a.gate_sigmoid);
      } else {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int c = (g.tid + j * a.tpr) * VW;
          if (c < a.d) vg.v[j].load(gate + grow * a.ldg + c);
        }
        float2 gv[NP];
        vg.get(gv);
        branch_gains();
#pragma unroll
        for (int p = 0; p < NP; ++p)
          wq[p] = mul2(wq[p], make_float2(act_of<T>(gv[p].x, a.gate_sigmoid), act_of<T>(gv[p].y, a.gate_sigmoid)));
      }
    }
    float2 x[NP];
    read(vh, st, 0);
    vh.get(x);
    if (o) {
      float2 q[NP];
      read(vo, st, 1);
      vo.get(q);
      const float ro = post ? gval * inv_sqrt(fmaf(s[0], inv_d, a.eps)) : gval;
      if (EACH) {
        float2 gv[NP];
        read(vg, st, 2);
        vg.get(gv);
        if (a.gate_sigmoid) {
#pragma unroll
          for (int p = 0; p < NP; ++p) gv[p] = sigmoid_of(exp_minus<T>(gv[p]));
        }
#pragma unroll
        for (int p = 0; p < NP; ++p) q[p] = mul2(q[p], gv[p]);
      }
#pragma unroll
      for (int p = 0; p < NP; ++p) x[p] = fma2(mul2(q[p], both(ro)), wq[p], mul2(x[p], alpha));
      L::put(sh, g.tid, a.tpr, a.d, x);
      sh += a.ldho;
    }
    if constexpr (S > 0) {
      load(r + S - 1, st == 0 ? S - 1 : st - 1);
      st = st + 1 == S ? 0 : st + 1;
      ring.wait();  // row r + 1 is there
    } else {
      load(r + 1, 0);
    }
    if (!n && !post) continue;
    s2 = both(0.f);
#pragma unroll
    for (int p = 0; p < NP; ++p) s2 = fma2(x[p], x[p], s2);
    s[1] = s2.x + s2.y;
    s[0] = 0.f;
    if (post) branch_sum(st);  // behind the last row: of what is there, not used
    exchange();
    if (n) {
      const float2 rn = both(inv_sqrt(fmaf(s[1], inv_d, a.eps)));
#pragma unroll
      for (int p = 0; p < NP; ++p) x[p] = mul2(mul2(x[p], rn), wn[p]);
      L::put(sn, g.tid, a.tpr, a.d, x);
      sn += a.ldn;
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

template <typename T, int VW, int NV, int S, int GK, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) joint_bwd_kernel(const JointBwdArgs a) {
  __shared__ __align__(16) float red[8][2][5 * 32];
  zero_slots(red[0][0], 8 * 2 * 5 * 32);
  const Group g(a.tpr);
  using L = Lane<T, VW, NV>;
  constexpr int NP = L::NP;
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
  constexpr bool EACH = GK == GK_EACH, SHARED = GK == GK_SHARED;
  const bool shared_gate = dgate && a.gate_rows > 1;
  float *slot = red[g.bar - 1][0], *other = red[g.bar - 1][1];
  float2 aq[NP], an[NP], ag[NP];  // column sums
  float ag_row = 0.f;
#pragma unroll
  for (int p = 0; p < NP; ++p) aq[p] = an[p] = ag[p] = both(0.f);
  const float inv_d = 1.f / float(a.d);
  const float2 alpha = both(o ? a.alpha : 1.f), beta = both(a.beta);
  L vo, vh, vd, vn, vg;
  vo.clear();
  vh.clear();
  vd.clear();
  vn.clear();
  vg.clear();
  const int sd = dn ? 2 : 0, so = sd + (dhp ? 1 : 0), sg = so + (o ? 1 : 0);  // places in the ring: h', dn first
  Ring<S, NV> ring;
  constexpr bool GR = EACH && S > 2;  // a gate of the row's own in the ring; with two stages there is no room for it
  if (S) {
    ring.init(sg + (GR ? 1 : 0));
    if (g.tid * VW >= a.d) ring.zero(S);
  }
  auto load = [&](int64_t r, int st) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (g.tid + j * a.tpr) * VW;
      if (c < a.d && r < r1) {
        if constexpr (S > 0) {
          if (dn) {
            ring.copy(ring.at(st, 0, j), hp + r * a.ldhp + c);
            ring.copy(ring.at(st, 1, j), dn + r * a.lddn + c);
          }
          if (dhp) ring.copy(ring.at(st, sd, j), dhp + r * a.lddhp + c);
          if (o) ring.copy(ring.at(st, so, j), o + r * a.ldo + c);
          if (GR) ring.copy(ring.at(st, sg, j), gate + r * a.ldg + c);
        } else {
          if (dn) {
            vh.v[j].load(hp + r * a.ldhp + c);
            vn.v[j].load(dn + r * a.lddn + c);
          }
          if (dhp) vd.v[j].load(dhp + r * a.lddhp + c);
          if (o) vo.v[j].load(o + r * a.ldo + c);
          if (EACH) vg.v[j].load(gate + r * a.ldg + c);
        }
      }
    }
    if constexpr (S > 0) ring.commit();
  };
  int st = 0;
  if constexpr (S > 0) {
#pragma unroll
    for (int k = 0; k < S - 1; ++k) load(r0 + k, k);
  } else {
    load(r0, 0);
  }
  Gains<VW, NV, (S > 0)> gq, gn;
  const uint32_t gains_at = ring.base - threadIdx.x * 16 + S * ring.stage;
  gq.init(a.w_post, gains_at, g.tid, a.tpr, a.d);
  gn.init(a.w_pre, gains_at + blockDim.x * VW * NV * 4, g.tid, a.tpr, a.d);
  // The gradient of the gate row in registers: to the result, or (where several
  // groups share the row) to this group's partial sums.
  int64_t grow = r0 / a.gate_rows;
  auto flush_gate = [&]() {
    if (EACH || !shared_gate) return;
    const bool part = a.chunks > 1;
    if (!SHARED) {
      if (g.tid == 0) {
        if (part) a.part_gate[g.id] = ag_row;
        else dgate[grow * a.lddg] = from_float<T>(ag_row);
      }
      ag_row = 0.f;
      return;
    }
    if (part) put_floats<VW, NV>(a.part_gate + g.id * a.d, g.tid, a.tpr, a.d, ag);
    else L::put(dgate + grow * a.lddg, g.tid, a.tpr, a.d, ag);
#pragma unroll
    for (int p = 0; p < NP; ++p) ag[p] = both(0.f);
  };
  auto fetch = [&](L &v, int place) {
    if constexpr (S > 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j) ring.read(v.v[j], ring.at(st, place, j));
    }
  };
  // The first sums of the row in stage st: h'^2, u h', o^2.  Each row's operands
  // are read from the ring twice, for its sums and for what follows from them,
  // rather than held in registers across the exchange.
  float s[5] = {0.f, 0.f, 0.f, 0.f, 0.f};
  auto first_sums = [&]() {
    if (dn) {
      float2 x[NP], y[NP], wn[NP], s0 = both(0.f), s1 = both(0.f);
      fetch(vh, 0);
      fetch(vn, 1);
      vh.get(x);
      vn.get(y);
      gn.get(wn);
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        s0 = fma2(x[p], x[p], s0);
        s1 = fma2(mul2(y[p], wn[p]), x[p], s1);
      }
      s[0] = s0.x + s0.y;
      s[1] = s1.x + s1.y;
    }
    if (o && a.post) {
      float2 x[NP], s2 = both(0.f);
      fetch(vo, so);
      vo.get(x);
#pragma unroll
      for (int p = 0; p < NP; ++p) s2 = fma2(x[p], x[p], s2);
      s[2] = s2.x + s2.y;
    }
  };
  // One exchange a row: the sums that row r's branch gradient needs (v ph, and
  // that of a row gate's gradient before its slope) with the first ones of row r + 1.
  const bool fifth = GK == GK_ROW && dgate;
  auto exchange = [&]() {
    row_sum_5(s, fifth, slot, g.warps, g.warp, g.bar, a.tpr);
    float *const was = slot;
    slot = other;
    other = was;
  };
  if constexpr (S > 0) ring.wait();
  if (r0 < r1) first_sums();
  exchange();
  float ga_row = 1.f, sl_row = 1.f;  // a row gate's value and slope
  int64_t gnext = a.gate_kind != POET_GATE_NONE && !EACH ? r0 : a.T;
  for (int64_t r = r0; r < r1; ++r) {
    if (r == gnext) {  // the next gate row
      if (r != r0) {
        flush_gate();
        ++grow;
      }
      gnext = (grow + 1) * a.gate_rows;
      if (!SHARED) {
        ga_row = to_float(gate[grow * a.ldg]);
        if (a.gate_sigmoid) {
          const float2 e = both(exp_minus<T>(ga_row)), r = both(sigmoid_of(e.x));
          ga_row = r.x;
          sl_row = slope_of(e, r).x;
        }
      } else {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int c = (g.tid + j * a.tpr) * VW;
          if (c < a.d) vg.v[j].load(gate + grow * a.ldg + c);
        }
      }
    }
    const float rn = inv_sqrt(fmaf(s[0], inv_d, a.eps)), mn = s[1] * rn * inv_d;  // 1 / r', mean(u nh)
    const float ro = a.post ? inv_sqrt(fmaf(s[2], inv_d, a.eps)) : 1.f;           // 1 / r
    if (EACH && S > 0 && !GR) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (g.tid + j * a.tpr) * VW;
        if (c < a.d) vg.v[j].load(gate + r * a.ldg + c);
      }
    }
    float2 t[NP], q[NP];  // t, then v; ph
    if (dhp) {
      fetch(vd, sd);
      vd.get(t);
    } else {
#pragma unroll
      for (int p = 0; p < NP; ++p) t[p] = both(0.f);
    }
    if (dn) {
      float2 x[NP], y[NP], wn[NP];
      fetch(vh, 0);
      fetch(vn, 1);
      vh.get(x);
      vn.get(y);
      gn.get(wn);
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const float2 nh = mul2(x[p], both(rn));
        an[p] = fma2(y[p], nh, an[p]);
        t[p] = fma2(mul2(y[p], wn[p]), both(rn), t[p]);
        t[p] = fma2(nh, both(-mn * rn), t[p]);
      }
    }
    {
      float2 out[NP];
#pragma unroll
      for (int p = 0; p < NP; ++p) out[p] = mul2(t[p], alpha);
      L::put(dh + r * a.lddh, g.tid, a.tpr, a.d, out);
    }
    s[3] = s[4] = 0.f;
    if (o) {
      float2 w0 = both(0.f), w1 = both(0.f), dg[NP], wq[NP];
      fetch(vo, so);
      if (GR) fetch(vg, sg);
      vo.get(q);
      if (EACH || SHARED) vg.get(dg);
      gq.get(wq);
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        float2 ga = both(ga_row), sl = both(1.f);
        if (EACH || SHARED) {
          ga = dg[p];
          if (a.gate_sigmoid) {
            const float2 e = exp_minus<T>(ga);
            ga = sigmoid_of(e);
            sl = slope_of(e, ga);
          }
        }
        const float2 da = mul2(t[p], beta), dp = mul2(da, ga);
        q[p] = mul2(q[p], both(ro));
        const float2 z = mul2(q[p], wq[p]);
        aq[p] = fma2(dp, q[p], aq[p]);
        t[p] = mul2(dp, wq[p]);
        w0 = fma2(dp, z, w0);
        if (EACH || SHARED) {
          dg[p] = mul2(da, z);
          if (a.gate_sigmoid) dg[p] = mul2(dg[p], sl);
          if (SHARED) ag[p] = add2(ag[p], dg[p]);
        } else {
          w1 = fma2(da, z, w1);
        }
      }
      if (EACH && dgate) L::put(dgate + r * a.lddg, g.tid, a.tpr, a.d, dg);
      s[3] = w0.x + w0.y;
      s[4] = w1.x + w1.y;
    }
    if constexpr (S > 0) {
      load(r + S - 1, st == 0 ? S - 1 : st - 1);
      st = st + 1 == S ? 0 : st + 1;
      ring.wait();  // row r + 1 is there
    } else {
      load(r + 1, 0);
    }
    first_sums();  // behind the last row: of what is there, not used
    exchange();
    if (!o) continue;
    if (a.post) {
      const float2 mo = both(-s[3] * inv_d);  // -mean(v ph)
#pragma unroll
      for (int p = 0; p < NP; ++p) t[p] = mul2(fma2(q[p], mo, t[p]), both(ro));
    }
    L::put(d_o + r * a.lddo, g.tid, a.tpr, a.d, t);
    if (!EACH && !SHARED && dgate) {
      if (a.gate_rows == 1) {
        if (g.tid == 0) dgate[r * a.lddg] = from_float<T>(s[4] * sl_row);
      } else {
        ag_row += s[4] * sl_row;
      }
    }
  }
  flush_gate();
  if (a.part_post) put_floats<VW, NV>(a.part_post + g.id * a.d, g.tid, a.tpr, a.d, aq);
  if (a.part_pre) put_floats<VW, NV>(a.part_pre + g.id * a.d, g.tid, a.tpr, a.d, an);
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
  if (col < width) {
    constexpr int AHEAD = 8;  // loads in flight
    const int64_t stride = int64_t(SUM_LANES) * width;
    const float *p = src + int64_t(threadIdx.y) * width + col;
    int left = int((count - threadIdx.y + SUM_LANES - 1) / SUM_LANES);
    for (; left >= AHEAD; left -= AHEAD, p += AHEAD * stride) {
      float v[AHEAD];
#pragma unroll
      for (int q = 0; q < AHEAD; ++q) v[q] = p[q * stride];
#pragma unroll
      for (int q = 0; q < AHEAD; ++q) s += v[q];
    }
    for (; left > 0; --left, p += stride) s += *p;
  }
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

// CTAs that an SM holds (what the kernels' launch bounds ask for: 80 registers a
// thread in the forward up to 256 threads).
int fwd_resident(int threads) { return threads <= 256 ? 65536 / (80 * threads) : 1; }
int bwd_resident(int threads) { return threads <= 320 ? 2 : 1; }

// Most groups of rows in the backward: what runs at once, and at least four rows
// each (a group's partial sums cost as much as a row).
int64_t bwd_most(int64_t T, const RowShape &s) {
  const int64_t fill = int64_t(num_sms()) * bwd_resident(s.threads) * s.groups_per_cta;
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

template <auto KERN, typename A>
poet_status launch_joint(const A &a, const RowShape &s, int64_t groups, size_t smem, cudaStream_t st, const char *what) {
  const unsigned grid = unsigned((groups + s.groups_per_cta - 1) / s.groups_per_cta);
  POET_TRY(allow_smem<KERN>(smem));
  KERN<<<grid, s.threads, smem, st>>>(a);
  count_launch();
  return launch_status(what);
}

// Rows of one 16-byte vector per thread go through the ring: four stages up to
// 512 threads (three in the backward with 257 to 320, where two CTAs share an
// SM); up to 1024, where four would not fit, three in the forward and two in the
// backward, which has more operands.  Wider rows, and rows that do not start on 16
// bytes, are read directly.  Measured (us on the GPU, 256 MB an operand, no gate;
// floors 164 and 245):
//   forward of 2560 bf16 (320 threads): four stages 264, two CTAs of two 322, direct 483
//           of 4096 bf16 209, 267, 384; of 2048 float 191, 236, 376
//           of 5120 bf16 (640 threads): three stages 231, two 369, direct 396
//           of 8192 bf16 243, 336, 379; of 4096 float 195, 318, 317
//   backward of 4096 bf16: four stages 405, two 567, direct 515; of 2048 float 314, 482, 453
//           of 5120 bf16: two stages 743, direct 902; of 8192 771, 772 (a gate each: 1245, 1046)
//           of 4096 float 569, 665
template <typename T, int VW, int GK>
poet_status launch_fwd(const JointFwdArgs &a, const RowShape &s, int64_t groups, int operands, cudaStream_t st) {
  const size_t stage = size_t(s.threads) * 16 * operands;
  if (s.nv == 1) {
    if (s.threads <= 256) return launch_joint<joint_fwd_kernel<T, VW, 1, 4, GK, 256, 3>>(a, s, groups, 4 * stage, st, "joint");
    if (s.threads <= 512) return launch_joint<joint_fwd_kernel<T, VW, 1, 4, GK, 512, 1>>(a, s, groups, 4 * stage, st, "joint");
    return launch_joint<joint_fwd_kernel<T, VW, 1, 3, GK, 1024, 1>>(a, s, groups, 3 * stage, st, "joint");
  }
  if (s.nv == 2) return launch_joint<joint_fwd_kernel<T, VW, 2, 0, GK, 1024, 1>>(a, s, groups, 0, st, "joint");
  return launch_joint<joint_fwd_kernel<T, VW, 4, 0, GK, 1024, 1>>(a, s, groups, 0, st, "joint");
}
template <typename T, int GK>
poet_status launch_fwd_scalar(const JointFwdArgs &a, const RowShape &s, int64_t groups, cudaStream_t st) {
  if (s.nv == 8) {
    if (s.threads <= 256) return launch_joint<joint_fwd_kernel<T, 1, 8, 0, GK, 256, 3>>(a, s, groups, 0, st, "joint");
    return launch_joint<joint_fwd_kernel<T, 1, 8, 0, GK, 1024, 1>>(a, s, groups, 0, st, "joint");
  }
  return launch_joint<joint_fwd_kernel<T, 1, 16, 0, GK, 1024, 1>>(a, s, groups, 0, st, "joint");
}

template <typename T, int VW, int GK>
poet_status launch_bwd(const JointBwdArgs &a, const RowShape &s, int64_t groups, int operands, cudaStream_t st) {
  const size_t stage = size_t(s.threads) * 16, gains = size_t(s.threads) * VW * 8;
  const int each = GK == GK_EACH ? 1 : 0;  // with two stages the gate is not in the ring
  const size_t four = 4 * stage * (operands + each) + gains, two = 2 * stage * operands + gains;
  if (s.nv == 1) {
    if (s.threads <= 256)
      return launch_joint<joint_bwd_kernel<T, VW, 1, 4, GK, 256, 2>>(a, s, groups, four, st, "joint_bwd");
    if (s.threads <= 320)
      return launch_joint<joint_bwd_kernel<T, VW, 1, 3, GK, 320, 2>>(a, s, groups, four - stage * (operands + each), st,
                          "joint_bwd");
    if (s.threads <= 512)
      return launch_joint<joint_bwd_kernel<T, VW, 1, 4, GK, 512, 1>>(a, s, groups, four, st, "joint_bwd");
    return launch_joint<joint_bwd_kernel<T, VW, 1, 2, GK, 1024, 1>>(a, s, groups, two, st, "joint_bwd");
  }
  if (s.nv == 2) return launch_joint<joint_bwd_kernel<T, VW, 2, 0, GK, 1024, 1>>(a, s, groups, 0, st, "joint_bwd");
  return launch_joint<joint_bwd_kernel<T, VW, 4, 0, GK, 1024, 1>>(a, s, groups, 0, st, "joint_bwd");
}
template <typename T, int GK>
poet_status launch_bwd_scalar(const JointBwdArgs &a, const RowShape &s, int64_t groups, cudaStream_t st) {
  if (s.nv == 8) {
    if (s.threads <= 256) return launch_joint<joint_bwd_kernel<T, 1, 8, 0, GK, 256, 2>>(a, s, groups, 0, st, "joint_bwd");
    return launch_joint<joint_bwd_kernel<T, 1, 8, 0, GK, 1024, 1>>(a, s, groups, 0, st, "joint_bwd");
  }
  return launch_joint<joint_bwd_kernel<T, 1, 16, 0, GK, 1024, 1>>(a, s, groups, 0, st, "joint_bwd");
}

template <int GK>
poet_status pick_fwd(const JointFwdArgs &a, const RowShape &s, int64_t groups, int operands, int dt, bool vec,
                     cudaStream_t st) {
  if (dt == POET_BF16)
    return vec ? launch_fwd<bf16, 8, GK>(a, s, groups, operands, st) : launch_fwd_scalar<bf16, GK>(a, s, groups, st);
  return vec ? launch_fwd<float, 4, GK>(a, s, groups, operands, st) : launch_fwd_scalar<float, GK>(a, s, groups, st);
}
template <int GK>
poet_status pick_bwd(const JointBwdArgs &a, const RowShape &s, int64_t groups, int operands, int dt, bool vec,
                     cudaStream_t st) {
  if (dt == POET_BF16)
    return vec ? launch_bwd<bf16, 8, GK>(a, s, groups, operands, st) : launch_bwd_scalar<bf16, GK>(a, s, groups, st);
  return vec ? launch_bwd<float, 4, GK>(a, s, groups, operands, st) : launch_bwd_scalar<float, GK>(a, s, groups, st);
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
  const int64_t fill = int64_t(num_sms()) * fwd_resident(s.threads) * s.groups_per_cta;
  a.rows_per_group = (T + fill - 1) / fill;
  const int64_t groups = (T + a.rows_per_group - 1) / a.rows_per_group;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int64_t G = T / J->gate_rows + (T % J->gate_rows ? 1 : 0);
  const double gate_elems = a.gate_kind == POET_GATE_CHANNEL ? double(G) * d : a.gate_kind == POET_GATE_ROW ? double(G) : 0.0;
  TraceScope ts("joint", 14.0 * double(T) * d,
                (double(T) * d * ((o ? 3 : 1) + (n ? 1 : 0)) + gate_elems) * double(esize(dt)), st);
  const bool channel = a.gate_kind == POET_GATE_CHANNEL;
  const int operands = 1 + (o ? 1 : 0) + (channel && J->gate_rows == 1 ? 1 : 0);
  if (!channel) return pick_fwd<GK_ROW>(a, s, groups, operands, dt, vec, st);
  return J->gate_rows == 1 ? pick_fwd<GK_EACH>(a, s, groups, operands, dt, vec, st)
                           : pick_fwd<GK_SHARED>(a, s, groups, operands, dt, vec, st);
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
    most = std::max(most, size_t(bwd_most(T, s)));
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
  const BwdPlan p = bwd_plan(J, T, bwd_most(T, s));
  a.seg_rows = p.seg_rows; a.chunks = p.chunks; a.segs_per_group = p.segs_per_group;
  const size_t part = align256(size_t(p.groups) * d * 4);
  char *wb = static_cast<char *>(ws);
  a.part_post = dw_post ? reinterpret_cast<float *>(wb) : nullptr;
  a.part_pre = dw_pre ? reinterpret_cast<float *>(wb + part) : nullptr;
  a.part_gate = reinterpret_cast<float *>(wb + 2 * part);
  const int64_t G = T / J->gate_rows + (T % J->gate_rows ? 1 : 0);
  const double gate_elems = channel ? 2.0 * double(G) * d : a.gate_kind == POET_GATE_ROW ? 2.0 * double(G) : 0.0;
  const int passes = 1 + (o ? 2 : 0) + (dn ? 2 : 0) + (dh_out ? 1 : 0);
  TraceScope ts("joint_bwd", 30.0 * double(T) * d, (double(T) * d * passes + gate_elems) * double(esize(dt)), st);
  const int operands = (dn ? 2 : 0) + (dh_out ? 1 : 0) + (o ? 1 : 0);
  if (!channel) POET_TRY(pick_bwd<GK_ROW>(a, s, p.groups, operands, dt, vec, st));
  else if (J->gate_rows == 1) POET_TRY(pick_bwd<GK_EACH>(a, s, p.groups, operands, dt, vec, st));
  else POET_TRY(pick_bwd<GK_SHARED>(a, s, p.groups, operands, dt, vec, st));
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
