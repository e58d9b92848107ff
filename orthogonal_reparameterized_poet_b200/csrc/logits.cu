// Operators on rows of logits: log probabilities of given tokens with entropy
// and top alternatives, distillation from a teacher's top logits, and their
// gradients.
//
// One pass over a row of V logits keeps, per thread, the running maximum m,
// s = sum exp(c (x - m)) and t = sum exp(c (x - m)) c (x - m); these are joined
// through shuffles, shared memory and the cluster's distributed shared memory,
// always in one order.  c = scale log2(e), so an exponential is one ex2;
// differences to the maximum are formed before they are scaled, so neither large
// logits nor masks of the type's lowest value lose anything.
//
// The forward operators are persistent: a CTA (or, with few rows, a cluster of
// CTAs, each with a contiguous slice) works through rows, and one warp of it
// streams their 16-byte vectors through a ring of stages in shared memory by
// bulk copies, so that the next rows are on their way while a row's sums are
// joined, its alternatives selected or its gradient written.  What they cannot go
// below: HBM (each logit is read once, each gradient written once) and, close
// behind, the exponential (16 a clock and SM: for a bf16 logit 73 % of the time
// that HBM needs) and instruction issue, hence the arithmetic in pairs.  None of
// them is saturated (issue slots 57 to 65 %, exponentials 51 to 63 %, DRAM 47 to
// 61 % of nominal): a row's join, and the second reading, from L2, of a row that
// does not fit the ring when its gradient is wanted, are not hidden entirely.
//
// Measured (bf16, on the GPU, every row live, of a copy's 6.56 TB/s): log
// probabilities and entropy of 4096 rows of 128000 170 us (6.2 TB/s), of 16384 of
// 32000 191 us (5.5; the stream without the arithmetic 156 us); with 64
// alternatives of 4096 x 128000 223 us; loss and gradient of 8192 x 32000 239 us
// (4.4), the loss alone 119, the gradient alone from saved sums 6.4 TB/s.  A call
// among others takes up to 7 % more, depending on the machine.  Tried and
// slower: a quarter of the exponentials by a polynomial (217 us against 197, issue
// and FMA bound), a cluster for rows that do not fit a CTA's ring (80 us against
// 64, the exchange of every row), the two passes of a loss with its gradient in
// different warps (274 us against 250, one CTA an SM).
#include <cmath>

#include <cooperative_groups.h>

#include "rows.cuh"

namespace cg = cooperative_groups;

namespace poet {
namespace {

constexpr int MAX_V = 2097152;
constexpr int MAX_K = 128;
constexpr int MAX_CLUSTER = 8;
constexpr int SLICE = 262144;  // most columns of one CTA
constexpr int NT = 256;        // threads of the element-wise gradients
constexpr int CAND = 1536;     // candidates kept at once by the selection: 192 vectors of 8
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr float LOWEST = -1e30f;

// scale log2(e), finite: an infinite one would make NaN of a difference of 0.
__device__ __forceinline__ float log2_scale(float scale) { return fminf(scale * LOG2E, 3.4028234e38f); }

// The hardware's exponential, off by two units in the last place, and 0 below
// 2^-126, where a probability counts for nothing beside the row's largest.  With the
// rounding of its argument a probability p is off by about 2^-23 (2 + |ln p|) of
// itself; CUDA's own function has the argument's error too.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 ex2(float2 x) { return make_float2(ex2(x.x), ex2(x.y)); }

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The aligned part of a row slice: elements [lo, lo + head) one by one, then
// `nv` 16-byte vectors, then elements [tail0, hi) one by one.
template <typename T>
struct Slice {
  static constexpr int E = 16 / int(sizeof(T));
  int lo, head, nv, tail0, hi;
};

// Slice `rank` of `size` of a row of V elements at p: the row's vectors are
// dealt out evenly, the elements before the first vector go to the first
// slice, those behind the last one to the last.
template <typename T>
__device__ __forceinline__ Slice<T> slice_of(const T *p, int V, int rank, int size) {
  constexpr int E = Slice<T>::E;
  Slice<T> s;
  int head = int(((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(T));
  if (head > V) head = V;
  const int nv = (V - head) / E;
  int b0 = 0, b1 = nv;
  if (size > 1) {  // nv * size < 2^32: V <= MAX_V, size <= 512
    b0 = int(unsigned(nv) * unsigned(rank) / unsigned(size));
    b1 = int(unsigned(nv) * unsigned(rank + 1) / unsigned(size));
  }
  s.lo = rank == 0 ? 0 : head + b0 * E;
  s.head = rank == 0 ? head : 0;
  s.nv = b1 - b0;
  s.tail0 = head + b1 * E;
  s.hi = rank == size - 1 ? V : s.tail0;
  return s;
}

// The running sums of some logits of a row, in pairs, relative to a base b that
// follows their maximum: it is moved only when an exponent would pass RISE, which
// after a thread's first logits is rare, and the sums' relative errors do not
// depend on it.
//
// An exponent is c x + k, one fused operation with k = -(b c) rounded: the sums
// are relative to -k / c instead of b, the same for all of them, so only the
// operation's own rounding counts, and at() gives the exponent of any other
// logit to convert by.  For a far base (|b c| >= FAR, where k's rounding alone
// would move the exponents, no base yet, or a scale so small or large that
// -2^100 would not do for a masked logit) it is c (x - b).
constexpr float RISE = 8.f, FAR = 1048576.f;
struct Run {
  float m, b, k;  // the largest, the base
  bool far;
  float2 s, t;
  __device__ __forceinline__ void clear() {
    m = b = -INFINITY;
    k = 0.f;
    far = true;
    s = t = both(0.f);
  }
  // the base for far exponents; without a base there are only masked logits
  __device__ __forceinline__ float origin() const { return b == -INFINITY ? 0.f : b; }
  __device__ __forceinline__ float at(float x, float c) const { return far ? (x - b) * c : fmaf(x, c, k); }
  // Moves the sums by D >= 0 (about) towards a larger base.
  __device__ __forceinline__ void shift(float D) {
    D = D < -LOWEST ? D : -LOWEST;  // no base yet: the sums are 0
    const float2 f = both(ex2(-D));
    t = mul2(fma2(s, both(-D), t), f);
    s = mul2(s, f);
  }
  // Takes mx into the maximum; call before adding logits up to mx.
  __device__ __forceinline__ void see(float mx, float c) {
    m = fmaxf(m, mx);
    const float d = at(mx, c);
    if (d > RISE) {
      b = mx;
      k = -(mx * c);
      far = !(fabsf(k) < FAR && c > 0x1p-60f && c < 0x1p27f);
      shift(d - (far ? 0.f : fmaf(mx, c, k)));
    }
  }
  // Adds exp(d) and exp(d) d for two logits.  Near: no logit below -2^100, k2 = k.
  template <bool ENT>
  __device__ __forceinline__ void add_near(float2 x, float2 k2, float2 c) {
    const float2 d = fma2(x, c, k2);
    const float2 e = ex2(d);
    s = add2(s, e);
    if (ENT) t = fma2(e, d, t);
  }
  template <bool ENT>
  __device__ __forceinline__ void add_far(float2 x, float2 minus_b, float2 c) {
    const float2 d = mul2(add2(x, minus_b), c);
    const float2 e = ex2(d);
    s = add2(s, e);
    if (ENT) t = fma2(e, make_float2(fmaxf(d.x, LOWEST), fmaxf(d.y, LOWEST)), t);
  }
  __device__ __forceinline__ void add1(float x, float c) {
    const float d = far ? (x - origin()) * c : fmaf(x, c, k), e = ex2(d);
    s.x += e;
    t.x = fmaf(e, fmaxf(d, LOWEST), t.x);
  }
};

// The joined sums of some logits.
struct Sums {
  float m, s, t;
  __device__ __forceinline__ float base() const { return m == -INFINITY ? 0.f : m; }
};

// Order of logits as unsigned integers (-0 and +0 equal; larger is larger).
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}
constexpr uint32_t KEY_MASKED = 0x007fffffu;  // key_of(-inf)

// Joins the sums that groups of 2^LOG lanes hold; every lane of a group gets the result.
template <int LOG>
__device__ __forceinline__ Sums join_lanes(Sums a, float c) {
  float m = a.m;
#pragma unroll
  for (int o = 1 << LOG >> 1; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float d = (a.m - (m == -INFINITY ? 0.f : m)) * c, f = ex2(d);
  float s = a.s * f, t = fmaf(a.s, fmaxf(d, LOWEST), a.t) * f;
#pragma unroll
  for (int o = 1 << LOG >> 1; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    t += __shfl_xor_sync(0xffffffffu, t, o);
  }
  return {m, s, t};
}
__device__ __forceinline__ Sums join_warp(Run &r, float c) {
  const float m = of_key(__reduce_max_sync(0xffffffffu, key_of(r.m)));
  if (m > -INFINITY) r.shift(r.at(m, c));
  float v[2] = {r.s.x + r.s.y, r.t.x + r.t.y};
  row_sum_2(v, nullptr, 1, 0, 0, 32);
  return {m, v[0], v[1]};
}

// A 16-byte vector of logits: its extremes (NaN ignored) and its pairs.
template <typename T>
struct Vec;
template <>
struct Vec<bf16> {
  static constexpr int E = 8;
  static constexpr uint32_t MASKED = 0xff80ff80u;
  // no element below -2^100; NaN stays
  static __device__ __forceinline__ uint4 bounded(const uint4 &v) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const Top t = __hmax2_nan(word(w[i]), word(0xf180f180u));
      w[i] = *reinterpret_cast<const uint32_t *>(&t);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  using Top = __nv_bfloat162;
  static __device__ __forceinline__ Top word(uint32_t w) { return *reinterpret_cast<const Top *>(&w); }
  static __device__ __forceinline__ Top largest(const uint4 &v) {
    return __hmax2(__hmax2(word(v.x), word(v.y)), __hmax2(word(v.z), word(v.w)));
  }
  static __device__ __forceinline__ Top larger(Top a, Top b) { return __hmax2(a, b); }
  static __device__ __forceinline__ float top(Top a) { return fmaxf(__low2float(a), __high2float(a)); }
  static __device__ __forceinline__ void get(const uint4 &v, float2 (&x)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  static __device__ __forceinline__ uint4 put(const float2 (&x)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __float22bfloat162_rn(x[i]);
      w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  // -inf in place of the elements whose bit is set
  static __device__ __forceinline__ void mask(uint4 &v, unsigned bits) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if ((bits >> (2 * i)) & 1u) w[i] = (w[i] & 0xffff0000u) | 0xff80u;
      if ((bits >> (2 * i + 1)) & 1u) w[i] = (w[i] & 0xffffu) | 0xff800000u;
    }
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec<float> {
  static constexpr int E = 4;
  static constexpr uint32_t MASKED = 0xff800000u;
  static __device__ __forceinline__ uint4 bounded(const uint4 &v) {
    auto g = [](uint32_t w) { return __float_as_uint(max_nan(f(w), -0x1p100f)); };
    return make_uint4(g(v.x), g(v.y), g(v.z), g(v.w));
  }
  using Top = float;
  static __device__ __forceinline__ float f(uint32_t w) { return __uint_as_float(w); }
  static __device__ __forceinline__ Top largest(const uint4 &v) {
    return fmaxf(fmaxf(f(v.x), f(v.y)), fmaxf(f(v.z), f(v.w)));
  }
  static __device__ __forceinline__ Top larger(Top a, Top b) { return fmaxf(a, b); }
  static __device__ __forceinline__ float top(Top a) { return a; }
  static __device__ __forceinline__ void get(const uint4 &v, float2 (&x)[2]) {
    x[0] = make_float2(f(v.x), f(v.y));
    x[1] = make_float2(f(v.z), f(v.w));
  }
  static __device__ __forceinline__ uint4 put(const float2 (&x)[2]) {
    return make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y), __float_as_uint(x[1].x), __float_as_uint(x[1].y));
  }
  static __device__ __forceinline__ void mask(uint4 &v, unsigned bits) {
    if (bits & 1u) v.x = MASKED;
    if (bits & 2u) v.y = MASKED;
    if (bits & 4u) v.z = MASKED;
    if (bits & 8u) v.w = MASKED;
  }
};

// ------------------------------------------------------------------ the stream of rows

constexpr int U = 4;             // vectors of a thread in one stage
constexpr int MAX_STAGES = 12;
// CTAs that share an SM, by the warps that compute (and what registers allow).
template <int NW>
constexpr int per_sm(bool lean) { return NW == 8 ? (lean ? 3 : 2) : NW == 4 ? (lean ? 5 : 4) : 6; }
constexpr int BAR = 1;           // the named barrier of the warps that compute
constexpr uint64_t TIMEOUT_NS = 4000000000ull;

__device__ __forceinline__ uint32_t smem_at(const void *p) { return uint32_t(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ uint32_t peer_at(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void bar_init(uint64_t *b, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_at(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t *b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_at(b)) : "memory");
}
__device__ __forceinline__ void bar_arrive_peer(uint64_t *b, int rank) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(peer_at(smem_at(b), rank)) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t at, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(at), "r"(parity)
      : "memory");
  return ok != 0;
}
// Waits for the phase of this parity.  Every wait ends: after TIMEOUT_NS it
// records ERR_TIMEOUT, and from then on the CTA's waits return at once (its
// results are void, and the producer issues nothing more).
__device__ __noinline__ bool bar_wait_long(uint32_t at, uint32_t parity, volatile int *abort, unsigned *errword) {
  const uint64_t t0 = now_ns();
  for (uint32_t it = 1;; ++it) {
    if (bar_try(at, parity)) return true;
    if ((it & 63) == 0) {
      if (*abort) return false;
      if (now_ns() - t0 > TIMEOUT_NS) {
        atomicOr(errword, unsigned(ERR_TIMEOUT));
        *abort = 1;
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool bar_wait(uint64_t *b, uint32_t parity, volatile int *abort, unsigned *errword) {
  const uint32_t at = smem_at(b);
  return bar_try(at, parity) || bar_wait_long(at, parity, abort, errword);
}

// The ring's barriers and the exchange of the cluster's CTAs.
struct Pipe {
  uint64_t full[MAX_STAGES], empty[MAX_STAGES];
  uint64_t join;             // the cluster's exchange of a row
  uint64_t hfull[2], hempty[2];  // two buffers handed from some warps to others
  float4 part[2][MAX_CLUSTER];
  float4 warp[2][8];
  int abort;
};
// from, to: warps that fill a buffer that is handed over, and that empty it.
template <int NW>
__device__ __forceinline__ void pipe_init(Pipe &P, int stages, int size, int from, int to, cg::cluster_group &cl) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      bar_init(&P.full[i], 1);
      bar_init(&P.empty[i], NW);
    }
    bar_init(&P.join, size);
    for (int i = 0; i < 2; ++i) {
      bar_init(&P.hfull[i], from);
      bar_init(&P.hempty[i], to);
    }
    P.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (size > 1) cl.sync();
  else __syncthreads();
}

// A place in the ring.
struct Spot {
  int st = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++st == stages) {
      st = 0;
      ph ^= 1;
    }
  }
};

// The producer: one thread copies the vectors of every row's slice, NW * 32 * U
// at a time, into the ring; `passes` times each row (a second time where a row
// does not fit the ring and is read again for its gradient).  rows.fetch(row)
// loads what decides whether a row is read at all, a row ahead, and rows.live()
// decides (the whole warp calls both).
template <typename T, int NW, typename F>
__device__ void produce(Pipe &P, const unsigned char *ring, int stages, const void *x0, int64_t ld, int V, int64_t T_rows,
                        int64_t first, int64_t step, int rank, int size, bool twice, unsigned *errword, F rows) {
  constexpr int SV = NW * 32 * U;
  Spot at;
  int64_t issued = 0;
  bool ok = true;
  if (first < T_rows) rows.fetch(first);
  for (int64_t row = first; row < T_rows && ok; row += step) {
    const bool live = rows.live();
    if (row + step < T_rows) rows.fetch(row + step);
    if (!live) continue;
    const T *x = static_cast<const T *>(x0) + row * ld;
    const Slice<T> sl = slice_of(x, V, rank, size);
    const T *body = x + sl.lo + sl.head;
    if ((threadIdx.x & 31) == 0) {
      const int nst = (sl.nv + SV - 1) / SV;
      const int passes = twice && nst > stages ? 2 : 1;
      for (int p = 0; p < passes && ok; ++p)
        for (int k = 0; k < nst; ++k) {
          if (!bar_wait(&P.empty[at.st], at.ph ^ 1, &P.abort, errword)) {
            ok = false;
            break;
          }
          const int n = min(sl.nv - k * SV, SV);
          const uint32_t bar = smem_at(&P.full[at.st]), bytes = uint32_t(n) * 16;
          asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
          asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                           smem_at(ring) + at.st * (SV * 16)),
                       "l"(body + int64_t(k) * SV * Vec<T>::E), "r"(bytes), "r"(bar)
                       : "memory");
          ++issued;
          at.next(stages);
        }
    }
    ok = __shfl_sync(0xffffffffu, ok, 0);
  }
  // after an abort: the copies in flight, with a limit
  if (!ok && (threadIdx.x & 31) == 0) {
    const uint64_t t0 = now_ns();
    for (int64_t k = issued > stages ? issued - stages : 0; k < issued; ++k)
      while (!bar_try(smem_at(&P.full[k % stages]), uint32_t(k / stages) & 1) && now_ns() - t0 < TIMEOUT_NS) {
      }
  }
  __syncwarp();
}

template <int NW>
__device__ __forceinline__ void warps_sync() {
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"n"(BAR), "n"(NW * 32) : "memory");
}

// Gives a stage back to the producer, by a warp that has used what it read from
// it.  The stage's next bytes come through the async proxy, so the reads, which
// are generic, are fenced against it; an arrival alone was seen to pass loads
// whose values were not used yet, and those then found the next bytes.
__device__ __forceinline__ void give_back(uint64_t *empty) {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  if ((threadIdx.x & 31) == 0) bar_arrive(empty);
}

// A stage's vectors of this thread; those behind the slice's end are masked.
template <typename T, int NW>
__device__ __forceinline__ void read_stage(uint4 (&v)[U], const unsigned char *ring, int st, int left) {
  const uint4 *p = reinterpret_cast<const uint4 *>(ring + st * (NW * 32 * U * 16)) + threadIdx.x;
  if (left >= NW * 32 * U) {
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = p[u * NW * 32];
  } else {
    constexpr uint32_t M = Vec<T>::MASKED;
#pragma unroll
    for (int u = 0; u < U; ++u)
      v[u] = u * NW * 32 + int(threadIdx.x) < left ? p[u * NW * 32] : make_uint4(M, M, M, M);
  }
}

// The sums with a thread's vectors added against a far base: rare, and out of
// line, because the loops over rows should stay in the instruction cache.
template <typename T, bool ENT>
__device__ __noinline__ Run add_far_vectors(Run r, uint4 v0, uint4 v1, uint4 v2, uint4 v3, float c) {
  using X = Vec<T>;
  static_assert(U == 4, "one argument a vector");
  const uint4 v[U] = {v0, v1, v2, v3};
  const float2 mb = both(-r.origin()), c2 = both(c);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float2 x[X::E / 2];
    X::get(v[u], x);
#pragma unroll
    for (int i = 0; i < X::E / 2; ++i) r.template add_far<ENT>(x[i], mb, c2);
  }
  return r;
}

// Adds a thread's vectors to its sums; returns their largest logit.
template <typename T, bool ENT>
__device__ __forceinline__ float add_vectors(Run &r, const uint4 (&v)[U], float c) {
  using X = Vec<T>;
  typename X::Top hi = X::largest(v[0]);
#pragma unroll
  for (int u = 1; u < U; ++u) hi = X::larger(hi, X::largest(v[u]));
  const float mx = X::top(hi);
  r.see(mx, c);
  const float2 c2 = both(c);
  if (!r.far) {
    const float2 k2 = both(r.k);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float2 x[X::E / 2];
      X::get(ENT ? X::bounded(v[u]) : v[u], x);
#pragma unroll
      for (int i = 0; i < X::E / 2; ++i) r.template add_near<ENT>(x[i], k2, c2);
    }
  } else {
    r = add_far_vectors<T, ENT>(r, v[0], v[1], v[2], v[3], c);
  }
  return mx;
}

// A row's sums from those of the NW warps in P.warp[par], and of the cluster's
// CTAs: by whole warps, of which `leads` says which exchanges with the others.
// The buffers of the exchange alternate with `par`: one is written again only
// after the exchange of the row between, for which each CTA's leading warp
// arrives after all its warps have read the first.
template <int NW>
__device__ __forceinline__ Sums join_warps(Pipe &P, float c, int par, int phase, bool leads, int rank, int size,
                                           unsigned *errword) {
  const int lane = threadIdx.x & 31;
  const float4 f = P.warp[par][lane % NW];
  Sums all = join_lanes<NW == 8 ? 3 : NW == 4 ? 2 : 1>({f.x, f.y, f.z}, c);
  if (size > 1) {
    if (leads && lane < size) {
      const uint32_t to = peer_at(smem_at(&P.part[par][rank]), lane);
      asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to), "f"(all.m), "f"(all.s), "f"(all.t),
                   "f"(0.f)
                   : "memory");
      bar_arrive_peer(&P.join, lane);
    }
    bar_wait(&P.join, phase, &P.abort, errword);
    const int q = lane % MAX_CLUSTER;
    const float4 g = q < size ? P.part[par][q] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
    all = join_lanes<3>({g.x, g.y, g.z}, c);
  }
  return all;
}
// The same with the warps that compute, all of whose threads get the sums.
template <int NW>
__device__ __forceinline__ Sums join_row(Pipe &P, Run &r, float c, int par, int rank, int size, unsigned *errword) {
  const Sums w = join_warp(r, c);
  if ((threadIdx.x & 31) == 0) P.warp[par][threadIdx.x >> 5] = make_float4(w.m, w.s, w.t, 0.f);
  warps_sync<NW>();
  return join_warps<NW>(P, c, par, par, threadIdx.x < 32, rank, size, errword);
}

// The ragged ends of a slice, at most E - 1 elements each, one per lane of the
// first warp, added to its sums.
template <typename T>
__device__ __forceinline__ void add_ends(Run &r, float xh, float xt, float c) {
  const float mx = fmaxf(xh, xt);
  r.see(mx, c);
  r.add1(xh, c);
  r.add1(xt, c);
}

// ------------------------------------------------------------------ selection of the largest

// Where a slice's largest logits are.  The logits of a thread in one stage are a
// group; the keys are the groups' largest (group k * NW * 32 + thread of stage
// k), tops the computing threads', ends those of the elements before and behind
// the slice's vectors.
struct Hand {
  float ends[2];
  float tops[256];
};
// Shared memory of the selection.
constexpr int LIST = 256;
constexpr unsigned MOST = 192;  // groups that are listed
struct Select {
  uint64_t gather[2];
  Hand hand[2];
  unsigned long long cand[CAND];
  unsigned long long best[MAX_K];
  unsigned short list[LIST];  // of fewer than 2^16 groups: SLICE / (4 U) and a stage
  unsigned counts[2][4];
  unsigned n, m;
};
constexpr int SELECT_BAR = 2;
// Warps that select beside NW that compute.
template <int NW>
constexpr int select_warps() { return NW == 8 ? 4 : 2; }

template <int NS>
__device__ __forceinline__ void select_sync() {
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"n"(SELECT_BAR), "n"(NS * 32) : "memory");
}
// The same; whether any thread brings true.
template <int NS>
__device__ __forceinline__ bool select_any(bool v) {
  unsigned any;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(unsigned(v)), "n"(SELECT_BAR), "n"(NS * 32)
      : "memory");
  return any != 0;
}
// The sum of a count over the selecting warps; one barrier, buffers alternate.
template <int NS>
__device__ __forceinline__ unsigned select_count(Select &S, unsigned v, int tid, int &flip) {
  v = __reduce_add_sync(0xffffffffu, v);
  if ((tid & 31) == 0) S.counts[flip][tid >> 5] = v;
  select_sync<NS>();
  unsigned total = 0;
#pragma unroll
  for (int w = 0; w < NS; ++w) total += S.counts[flip][w];
  flip ^= 1;
  return total;
}
// Where a lane's n items go in a list that `cell` counts; the whole warp.
__device__ __forceinline__ unsigned place_of(unsigned n, unsigned *cell) {
  const int lane = threadIdx.x & 31;
  unsigned upto = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  unsigned base = 0;
  if (lane == 31 && upto) base = atomicAdd(cell, upto);
  return __shfl_sync(0xffffffffu, base, 31) + upto - n;
}

__device__ __forceinline__ unsigned long long order_of(float x, unsigned index) {
  return (static_cast<unsigned long long>(key_of(x)) << 32) | (0xffffffffu - index);
}

// The K largest logits of a slice (equal ones: the lower index first), in
// falling order, as order_of, to S.best, 0 where there are fewer; -inf is never
// among them.  floor: the smallest of the computing threads' maxima; top: no
// logit is larger; no NaN.
//
// The K-th largest of some maxima of disjoint parts is a bound that at least K
// logits reach and few others.  The parts are first the computing threads'
// logits (G values, found about by bisection); only the groups that reach that
// bound are read again (from L2).  Where more than MOST groups do, the bound is
// drawn closer with the groups' maxima; where equal logits or a few crowded
// groups leave too many candidates, the exact bound is found by bisection over
// the slice's elements.
template <typename T, int NW>
__device__ void select_largest(Select &S, const Hand &H, const float *keys, const T *x, const Slice<T> &sl, unsigned K,
                               float floor, float top, int tid) {
  constexpr int G = NW * 32, SV = G * U, E = Vec<T>::E, NS = select_warps<NW>(), NN = NS * 32;
  const T *body = x + sl.lo + sl.head;
  const int groups = (sl.nv + SV - 1) / SV * G;
  int flip = 0;
  const unsigned most = K + K / 2 < 32 ? 32 : K + K / 2;  // <= 192 < 256
  auto groups_at = [&](float b) {
    unsigned n = 0;
#pragma unroll 4
    for (int k = tid; k < groups; k += NN) n += keys[k] >= b;
    if (tid == 0) n += (H.ends[0] >= b) + (H.ends[1] >= b);
    return select_count<NS>(S, n, tid, flip);
  };
  uint32_t lo = KEY_MASKED + 1, hi = key_of(top) + 1;  // none reach hi
  // A value between lo and hi, of values for some steps, then of the order of floats.
  auto between = [&](int step) {
    const float v = 0.5f * of_key(lo) + 0.5f * of_key(hi - 1);
    return step < 12 ? min(max(key_of(v), lo + 1), hi - 1) : lo + (hi - lo) / 2;
  };
  if (tid == 0) { S.n = 0; S.m = 0; }
  select_sync<NS>();
  if (K <= unsigned(G) && floor > -INFINITY) {
    // every computing thread has logits: the K-th largest of their maxima first
    float t[G / NN];
#pragma unroll
    for (int i = 0; i < G / NN; ++i) t[i] = H.tops[tid + i * NN];
    lo = max(lo, key_of(floor));
    for (int step = 0; hi - lo > 1; ++step) {
      const uint32_t mid = between(step);
      unsigned n = 0;
#pragma unroll
      for (int i = 0; i < G / NN; ++i) n += t[i] >= of_key(mid);
      n = select_count<NS>(S, n, tid, flip);
      if (n < K) hi = mid;
      else {
        lo = mid;
        if (n <= K + K / 8 + 2) break;
      }
    }
    hi = key_of(top) + 1;
  }
  // the groups that reach the bound
  unsigned mine = 0, at = 0;
  bool crowded = false;
  auto count_mine = [&]() {
    mine = 0;
#pragma unroll 4
    for (int k = tid; k < groups; k += NN) mine += keys[k] >= of_key(lo);
    at = place_of(mine, &S.m);
    select_sync<NS>();
  };
  count_mine();
  if (S.m + 2 > MOST) {  // a closer one: at least K reach it, no more than `most`
    for (int step = 0;; ++step) {
      if (hi - lo <= 1) {
        crowded = true;
        break;
      }
      const uint32_t mid = between(step);
      const unsigned n = groups_at(of_key(mid));
      if (n < K) hi = mid;
      else {
        lo = mid;
        if (n <= most) break;
      }
    }
    if (!crowded) {
      if (tid == 0) S.m = 0;
      select_sync<NS>();
      count_mine();
    }
  }
  const float bound = of_key(lo);
  unsigned n = 0;
  if (!crowded) {
    if (mine)
      for (int k = tid; k < groups; k += NN)
        if (keys[k] >= bound && at < LIST) S.list[at++] = (unsigned short)k;
    select_sync<NS>();
    const unsigned items = min(S.m, unsigned(LIST)) * U;
    constexpr int AHEAD = 2;  // vectors that a thread reads at once
    for (unsigned j0 = 0; j0 < items; j0 += AHEAD * NN) {
      uint4 w[AHEAD];
      int from[AHEAD];
#pragma unroll
      for (int q = 0; q < AHEAD; ++q) {
        constexpr uint32_t M = Vec<T>::MASKED;
        const unsigned j = j0 + q * NN + tid;
        w[q] = make_uint4(M, M, M, M);
        from[q] = 0;
        if (j < items) {
          const int g = int(S.list[j / U]), v = g / G * SV + int(j % U) * G + g % G;
          if (v < sl.nv) {
            w[q] = *reinterpret_cast<const uint4 *>(body + int64_t(v) * E);
            from[q] = sl.lo + sl.head + v * E;
          }
        }
      }
#pragma unroll
      for (int q = 0; q < AHEAD; ++q) {
        float2 f[E / 2];
        Vec<T>::get(w[q], f);
        unsigned bits = 0;
#pragma unroll
        for (int i = 0; i < E / 2; ++i) bits |= unsigned(f[i].x >= bound) << (2 * i) | unsigned(f[i].y >= bound) << (2 * i + 1);
        unsigned to = place_of(__popc(bits), &S.n);
#pragma unroll
        for (int i = 0; i < E; ++i)
          if (bits >> i & 1u) {
            if (to < CAND) S.cand[to] = order_of(i & 1 ? f[i / 2].y : f[i / 2].x, unsigned(from[q] + i));
            ++to;
          }
      }
    }
    if (tid < 32) {  // the ends
      const int ih = sl.lo + tid, it = sl.tail0 + tid;
      const float xh = tid < sl.head ? to_float(x[ih]) : -INFINITY, xt = it < sl.hi ? to_float(x[it]) : -INFINITY;
      unsigned to = place_of(unsigned(xh >= bound) + unsigned(xt >= bound), &S.n);
      if (xh >= bound && to < CAND) S.cand[to] = order_of(xh, unsigned(ih));
      to += xh >= bound;
      if (xt >= bound && to < CAND) S.cand[to] = order_of(xt, unsigned(it));
    }
    select_sync<NS>();
    n = S.n;
  }
  if (crowded || n > CAND) {
    // the exact bound: the largest that K elements reach (elements of groups below it need not be read)
    auto each = [&](float from, auto &&f) {
      for (int k = tid; k < groups; k += NN)
        if (keys[k] >= from)
          for (int u = 0; u < U; ++u) {
            const int v = k / G * SV + u * G + k % G;
            if (v < sl.nv) {
              float2 e[E / 2];
              Vec<T>::get(*reinterpret_cast<const uint4 *>(body + int64_t(v) * E), e);
#pragma unroll
              for (int i = 0; i < E; ++i) f(i & 1 ? e[i / 2].y : e[i / 2].x, sl.lo + sl.head + v * E + i);
            }
          }
      if (tid < 32) {
        if (tid < sl.head) f(to_float(x[sl.lo + tid]), sl.lo + tid);
        if (sl.tail0 + tid < sl.hi) f(to_float(x[sl.tail0 + tid]), sl.tail0 + tid);
      }
    };
    uint32_t l = lo, h = key_of(top) + 1;  // at least K reach l, none h
    for (int step = 0; h - l > 1; ++step) {
      const float v = 0.5f * of_key(l) + 0.5f * of_key(h - 1);
      const uint32_t mid = step < 8 ? min(max(key_of(v), l + 1), h - 1) : l + (h - l) / 2;
      unsigned c = 0;
      each(of_key(mid), [&](float v, int) { c += v >= of_key(mid); });
      if (select_count<NS>(S, c, tid, flip) >= K) l = mid;
      else h = mid;
    }
    // what is above it
    const float b = of_key(l);
    select_sync<NS>();  // all have read S.n
    if (tid == 0) S.n = 0;
    select_sync<NS>();
    each(b, [&](float v, int i) {
      if (v > b) {
        const unsigned to = atomicAdd(&S.n, 1u);
        if (to < CAND) S.cand[to] = order_of(v, unsigned(i));
      }
    });
    select_sync<NS>();
    // and the first of those equal to it, in their order, as many as are left
    unsigned taken = S.n;
    for (int v0 = -1; v0 <= sl.nv && taken < K; v0 = v0 < 0 ? 0 : v0 + NN) {
      // items of this thread: the elements before the vectors (v0 = -1), a vector, or the elements behind
      const int v = v0 + tid;
      float e[E];
      int at0 = 0;
#pragma unroll
      for (int i = 0; i < E; ++i) e[i] = -INFINITY;
      if (v0 < 0) {
        at0 = sl.lo + tid;
        if (tid < sl.head) e[0] = to_float(x[at0]);
      } else if (v < sl.nv) {
        at0 = sl.lo + sl.head + v * E;
        float2 f[E / 2];
        Vec<T>::get(*reinterpret_cast<const uint4 *>(body + int64_t(v) * E), f);
#pragma unroll
        for (int i = 0; i < E; ++i) e[i] = i & 1 ? f[i / 2].y : f[i / 2].x;
      } else if (v == sl.nv) {
        at0 = sl.tail0;
        for (int i = 0; i < E; ++i)
          if (sl.tail0 + i < sl.hi) e[i] = to_float(x[sl.tail0 + i]);
      }
      unsigned mine = 0;
#pragma unroll
      for (int i = 0; i < E; ++i) mine += e[i] == b;
      unsigned upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned u = __shfl_up_sync(0xffffffffu, upto, o);
        if ((tid & 31) >= o) upto += u;
      }
      if ((tid & 31) == 31) S.counts[flip][tid >> 5] = upto;
      select_sync<NS>();
      unsigned to = taken + upto - mine, all = 0;
#pragma unroll
      for (int w = 0; w < NS; ++w) {
        if (w < (tid >> 5)) to += S.counts[flip][w];
        all += S.counts[flip][w];
      }
      flip ^= 1;
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (e[i] == b) {
          if (to < K) S.cand[to] = order_of(b, unsigned(at0 + i));
          ++to;
        }
      taken += all;
    }
    select_sync<NS>();
    n = min(taken, K);
  } else if (n > 2 * most) {
    // many in the listed groups: a closer bound among the candidates (their order has no ties)
    unsigned long long l = 0, h = ~0ull;
    while (h - l > 1) {
      const unsigned long long mid = l + (h - l) / 2;
      unsigned c = 0;
      for (unsigned i = tid; i < n; i += NN) c += S.cand[i] >= mid;
      c = select_count<NS>(S, c, tid, flip);
      if (c < K) h = mid;
      else if (c > most) l = mid;
      else { l = mid; break; }
    }
    if (tid == 0) S.n = 0;
    for (unsigned i0 = 0; i0 < n; i0 += NN) {  // those that reach it move to the front: never past what is read
      const unsigned i = i0 + tid;
      const unsigned long long mine = i < n ? S.cand[i] : 0;
      select_sync<NS>();
      if (i < n && mine >= l) S.cand[atomicAdd(&S.n, 1u)] = mine;
    }
    select_sync<NS>();
    n = S.n;
  }
  for (unsigned i = tid; i < K; i += NN)
    if (i >= n) S.best[i] = 0;
  for (unsigned i = tid; i < n; i += NN) {
    const unsigned long long mine = S.cand[i];
    unsigned above = 0;
#pragma unroll 8
    for (unsigned j = 0; j < n; ++j) above += S.cand[j] > mine;
    if (above < K) S.best[above] = mine;
  }
  select_sync<NS>();
}

// ------------------------------------------------------------------ log probabilities

struct LogpArgs {
  const void *x;
  int64_t ld, T;
  int V, K, stages;
  int key_floats;  // of one of the two buffers of keys
  float scale;
  const int32_t *tokens;
  float *logp, *entropy, *top_logp, *saved;
  int32_t *top_tokens;
  unsigned *errword;
};

struct GivenTokens {
  const int32_t *tokens;
  int V, token;
  __device__ __forceinline__ void fetch(int64_t row) { token = tokens ? tokens[row] : 0; }
  __device__ __forceinline__ bool live() const { return token >= 0 && token < V; }
};

// The computing warps' part: each warp's sums of every row, and what the
// selection needs.  They never wait for one another.
template <typename T, int NW, bool TOP, bool ENT>
__device__ __forceinline__ void logp_rows(const LogpArgs &a, Pipe &P, Select &S, float *keys0, const unsigned char *ring,
                                          int rank, int size, int64_t first, int64_t step) {
  constexpr int G = NW * 32, SV = G * U;
  const int tid = threadIdx.x;
  const float c = log2_scale(a.scale);
  Spot at;
  uint32_t round = 0;  // rows handed over
  int token = a.tokens && first < a.T ? a.tokens[first] : 0;
  for (int64_t row = first; row < a.T; row += step) {
    const T *x = static_cast<const T *>(a.x) + row * a.ld;
    const int y = token;
    if (a.tokens && row + step < a.T) token = a.tokens[row + step];
    if (y < 0 || y >= a.V) continue;
    const Slice<T> sl = slice_of(x, a.V, rank, size);
    const int nst = (sl.nv + SV - 1) / SV;
    Run r;
    r.clear();
    float xh = -INFINITY, xt = -INFINITY;
    if (tid < 32) {
      if (tid < sl.head) xh = to_float(x[sl.lo + tid]);
      if (sl.tail0 + tid < sl.hi) xt = to_float(x[sl.tail0 + tid]);
    }
    const int buf = int(round & 1);
    float *keys = keys0 + buf * a.key_floats;
    if (TOP) bar_wait(&P.hempty[buf], (round >> 1 & 1) ^ 1, &P.abort, a.errword);
    for (int k = 0; k < nst; ++k) {
      uint4 v[U];
      bar_wait(&P.full[at.st], at.ph, &P.abort, a.errword);
      read_stage<T, NW>(v, ring, at.st, sl.nv - k * SV);
      const float mx = add_vectors<T, ENT>(r, v, c);
      give_back(&P.empty[at.st]);
      at.next(a.stages);
      if (TOP) keys[k * G + tid] = mx;
    }
    float floor = 0.f;
    if (TOP) {
      S.hand[buf].tops[tid] = r.m;
      floor = of_key(__reduce_min_sync(0xffffffffu, key_of(r.m)));
    }
    if (tid < 32) {
      add_ends<T>(r, xh, xt, c);
      if (TOP) {
        const uint32_t kh = __reduce_max_sync(0xffffffffu, key_of(xh)), kt = __reduce_max_sync(0xffffffffu, key_of(xt));
        if (tid == 0) {
          S.hand[buf].ends[0] = of_key(kh);
          S.hand[buf].ends[1] = of_key(kt);
        }
      }
    }
    const Sums w = join_warp(r, c);
    if (!TOP) bar_wait(&P.hempty[buf], (round >> 1 & 1) ^ 1, &P.abort, a.errword);
    if ((tid & 31) == 0) P.warp[buf][tid >> 5] = make_float4(w.m, w.s, w.t, floor);
    __syncwarp();
    if ((tid & 31) == 0) bar_arrive(&P.hfull[buf]);
    ++round;
  }
}

// The finishing warps' part, a row behind: the join of the sums, the results and
// the selection of the alternatives.
template <typename T, int NW, bool TOP, bool ENT>
__device__ __forceinline__ void finish_rows(const LogpArgs &a, Pipe &P, Select &S, const float *keys0,
                                            unsigned long long *gather0, int rank, int size, int64_t first, int64_t step,
                                            int tid) {
  constexpr int NS = select_warps<NW>(), NN = (TOP ? NS : 1) * 32;
  const unsigned K = unsigned(a.K);
  const float c = log2_scale(a.scale);
  uint32_t round = 0;
  int token = a.tokens && first < a.T ? a.tokens[first] : 0;
  for (int64_t row = first; row < a.T; row += step) {
    const T *x = static_cast<const T *>(a.x) + row * a.ld;
    const int y = token;
    if (a.tokens && row + step < a.T) token = a.tokens[row + step];
    if (y < 0 || y >= a.V) {  // the whole cluster takes this way
      if (rank != 0) continue;
      if (tid == 0) {
        if (y >= a.V) atomicOr(a.errword, unsigned(ERR_BOUNDS));
        if (a.logp) a.logp[row] = 0.f;
        if (a.entropy) a.entropy[row] = 0.f;
        if (a.saved) reinterpret_cast<float4 *>(a.saved)[row] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      if (TOP)
        for (unsigned k = tid; k < K; k += NN) {
          a.top_tokens[row * K + k] = -1;
          a.top_logp[row * K + k] = -INFINITY;
        }
      continue;
    }
    const int buf = int(round & 1);
    const uint32_t phase = round >> 1 & 1;
    float xy = 0.f;
    if (a.logp && rank == 0 && tid == 0) xy = to_float(x[y]);
    const bool ok = bar_wait(&P.hfull[buf], phase, &P.abort, a.errword);
    // all leave together: a warp that stayed would wait for the others
    if (TOP ? select_any<NS>(!ok) : !__all_sync(0xffffffffu, ok)) break;
    const Sums all = join_warps<NW>(P, c, buf, buf, tid < 32, rank, size, a.errword);
    const bool bad = !(all.s < INFINITY);  // a NaN or +inf among the logits
    const float logs = logf(all.s);        // -inf for a row of masks
    if (rank == 0 && tid == 0) {
      float H = 0.f;
      if (bad) H = NAN;
      else if (ENT && all.s > 0.f) H = fmaxf(logs - LN2 * (all.t / all.s), 0.f);
      if (a.logp) a.logp[row] = bad ? NAN : xy == -INFINITY ? -INFINITY : (xy - all.m) * a.scale - logs;
      if (a.entropy) a.entropy[row] = H;
      if (a.saved)
        reinterpret_cast<float4 *>(a.saved)[row] = make_float4(bad ? NAN : all.m, bad ? NAN : logs, H, 0.f);
    }
    auto release = [&]() {
      __syncwarp();
      if ((tid & 31) == 0) bar_arrive(&P.hempty[buf]);
    };
    ++round;
    if (!TOP) {
      release();
      continue;
    }
    auto put = [&](unsigned k, unsigned long long b) {
      a.top_tokens[row * K + k] = b ? int32_t(0xffffffffu - uint32_t(b)) : -1;
      a.top_logp[row * K + k] = bad ? NAN : b ? (of_key(uint32_t(b >> 32)) - all.m) * a.scale - logs : -INFINITY;
    };
    if (bad) {
      for (unsigned k = tid; k < K; k += NN) S.best[k] = 0;
      select_sync<NS>();
    } else {
      float floor = P.warp[buf][tid % NW].w;
#pragma unroll
      for (int o = NW / 2; o > 0; o >>= 1) floor = fminf(floor, __shfl_xor_sync(0xffffffffu, floor, o));
      select_largest<T, NW>(S, S.hand[buf], keys0 + buf * a.key_floats, x, slice_of(x, a.V, rank, size), K, floor, all.m,
                            tid);
    }
    if (size == 1) {
      for (unsigned k = tid; k < K; k += NN) put(k, S.best[k]);
      release();
      select_sync<NS>();  // S.best is written again in the next row
      continue;
    }
    // the CTAs' lists to the first one, which merges them: an element's place is its place in its list plus the
    // numbers of larger elements in the others.  Two buffers: the others are at most one row ahead of the first.
    unsigned long long *gather = gather0 + buf * size * K;
    for (unsigned k = tid; k < K; k += NN)
      asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(peer_at(smem_at(gather + rank * K + k), 0)), "l"(S.best[k])
                   : "memory");
    select_sync<NS>();
    if (tid == 0) bar_arrive_peer(&S.gather[buf], 0);
    if (rank == 0) {
      bar_wait(&S.gather[buf], phase, &P.abort, a.errword);
      unsigned found = 0;
      for (unsigned i = tid; i < size * K; i += NN) {
        const unsigned long long mine = gather[i];
        if (!mine) continue;
        ++found;
        unsigned place = i % K;
        for (int q = 0; q < size; ++q) {
          if (q == int(i / K)) continue;
          unsigned l = 0, hi = K;  // the first place of list q that is not larger
          while (l < hi) {
            const unsigned mid = (l + hi) / 2;
            if (gather[q * K + mid] > mine) l = mid + 1;
            else hi = mid;
          }
          place += l;
        }
        if (place < K) put(place, mine);
      }
      int flip = 0;
      found = select_count<NS>(S, found, tid, flip);
      for (unsigned k = found + tid; k < K; k += NN) put(k, 0);
    }
    release();
    select_sync<NS>();
  }
}

template <int NW, bool TOP>
constexpr int finish_warps() { return TOP ? select_warps<NW>() : 1; }
template <int NW, bool TOP>
constexpr int logp_threads() { return (NW + 1 + finish_warps<NW, TOP>()) * 32; }

// NW warps compute, one streams the rows, and one (or, where alternatives are
// wanted, a few) finishes them, a row behind: joining a row's sums and selecting
// its largest are chains of short steps, which the next row's sums hide.
template <typename T, int NW, bool TOP, bool ENT>
__global__ void __launch_bounds__(logp_threads<NW, TOP>(), per_sm<NW>(!TOP)) logp_kernel(const LogpArgs a) {
  constexpr int G = NW * 32;
  __shared__ Pipe P;
  extern __shared__ __align__(128) unsigned char ring[];
  cg::cluster_group cl = cg::this_cluster();
  const int size = int(cl.num_blocks()), rank = int(cl.block_rank());
  const int64_t first = blockIdx.x / size, step = gridDim.x / size;
  const int tid = threadIdx.x;
  Select &S = *reinterpret_cast<Select *>(ring + a.stages * (G * U * 16));
  unsigned long long *gather = reinterpret_cast<unsigned long long *>(&S + 1);  // [2][size][K], the first CTA's
  float *keys = reinterpret_cast<float *>(gather + (size > 1 ? 2 * size * a.K : 0));
  if (TOP && tid == 0)
    for (int i = 0; i < 2; ++i) bar_init(&S.gather[i], size);
  pipe_init<NW>(P, a.stages, size, NW, finish_warps<NW, TOP>(), cl);
  if (tid < G)
    logp_rows<T, NW, TOP, ENT>(a, P, S, keys, ring, rank, size, first, step);
  else if (tid < G + 32)
    produce<T, NW>(P, ring, a.stages, a.x, a.ld, a.V, a.T, first, step, rank, size, false, a.errword,
                   GivenTokens{a.tokens, a.V, 0});
  else
    finish_rows<T, NW, TOP, ENT>(a, P, S, keys, gather, rank, size, first, step, tid - G - 32);
  if (size > 1) cl.sync();  // no CTA leaves while another may still write to its shared memory
}

// ------------------------------------------------------------------ writing a gradient row

// out[i] = f(x[i]) over a slice, in 16-byte units where out's rows are aligned
// as x's are.  f(index, value).
template <typename T, typename F>
__device__ __forceinline__ void map_slice(const T *x, T *out, const Slice<T> &sl, F f) {
  constexpr int E = Slice<T>::E;
  if (threadIdx.x < 32) {
    const int ih = sl.lo + int(threadIdx.x), it = sl.tail0 + int(threadIdx.x);
    if (int(threadIdx.x) < sl.head) out[ih] = from_float<T>(f(ih, to_float(x[ih])));
    if (it < sl.hi) out[it] = from_float<T>(f(it, to_float(x[it])));
  }
  const int b0 = sl.lo + sl.head;
  const bool same = ((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
  constexpr int U = 4;
  for (int i0 = 0; i0 < sl.nv; i0 += NT * U) {
    RowVec<T, E> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * NT + int(threadIdx.x);
      if (i < sl.nv) v[u].load(x + b0 + int64_t(i) * E);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * NT + int(threadIdx.x);
      if (i >= sl.nv) break;
      float g[E];
      v[u].get(g);
      const int at = b0 + i * E;
#pragma unroll
      for (int e = 0; e < E; ++e) g[e] = f(at + e, g[e]);
      if (same) {
        RowVec<T, E>::store(out + at, g);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) out[at + e] = from_float<T>(g[e]);
      }
    }
  }
}

template <typename T, int N>
__device__ __forceinline__ void zero_slice(T *out, int lo, int hi) {
  constexpr int E = Slice<T>::E;
  int head = int(((16 - (reinterpret_cast<uintptr_t>(out + lo) & 15)) & 15) / sizeof(T));
  if (head > hi - lo) head = hi - lo;
  if (int(threadIdx.x) < head) out[lo + threadIdx.x] = from_float<T>(0.f);
  const int nv = (hi - lo - head) / E;
  for (int i = threadIdx.x; i < nv; i += N)
    *reinterpret_cast<uint4 *>(out + lo + head + int64_t(i) * E) = make_uint4(0u, 0u, 0u, 0u);
  for (int i = lo + head + nv * E + int(threadIdx.x); i < hi; i += N) out[i] = from_float<T>(0.f);
}

struct LogpGradArgs {
  const void *x;
  void *out;
  int64_t ld, ldd;
  int V, parts;
  float scale;
  const int32_t *tokens;
  const float *saved, *dlogp, *dentropy;
  unsigned *errword;
};

// Part blockIdx % parts of row blockIdx / parts: element-wise given the
// forward's sums; the given token's element is put right last.
template <typename T>
__global__ void __launch_bounds__(NT) logp_grad_kernel(const LogpGradArgs a) {
  const int64_t row = blockIdx.x / a.parts;
  const int part = int(blockIdx.x % a.parts);
  const T *x = static_cast<const T *>(a.x) + row * a.ld;
  T *out = static_cast<T *>(a.out) + row * a.ldd;
  const Slice<T> sl = slice_of(x, a.V, part, a.parts);
  int token = -1;
  bool skip = false;
  if (a.tokens) {
    token = a.tokens[row];
    if (token >= a.V && threadIdx.x == 0 && part == 0) atomicOr(a.errword, unsigned(ERR_BOUNDS));
    skip = token < 0 || token >= a.V;
  }
  const float4 sv = reinterpret_cast<const float4 *>(a.saved)[row];
  if (skip || sv.x == -INFINITY) {
    zero_slice<T, NT>(out, sl.lo, sl.hi);
    return;
  }
  const float c = log2_scale(a.scale), L = sv.y * LOG2E;
  const float gl = a.dlogp ? a.dlogp[row] : 0.f, gh = a.dentropy ? a.dentropy[row] : 0.f;
  const bool mine = a.dlogp && token >= sl.lo && token < sl.hi;
  const float xt = mine ? to_float(x[token]) : 0.f;
  if (mine) __syncthreads();  // out may be x: every thread has read the token's logit
  const float M = sv.x;
  const float A = -gl * a.scale;
  float k;
  if (a.dentropy) {
    // -gl p - gh p (ln p + H) = p (B + C log2 p)
    // where p is 0 in float (below 2^-126), ln p stays small enough for its product with a large weight
    const float B = A - gh * a.scale * sv.z, C = -gh * a.scale * LN2;
    constexpr float NONE = -200.f;
    map_slice(x, out, sl, [=](int, float v) {
      const float d = fmaf(v - M, c, -L);
      return ex2(d) * fmaf(C, fmaxf(d, NONE), B);
    });
    const float d = fmaf(xt - M, c, -L);
    k = ex2(d) * fmaf(C, fmaxf(d, NONE), B);
  } else {
    map_slice(x, out, sl, [=](int, float v) { return A * ex2(fmaf(v - M, c, -L)); });
    k = A * ex2(fmaf(xt - M, c, -L));
  }
  if (mine) {
    __syncthreads();
    if (threadIdx.x == 0) out[token] = from_float<T>(k + gl * a.scale);
  }
}

// ------------------------------------------------------------------ distillation

struct DistillArgs {
  const void *x;
  void *out;
  int64_t ld, ldd, T;
  int V, K, tail, parts, stages;
  float scale, value_scale;
  const int32_t *tokens;
  const float *values, *dloss;
  float *loss, *saved;
  unsigned *errword;
};

// A row's teacher entries in shared memory.
constexpr int HASH = 256;
struct Teacher {
  int hash[HASH];    // -1 between rows
  float q[MAX_K], lq[MAX_K], x[MAX_K];
  float sum[MAX_K];  // of a token's first entry: the q of all its entries
  int idx[MAX_K];    // -1: left out
  int first[MAX_K];  // whether no earlier entry has the same token
  float rest;        // q_r where it counts: 0 with every token listed
  float mass;        // sum q + q_r, the mass that the loss counts: 1 unless the values sum to more, or leave nothing outside
  float m, s;        // running sum of the student's logits at the distinct tokens
  int live;          // entries that count
  // tail: the slice's vectors that the marks are of, and the marks of its ends
  int base, nv;
  unsigned head, behind;
};

// A row's entries as they are given, some to each lane of a warp, and the
// student's logits at those in [lo, hi).
struct Entries {
  static constexpr int Q = MAX_K / 32;  // entries of a lane: lane, lane + 32, ...
  int t[Q];
  float v[Q], x[Q];
  __device__ __forceinline__ void fetch(const DistillArgs &a, int64_t row) {
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      const int k = int(threadIdx.x & 31) + 32 * i;
      t[i] = k < a.K ? a.tokens[row * a.K + k] : -1;
      v[i] = k < a.K ? a.values[row * a.K + k] : 0.f;
    }
  }
  template <typename T>
  __device__ __forceinline__ void gather(const T *row, int lo, int hi) {
#pragma unroll
    for (int i = 0; i < Q; ++i) x[i] = t[i] >= lo && t[i] < hi ? to_float(row[t[i]]) : -INFINITY;
  }
};

// The entries' probabilities q and ln q.  One warp.
__device__ __forceinline__ void load_teacher(Teacher &S, const DistillArgs &a, const Entries &e, bool report) {
  constexpr int Q = Entries::Q;
  const int lane = threadIdx.x & 31;
  const float c = log2_scale(a.scale);
  int t[Q];
  float lq[Q], xs[Q], q[Q];
  float mx = -INFINITY;
  int n = 0;
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    t[i] = e.t[i];
    xs[i] = e.x[i];
    lq[i] = e.v[i];
    if (t[i] >= a.V && report) atomicOr(a.errword, unsigned(ERR_BOUNDS));
    if (t[i] < 0 || t[i] >= a.V) {
      t[i] = -1;
      lq[i] = -INFINITY;
    }
    if (lane + 32 * i < a.K) S.idx[lane + 32 * i] = t[i];
    mx = fmaxf(mx, lq[i]);
    n += t[i] >= 0;
  }
  n = __reduce_add_sync(0xffffffffu, n);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (a.tail || mx == -INFINITY) mx = 0.f;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    q[i] = 0.f;
    lq[i] = (lq[i] - mx) * a.value_scale;  // the difference first: the products alone may overflow
    if (32 * i < a.K && t[i] >= 0) q[i] = expf(lq[i]);
    s += q[i];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (!a.tail && s == 0.f) n = 0;  // nothing but -inf: no teacher
  const float ls = a.tail ? 0.f : logf(s), inv_s = n ? 1.f / s : 0.f;
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const int k = lane + 32 * i;
    lq[i] -= ls;
    if (!a.tail) q[i] *= inv_s;
    if (k < a.K) {
      S.q[k] = q[i];
      S.lq[k] = lq[i];
      S.x[k] = xs[i];
    }
  }
  __syncwarp();
  // a token's first entry, and the sum over all its entries: every entry's own unless a hash table (empty between
  // rows, at most half full) shows that a token is listed twice
  float sum[Q];
  bool first[Q], twice = false;
  int slot[Q];
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    first[i] = t[i] >= 0;
    sum[i] = q[i];
    slot[i] = -1;
    if (32 * i >= a.K || !first[i]) continue;
    for (int h = int((unsigned(t[i]) * 2654435761u) >> 24);; h = (h + 1) % HASH) {
      const int was = atomicCAS(&S.hash[h], -1, t[i]);
      if (was == -1) slot[i] = h;
      if (was == t[i]) twice = true;
      if (was == -1 || was == t[i]) break;
    }
  }
  twice = __any_sync(0xffffffffu, twice);
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    if (slot[i] >= 0) S.hash[slot[i]] = -1;
    if (twice) sum[i] = 0.f;
  }
  for (int j = 0; twice && j < a.K; ++j) {
    const int tj = S.idx[j];
    const float qj = S.q[j];
#pragma unroll
    for (int i = 0; i < Q; ++i)
      if (tj == t[i]) {
        first[i] = first[i] && j >= lane + 32 * i;
        sum[i] += qj;
      }
  }
  float m = -INFINITY, es = 0.f;
  int distinct = 0;
#pragma unroll
  for (int i = 0; i < Q; ++i)
    if (first[i]) {
      m = fmaxf(m, xs[i]);
      ++distinct;
    }
  m = of_key(__reduce_max_sync(0xffffffffu, key_of(m)));
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const int k = lane + 32 * i;
    if (first[i]) es += ex2((xs[i] - (m == -INFINITY ? 0.f : m)) * c);
    if (k < a.K) {
      S.first[k] = first[i];
      S.sum[k] = sum[i];
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) es += __shfl_xor_sync(0xffffffffu, es, o);
  distinct = __reduce_add_sync(0xffffffffu, distinct);
  if (lane == 0) {
    S.live = n;
    const float rest = 1.f - s;
    S.rest = a.tail && distinct < a.V && !(rest < float(n) * 1.1920929e-7f) ? rest : 0.f;
    S.mass = a.tail ? s + S.rest : 1.f;
    S.m = m;
    S.s = es;
  }
  __syncwarp();
}

// Puts the teacher's tokens of the slice [lo, hi) right after the other
// elements were written: (p (sum q + q_r) - q) g, all NaN in a row whose M is.
// All threads of the CTA that compute.
template <typename T>
__device__ __forceinline__ void write_teacher(const Teacher &S, const DistillArgs &a, T *out, int lo, int hi, float M,
                                              float logs, float g, int threads) {
  for (int k = threadIdx.x; k < a.K; k += threads)
    if (S.first[k] && S.idx[k] >= lo && S.idx[k] < hi) {
      const float p = S.x[k] == -INFINITY && M == M ? 0.f : ex2(fmaf(S.x[k] - M, log2_scale(a.scale), -logs * LOG2E));
      out[S.idx[k]] = from_float<T>((p * S.mass - S.sum[k]) * g);
    }
}

// The gradient of the tokens outside the teacher's: f exp(scale (x - M) - L).
struct Outside {
  float f, L;
};
__device__ __forceinline__ Outside outside_of(const Teacher &S, int tail, float logs, float ltail) {
  Outside o{1.f, logs};
  if (tail) {
    if (ltail == -INFINITY) {  // no token there, or only masked ones
      o.f = 0.f;
    } else {  // p_v (sum q + q_r - q_r / p_r) = exp(z_v - ltail) (p_r (sum q + q_r) - q_r)
      o.f = ex2((ltail - logs) * LOG2E) * S.mass - S.rest;
      o.L = ltail;
    }
  }
  return o;
}

// Whether a row has a teacher: the same decision as load_teacher's live.
struct HasTeacher {
  const DistillArgs &a;
  Entries e;
  __device__ __forceinline__ void fetch(int64_t row) { e.fetch(a, row); }
  __device__ __forceinline__ bool live() const {
    bool any = false;
#pragma unroll
    for (int i = 0; i < Entries::Q; ++i)
      any = any || (e.t[i] >= 0 && e.t[i] < a.V && (a.tail || e.v[i] != -INFINITY));
    return __any_sync(0xffffffffu, any);
  }
};

// The marks of a slice's vectors, a byte each.
template <typename T>
__host__ __device__ inline int mark_bytes_of(int V, int size) { return (V / Vec<T>::E / size + 2 + 15) / 16 * 16; }

// The part of two warps, every second row each: the teacher's entries of the
// rows to come (one warp alone would hold up the others: a row's entries are a
// long chain of few instructions).
template <typename T>
__device__ __forceinline__ void teacher_rows(const DistillArgs &a, Pipe &P, Teacher (&teachers)[2], unsigned char *marks,
                                             int mark_bytes, int rank, int size, int64_t first, int64_t step, int odd) {
  constexpr int E = Vec<T>::E;
  first += odd * step;
  step *= 2;
  Teacher &S = teachers[odd];
  unsigned *words = reinterpret_cast<unsigned *>(marks + odd * mark_bytes);
  // the entries are loaded two rows ahead, the logits at them one
  const T *x0 = static_cast<const T *>(a.x);
  Entries e, ahead;
  if (first < a.T) {
    e.fetch(a, first);
    e.gather(x0 + first * a.ld, 0, a.V);
    if (first + step < a.T) ahead.fetch(a, first + step);
  }
  uint32_t phase = 1;
  for (int64_t row = first; row < a.T; row += step, phase ^= 1) {
    const Entries now = e;
    if (row + step < a.T) {
      e = ahead;
      e.gather(x0 + (row + step) * a.ld, 0, a.V);
      if (row + 2 * step < a.T) ahead.fetch(a, row + 2 * step);
    }
    bar_wait(&P.hempty[odd], phase, &P.abort, a.errword);
    const T *x = static_cast<const T *>(a.x) + row * a.ld;
    const int lane = threadIdx.x & 31;
    if (a.tail)  // the marks of the buffer's last row
      for (int k = lane; k < a.K; k += 32) {
        const int i = S.idx[k] - S.base;
        if (S.nv && S.idx[k] >= 0 && i >= 0 && i < S.nv * E) words[i / E / 4] = 0u;
      }
    __syncwarp();
    load_teacher(S, a, now, rank == 0);
    if (a.tail) {
      const Slice<T> sl = slice_of(x, a.V, rank, size);
      const int base = sl.lo + sl.head;
      unsigned head = 0, behind = 0;
      for (int k = lane; k < a.K; k += 32) {
        const int t = S.idx[k], i = t - base;
        if (t < 0) continue;
        if (i >= 0 && i < sl.nv * E) atomicOr(&words[i / E / 4], 1u << (i / E % 4 * 8 + i % E));
        else if (t >= sl.lo && t < base) head |= 1u << (t - sl.lo);
        else if (t >= sl.tail0 && t < sl.hi) behind |= 1u << (t - sl.tail0);
      }
      __syncwarp();
      head = __reduce_or_sync(0xffffffffu, head);
      behind = __reduce_or_sync(0xffffffffu, behind);
      if (lane == 0) {
        S.base = base;
        S.nv = sl.nv;
        S.head = head;
        S.behind = behind;
      }
    }
    __syncwarp();
    if (lane == 0) bar_arrive(&P.hfull[odd]);
  }
}

// The computing warps' part.
template <typename T, int NW, bool GRAD>
__device__ __forceinline__ void distill_rows(const DistillArgs &a, Pipe &P, const Teacher (&teachers)[2],
                                             const unsigned char *ring, const unsigned char *marks, int mark_bytes,
                                             int rank, int size, int64_t first, int64_t step) {
  constexpr int G = NW * 32, SV = G * U, E = Vec<T>::E;
  const int tid = threadIdx.x;
  const float c = log2_scale(a.scale);
  Spot at;
  int par = 0;
  int64_t n = 0;
  for (int64_t row = first; row < a.T; row += step, ++n) {
    const T *x = static_cast<const T *>(a.x) + row * a.ld;
    const Slice<T> sl = slice_of(x, a.V, rank, size);
    T *out = GRAD ? static_cast<T *>(a.out) + row * a.ldd : nullptr;
    const Teacher &S = teachers[n & 1];
    bar_wait(&P.hfull[n & 1], uint32_t(n >> 1 & 1), &P.abort, a.errword);
    auto release = [&]() {
      __syncwarp();
      if ((tid & 31) == 0) bar_arrive(&P.hempty[n & 1]);
    };
    if (S.live == 0) {
      if (rank == 0 && tid == 0) {
        a.loss[row] = 0.f;
        if (a.saved) reinterpret_cast<float4 *>(a.saved)[row] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      if (GRAD) zero_slice<T, G>(out, sl.lo, sl.hi);
      release();
      continue;
    }
    const int nst = (sl.nv + SV - 1) / SV;
    const bool stays = GRAD && nst <= a.stages;
    const unsigned char *mark = marks + (n & 1) * mark_bytes;
    Run r;
    r.clear();
    float xh = -INFINITY, xt = -INFINITY;
    if (tid < 32) {
      if (tid < sl.head) xh = to_float(x[sl.lo + tid]);
      if (sl.tail0 + tid < sl.hi) xt = to_float(x[sl.tail0 + tid]);
      const bool mh = a.tail && (S.head >> tid & 1u), mt = a.tail && (S.behind >> tid & 1u);
      add_ends<T>(r, mh ? -INFINITY : xh, mt ? -INFINITY : xt, c);
    }
    Spot again = at;
    for (int k = 0; k < nst; ++k) {
      uint4 v[U];
      bar_wait(&P.full[at.st], at.ph, &P.abort, a.errword);
      read_stage<T, NW>(v, ring, at.st, sl.nv - k * SV);
      if (a.tail) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = k * SV + u * G + tid;
          const unsigned b = i < sl.nv ? mark[i] : 0u;
          if (b) Vec<T>::mask(v[u], b);
        }
      }
      add_vectors<T, false>(r, v, c);
      if (!stays) give_back(&P.empty[at.st]);
      at.next(a.stages);
    }
    Sums all = join_row<NW>(P, r, c, par, rank, size, a.errword);
    par ^= 1;
    // tail: `all` is the sum over the tokens outside the teacher's; add the teacher's
    float ltail = 0.f;
    if (a.tail) {
      const Sums o = all;
      all.m = fmaxf(o.m, S.m);
      all.s = o.s * ex2((o.m - all.base()) * c) + S.s * ex2((S.m - all.base()) * c);
      ltail = o.s == 0.f ? -INFINITY : (o.m - all.base()) * a.scale + logf(o.s);
    }
    const bool bad = !(all.s < INFINITY);
    const bool empty = all.s == 0.f;
    const float logs = logf(all.s);
    const float M = all.m;
    if (rank == 0 && tid < 32) {
      float l = 0.f;
      for (int k = tid; k < a.K; k += 32)
        if (S.idx[k] >= 0 && S.q[k] != 0.f)
          l += S.q[k] * (S.lq[k] - (empty || S.x[k] == -INFINITY ? -INFINITY : (S.x[k] - M) * a.scale - logs));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      if (tid == 0) {
        if (S.rest > 0.f)
          l += S.rest * (logf(S.rest) - (empty ? -INFINITY : ltail - logs));
        a.loss[row] = bad ? NAN : l;
        if (a.saved)
          reinterpret_cast<float4 *>(a.saved)[row] = make_float4(bad ? NAN : M, bad ? NAN : logs, 0.f, bad ? NAN : ltail);
      }
    }
    if (GRAD) {
      const float g = (a.dloss ? a.dloss[row] : 1.f) * a.scale;
      Outside o = outside_of(S, a.tail, logs, ltail);
      if (bad) o.f = NAN;
      // a row of masks: 0 everywhere
      const float A = empty ? 0.f : o.f * g, L = empty ? 0.f : o.L * LOG2E, base = empty ? 0.f : M;
      // the exponent c (v - M) - L as c v + k, with what k's rounding leaves taken into the factor; where M is far,
      // in two steps
      const bool far = !(fabsf(base * c) < FAR);
      const float mc = base * c, k = -mc - L, kb = k + mc;
      const float left = fmaf(-base, c, mc) + ((-mc - (k - kb)) + (-L - kb));  // -base c - L - k
      const float2 A2 = both(far ? A : A * ex2(left)), k2 = both(far ? -base : k), nL = both(-L), c2 = both(c);
      auto grad = [&](float2 v) {
        const float2 d = far ? fma2(add2(v, k2), c2, nL) : fma2(v, c2, k2);
        return mul2(ex2(d), A2);
      };
      T *to = out + sl.lo + sl.head;
      const bool aligned = (reinterpret_cast<uintptr_t>(to) & 15) == 0;
      if (tid < 32) {
        if (tid < sl.head) out[sl.lo + tid] = from_float<T>(grad(both(xh)).x);
        if (sl.tail0 + tid < sl.hi) out[sl.tail0 + tid] = from_float<T>(grad(both(xt)).x);
      }
      Spot &from = stays ? again : at;
      for (int k = 0; k < nst; ++k) {
        uint4 v[U];
        if (!stays) bar_wait(&P.full[from.st], from.ph, &P.abort, a.errword);
        read_stage<T, NW>(v, ring, from.st, sl.nv - k * SV);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = k * SV + u * G + tid;
          if (i >= sl.nv) break;
          float2 f[E / 2];
          Vec<T>::get(v[u], f);
#pragma unroll
          for (int e = 0; e < E / 2; ++e) f[e] = grad(f[e]);
          if (aligned) {
            *reinterpret_cast<uint4 *>(to + int64_t(i) * E) = Vec<T>::put(f);
          } else {
#pragma unroll
            for (int e = 0; e < E; ++e) to[int64_t(i) * E + e] = from_float<T>(e & 1 ? f[e / 2].y : f[e / 2].x);
          }
        }
        give_back(&P.empty[from.st]);
        from.next(a.stages);
      }
      warps_sync<NW>();
      if (!empty) write_teacher(S, a, out, sl.lo, sl.hi, bad ? NAN : M, logs, g, G);
    }
    release();
  }
}

// NW warps compute, one streams the rows, two load the teacher's entries of the
// rows to come.  With the tail as one more outcome the sum runs over the
// tokens outside the teacher's alone (they may be all that is left of 1 in
// float), so the teacher's are marked, a bit each, and masked as they are read.
// A row whose slice fits the ring stays there for its gradient; a longer one is
// streamed a second time (from L2).
template <typename T, int NW, bool GRAD>
__global__ void __launch_bounds__((NW + 3) * 32, per_sm<NW>(false)) distill_kernel(const DistillArgs a) {
  constexpr int G = NW * 32;
  __shared__ Pipe P;
  __shared__ Teacher teachers[2];
  extern __shared__ __align__(128) unsigned char ring[];
  cg::cluster_group cl = cg::this_cluster();
  const int size = int(cl.num_blocks()), rank = int(cl.block_rank());
  const int64_t first = blockIdx.x / size, step = gridDim.x / size;
  const int tid = threadIdx.x;
  const int mark_bytes = a.tail ? mark_bytes_of<T>(a.V, size) : 0;
  unsigned char *marks = ring + a.stages * (G * U * 16);
  for (int i = tid; i < 2 * mark_bytes / 4; i += (NW + 3) * 32) reinterpret_cast<unsigned *>(marks)[i] = 0u;
  if (tid < 2) teachers[tid].nv = 0;
  for (int i = tid; i < 2 * HASH; i += (NW + 3) * 32) teachers[i / HASH].hash[i % HASH] = -1;
  pipe_init<NW>(P, a.stages, size, 1, NW, cl);
  if (tid >= G + 32)
    teacher_rows<T>(a, P, teachers, marks, mark_bytes, rank, size, first, step, (tid - G - 32) / 32);
  else if (tid >= G)
    produce<T, NW>(P, ring, a.stages, a.x, a.ld, a.V, a.T, first, step, rank, size, GRAD, a.errword,
                   HasTeacher{a, {}});
  else
    distill_rows<T, NW, GRAD>(a, P, teachers, ring, marks, mark_bytes, rank, size, first, step);
  if (size > 1) cl.sync();  // no CTA leaves while another may still write to its shared memory
}

template <typename T>
__global__ void __launch_bounds__(NT) distill_grad_kernel(const DistillArgs a) {
  __shared__ Teacher S;
  const int64_t row = blockIdx.x / a.parts;
  const int part = int(blockIdx.x % a.parts);
  const T *x = static_cast<const T *>(a.x) + row * a.ld;
  T *out = static_cast<T *>(a.out) + row * a.ldd;
  const Slice<T> sl = slice_of(x, a.V, part, a.parts);
  for (int i = threadIdx.x; i < HASH; i += NT) S.hash[i] = -1;
  __syncthreads();
  // only this part's logits: in place, the other parts may already be gradients
  if (threadIdx.x < 32) {
    Entries e;
    e.fetch(a, row);
    e.gather(x, sl.lo, sl.hi);
    load_teacher(S, a, e, part == 0);
  }
  __syncthreads();
  const float4 sv = reinterpret_cast<const float4 *>(a.saved)[row];
  if (S.live == 0 || sv.x == -INFINITY) {
    zero_slice<T, NT>(out, sl.lo, sl.hi);
    return;
  }
  const float c = log2_scale(a.scale);
  const float g = (a.dloss ? a.dloss[row] : 1.f) * a.scale;
  const Outside o = outside_of(S, a.tail, sv.y, sv.w);
  const float A = o.f * g, L = o.L * LOG2E, M = sv.x;
  map_slice(x, out, sl, [=](int, float v) { return A * ex2(fmaf(v - M, c, -L)); });
  __syncthreads();
  write_teacher(S, a, out, sl.lo, sl.hi, M, sv.y, g, NT);
}

// ------------------------------------------------------------------ launch shapes and checks

// CTAs of a row.  One per row where there are rows enough for every SM; with
// fewer, a row is split so that the GPU has two CTAs per SM or the slices fall
// to 4096 columns, whichever comes first.  Alternatives are selected from every
// slice and merged, which costs more the more of both there are: their slices
// stay above 16384 columns, and at most four and 256 / K share a row.  Measured
// (us, 1 / 2 / 4 / 8 CTAs a row of four warps): 4 rows of 32000 without 4.8 / 4.7
// / 4.2 / 4.3, with 20 10.7 / 10.8 / 11.5 / 16.5; 4 of 128000 without 10.4 / 7.5 /
// 5.7 / 4.8, with 20 22.5 / 16.6 / 14.5 / 17.9, with 128 23.5 / 21.2 / 22.6 / 40.9.  A slice
// has at most SLICE columns.
int cluster_of(int64_t T, int V, int K = 0) {
  const int least = K ? 16384 : 4096, most = K ? std::max(1, std::min(4, 256 / K)) : MAX_CLUSTER;
  int c = 1;
  while (c < MAX_CLUSTER &&
         ((2 * c <= most && T * c < int64_t(num_sms()) * 2 && V / (2 * c) >= least) || V > int64_t(SLICE) * c))
    c *= 2;
  return c;
}

// Parts of a row for the element-wise gradients: at most 32768 columns each,
// and enough CTAs for every SM where a part keeps 4096.
int parts_of(int64_t T, int V) {
  int64_t p = (V + 32767) / 32768;
  while (T * p < int64_t(num_sms()) * 2 && V / (2 * p) >= 4096) p *= 2;
  return int(p);
}

poet_status check_logits(const char *what, const void *x, int64_t ld, int32_t dtype, int64_t T, int32_t V, float scale) {
  POET_REQUIRE(dtype == POET_F32 || dtype == POET_BF16, "%s: bad dtype %d", what, dtype);
  POET_REQUIRE(V >= 1 && V <= MAX_V, "%s: V=%d outside 1..%d", what, V, MAX_V);
  POET_REQUIRE(T >= 0 && T <= (int64_t(1) << 24), "%s: T=%lld outside 0..2^24", what, (long long)T);
  POET_REQUIRE(std::isfinite(scale) && scale > 0.f, "%s: scale must be positive", what);
  if (T == 0) return POET_OK;
  POET_REQUIRE(x != nullptr, "%s: logits is NULL", what);
  POET_REQUIRE((reinterpret_cast<uintptr_t>(x) & (esize(dtype) - 1)) == 0, "%s: logits not aligned to its elements", what);
  POET_REQUIRE(ld >= V, "%s: row stride %lld below V=%d", what, (long long)ld, V);
  return POET_OK;
}
poet_status check_out(const char *what, const void *x, int64_t ld, const void *out, int64_t ldd, int32_t dtype, int32_t V) {
  POET_REQUIRE(out != nullptr, "%s: dlogits is NULL", what);
  POET_REQUIRE((reinterpret_cast<uintptr_t>(out) & (esize(dtype) - 1)) == 0, "%s: dlogits not aligned to its elements", what);
  POET_REQUIRE(ldd >= V, "%s: row stride %lld of dlogits below V=%d", what, (long long)ldd, V);
  POET_REQUIRE(out != x || ldd == ld, "%s: dlogits is logits with another row stride", what);
  return POET_OK;
}
bool al(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// How the rows are spread: CTAs of NW computing warps, clusters of `cluster` of
// them, and the stages that fit beside `extra` bytes (and the `fixed` ones of the
// kernel's static shared memory and the system) where `per_sm` CTAs share an SM.
struct Spread {
  int cluster, stages;
  unsigned grid;
  size_t smem;
};
template <int NW>
Spread spread(int64_t rows, int cluster, size_t extra, size_t fixed, int per_sm) {
  constexpr size_t STAGE = size_t(NW) * 32 * U * 16, SM = 228 * 1024;
  Spread s;
  s.cluster = cluster;
  size_t left = 0;
  for (;; --per_sm) {  // at least three stages, or two of one CTA alone
    left = std::min<size_t>(SM / per_sm, 227 * 1024) - fixed;
    if (left >= extra + 3 * STAGE || per_sm == 1) break;
  }
  s.stages = int(std::min<size_t>((left - extra) / STAGE, MAX_STAGES));
  s.smem = s.stages * STAGE + extra;
  s.grid = unsigned(std::max<int64_t>(1, std::min<int64_t>(rows, int64_t(num_sms()) * per_sm / cluster)) * cluster);
  return s;
}

template <auto KERN, typename A>
poet_status launch_rows(const A &a, const Spread &s, int threads, cudaStream_t st, const char *what) {
  POET_TRY(allow_smem<KERN>(s.smem));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(s.cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(s.grid);
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = s.smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  POET_CUDA_TRY(cudaLaunchKernelEx(&cfg, KERN, a));
  count_launch();
  return launch_status(what);
}

// How many warps work on a row, by its bytes: fewer of them let more rows share an
// SM, which hides what comes between a row's passes, and more read a long row
// faster.  Measured (us on the GPU, 512 MB of logits, two / four / eight warps):
//   loss and gradient, bf16: rows of 4096 467 / 470 / 749, of 6000 420 / 425 / 526, of 7000 422 / 379 / 467, of
//     50257 285 / 232 / 247, of 56000 276 / 257 / 229, of 128000 301 / 281 / 268
//   float: of 3000 313 / 340 / 470, of 4096 265 / 255 / 336, of 8192 221 / 190 / 218, of 15000 223 / 186 / 187, of
//     16000 237 / 209 / 181, of 28000 272 / 247 / 195
//   log probabilities without alternatives, bf16: of 6000 152 / 173 / 197, of 7000 163 / 150 / 170, of 12000 134 /
//     119 / 152, of 28000 119 / 105 / 113, of 32000 121 / 103 / 101, of 128000 114 / 101 / 95
//   float: of 3000 114 / 136 / 164, of 4096 101 / 97 / 115, of 8192 88 / 91 / 86, of 16000 97 / 92 / 89
// The loss alone takes the warps of the loss with its gradient, and so its bits.
constexpr int64_t KB = 1024, NARROW = 13 * KB, LOGP_FOUR = 56 * KB, ALTERNATIVES_FOUR = 112 * KB;
template <typename T>
constexpr int64_t DISTILL_FOUR = (sizeof(T) == 2 ? 104 : 60) * KB;
constexpr int NARROW_SELECT = 8192;  // columns, with alternatives

template <typename T, int NW>
poet_status run_logp(LogpArgs &a, int cluster, cudaStream_t st) {
  const int64_t nv = a.V / Vec<T>::E / cluster + 1, nst = (nv + NW * 32 * U - 1) / (NW * 32 * U);
  a.key_floats = int(nst) * NW * 32;
  size_t extra = 0;
  if (a.K) extra = sizeof(Select) + (cluster > 1 ? size_t(2) * cluster * a.K * 8 : 0) + size_t(2) * a.key_floats * 4;
  const Spread s = spread<NW>(a.T, cluster, extra, 2048, per_sm<NW>(!a.K));
  a.stages = s.stages;
  // A caller that wants neither the entropy nor saved (which holds it) does without its sum.  Measured with / without
  // (us on the GPU, bf16): 16384 rows of 32000 191 / 180, 4096 of 128000 with 64 alternatives 223 / 210.
  const bool ent = a.entropy || a.saved;
  if (a.K)
    return ent ? launch_rows<logp_kernel<T, NW, true, true>>(a, s, logp_threads<NW, true>(), st, "logprobs")
               : launch_rows<logp_kernel<T, NW, true, false>>(a, s, logp_threads<NW, true>(), st, "logprobs");
  return ent ? launch_rows<logp_kernel<T, NW, false, true>>(a, s, logp_threads<NW, false>(), st, "logprobs")
             : launch_rows<logp_kernel<T, NW, false, false>>(a, s, logp_threads<NW, false>(), st, "logprobs");
}
template <typename T>
poet_status run_logp(LogpArgs &a, cudaStream_t st) {
  const int cluster = cluster_of(a.T, a.V, a.K);
  // A selection takes as long for short rows as for long ones, so with few alternatives more and smaller CTAs share
  // an SM; many need the maxima of many threads.  Measured with four warps / eight (us): 8192 rows of 32000 bf16
  // with 20 142 / 192, with 64 232 / 248; 4096 of 64000 with 20 117 / 127, with 64 173 / 161; 4096 of 128000 with
  // 64 232 / 223; of float 5592 of 24000 with 64 157 / 169, 4194 of 32000 159 / 146.  With two / four warps and 20:
  // bf16 44739 of 6000 372 / 460, 32768 of 8192 295 / 337, 22369 of 12000 233 / 256 but 400 of 12000 12.9 / 11.0; float
  // 16384 of 8192 151 / 170, 400 of 12000 14.9 / 13.0; with 64, 32768 of 8192 973 / 603.
  // With a row an SM at most there is nothing to share and eight warps are the quickest (two or four / eight on the
  // GPU, with 20: 4 rows of 8000 8.2 / 7.4, of 32000 10.6 / 9.4, of 128000 14.8 / 12.2; of 1000, where eight warps
  // have no logits for every thread, 6.6 / 13.7).
  if (a.K && a.T <= num_sms() && a.V >= 4096) return run_logp<T, 8>(a, cluster, st);
  const int64_t bytes = int64_t(a.V) * int64_t(sizeof(T));
  if (a.K ? a.V <= NARROW_SELECT && a.K <= 32 : bytes <= NARROW) return run_logp<T, 2>(a, cluster, st);
  if (a.K ? a.K <= 32 || (a.K <= 64 && bytes <= ALTERNATIVES_FOUR) : bytes <= LOGP_FOUR)
    return run_logp<T, 4>(a, cluster, st);
  return run_logp<T, 8>(a, cluster, st);
}

template <typename T, int NW>
poet_status run_distill(DistillArgs &a, int cluster, cudaStream_t st) {
  constexpr int THREADS = (NW + 3) * 32;
  const size_t marks = a.tail ? mark_bytes_of<T>(a.V, cluster) : 0;
  const Spread s = spread<NW>(a.T, cluster, 2 * marks, 11 * 1024, per_sm<NW>(false));
  a.stages = s.stages;
  return a.out ? launch_rows<distill_kernel<T, NW, true>>(a, s, THREADS, st, "distill")
               : launch_rows<distill_kernel<T, NW, false>>(a, s, THREADS, st, "distill");
}
template <typename T>
poet_status run_distill(DistillArgs &a, cudaStream_t st) {
  const int cluster = cluster_of(a.T, a.V);
  const int64_t bytes = int64_t(a.V) * int64_t(sizeof(T));
  if (bytes <= NARROW) return run_distill<T, 2>(a, cluster, st);
  return bytes <= DISTILL_FOUR<T> ? run_distill<T, 4>(a, cluster, st) : run_distill<T, 8>(a, cluster, st);
}

poet_status check_teacher(const char *what, const int32_t *tokens, const float *values, int32_t K, float value_scale,
                          int32_t tail, const float *dloss, int64_t T) {
  POET_REQUIRE(K >= 1 && K <= MAX_K, "%s: K=%d outside 1..%d", what, K, MAX_K);
  POET_REQUIRE(std::isfinite(value_scale) && value_scale > 0.f, "%s: value_scale must be positive", what);
  POET_REQUIRE(tail == 0 || tail == 1, "%s: tail %d must be 0 or 1", what, tail);
  if (T == 0) return POET_OK;
  POET_REQUIRE(tokens && values && al(tokens, 4) && al(values, 4),
               "%s: teacher_tokens / teacher_values NULL or not 4-byte aligned", what);
  POET_REQUIRE(al(dloss, 4), "%s: dloss not 4-byte aligned", what);
  return POET_OK;
}

}  // namespace
}  // namespace poet

using namespace poet;

extern "C" {

poet_status poet_token_logprobs(const void *logits, int64_t ld, int32_t dtype, int64_t T, int32_t V, float scale,
                                const int32_t *tokens, int32_t topk, float *logp, float *entropy, int32_t *top_tokens,
                                float *top_logp, float *saved, poet_stream stream) {
  CallRange nvtx_range("poet_token_logprobs");
  clear_error();
  const char *what = "poet_token_logprobs";
  POET_TRY(check_logits(what, logits, ld, dtype, T, V, scale));
  POET_REQUIRE(topk >= 0 && topk <= MAX_K, "%s: topk=%d outside 0..%d", what, topk, MAX_K);
  if (T == 0) return POET_OK;
  POET_REQUIRE(al(tokens, 4) && al(logp, 4) && al(entropy, 4) && al(top_tokens, 4) && al(top_logp, 4),
               "%s: a buffer is not 4-byte aligned", what);
  POET_REQUIRE(al(saved, 16), "%s: saved not 16-byte aligned", what);
  POET_REQUIRE(tokens || !logp, "%s: logp without tokens", what);
  POET_REQUIRE(topk ? (top_tokens && top_logp) : (!top_tokens && !top_logp),
               "%s: top_tokens and top_logp go with topk > 0", what);
  LogpArgs a{};
  a.x = logits; a.ld = ld; a.T = T; a.V = V; a.K = topk; a.scale = scale; a.tokens = tokens;
  a.logp = logp; a.entropy = entropy; a.top_tokens = top_tokens; a.top_logp = top_logp; a.saved = saved;
  a.errword = device_errword();
  POET_REQUIRE(a.errword != nullptr, "%s: no device status word", what);
  TraceScope ts("logprobs", 6.0 * double(T) * V, double(T) * V * double(esize(dtype)),
                reinterpret_cast<cudaStream_t>(stream));
  return dtype == POET_BF16 ? run_logp<bf16>(a, reinterpret_cast<cudaStream_t>(stream))
                            : run_logp<float>(a, reinterpret_cast<cudaStream_t>(stream));
}

poet_status poet_token_logprobs_grad(const void *logits, int64_t ld, int32_t dtype, int64_t T, int32_t V, float scale,
                                     const int32_t *tokens, const float *saved, const float *dlogp,
                                     const float *dentropy, void *dlogits, int64_t ldd, poet_stream stream) {
  CallRange nvtx_range("poet_token_logprobs_grad");
  clear_error();
  const char *what = "poet_token_logprobs_grad";
  POET_TRY(check_logits(what, logits, ld, dtype, T, V, scale));
  if (T == 0) return POET_OK;
  POET_TRY(check_out(what, logits, ld, dlogits, ldd, dtype, V));
  POET_REQUIRE(saved && al(saved, 16), "%s: saved NULL or not 16-byte aligned", what);
  POET_REQUIRE(al(tokens, 4) && al(dlogp, 4) && al(dentropy, 4), "%s: a buffer is not 4-byte aligned", what);
  POET_REQUIRE(dlogp || dentropy, "%s: dlogp and dentropy are both NULL", what);
  POET_REQUIRE(tokens || !dlogp, "%s: dlogp without tokens", what);
  LogpGradArgs a{};
  a.x = logits; a.out = dlogits; a.ld = ld; a.ldd = ldd; a.V = V; a.parts = parts_of(T, V); a.scale = scale;
  a.tokens = tokens; a.saved = saved; a.dlogp = dlogp; a.dentropy = dentropy;
  a.errword = device_errword();
  POET_REQUIRE(a.errword != nullptr, "%s: no device status word", what);
  POET_REQUIRE(T * a.parts < (int64_t(1) << 31), "%s: T=%lld rows of %d columns are too many for one call", what,
               (long long)T, V);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  TraceScope ts("logprobs_grad", 8.0 * double(T) * V, 2.0 * double(T) * V * double(esize(dtype)), st);
  const unsigned grid = unsigned(T * a.parts);
  if (dtype == POET_BF16) logp_grad_kernel<bf16><<<grid, NT, 0, st>>>(a);
  else logp_grad_kernel<float><<<grid, NT, 0, st>>>(a);
  count_launch();
  return launch_status("logprobs_grad");
}

poet_status poet_distill_topk(const void *logits, int64_t ld, int32_t dtype, int64_t T, int32_t V, float scale,
                              const int32_t *teacher_tokens, const float *teacher_values, int32_t K, float value_scale,
                              int32_t tail, const float *dloss, float *loss, float *saved, void *dlogits, int64_t ldd,
                              poet_stream stream) {
  CallRange nvtx_range("poet_distill_topk");
  clear_error();
  const char *what = "poet_distill_topk";
  POET_TRY(check_logits(what, logits, ld, dtype, T, V, scale));
  POET_TRY(check_teacher(what, teacher_tokens, teacher_values, K, value_scale, tail, dloss, T));
  if (T == 0) return POET_OK;
  POET_REQUIRE(loss && al(loss, 4), "%s: loss NULL or not 4-byte aligned", what);
  POET_REQUIRE(al(saved, 16), "%s: saved not 16-byte aligned", what);
  if (dlogits) POET_TRY(check_out(what, logits, ld, dlogits, ldd, dtype, V));
  DistillArgs a{};
  a.x = logits; a.out = dlogits; a.ld = ld; a.ldd = ldd; a.T = T; a.V = V; a.K = K; a.tail = tail; a.scale = scale;
  a.value_scale = value_scale; a.tokens = teacher_tokens; a.values = teacher_values; a.dloss = dloss;
  a.loss = loss; a.saved = saved;
  a.errword = device_errword();
  POET_REQUIRE(a.errword != nullptr, "%s: no device status word", what);
  TraceScope ts("distill", 10.0 * double(T) * V, (dlogits ? 2.0 : 1.0) * double(T) * V * double(esize(dtype)),
                reinterpret_cast<cudaStream_t>(stream));
  return dtype == POET_BF16 ? run_distill<bf16>(a, reinterpret_cast<cudaStream_t>(stream))
                            : run_distill<float>(a, reinterpret_cast<cudaStream_t>(stream));
}

poet_status poet_distill_topk_grad(const void *logits, int64_t ld, int32_t dtype, int64_t T, int32_t V, float scale,
                                   const int32_t *teacher_tokens, const float *teacher_values, int32_t K,
                                   float value_scale, int32_t tail, const float *saved, const float *dloss,
                                   void *dlogits, int64_t ldd, poet_stream stream) {
  CallRange nvtx_range("poet_distill_topk_grad");
  clear_error();
  const char *what = "poet_distill_topk_grad";
  POET_TRY(check_logits(what, logits, ld, dtype, T, V, scale));
  POET_TRY(check_teacher(what, teacher_tokens, teacher_values, K, value_scale, tail, dloss, T));
  if (T == 0) return POET_OK;
  POET_TRY(check_out(what, logits, ld, dlogits, ldd, dtype, V));
  POET_REQUIRE(saved && al(saved, 16), "%s: saved NULL or not 16-byte aligned", what);
  DistillArgs a{};
  a.x = logits; a.out = dlogits; a.ld = ld; a.ldd = ldd; a.T = T; a.V = V; a.K = K; a.tail = tail; a.scale = scale;
  a.value_scale = value_scale; a.tokens = teacher_tokens; a.values = teacher_values; a.dloss = dloss;
  a.saved = const_cast<float *>(saved);
  a.parts = parts_of(T, V);
  a.errword = device_errword();
  POET_REQUIRE(a.errword != nullptr, "%s: no device status word", what);
  POET_REQUIRE(T * a.parts < (int64_t(1) << 31), "%s: T=%lld rows of %d columns are too many for one call", what,
               (long long)T, V);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  TraceScope ts("distill_grad", 5.0 * double(T) * V, 2.0 * double(T) * V * double(esize(dtype)), st);
  const unsigned grid = unsigned(T * a.parts);
  if (dtype == POET_BF16) distill_grad_kernel<bf16><<<grid, NT, 0, st>>>(a);
  else distill_grad_kernel<float><<<grid, NT, 0, st>>>(a);
  count_launch();
  return launch_status("distill_grad");
}

}  // extern "C"
