// Operators on rows of logits: log probabilities of given tokens with entropy
// and top alternatives, distillation from a teacher's top logits, and their
// gradients.
//
// A row of V logits is worked on by a cluster of C CTAs (C = 1 where there are
// rows enough to fill the GPU), each with a contiguous slice.  One pass over
// the slice keeps, per thread, the running maximum m, s = sum exp(c (x - m))
// and t = sum exp(c (x - m)) c (x - m); these are joined through shuffles,
// shared memory and the cluster's distributed shared memory, always in one
// order.  c = scale log2(e), so an exponential is one ex2; differences to the
// maximum are formed before they are scaled, so neither large logits nor masks
// of the type's lowest value lose anything.
//
// HBM-bound: the forward reads the logits once.  The fused loss + gradient
// reads them again in its second pass, from L2.
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
constexpr int NT = 256;
constexpr int NW = NT / 32;
constexpr int CAND = 1024;     // candidates kept at once by the selection
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr float LOWEST = -1e30f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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
  const int b0 = int(int64_t(nv) * rank / size), b1 = int(int64_t(nv) * (rank + 1) / size);
  s.lo = rank == 0 ? 0 : head + b0 * E;
  s.head = rank == 0 ? head : 0;
  s.nv = b1 - b0;
  s.tail0 = head + b1 * E;
  s.hi = rank == size - 1 ? V : s.tail0;
  return s;
}

// The running sums of some logits of a row.
struct Run {
  float m, s, t;
  __device__ __forceinline__ void clear() { m = -INFINITY; s = 0.f; t = 0.f; }
  // Move to maximum mx >= m.
  __device__ __forceinline__ void raise(float mx, float c) {
    const float base = mx == -INFINITY ? 0.f : mx;
    const float d = fmaxf((m - base) * c, LOWEST);
    const float f = ex2((m - base) * c);
    t = fmaf(s, d, t) * f;
    s *= f;
    m = mx;
  }
  __device__ __forceinline__ float base() const { return m == -INFINITY ? 0.f : m; }
  template <bool ENT>
  __device__ __forceinline__ void add(float x, float b, float c) {
    const float d = (x - b) * c;
    const float e = ex2(d);
    s += e;
    if (ENT) t = fmaf(e, fmaxf(d, LOWEST), t);
  }
  __device__ __forceinline__ void join(float om, float os, float ot, float c) {
    Run o{om, os, ot};
    const float mx = fmaxf(m, om);
    raise(mx, c);
    o.raise(mx, c);
    s += o.s;
    t += o.t;
  }
  __device__ __forceinline__ void join_warp(float c) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float om = __shfl_xor_sync(0xffffffffu, m, o), os = __shfl_xor_sync(0xffffffffu, s, o),
                  ot = __shfl_xor_sync(0xffffffffu, t, o);
      // both sides of a pair join in the same order, so that they agree to the bit
      if ((threadIdx.x & o) == 0) {
        join(om, os, ot, c);
      } else {
        Run a{om, os, ot};
        a.join(m, s, t, c);
        *this = a;
      }
    }
  }
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

template <typename T>
__device__ __forceinline__ void load_vec(const T *p, float (&f)[16 / sizeof(T)]) {
  RowVec<T, 16 / sizeof(T)> v;
  v.load(p);
  v.get(f);
}

// ------------------------------------------------------------------ selection of the largest

struct SelectSmem {
  unsigned long long cand[CAND];
  unsigned long long best[MAX_K];
  unsigned list[256];
  unsigned n, m;
  unsigned count;
};

// Number of items for which the predicate holds over the CTA's threads.
__device__ __forceinline__ unsigned cta_sum(unsigned v, unsigned *cell) {
  v = __reduce_add_sync(0xffffffffu, v);
  if (threadIdx.x == 0) *cell = 0;
  __syncthreads();
  if ((threadIdx.x & 31) == 0 && v) atomicAdd(cell, v);
  __syncthreads();
  const unsigned total = *cell;
  __syncthreads();
  return total;
}

// A bound with between `least` and `most` items at or above it, by bisection of
// the 64-bit order (which has no ties, so it ends); 0 if there are no more than
// `most` items.  count(b): the thread's number of items >= b.
template <typename F>
__device__ unsigned long long bound_for(unsigned least, unsigned most, unsigned long long hi, unsigned *cell, F count) {
  unsigned long long lo = 0;  // count(lo) > most, count(hi) < least
  for (;;) {
    const unsigned long long mid = lo + (hi - lo) / 2;
    const unsigned c = cta_sum(count(mid), cell);
    if (c < least) hi = mid;
    else if (c > most) lo = mid;
    else return mid;
    if (hi - lo <= 1) return lo;  // not reached: orders are distinct
  }
}

// From n candidates in S.cand (distinct) the K largest, in falling order, to
// S.best (0 where there are fewer); n <= CAND.
__device__ void rank_candidates(SelectSmem &S, unsigned n, unsigned K) {
  for (unsigned i = threadIdx.x; i < K; i += NT)
    if (i >= n) S.best[i] = 0;
  for (unsigned i = threadIdx.x; i < n; i += NT) {
    const unsigned long long mine = S.cand[i];
    unsigned above = 0;
    for (unsigned j = 0; j < n; ++j) above += S.cand[j] > mine;
    if (above < K) S.best[above] = mine;
  }
  __syncthreads();
}

// ------------------------------------------------------------------ log probabilities

struct LogpArgs {
  const void *x;
  int64_t ld;
  int V, K;
  float scale;
  const int32_t *tokens;
  float *logp, *entropy, *top_logp, *saved;
  int32_t *top_tokens;
  unsigned *errword;
};

// Shared memory of a row's slice when alternatives are wanted: the largest
// logit of every chunk of CHUNK vectors (as ordered keys), chunk 0 being the
// elements before the first vector and the last one those behind the last.
constexpr int CHUNK = 4;
template <typename T>
__device__ __host__ inline int chunks_of(int nv) { return (nv + CHUNK - 1) / CHUNK + 2; }

template <typename T, bool TOP, bool ENT>
__global__ void __launch_bounds__(NT) logp_kernel(const LogpArgs a) {
  constexpr int E = Slice<T>::E;
  __shared__ float sm_m[NW], sm_s[NW], sm_t[NW];
  __shared__ float part[3];
  extern __shared__ __align__(16) unsigned char dyn[];
  cg::cluster_group cl = cg::this_cluster();
  const int size = int(cl.num_blocks()), rank = int(cl.block_rank());
  const int64_t row = blockIdx.x / size;
  const T *x = static_cast<const T *>(a.x) + row * a.ld;
  const float c = a.scale * LOG2E;
  int token = -1;
  bool skip = false;
  if (a.tokens) {
    token = a.tokens[row];
    if (token >= a.V && threadIdx.x == 0 && rank == 0) atomicOr(a.errword, unsigned(ERR_BOUNDS));
    skip = token < 0 || token >= a.V;
  }
  if (skip) {  // the whole cluster takes this way
    if (rank != 0) return;
    if (threadIdx.x == 0) {
      if (a.logp) a.logp[row] = 0.f;
      if (a.entropy) a.entropy[row] = 0.f;
      if (a.saved) reinterpret_cast<float4 *>(a.saved)[row] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int k = threadIdx.x; k < a.K; k += NT) {
      a.top_tokens[row * a.K + k] = -1;
      a.top_logp[row * a.K + k] = -INFINITY;
    }
    return;
  }
  const Slice<T> sl = slice_of(x, a.V, rank, size);
  SelectSmem &S = *reinterpret_cast<SelectSmem *>(dyn);
  uint32_t *keys = reinterpret_cast<uint32_t *>(dyn + (TOP ? sizeof(SelectSmem) : 0));
  const int nchunks = chunks_of<T>(sl.nv);
  Run r;
  r.clear();
  // the ragged ends: at most E - 1 elements each, one per thread of the first warp
  if (threadIdx.x < 32) {
    const int ih = sl.lo + int(threadIdx.x), it = sl.tail0 + int(threadIdx.x);
    const bool ph = int(threadIdx.x) < sl.head, pt = it < sl.hi;
    const float xh = ph ? to_float(x[ih]) : -INFINITY, xt = pt ? to_float(x[it]) : -INFINITY;
    if (ph || pt) {
      r.raise(fmaxf(xh, xt), c);
      const float b = r.base();
      if (ph) r.add<ENT>(xh, b, c);
      if (pt) r.add<ENT>(xt, b, c);
    }
    if (TOP) {
      const uint32_t kh = __reduce_max_sync(0xffffffffu, key_of(xh)), kt = __reduce_max_sync(0xffffffffu, key_of(xt));
      if (threadIdx.x == 0) {
        keys[0] = kh;
        keys[nchunks - 1] = kt;
      }
    }
  }
  const T *body = x + sl.lo + sl.head;
  constexpr int U = 4;
  for (int i0 = 0; i0 < sl.nv; i0 += NT * U) {
    RowVec<T, E> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * NT + int(threadIdx.x);
      if (i < sl.nv) v[u].load(body + int64_t(i) * E);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * NT + int(threadIdx.x);
      if (i0 + u * NT >= sl.nv) break;
      float f[E];
      float mx = -INFINITY;
      if (i < sl.nv) {
        v[u].get(f);
#pragma unroll
        for (int e = 0; e < E; ++e) mx = fmaxf(mx, f[e]);
        if (mx > r.m) r.raise(mx, c);
        const float b = r.base();
#pragma unroll
        for (int e = 0; e < E; ++e) r.add<ENT>(f[e], b, c);
      }
      if (TOP) {
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        if ((threadIdx.x & 3) == 0 && i < sl.nv) keys[1 + i / CHUNK] = key_of(mx);
      }
    }
  }
  // join: warp, CTA, cluster
  r.join_warp(c);
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) { sm_m[warp] = r.m; sm_s[warp] = r.s; sm_t[warp] = r.t; }
  __syncthreads();
  Run all{sm_m[0], sm_s[0], sm_t[0]};
#pragma unroll
  for (int w = 1; w < NW; ++w) all.join(sm_m[w], sm_s[w], sm_t[w], c);
  if (size > 1) {
    if (threadIdx.x == 0) { part[0] = all.m; part[1] = all.s; part[2] = all.t; }
    cl.sync();
    all.clear();
    for (int q = 0; q < size; ++q) {
      const float *o = cl.map_shared_rank(part, q);
      all.join(o[0], o[1], o[2], c);
    }
  }
  const bool bad = !(all.s < INFINITY);  // a NaN or +inf among the logits
  const float logs = logf(all.s);        // -inf for a row of masks
  if (rank == 0 && threadIdx.x == 0) {
    float H = 0.f;
    if (bad) H = NAN;
    else if (ENT && all.s > 0.f) H = fmaxf(logs - LN2 * (all.t / all.s), 0.f);
    if (a.logp) {
      const float xy = to_float(x[token]);
      a.logp[row] = bad ? NAN : xy == -INFINITY ? -INFINITY : (xy - all.m) * a.scale - logs;
    }
    if (a.entropy) a.entropy[row] = H;
    if (a.saved)
      reinterpret_cast<float4 *>(a.saved)[row] = make_float4(bad ? NAN : all.m, bad ? NAN : logs, H, 0.f);
  }
  if (!TOP) {
    if (size > 1) cl.sync();  // part is read by the others until here
    return;
  }
  const unsigned K = unsigned(a.K);
  if (bad) {
    if (rank == 0)
      for (unsigned k = threadIdx.x; k < K; k += NT) {
        a.top_tokens[row * K + k] = -1;
        a.top_logp[row * K + k] = NAN;
      }
    if (size > 1) cl.sync();
    return;
  }
  // The K largest of the slice.  Elements are ordered by (logit, lower index
  // first), chunks by (their largest logit, lower chunk first): each of the K
  // best chunks holds an element that is above every element of a chunk behind
  // them, so the K best elements lie in the K best chunks.
  auto order = [](uint32_t key, uint32_t index) { return (static_cast<unsigned long long>(key) << 32) | (0xffffffffu - index); };
  const unsigned most = K + K / 2 < 32 ? 32 : K + K / 2;  // <= 192 <= 256
  unsigned long long cb = 0;
  if (unsigned(nchunks) > most)
    cb = bound_for(K, most, ~0ull, &S.count, [&](unsigned long long b) {
      unsigned n = 0;
      for (int i = threadIdx.x; i < nchunks; i += NT) n += order(keys[i], i) >= b;
      return n;
    });
  if (threadIdx.x == 0) { S.n = 0; S.m = 0; }
  __syncthreads();
  for (int i = threadIdx.x; i < nchunks; i += NT)
    if (keys[i] > KEY_MASKED && order(keys[i], i) >= cb) S.list[atomicAdd(&S.m, 1u)] = unsigned(i);
  __syncthreads();
  const unsigned nlist = S.m;
  const uint32_t floor_key = max(uint32_t(cb >> 32), KEY_MASKED + 1);
  // visit the elements of the listed chunks
  auto visit = [&](auto &&f) {
    for (unsigned j = threadIdx.x; j < nlist * (CHUNK * E); j += NT) {
      const int ch = int(S.list[j / (CHUNK * E)]), w = int(j % (CHUNK * E));
      int idx;
      bool in;
      if (ch == 0) { idx = sl.lo + w; in = w < sl.head; }
      else if (ch == nchunks - 1) { idx = sl.tail0 + w; in = idx < sl.hi; }
      else { idx = sl.lo + sl.head + (ch - 1) * (CHUNK * E) + w; in = idx < sl.tail0; }
      if (in) f(key_of(to_float(x[idx])), unsigned(idx));
    }
  };
  visit([&](uint32_t key, unsigned idx) {
    if (key >= floor_key) {
      const unsigned at = atomicAdd(&S.n, 1u);
      if (at < CAND) S.cand[at] = order(key, idx);
    }
  });
  __syncthreads();
  unsigned n = S.n;
  __syncthreads();
  if (n > most) {
    // too many at or above the chunks' bound (ties, or many large logits in few
    // chunks): a closer bound, from the candidates or, if they did not all fit, the row
    unsigned long long eb;
    if (n <= CAND) {
      eb = bound_for(K, most, ~0ull, &S.count, [&](unsigned long long b) {
        unsigned k = 0;
        for (unsigned i = threadIdx.x; i < n; i += NT) k += S.cand[i] >= b;
        return k;
      });
    } else {
      eb = bound_for(K, most, ~0ull, &S.count, [&](unsigned long long b) {
        unsigned k = 0;
        visit([&](uint32_t key, unsigned idx) { k += key >= floor_key && order(key, idx) >= b; });
        return k;
      });
    }
    if (threadIdx.x == 0) S.n = 0;
    __syncthreads();
    visit([&](uint32_t key, unsigned idx) {
      if (key >= floor_key && order(key, idx) >= eb) S.cand[atomicAdd(&S.n, 1u)] = order(key, idx);
    });
    __syncthreads();
    n = S.n;
    __syncthreads();
  }
  rank_candidates(S, n, K);
  if (size > 1) {
    cl.sync();  // every slice's best is there (and `part` read)
    if (rank == 0) {
      // K from each slice: size * K <= CAND
      for (unsigned i = threadIdx.x; i < size * K; i += NT) {
        const unsigned long long *o = cl.map_shared_rank(S.best, i / K);
        S.cand[i] = o[i % K];
      }
      __syncthreads();
      // empty places (0) are equal to one another: rank only what is there
      for (unsigned i = threadIdx.x; i < size * K; i += NT) {
        const unsigned long long mine = S.cand[i];
        unsigned above = 0;
        for (unsigned j = 0; j < size * K; ++j) above += S.cand[j] > mine;
        if (mine && above < K) {
          a.top_tokens[row * K + above] = int32_t(0xffffffffu - uint32_t(mine));
          a.top_logp[row * K + above] = (of_key(uint32_t(mine >> 32)) - all.m) * a.scale - logs;
        }
      }
      // the places behind the last one found
      unsigned have = 0;
      for (unsigned i = threadIdx.x; i < size * K; i += NT) have += S.cand[i] != 0;
      have = cta_sum(have, &S.count);
      for (unsigned k = have + threadIdx.x; k < K; k += NT) {
        a.top_tokens[row * K + k] = -1;
        a.top_logp[row * K + k] = -INFINITY;
      }
    }
    cl.sync();  // S.best is read by the first CTA until here
    return;
  }
  for (unsigned k = threadIdx.x; k < K; k += NT) {
    const unsigned long long b = S.best[k];
    a.top_tokens[row * K + k] = b ? int32_t(0xffffffffu - uint32_t(b)) : -1;
    a.top_logp[row * K + k] = b ? (of_key(uint32_t(b >> 32)) - all.m) * a.scale - logs : -INFINITY;
  }
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

template <typename T>
__device__ __forceinline__ void zero_slice(T *out, int lo, int hi) {
  constexpr int E = Slice<T>::E;
  int head = int(((16 - (reinterpret_cast<uintptr_t>(out + lo) & 15)) & 15) / sizeof(T));
  if (head > hi - lo) head = hi - lo;
  if (int(threadIdx.x) < head) out[lo + threadIdx.x] = from_float<T>(0.f);
  const int nv = (hi - lo - head) / E;
  for (int i = threadIdx.x; i < nv; i += NT)
    *reinterpret_cast<uint4 *>(out + lo + head + int64_t(i) * E) = make_uint4(0u, 0u, 0u, 0u);
  for (int i = lo + head + nv * E + int(threadIdx.x); i < hi; i += NT) out[i] = from_float<T>(0.f);
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
    zero_slice(out, sl.lo, sl.hi);
    return;
  }
  const float c = a.scale * LOG2E, L = sv.y * LOG2E;
  const float gl = a.dlogp ? a.dlogp[row] : 0.f, gh = a.dentropy ? a.dentropy[row] : 0.f;
  const bool mine = a.dlogp && token >= sl.lo && token < sl.hi;
  const float xt = mine ? to_float(x[token]) : 0.f;
  if (mine) __syncthreads();  // out may be x: every thread has read the token's logit
  const float M = sv.x;
  const float A = -gl * a.scale;
  float k;
  if (a.dentropy) {
    // -gl p - gh p (ln p + H) = p (B + C log2 p)
    const float B = A - gh * a.scale * sv.z, C = -gh * a.scale * LN2;
    map_slice(x, out, sl, [=](int, float v) {
      const float d = fmaf(v - M, c, -L);
      return ex2(d) * fmaf(C, fmaxf(d, LOWEST), B);
    });
    const float d = fmaf(xt - M, c, -L);
    k = ex2(d) * fmaf(C, fmaxf(d, LOWEST), B);
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
  int64_t ld, ldd;
  int V, K, tail, parts;
  float scale, value_scale;
  const int32_t *tokens;
  const float *values, *dloss;
  float *loss, *saved;
  unsigned *errword;
};

// A row's teacher entries in shared memory.
struct Teacher {
  float q[MAX_K], lq[MAX_K], x[MAX_K];
  int idx[MAX_K];    // -1: left out
  int first[MAX_K];  // whether no earlier entry has the same token
  float rest;        // q_r
  float m, s;        // running sum of the student's logits at the distinct tokens
  int live;          // entries that count
  int distinct;      // tokens among them
};

// Loads the entries, their probabilities q and ln q, and the student's logits
// at those in [lo, hi).  All NT threads; returns after a barrier.
template <typename T>
__device__ void load_teacher(Teacher &S, const DistillArgs &a, int64_t row, const T *x, int lo, int hi, bool report) {
  const int k = threadIdx.x;
  if (k < a.K) {
    int t = a.tokens[row * a.K + k];
    if (t >= a.V && report) atomicOr(a.errword, unsigned(ERR_BOUNDS));
    if (t >= a.V || t < 0) t = -1;
    S.idx[k] = t;
    S.lq[k] = t < 0 ? -INFINITY : a.values[row * a.K + k] * a.value_scale;
    S.x[k] = t >= lo && t < hi ? to_float(x[t]) : -INFINITY;
  }
  __syncthreads();
  if (k < a.K) {
    bool first = true;
    for (int j = 0; j < k; ++j) first = first && S.idx[j] != S.idx[k];
    S.first[k] = first && S.idx[k] >= 0;
  }
  if (threadIdx.x < 32) {
    // the sums of up to four entries per lane
    float mx = -INFINITY;
    int n = 0;
    for (int j = threadIdx.x; j < a.K; j += 32) {
      mx = fmaxf(mx, S.lq[j]);
      n += S.idx[j] >= 0;
    }
    n = __reduce_add_sync(0xffffffffu, n);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (a.tail || mx == -INFINITY) mx = 0.f;
    float s = 0.f;
    for (int j = threadIdx.x; j < a.K; j += 32) s += S.idx[j] >= 0 ? expf(S.lq[j] - mx) : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (!a.tail && s == 0.f) n = 0;  // nothing but -inf: no teacher
    const float ls = a.tail ? 0.f : mx + logf(s);
    for (int j = threadIdx.x; j < a.K; j += 32) {
      const float l = S.lq[j] - ls;
      S.lq[j] = l;
      S.q[j] = S.idx[j] >= 0 && n ? (a.tail ? expf(l) : expf(l + ls - mx) / s) : 0.f;
    }
    if (threadIdx.x == 0) {
      S.live = n;
      const float rest = 1.f - s;
      S.rest = a.tail && !(rest < float(n) * 1.1920929e-7f) ? rest : 0.f;
    }
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    Run r;
    r.clear();
    int n = 0;
    const float c = a.scale * LOG2E;
    for (int j = threadIdx.x; j < a.K; j += 32)
      if (S.first[j]) {
        r.raise(fmaxf(r.m, S.x[j]), c);
        r.add<false>(S.x[j], r.base(), c);
        ++n;
      }
    r.t = 0.f;
    r.join_warp(c);
    n = __reduce_add_sync(0xffffffffu, n);
    if (threadIdx.x == 0) {
      S.m = r.m;
      S.s = r.s;
      S.distinct = n;
    }
  }
  __syncthreads();
}

// Puts the teacher's tokens of the slice [lo, hi) right after the other
// elements were written: (p - q) g.
template <typename T>
__device__ __forceinline__ void write_teacher(const Teacher &S, const DistillArgs &a, T *out, int lo, int hi, float M,
                                              float logs, float g) {
  const int k = threadIdx.x;
  if (k < a.K && S.first[k] && S.idx[k] >= lo && S.idx[k] < hi) {
    float q = 0.f;
    for (int j = k; j < a.K; ++j) q += S.idx[j] == S.idx[k] ? S.q[j] : 0.f;
    const float p = S.x[k] == -INFINITY ? 0.f : ex2(fmaf(S.x[k] - M, a.scale * LOG2E, -logs * LOG2E));
    out[S.idx[k]] = from_float<T>((p - q) * g);
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
    } else {  // p_v (1 - q_r / p_r) = exp(z_v - ltail) (p_r - q_r)
      o.f = ex2((ltail - logs) * LOG2E) - S.rest;
      o.L = ltail;
    }
  }
  return o;
}

template <typename T, bool GRAD>
__global__ void __launch_bounds__(NT) distill_kernel(const DistillArgs a) {
  constexpr int E = Slice<T>::E;
  __shared__ Teacher S;
  __shared__ float sm_m[NW], sm_s[NW];
  __shared__ float part[2];
  extern __shared__ __align__(16) unsigned bits[];  // tail: one bit per element of the slice, a vector's E bits side by side
  cg::cluster_group cl = cg::this_cluster();
  const int size = int(cl.num_blocks()), rank = int(cl.block_rank());
  const int64_t row = blockIdx.x / size;
  const T *x = static_cast<const T *>(a.x) + row * a.ld;
  const Slice<T> sl = slice_of(x, a.V, rank, size);
  const float c = a.scale * LOG2E;
  load_teacher(S, a, row, x, 0, a.V, rank == 0);
  T *out = GRAD ? static_cast<T *>(a.out) + row * a.ldd : nullptr;
  if (S.live == 0) {
    if (rank == 0 && threadIdx.x == 0) {
      a.loss[row] = 0.f;
      if (a.saved) reinterpret_cast<float4 *>(a.saved)[row] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (GRAD) {
      if (size > 1) cl.sync();  // out may be x: the entries' logits have been read
      zero_slice(out, sl.lo, sl.hi);
    }
    return;
  }
  // mark the teacher's tokens of this slice: element sl.lo + sl.head + i at bit E + i,
  // the elements before the first vector below, those behind the last above
  const int base = sl.lo + sl.head - E;
  if (a.tail) {
    const int words = ((sl.nv + 2) * E + 31) / 32;
    for (int i = threadIdx.x; i < words; i += NT) bits[i] = 0u;
    __syncthreads();
    const int k = threadIdx.x;
    if (k < a.K && S.idx[k] >= sl.lo && S.idx[k] < sl.hi)
      atomicOr(&bits[(S.idx[k] - base) >> 5], 1u << ((S.idx[k] - base) & 31));
    __syncthreads();
  }
  auto marked = [&](int idx) { return a.tail && ((bits[(idx - base) >> 5] >> ((idx - base) & 31)) & 1u); };
  Run r;
  r.clear();
  if (threadIdx.x < 32) {
    const int ih = sl.lo + int(threadIdx.x), it = sl.tail0 + int(threadIdx.x);
    const bool ph = int(threadIdx.x) < sl.head, pt = it < sl.hi;
    const float xh = ph && !marked(ih) ? to_float(x[ih]) : -INFINITY;
    const float xt = pt && !marked(it) ? to_float(x[it]) : -INFINITY;
    if (ph || pt) {
      r.raise(fmaxf(xh, xt), c);
      const float b = r.base();
      r.add<false>(xh, b, c);
      r.add<false>(xt, b, c);
    }
  }
  const T *body = x + sl.lo + sl.head;
  constexpr int U = 4;
  for (int i0 = 0; i0 < sl.nv; i0 += NT * U) {
    RowVec<T, E> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * NT + int(threadIdx.x);
      if (i < sl.nv) v[u].load(body + int64_t(i) * E);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * NT + int(threadIdx.x);
      if (i >= sl.nv) break;
      float f[E];
      v[u].get(f);
      if (a.tail) {
        const unsigned mk = (bits[((i + 1) * E) >> 5] >> (((i + 1) * E) & 31)) & ((1u << E) - 1u);
        if (mk)
#pragma unroll
          for (int e = 0; e < E; ++e)
            if ((mk >> e) & 1u) f[e] = -INFINITY;
      }
      float mx = -INFINITY;
#pragma unroll
      for (int e = 0; e < E; ++e) mx = fmaxf(mx, f[e]);
      if (mx > r.m) r.raise(mx, c);
      const float b = r.base();
#pragma unroll
      for (int e = 0; e < E; ++e) r.add<false>(f[e], b, c);
    }
  }
  r.t = 0.f;
  r.join_warp(c);
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) { sm_m[warp] = r.m; sm_s[warp] = r.s; }
  __syncthreads();
  Run all{sm_m[0], sm_s[0], 0.f};
#pragma unroll
  for (int w = 1; w < NW; ++w) all.join(sm_m[w], sm_s[w], 0.f, c);
  if (size > 1) {
    if (threadIdx.x == 0) { part[0] = all.m; part[1] = all.s; }
    cl.sync();
    all.clear();
    for (int q = 0; q < size; ++q) {
      const float *o = cl.map_shared_rank(part, q);
      all.join(o[0], o[1], 0.f, c);
    }
    cl.sync();  // everything of the row that the first pass reads has been read
  } else {
    __syncthreads();
  }
  // tail: `all` is the sum over the tokens outside the teacher's; add the teacher's
  float ltail = 0.f;
  if (a.tail) {
    const Run others = all;
    all.join(S.m, S.s, 0.f, c);
    ltail = others.s == 0.f ? -INFINITY : (others.m - all.base()) * a.scale + logf(others.s);
  }
  const bool bad = !(all.s < INFINITY);
  const bool empty = all.s == 0.f;
  const float logs = logf(all.s);
  const float M = all.m;
  if (rank == 0 && threadIdx.x < 32) {
    float l = 0.f;
    for (int k = threadIdx.x; k < a.K; k += 32)
      if (S.idx[k] >= 0 && S.q[k] != 0.f)
        l += S.q[k] * (S.lq[k] - (empty || S.x[k] == -INFINITY ? -INFINITY : (S.x[k] - M) * a.scale - logs));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (threadIdx.x == 0) {
      if (a.tail && S.rest > 0.f && S.distinct < a.V)
        l += S.rest * (logf(S.rest) - (empty ? -INFINITY : ltail - logs));
      a.loss[row] = bad ? NAN : l;
      if (a.saved)
        reinterpret_cast<float4 *>(a.saved)[row] =
            make_float4(bad ? NAN : M, bad ? NAN : logs, 0.f, bad ? NAN : ltail);
    }
  }
  if (!GRAD) return;
  if (empty) {
    zero_slice(out, sl.lo, sl.hi);
    return;
  }
  const float g = (a.dloss ? a.dloss[row] : 1.f) * a.scale;
  Outside o = outside_of(S, a.tail, logs, ltail);
  if (bad) o.f = NAN;
  const float A = o.f * g, L = o.L * LOG2E;
  map_slice(x, out, sl, [=](int, float v) { return A * ex2(fmaf(v - M, c, -L)); });
  __syncthreads();
  write_teacher(S, a, out, sl.lo, sl.hi, bad ? NAN : M, logs, g);
}

template <typename T>
__global__ void __launch_bounds__(NT) distill_grad_kernel(const DistillArgs a) {
  __shared__ Teacher S;
  const int64_t row = blockIdx.x / a.parts;
  const int part = int(blockIdx.x % a.parts);
  const T *x = static_cast<const T *>(a.x) + row * a.ld;
  T *out = static_cast<T *>(a.out) + row * a.ldd;
  const Slice<T> sl = slice_of(x, a.V, part, a.parts);
  // only this part's logits: in place, the other parts may already be gradients
  load_teacher(S, a, row, x, sl.lo, sl.hi, part == 0);
  const float4 sv = reinterpret_cast<const float4 *>(a.saved)[row];
  if (S.live == 0 || sv.x == -INFINITY) {
    zero_slice(out, sl.lo, sl.hi);
    return;
  }
  const float c = a.scale * LOG2E;
  const float g = (a.dloss ? a.dloss[row] : 1.f) * a.scale;
  const Outside o = outside_of(S, a.tail, sv.y, sv.w);
  const float A = o.f * g, L = o.L * LOG2E, M = sv.x;
  map_slice(x, out, sl, [=](int, float v) { return A * ex2(fmaf(v - M, c, -L)); });
  __syncthreads();
  write_teacher(S, a, out, sl.lo, sl.hi, M, sv.y, g);
}

// ------------------------------------------------------------------ launch shapes and checks

// CTAs of a row.  One per row where there are rows enough for every SM; with
// fewer, a row is split so that the GPU has two CTAs per SM or the slices fall
// to 4096 columns, whichever comes first.  A slice has at most SLICE columns.
int cluster_of(int64_t T, int V) {
  int c = 1;
  while (c < MAX_CLUSTER && ((T * c < int64_t(num_sms()) * 2 && V / (2 * c) >= 4096) || V > int64_t(SLICE) * c)) c *= 2;
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

template <typename K, typename A>
poet_status launch_rows(K kern, const A &a, int64_t T, int cluster, size_t smem, cudaStream_t st, const char *what) {
  if (smem > 32 * 1024) POET_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(unsigned(T * cluster));
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  POET_CUDA_TRY(cudaLaunchKernelEx(&cfg, kern, a));
  count_launch();
  return launch_status(what);
}

template <typename T>
poet_status run_logp(const LogpArgs &a, int64_t rows, cudaStream_t st) {
  const int cluster = cluster_of(rows, a.V);
  const int nv = a.V / Slice<T>::E / cluster + 1;
  const size_t smem = a.K ? sizeof(SelectSmem) + size_t(chunks_of<T>(nv)) * 4 : 0;
  const bool ent = a.entropy || a.saved;
  if (a.K)
    return ent ? launch_rows(logp_kernel<T, true, true>, a, rows, cluster, smem, st, "logprobs")
               : launch_rows(logp_kernel<T, true, false>, a, rows, cluster, smem, st, "logprobs");
  return ent ? launch_rows(logp_kernel<T, false, true>, a, rows, cluster, smem, st, "logprobs")
             : launch_rows(logp_kernel<T, false, false>, a, rows, cluster, smem, st, "logprobs");
}

template <typename T>
poet_status run_distill(const DistillArgs &a, int64_t rows, cudaStream_t st) {
  const int cluster = cluster_of(rows, a.V);
  const int nv = a.V / Slice<T>::E / cluster + 1;
  const size_t smem = a.tail ? size_t(((nv + 2) * Slice<T>::E + 31) / 32) * 4 : 0;
  return a.out ? launch_rows(distill_kernel<T, true>, a, rows, cluster, smem, st, "distill")
               : launch_rows(distill_kernel<T, false>, a, rows, cluster, smem, st, "distill");
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
  a.x = logits; a.ld = ld; a.V = V; a.K = topk; a.scale = scale; a.tokens = tokens;
  a.logp = logp; a.entropy = entropy; a.top_tokens = top_tokens; a.top_logp = top_logp; a.saved = saved;
  a.errword = device_errword();
  POET_REQUIRE(a.errword != nullptr, "%s: no device status word", what);
  TraceScope ts("logprobs", 6.0 * double(T) * V, double(T) * V * double(esize(dtype)),
                reinterpret_cast<cudaStream_t>(stream));
  return dtype == POET_BF16 ? run_logp<bf16>(a, T, reinterpret_cast<cudaStream_t>(stream))
                            : run_logp<float>(a, T, reinterpret_cast<cudaStream_t>(stream));
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
  a.x = logits; a.out = dlogits; a.ld = ld; a.ldd = ldd; a.V = V; a.K = K; a.tail = tail; a.scale = scale;
  a.value_scale = value_scale; a.tokens = teacher_tokens; a.values = teacher_values; a.dloss = dloss;
  a.loss = loss; a.saved = saved;
  a.errword = device_errword();
  POET_REQUIRE(a.errword != nullptr, "%s: no device status word", what);
  TraceScope ts("distill", 10.0 * double(T) * V, (dlogits ? 2.0 : 1.0) * double(T) * V * double(esize(dtype)),
                reinterpret_cast<cudaStream_t>(stream));
  return dtype == POET_BF16 ? run_distill<bf16>(a, T, reinterpret_cast<cudaStream_t>(stream))
                            : run_distill<float>(a, T, reinterpret_cast<cudaStream_t>(stream));
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
  a.x = logits; a.out = dlogits; a.ld = ld; a.ldd = ldd; a.V = V; a.K = K; a.tail = tail; a.scale = scale;
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
