// Sampling under a request's parameters (temperature, top-k, top-p, min-p) from
// given random numbers: a token per logit row, and the acceptance walk with the
// target distribution so filtered.
//
// One row, with x its logits, M their maximum, T the temperature:
//   weight     w(x) = 2^44 exp((x - M) / T), rounded to an integer (a token whose
//              weight rounds to 0, less likely than 2^-45 of the likeliest, is
//              never drawn)
//   order      larger logit first, equal logits by lower id
//   top-k      the first k tokens; Z = the sum of their weights
//   top-p      of those, the fewest first ones whose weights sum to >= p Z
//   min-p      of those, the ones with exp((x - M) / T) >= min_p
//   draw       S = the sum of the weights kept: the smallest id whose cumulative
//              kept weight (in id order) exceeds u S
// With integer weights every sum is exact whatever its order, so the totals, the
// cumulative sums of any split of the row and a second pass over part of it all
// agree, and a draw cannot fall between two partial sums.
//
// One thread-block cluster holds a row in its shared memory (each logit is read
// from memory once) and passes over it there; a CTA has a contiguous slice, its
// threads take the slice's 16-byte vectors in turn.
#include <cooperative_groups.h>

#include <map>
#include <mutex>
#include <utility>

#include "eagle_internal.h"

namespace cg = cooperative_groups;

namespace eagle {

constexpr int kSmpThreads = 256;
constexpr int kSmpWarps = kSmpThreads / 32;
constexpr int kSmpMaxCluster = 16;
constexpr int kSmpSliceBytes = 32 * 1024;     // of a row per CTA, up to kSmpMaxCluster CTAs
constexpr int kSmpMaxSliceBytes = 64 * 1024;  // the most a CTA holds (the widest fp32 rows)
constexpr int kSmpMaxRounds = kSmpMaxSliceBytes / 16 / kSmpThreads + 1;
constexpr int kWeightBits = 44;

struct SmpShared {
  double tab[32];                                 // 2^(44 - j/32)
  unsigned long long xch[2][2][kSmpMaxCluster];  // [parity][value][rank]: what the CTAs tell one another
  unsigned long long warp_part[2][kSmpWarps];
  unsigned long long round_part[kSmpMaxRounds * kSmpWarps];
  unsigned long long pick_base;
  int pick_entry;
  int cut_id;
};

// A CTA's slice of a row: vectors of 16 bytes in shared memory; what lies
// outside the row is -inf.  Element e of vector v is token first + v * kPerVec + e.
template <typename T>
struct RowSlice {
  uint4* vec;
  int nvec;
  int first;
};

// Per-row constants.
struct RowStat {
  float top;       // M
  bool infinite;   // the row held +inf: those tokens count as 0, all others as -inf
  double c32;      // 32 log2(e) / T
  float c;         // log2(e) / T, for skipping weights that round to 0
  float vcut;      // kept: x > vcut, or x == vcut and id <= idcut, and x >= floor
  int idcut;
  float floor;
  unsigned long long total;  // S (0: nothing to draw)
};

__device__ __forceinline__ bool kept(const RowStat& s, float x, int id) {
  return (x > s.vcut || (x == s.vcut && id <= s.idcut)) && x >= s.floor;
}

// 2^44 e^{-d/T} for d = M - x >= 0, rounded to an integer.  t = 32 d log2(e)/T =
// n - r with n an integer and |r| <= 1/2; 2^(-n/32) comes from a table of 32
// and an exponent, 2^(r/32) = exp(r ln2/32) from its series up to r^3 (the next
// term is below 6e-10 relative), all in fp64: an fp32 weight (error 2^-24) would
// move the cumulative sums of a wide row by more than a small weight's width and
// with it the token.
__device__ __forceinline__ unsigned long long weight(const RowStat& s, const double* tab, float x) {
  if (!((s.top - x) * s.c < 45.5f)) return 0ull;  // also NaN and -inf
  constexpr double kMagic = 6755399441055744.0;   // 1.5 * 2^52: adding it rounds to an integer in the low bits
  constexpr double k1 = kLn2 / 32, k2 = k1 * k1 / 2, k3 = k1 * k1 * k1 / 6;
  const double t = ((double)s.top - (double)x) * s.c32;
  const double nm = t + kMagic;
  const int n = __double2loint(nm);
  const double r = (nm - kMagic) - t;
  const double p = r * fma(r, fma(r, k3, k2), k1);
  const double b = tab[n & 31];
  const double e = __hiloint2double(__double2hiint(b) - ((n >> 5) << 20), __double2loint(b));
  const double w = fma(e, p, e) + 4503599627370496.0;  // + 2^52: rounds, integer in the low 52 bits
  return (unsigned long long)(__double_as_longlong(w) & 0xfffffffffffffll);
}

__device__ __forceinline__ unsigned long long warp_sum_u64(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// The cluster as seen by the passes over one row.
struct Team {
  cg::cluster_group cl;
  SmpShared* sm;
  int rank, size, parity;

  // Two numbers per CTA (each thread's a and b summed over the CTA, or their
  // maxima) told to every CTA: xch[.][0 / 1][rank] after it.  Buffers alternate:
  // a CTA writes a buffer again only after the call between, whose barrier every
  // CTA reached after its last read.
  template <bool MAX>
  __device__ __forceinline__ const unsigned long long (*tell(unsigned long long a, unsigned long long b))[kSmpMaxCluster] {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (MAX) {
      a = warp_max_u64(a);
      b = warp_max_u64(b);
    } else {
      a = warp_sum_u64(a);
      b = warp_sum_u64(b);
    }
    if (lane == 0) {
      sm->warp_part[0][warp] = a;
      sm->warp_part[1][warp] = b;
    }
    __syncthreads();
    parity ^= 1;
    if ((int)threadIdx.x < 2 * size) {
      const int which = threadIdx.x & 1, to = threadIdx.x >> 1;
      unsigned long long v = 0;
      for (int w = 0; w < kSmpWarps; ++w) {
        const unsigned long long y = sm->warp_part[which][w];
        v = MAX ? umax64(v, y) : v + y;
      }
      *cl.map_shared_rank(&sm->xch[parity][which][rank], to) = v;
    }
    cl.sync();
    return sm->xch[parity];
  }
  __device__ __forceinline__ void sums(unsigned long long& a, unsigned long long& b) {
    const auto x = tell<false>(a, b);
    a = b = 0;
    for (int r = 0; r < size; ++r) {
      a += x[0][r];
      b += x[1][r];
    }
  }
  __device__ __forceinline__ unsigned long long max1(unsigned long long a) {
    const auto x = tell<true>(a, 0);
    a = 0;
    for (int r = 0; r < size; ++r) a = umax64(a, x[0][r]);
    return a;
  }
};

template <typename T, typename F>
__device__ __forceinline__ void each(const RowSlice<T>& sl, F&& f) {
  constexpr int E = Elem<T>::kPerVec;
  for (int v = threadIdx.x; v < sl.nvec; v += kSmpThreads) {
    float x[E];
    Elem<T>::unpack(sl.vec[v], x);
    const int id = sl.first + v * E;
#pragma unroll
    for (int e = 0; e < E; ++e) f(x[e], id + e);
  }
}

// The smallest id whose cumulative g(x, id) (a non-negative integer) exceeds
// thr, in the CTA that holds it: the thread with that token calls hit(id, x).
// thr < the total over the row.
template <typename T, typename G, typename H>
__device__ __forceinline__ void select(Team& tm, const RowSlice<T>& sl, unsigned long long thr, G&& g, H&& hit) {
  constexpr int E = Elem<T>::kPerVec;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  SmpShared& sm = *tm.sm;
  unsigned long long mine = 0;
  each<T>(sl, [&](float x, int id) { mine += g(x, id); });
  const auto x = tm.tell<false>(mine, 0);
  unsigned long long before = 0;
  int owner = -1;
  for (int r = 0; r < tm.size; ++r) {
    const unsigned long long c = x[0][r];
    if (owner < 0 && thr < before + c) owner = r;
    if (owner < 0) before += c;
  }
  if (owner != tm.rank) return;  // the same in every thread of the CTA
  // rounds of 256 vectors in id order, a warp's 32 at a time
  const int rounds = (sl.nvec + kSmpThreads - 1) / kSmpThreads;
  auto lane_sum = [&](int v) {
    unsigned long long s = 0;
    if (v < sl.nvec) {
      float y[E];
      Elem<T>::unpack(sl.vec[v], y);
#pragma unroll
      for (int e = 0; e < E; ++e) s += g(y[e], sl.first + v * E + e);
    }
    return s;
  };
  for (int q = 0; q < rounds; ++q) {
    const unsigned long long s = warp_sum_u64(lane_sum(q * kSmpThreads + tid));
    if (lane == 0) sm.round_part[q * kSmpWarps + warp] = s;
  }
  __syncthreads();
  if (warp == 0) {
    unsigned long long base = before;
    for (int e0 = 0; e0 < rounds * kSmpWarps; e0 += 32) {
      const unsigned long long c = e0 + lane < rounds * kSmpWarps ? sm.round_part[e0 + lane] : 0;
      unsigned long long inc = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(kFull, inc, o);
        if (lane >= o) inc += y;
      }
      const unsigned m = __ballot_sync(kFull, thr < base + inc);
      if (m) {
        if (lane == __ffs(m) - 1) {
          sm.pick_entry = e0 + lane;
          sm.pick_base = base + inc - c;
        }
        break;
      }
      base += __shfl_sync(kFull, inc, 31);
    }
  }
  __syncthreads();
  if (sm.pick_entry % kSmpWarps != warp) return;
  const int v = sm.pick_entry / kSmpWarps * kSmpThreads + tid;
  const unsigned long long c = lane_sum(v);
  unsigned long long inc = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(kFull, inc, o);
    if (lane >= o) inc += y;
  }
  unsigned long long cum = sm.pick_base + inc - c;
  if (thr < cum || thr >= cum + c) return;
  float y[E];
  Elem<T>::unpack(sl.vec[v], y);
  const int id = sl.first + v * E;
  bool done = false;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    cum += g(y[e], id + e);
    if (!done && thr < cum) {
      done = true;
      hit(id + e, y[e]);
    }
  }
}

// A CTA's part of a row at `row` (element aligned), and filling it: 16-byte copies
// where the row covers the whole vector, single elements at its two ends.
template <typename T>
__device__ __forceinline__ void place_slice(RowSlice<T>& sl, const T* row, int V, int per, int rank) {
  constexpr int E = Elem<T>::kPerVec;
  const int off = (int)(((uintptr_t)row & 15u) / sizeof(T));  // the row starts inside its first vector
  sl.first = rank * per * E - off;
  const int all = (V + off + E - 1) / E;
  sl.nvec = max(0, min(per, all - rank * per));
}
template <typename T>
__device__ __forceinline__ void fill_slice(RowSlice<T>& sl, const T* row, int V) {
  constexpr int E = Elem<T>::kPerVec;
  const bool aligned = ((uintptr_t)(row + sl.first) & 15u) == 0;  // else another row's placement, out of step with this one's
  for (int v = threadIdx.x; v < sl.nvec; v += kSmpThreads) {
    const int id = sl.first + v * E;
    if (aligned && id >= 0 && id + E <= V) {
      const uint32_t dst = (uint32_t)__cvta_generic_to_shared(sl.vec + v);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(row + id) : "memory");
    } else {
      uint4 u = Elem<T>::neg_inf_vec();
      T* p = reinterpret_cast<T*>(&u);
      for (int e = 0; e < E; ++e)
        if (id + e >= 0 && id + e < V) p[e] = row[id + e];
      sl.vec[v] = u;
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  // (each thread reads only vectors it copied itself until the next barrier)
}

struct RowParams {
  float temperature, top_p, min_p;
  int top_k;
};

__device__ __forceinline__ RowParams row_params(const eagle_sampling_t& s, long long row) {
  RowParams p;
  p.temperature = s.temperature ? __ldg(s.temperature + row) : 1.f;
  p.top_k = s.top_k ? __ldg(s.top_k + row) : 0;
  p.top_p = s.top_p ? __ldg(s.top_p + row) : 1.f;
  p.min_p = s.min_p ? __ldg(s.min_p + row) : 0.f;
  return p;
}

// The row's maximum, cut and total (every thread of every CTA gets the same).
template <typename T>
__device__ void filter_row(Team& tm, RowSlice<T>& sl, const RowParams& pr, int V, RowStat& s) {
  const SmpShared& sm = *tm.sm;
  {
    float m = -INFINITY;
    for (int v = threadIdx.x; v < sl.nvec; v += kSmpThreads) m = fmaxf(m, Elem<T>::vec_max(sl.vec[v]));
    m = order_value((uint32_t)tm.max1(order_bits(m)));
    s.infinite = m == INFINITY;
    if (s.infinite) {  // the likeliest tokens are the infinite ones, alike
      constexpr int E = Elem<T>::kPerVec;
      for (int v = threadIdx.x; v < sl.nvec; v += kSmpThreads) {
        T* p = reinterpret_cast<T*>(sl.vec + v);
        for (int e = 0; e < E; ++e) p[e] = (float)p[e] == INFINITY ? (T)0.f : (T)-INFINITY;
      }
      m = 0.f;
    }
    s.top = m;
  }
  s.vcut = -INFINITY;
  s.idcut = 0x7fffffff;
  s.floor = -INFINITY;
  s.total = 0;
  if (s.top == -INFINITY) return;
  const bool greedy = !(pr.temperature > 0.f);
  const double T_ = greedy ? 1.0 : (double)pr.temperature;
  s.c32 = 32.0 * 1.4426950408889634 / T_;
  s.c = (float)fmin(s.c32 / 32.0, 1e30);
  const bool by_p = !greedy && pr.top_p < 1.f;  // (NaN: off)
  long long k = greedy || (by_p && !(pr.top_p > 0.f)) ? 1 : (pr.top_k > 0 && pr.top_k < V ? pr.top_k : 0);
  if (!greedy && pr.min_p > 0.f) {
    // e >= min_p where x >= M + T ln(min_p): the smallest float at or above it
    const double at = pr.min_p >= 1.f ? (double)s.top : (double)s.top + T_ * log((double)pr.min_p);
    float f = __double2float_ru(at);
    s.floor = f;
  }
  auto count_mass = [&](float cut, unsigned long long& n, unsigned long long& m, bool strict, bool mass) {
    n = m = 0;
    each<T>(sl, [&](float x, int id) {
      if (kept(s, x, id) && (strict ? x > cut : x >= cut)) {
        ++n;
        if (mass) m += weight(s, sm.tab, x);
      }
    });
    tm.sums(n, m);
  };
  const float floor_ = s.floor;
  s.floor = -INFINITY;  // min-p comes last: it takes nothing from the sums before it
  // The largest cut value v with measure(x >= v) >= need, by halving the ordered
  // bit patterns; then how many of the tokens equal to v belong, by id.
  auto cut_at = [&](unsigned long long need, bool mass) {
    uint32_t lo = order_bits(-INFINITY) + 1, hi = order_bits(s.top);  // lo always holds enough
    unsigned long long n, m;
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo + 1) / 2;
      count_mass(order_value(mid), n, m, false, mass);
      if ((mass ? m : n) >= need) lo = mid;
      else hi = mid - 1;
    }
    const float v = order_value(lo);
    count_mass(v, n, m, true, mass);
    const unsigned long long one = mass ? weight(s, sm.tab, v) : 1ull;
    const unsigned long long ties = (need - (mass ? m : n) + one - 1) / one;  // >= 1 of them
    select<T>(tm, sl, ties - 1, [&](float x, int id) { return (unsigned long long)(x == v && kept(s, x, id)); },
              [&](int id, float) {
                for (int r = 0; r < tm.size; ++r) *tm.cl.map_shared_rank(&tm.sm->cut_id, r) = id;
              });
    tm.cl.sync();
    s.vcut = v;
    s.idcut = tm.sm->cut_id;
    tm.cl.sync();
  };
  if (k == 1) {
    // the first of the largest
    const float v = s.top;
    select<T>(tm, sl, 0ull, [&](float x, int) { return (unsigned long long)(x == v); },
              [&](int id, float) {
                for (int r = 0; r < tm.size; ++r) *tm.cl.map_shared_rank(&tm.sm->cut_id, r) = id;
              });
    tm.cl.sync();
    s.vcut = v;
    s.idcut = tm.sm->cut_id;
    tm.cl.sync();
  } else if (k > 1) {
    unsigned long long n, m;
    count_mass(-INFINITY, n, m, true, false);
    if (n > (unsigned long long)k) cut_at((unsigned long long)k, false);
  }
  if (by_p && k != 1) {
    unsigned long long n, Z;
    count_mass(-INFINITY, n, Z, true, true);
    const unsigned long long need = (unsigned long long)ceil((double)pr.top_p * (double)Z);
    cut_at(need < 1 ? 1 : (need > Z ? Z : need), true);
  }
  s.floor = floor_;
  unsigned long long S = 0, unused = 0;
  each<T>(sl, [&](float x, int id) {
    if (kept(s, x, id)) S += weight(s, sm.tab, x);
  });
  tm.sums(S, unused);
  s.total = S;
}

// u as the draws read it: NaN and negative as 0, 1 and above as the largest float below 1
__device__ __forceinline__ double draw_u(float u) { return u >= 0.f ? (double)fminf(u, 0x1.fffffep-1f) : 0.0; }

__device__ __forceinline__ void team_init(Team& tm, SmpShared& sm) {
  tm.sm = &sm;
  tm.rank = (int)tm.cl.block_rank();
  tm.size = (int)tm.cl.num_blocks();
  tm.parity = 0;
  if (threadIdx.x < 32) sm.tab[threadIdx.x] = exp2((double)kWeightBits - threadIdx.x / 32.0);
}

template <typename T>
__global__ void __launch_bounds__(kSmpThreads)
sample_kernel(const T* __restrict__ logits, int V, long long stride, eagle_sampling_t params,
              const float* __restrict__ uniforms, int32_t* __restrict__ tokens, float* __restrict__ logprob, int per) {
  __shared__ SmpShared sm;
  extern __shared__ __align__(16) unsigned char dyn[];
  griddep_wait();
  griddep_launch_dependents();
  Team tm{cg::this_cluster(), &sm, 0, 0, 0};
  team_init(tm, sm);
  const long long row = blockIdx.x / tm.size;
  RowSlice<T> sl;
  sl.vec = reinterpret_cast<uint4*>(dyn);
  place_slice<T>(sl, logits + row * stride, V, per, tm.rank);
  fill_slice<T>(sl, logits + row * stride, V);
  const RowParams pr = row_params(params, row);
  const float u = uniforms[row];
  __syncthreads();
  RowStat s;
  filter_row<T>(tm, sl, pr, V, s);
  if (s.total == 0) {
    if (tm.rank == 0 && threadIdx.x == 0) {
      tokens[row] = -1;
      if (logprob) logprob[row] = -INFINITY;
    }
    tm.cl.sync();
    return;
  }
  const unsigned long long thr = (unsigned long long)(draw_u(u) * (double)s.total);
  select<T>(tm, sl, thr, [&](float x, int id) { return kept(s, x, id) ? weight(s, sm.tab, x) : 0ull; },
            [&](int id, float x) {
              tokens[row] = id;
              if (logprob) {
                // log of the kept probability: (x - M) / T - ln(S / 2^44)
                const double z = ((double)x - (double)s.top) * (s.c32 * (kLn2 / 32.0));
                logprob[row] = (float)(z - log(ldexp((double)s.total, -kWeightBits)));
              }
            });
  tm.cl.sync();  // no CTA leaves while another may still write to its shared memory
}

// The acceptance walk (accept.cu's rules) with p = the filtered target
// distribution kept(x) w(x) / S: one cluster per sequence goes down the tree
// and filters the target rows that the walk visits, and only those.  At node j
// the current target after r rejections is max(0, p - t q) / F(t), F(t) = sum
// max(0, p - t q); q = the draft row's softmax, unfiltered.
struct WalkShared {
  int tok[EAGLE_MAX_NODES], par[EAGLE_MAX_NODES], drow[EAGLE_MAX_NODES + 1];
  float u_acc[EAGLE_MAX_NODES + 1];
  double px[EAGLE_MAX_NODES + 1], qx[EAGLE_MAX_NODES + 1];  // of the current node's children
  double part[kSmpWarps];
  double xd[2][kSmpMaxCluster];
};

// Sum of one double per thread over the cluster, in a fixed order (every thread
// of every CTA gets the same bits).
__device__ __forceinline__ double team_sum(Team& tm, WalkShared& ws, double v) {
  v = warp_sum_d(v);
  if ((threadIdx.x & 31) == 0) ws.part[threadIdx.x >> 5] = v;
  __syncthreads();
  tm.parity ^= 1;
  if ((int)threadIdx.x < tm.size) {
    double a = 0.0;
    for (int w = 0; w < kSmpWarps; ++w) a += ws.part[w];
    *tm.cl.map_shared_rank(&ws.xd[tm.parity][tm.rank], threadIdx.x) = a;
  }
  tm.cl.sync();
  double a = 0.0;
  for (int r = 0; r < tm.size; ++r) a += ws.xd[tm.parity][r];
  return a;
}

template <typename T>
__global__ void __launch_bounds__(kSmpThreads)
accept_sampling_kernel(const T* __restrict__ tgt, const T* __restrict__ dft, const double* __restrict__ dlse, int R, int V,
                       int n, int depth, const int32_t* __restrict__ tokens, const int32_t* __restrict__ parents,
                       const int32_t* __restrict__ draft_row, const float* __restrict__ uniforms,
                       eagle_sampling_t params, int without_replacement, int32_t* __restrict__ accepted_len,
                       int32_t* __restrict__ path, int32_t* __restrict__ bonus, int per) {
  __shared__ SmpShared sm;
  __shared__ WalkShared ws;
  extern __shared__ __align__(16) unsigned char dyn[];
  griddep_wait();
  griddep_launch_dependents();
  Team tm{cg::this_cluster(), &sm, 0, 0, 0};
  team_init(tm, sm);
  const int b = blockIdx.x / tm.size, tid = threadIdx.x;
  const bool leader = tm.rank == 0 && tid == 0;
  const size_t trow0 = (size_t)b * (n + 1);
  const float* u_res = uniforms + (size_t)b * 2 * (n + 1) + (n + 1);
  if (tid < n) {
    ws.tok[tid] = tokens[(size_t)b * n + tid];
    ws.par[tid] = parents[(size_t)b * n + tid];
  }
  if (tid <= n) {
    const int r = draft_row[trow0 + tid];
    ws.drow[tid] = r >= 0 && r < R ? r : -1;  // an out-of-range row counts as "not expanded"
    ws.u_acc[tid] = uniforms[(size_t)b * 2 * (n + 1) + tid];
  }
  const RowParams pr = row_params(params, b);
  RowSlice<T> sl, dl;
  sl.vec = reinterpret_cast<uint4*>(dyn);
  dl.vec = sl.vec + per;
  __syncthreads();

  int j = 0, len = 0;
  RowStat s;
  while (true) {
    const T* trow = tgt + (trow0 + j) * (size_t)V;
    const int r = ws.drow[j];
    const T* drow = r >= 0 ? dft + ((size_t)b * R + r) * (size_t)V : nullptr;
    const double lse = r >= 0 ? dlse[(size_t)b * R + r] : 0.0;
    place_slice<T>(sl, trow, V, per, tm.rank);
    fill_slice<T>(sl, trow, V);
    dl.first = sl.first;
    dl.nvec = sl.nvec;
    filter_row<T>(tm, sl, pr, V, s);
    const double inv_S = s.total ? 1.0 / (double)s.total : 0.0;
    // p and q of every child's token (0 for a token outside the vocabulary)
    if (tid < n && ws.par[tid] == j) {
      const int x = ws.tok[tid];
      double p = 0.0, q = 0.0;
      if (x >= 0 && x < V && r >= 0) {
        float xt = (float)trow[x];
        if (s.infinite) xt = xt == INFINITY ? 0.f : -INFINITY;  // as in the slice
        if (kept(s, xt, x)) p = (double)weight(s, sm.tab, xt) * inv_S;
        q = exp((double)(float)drow[x] - lse);
      }
      ws.px[tid + 1] = p;
      ws.qx[tid + 1] = q;
    }
    __syncthreads();
    double t = 0.0, F = 1.0, Q = 1.0;  // Q: draft mass not yet rejected at j (1 with replacement)
    bool rejected = false, spent = false, have_draft = false;
    int moved = 0;
    // max(0, p - t q) of a token of this slice (the draft slice lies under the target's)
    auto residual = [&](float x, int id) {
      if (!kept(s, x, id)) return 0.0;
      const unsigned long long w = weight(s, sm.tab, x);
      if (w == 0) return 0.0;
      const float y = (float)reinterpret_cast<const T*>(dl.vec)[id - dl.first];
      return fmax(0.0, (double)w * inv_S - t * exp((double)y - lse));
    };
    if (len < depth && s.total) {
      int c = 1;
      while (c <= n && ws.par[c - 1] != j) ++c;
      while (c <= n && r >= 0) {
        const double px = ws.px[c], qx = ws.qx[c];
        const double rho = t == 0.0 ? px : fmax(0.0, px - t * qx);
        if (qx > 0.0 && (double)ws.u_acc[c] * (F * qx) < Q * rho) {
          moved = c;
          break;
        }
        t += F / Q;
        rejected = true;
        if (without_replacement) {
          Q -= qx;
          if (!(Q > 0.0)) {
            spent = true;
            break;
          }
        }
        ++c;
        while (c <= n && ws.par[c - 1] != j) ++c;
        if (c <= n) {  // another sibling will be tested: F at the new t
          if (!have_draft) fill_slice<T>(dl, drow, V);
          have_draft = true;
          double f = 0.0;
          each<T>(sl, [&](float x, int id) { f += residual(x, id); });
          F = team_sum(tm, ws, f);
          if (!(F > 0.0)) break;  // p = t q left nothing: the walk stays here
        }
      }
    }
    if (moved) {
      if (leader) path[(size_t)b * depth + len] = moved;
      ++len;
      j = moved;
      __syncthreads();  // px, qx and the slices are read above and written for the next node
      continue;
    }
    // the walk ends at j
    if (leader) {
      accepted_len[b] = len;
      for (int i = len; i < depth; ++i) path[(size_t)b * depth + i] = -1;
    }
    const double u = draw_u(u_res[j]);
    bool drawn = false;
    if (s.total && !spent) {
      if (!rejected) {
        select<T>(tm, sl, (unsigned long long)(u * (double)s.total),
                  [&](float x, int id) { return kept(s, x, id) ? weight(s, sm.tab, x) : 0ull; },
                  [&](int id, float) { bonus[b] = id; });
        drawn = true;
      } else {
        if (!have_draft) fill_slice<T>(dl, drow, V);
        double f = 0.0;
        each<T>(sl, [&](float x, int id) { f += residual(x, id); });
        F = team_sum(tm, ws, f);
        if (F > 0.0) {
          // integer weights of the residual, their sum about 2^60
          const double scale = 1152921504606846976.0 / F;
          auto g = [&](float x, int id) { return (unsigned long long)(residual(x, id) * scale); };
          unsigned long long W = 0, unused = 0;
          each<T>(sl, [&](float x, int id) { W += g(x, id); });
          tm.sums(W, unused);
          select<T>(tm, sl, (unsigned long long)(u * (double)W), g, [&](int id, float) { bonus[b] = id; });
          drawn = true;
        }
      }
    }
    if (!drawn) {
      // nothing left to draw from: the target's argmax (-1 in a row without a finite logit)
      if (s.top == -INFINITY) {
        if (leader) bonus[b] = -1;
      } else {
        select<T>(tm, sl, 0ull, [&](float x, int) { return (unsigned long long)(x == s.top); },
                  [&](int id, float) { bonus[b] = id; });
      }
    }
    break;
  }
  tm.cl.sync();  // no CTA leaves while another may still write to its shared memory
}

// ------------------------------------------------------------------- host
namespace {

// Clusters of more than 8 CTAs are opt-in per kernel and device.
cudaError_t ensure_wide_cluster(const void* kernel) {
  static std::mutex mu;
  static std::map<std::pair<const void*, int>, bool> done;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  bool& ok = done[std::make_pair(kernel, dev)];
  if (ok) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) ok = true;
  return e;
}

// CTAs per row and 16-byte vectors per CTA.
struct RowPlan {
  int cluster, per;
};
RowPlan plan_row(long long rows, int V, int elem_bytes) {
  const int E = 16 / elem_bytes;
  const int all = (V + 2 * E - 2) / E;  // a row may start inside its first vector
  int cl = (all * 16 + kSmpSliceBytes - 1) / kSmpSliceBytes;
  // few rows: more CTAs each, as long as all fit at two per SM
  const long long want = 2LL * device_sm_count() / rows;
  if (cl < want) cl = (int)(want < kSmpMaxCluster ? want : kSmpMaxCluster);
  if (cl > kSmpMaxCluster) cl = kSmpMaxCluster;
  if (cl > all) cl = all;
  return {cl, (all + cl - 1) / cl};
}

template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), long long grid, int cluster, size_t smem, bool pdl, cudaStream_t s,
                           Args... args) {
  cudaError_t e = ensure_smem_limit((const void*)kernel, smem + 4096);
  if (e == cudaSuccess && cluster > 8) e = ensure_wide_cluster((const void*)kernel);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kSmpThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_sample(const void* logits, int dtype, long long rows, int V, long long stride,
                          const eagle_sampling_t& params, const float* uniforms, int32_t* tokens, float* logprob,
                          cudaStream_t s) {
  const RowPlan pl = plan_row(rows, V, dtype_bytes(dtype));
  const size_t smem = (size_t)pl.per * 16;
  if (dtype == EAGLE_F32)
    return launch_cluster(sample_kernel<float>, rows * pl.cluster, pl.cluster, smem, false, s,
                          static_cast<const float*>(logits), V, stride, params, uniforms, tokens, logprob, pl.per);
  return launch_cluster(sample_kernel<__nv_bfloat16>, rows * pl.cluster, pl.cluster, smem, false, s,
                        static_cast<const __nv_bfloat16*>(logits), V, stride, params, uniforms, tokens, logprob, pl.per);
}

cudaError_t launch_accept_sampling(const void* tgt, int dtype, const void* dft, const double* dlse, int R,
                                   const int32_t* tokens, const int32_t* parents, const int32_t* draft_row,
                                   const float* uniforms, const eagle_sampling_t& params, bool without_replacement, int B,
                                   int n, int V, int depth, int32_t* accepted_len, int32_t* path, int32_t* bonus,
                                   bool pdl, cudaStream_t s) {
  const RowPlan pl = plan_row(B, V, dtype_bytes(dtype));
  const size_t smem = (size_t)pl.per * 32;  // a target and a draft slice
  const long long grid = (long long)B * pl.cluster;
  if (dtype == EAGLE_F32)
    return launch_cluster(accept_sampling_kernel<float>, grid, pl.cluster, smem, pdl, s, static_cast<const float*>(tgt),
                          static_cast<const float*>(dft), dlse, R, V, n, depth, tokens, parents, draft_row, uniforms,
                          params, (int)without_replacement, accepted_len, path, bonus, pl.per);
  return launch_cluster(accept_sampling_kernel<__nv_bfloat16>, grid, pl.cluster, smem, pdl, s,
                        static_cast<const __nv_bfloat16*>(tgt), static_cast<const __nv_bfloat16*>(dft), dlse, R, V, n,
                        depth, tokens, parents, draft_row, uniforms, params, (int)without_replacement, accepted_len, path,
                        bonus, pl.per);
}

}  // namespace eagle
