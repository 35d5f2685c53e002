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
// One thread-block cluster takes a row, each CTA a contiguous slice.  The row is
// read once in full, into counts by value: a bin per pattern of a logit's upper
// 16 bits (sign, exponent, 7 mantissa bits), kept in shared memory and summed
// over the cluster.
//   bf16  a bin is one value, so the counts hold all there is to know: weights are
//         evaluated once per bin, the cuts of top-k and top-p fall out of prefix
//         sums over the bins, and each CTA's share of S out of its own counts.
//         Only the CTA that the draw falls into reads its slice again.
//   fp32  the bins tell where a cut lies; the few tokens in the bins around it are
//         gathered into a list, sorted and cut exactly, in a second pass that also
//         adds up the exact weights (fp64 exponentials) of the tokens above them.
// What the bins cannot place (logits of 512 and more, a list that overflows, an
// estimate that missed) is cut by halving the ordered bit patterns of the logits,
// one pass over the slices per step.
//
// What bounds it (bf16, V = 128256).  1056 rows, 271 MB: a CTA per row, in two
// waves of 592.  Per wave and p = 0.9 the counting pass takes 27 us (one shared
// atomic per logit; HBM alone would need 21), the second count of the CTA the
// draw falls into (narrow) 36, the cuts 14, the weights 12 and the draw 6:
// 255 us in all, instruction issue rather than memory.  One fp32 row of 32000
// (top-p): eleven cluster exchanges of about 1.5 us, half of its 33 us; 32 rows 35.
// An unfiltered row of small positive and negative logits has no short list of
// values: its draw is bound by the fp64 weights of its own slice (1056 rows: 400 us).
// Rows cut by halving take 2 to 6 times as long where there are 1 to 32, 5 to 18
// times where there are hundreds (1056 rows with a logit of 600, top-p: 5 ms).
#include <cooperative_groups.h>

#include <map>
#include <mutex>
#include <utility>

#include "eagle_internal.h"

namespace cg = cooperative_groups;

namespace eagle {

typedef unsigned long long u64;

constexpr int kSmpThreads = 256;
constexpr int kSmpWarps = kSmpThreads / 32;
constexpr int kSmpMaxCluster = 16;
constexpr int kSmpBatch = 4;  // 16-byte loads a thread has in flight (passes that only count: twice as many)
constexpr int kWeightBits = 44;
constexpr int kListCap = 1024;  // fp32: tokens gathered around a cut

// Bins in descending order of value: 0 = 512 and above (and NaN), then the
// positive patterns down to 2^-16, one bin for everything smaller in magnitude
// (kZeroBin, read as 0), the negative patterns down, and last = -512 and below.
constexpr int kPatLow = (127 - 16) << 7, kPatHigh = (127 + 9) << 7;
constexpr int kZeroBin = kPatHigh - kPatLow + 1;
constexpr int kLastBin = 2 * kZeroBin;
constexpr int kBins = kLastBin + 1;
// In shared memory a bin's count sits at its distance from the zero bin, those
// of negative values kNegative further on.
constexpr int kNegative = 4096;
constexpr int kBinWords = 2 * kNegative;
static_assert(kZeroBin < kNegative, "a slot per bin");

struct SmpShared {
  double tab[32];                   // 2^(44 - j/32)
  u64 xch[2][2][kSmpMaxCluster];    // [parity][value][rank]: what the CTAs tell one another
  u64 word[2][2];                   // [parity]: what one CTA tells all
  u64 warp_part[2][kSmpWarps];
  u64 cta_mass[kSmpMaxCluster];     // kept weight of each CTA's slice
  u64 list[kListCap];               // CTA 0: (order bits, ~id) of the tokens gathered
  int pick_entry, pick_id;
  int list_n;
};

// A CTA's slice of a row in global memory: vectors of 16 bytes; element e of
// vector v is token first + v * kPerVec + e; what lies outside the row reads as -inf.
template <typename T>
struct RowSlice {
  const T* row;
  int V, first, nvec;
  __device__ __forceinline__ uint4 get(int v) const {
    constexpr int E = Elem<T>::kPerVec;
    const int id = first + v * E;
    if (id >= 0 && id + E <= V) return __ldg(reinterpret_cast<const uint4*>(row + id));
    const uint4 none = Elem<T>::neg_inf_vec();
    uint32_t w[4] = {none.x, none.y, none.z, none.w};
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (id + e >= 0 && id + e < V) {
        if (sizeof(T) == 4) {
          w[e] = __ldg(reinterpret_cast<const unsigned*>(row) + id + e);
        } else {
          const uint32_t h = __ldg(reinterpret_cast<const unsigned short*>(row) + id + e);
          w[e / 2] = (e & 1) ? (w[e / 2] & 0xffffu) | (h << 16) : (w[e / 2] & 0xffff0000u) | h;
        }
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// A CTA's part of the row at `row` (element aligned; it may start inside a vector,
// so that the vectors inside it are aligned).
template <typename T>
__device__ __forceinline__ void place_slice(RowSlice<T>& sl, const T* row, int V, int per, int rank) {
  constexpr int E = Elem<T>::kPerVec;
  const int off = (int)(((uintptr_t)row & 15u) / sizeof(T));
  sl.row = row;
  sl.V = V;
  sl.first = rank * per * E - off;
  sl.nvec = max(0, min(per, (V + off + E - 1) / E - rank * per));
}

// Per-row constants.
struct RowStat {
  float top;       // M
  bool infinite;   // the row holds +inf: those tokens count as 0, all others as -inf
  bool merged;     // bf16: values below 2^-16 in magnitude are read as 0, as the bins do
  double c32;      // 32 log2(e) / T
  float c;         // log2(e) / T, for skipping weights that round to 0 (T >= 2^-100, so finite and within c32's reach)
  float vcut;      // kept: x > vcut, or x == vcut and id <= idcut, and x >= floor
  int idcut;
  float floor;
  u64 total;       // S (0: nothing to draw)
  // bf16 rows settled by the bins: kept values lie in bins [bin0, bin1] (-1: not settled so); of the tokens equal
  // to vcut the CTA's slice keeps the first `ties` of its own
  int bin0, bin1;
  u64 ties;
};

// A logit's own value (in a row that holds +inf, see RowStat::infinite).
__device__ __forceinline__ float own(const RowStat& s, float x) {
  return s.infinite ? (x == INFINITY ? 0.f : -INFINITY) : x;
}
// A logit as the passes that have to agree with the bins read it, see
// RowStat::merged (cut_by_bins makes sure that no sum notices, nor what is kept).
template <typename T>
__device__ __forceinline__ float canon(const RowStat& s, float x) {
  if (sizeof(T) == 2 && s.merged) return fabsf(x) < 0x1p-16f ? 0.f : x;
  return own(s, x);
}

__device__ __forceinline__ bool kept(const RowStat& s, float x, int id) {
  return (x > s.vcut || (x == s.vcut && id <= s.idcut)) && x >= s.floor;
}

// 2^44 e^{-d/T} for d = M - x >= 0, rounded to an integer.  t = 32 d log2(e)/T =
// n - r with n an integer and |r| <= 1/2; 2^(-n/32) comes from a table of 32
// and an exponent, 2^(r/32) = exp(r ln2/32) from its series up to r^3 (the next
// term is below 6e-10 relative), all in fp64: an fp32 weight (error 2^-24) would
// move the cumulative sums of a wide row by more than a small weight's width and
// with it the token.  Every product that is added to something is an explicit fma:
// the passes over a row have to find the same sums, so a weight must not depend on
// what the compiler makes of each copy of this code.
__device__ __forceinline__ u64 weight(const RowStat& s, const double* tab, float x) {
  if (!((s.top - x) * s.c < 45.5f)) return 0ull;  // also NaN and -inf
  constexpr double kMagic = 6755399441055744.0;   // 1.5 * 2^52: adding it rounds to an integer in the low bits
  constexpr double k1 = kLn2 / 32, k2 = k1 * k1 / 2, k3 = k1 * k1 * k1 / 6;
  const double d = (double)s.top - (double)x;
  const double nm = fma(d, s.c32, kMagic);
  const int n = __double2loint(nm);
  const double r = fma(-d, s.c32, nm - kMagic);
  const double p = r * fma(r, fma(r, k3, k2), k1);
  const double b = tab[n & 31];
  const double e = __hiloint2double(__double2hiint(b) - ((n >> 5) << 20), __double2loint(b));
  const double w = fma(e, p, e) + 4503599627370496.0;  // + 2^52: rounds, integer in the low 52 bits
  return (u64)(__double_as_longlong(w) & 0xfffffffffffffll);
}

// ------------------------------------------------------------------- bins
// The bin of a logit with upper half `pat`.
__device__ __forceinline__ int bin_of(uint32_t pat) {
  const int t = min(max((int)(pat & 0x7fffu), kPatLow - 1), kPatHigh) - (kPatLow - 1);
  return (pat & 0x8000u) ? kZeroBin + t : kZeroBin - t;
}
__device__ __forceinline__ int slot_of(int j) { return j <= kZeroBin ? kZeroBin - j : kNegative + j - kZeroBin; }
__device__ __forceinline__ void count_at(uint32_t a) { asm volatile("red.shared.add.u32 [%0], 1;" ::"r"(a) : "memory"); }
// The pattern of a bin (both ends: beyond the range), as the value whose lower
// half is `low`: for bf16 (low = 0) the bin's one value.
__device__ __forceinline__ float bin_value(int j, uint32_t low) {
  const int t = j < kZeroBin ? kZeroBin - j : j - kZeroBin;
  if (t == 0) return 0.f;
  return __uint_as_float((j > kZeroBin ? 0x80000000u : 0u) | ((uint32_t)(t + kPatLow - 1) << 16) | low);
}

// ------------------------------------------------------------------- team
__device__ __forceinline__ u64 warp_sum_u64(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
__device__ __forceinline__ u64 warp_scan_u64(u64 v) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 y = __shfl_up_sync(kFull, v, o);
    if ((int)(threadIdx.x & 31) >= o) v += y;
  }
  return v;
}

// Another CTA's shared memory: one word per access, in the cluster's window.
__device__ __forceinline__ uint32_t remote(const void* p, int rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void remote_store(uint32_t a, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
__device__ __forceinline__ u64 remote_load(uint32_t a) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t remote_load32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ int remote_add(uint32_t a, int v) {
  int o;
  asm volatile("atom.shared::cluster.add.s32 %0, [%1], %2;" : "=r"(o) : "r"(a), "r"(v) : "memory");
  return o;
}
// Cluster barrier for warps whose lanes may arrive at different times (a pass
// over a ragged slice comes right before it): the warp is brought together first
// and the barrier is the form without .aligned.
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  __syncwarp();
}

// The cluster as seen by the passes over one row.
struct Team {
  cg::cluster_group cl;
  SmpShared* sm;
  uint32_t* bins;  // this CTA's counts, by slot [kBinWords]
  uint32_t* sums;  // the cluster's counts of this CTA's segment of the bins (one CTA: unused)
  uint32_t* lows;  // fp32: per positive slot, the sum of the logits' lower 16 bits (/ 16) [kNegative], then the segment's
  int rank, size, parity;

  // Two numbers per CTA (each thread's a and b summed over the CTA, or their
  // maxima) told to every CTA: result[0 / 1][rank].  Buffers alternate: a CTA
  // writes a buffer again only after the call between, whose barrier every CTA
  // reached after its last read.
  template <bool MAX>
  __device__ __forceinline__ const u64 (*tell(u64 a, u64 b))[kSmpMaxCluster] {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    a = MAX ? warp_max_u64(a) : warp_sum_u64(a);
    b = MAX ? warp_max_u64(b) : warp_sum_u64(b);
    if (lane == 0) {
      sm->warp_part[0][warp] = a;
      sm->warp_part[1][warp] = b;
    }
    __syncthreads();
    parity ^= 1;
    if ((int)threadIdx.x < 2 * size) {
      const int which = threadIdx.x & 1, to = threadIdx.x >> 1;
      u64 v = 0;
      for (int w = 0; w < kSmpWarps; ++w) {
        const u64 y = sm->warp_part[which][w];
        v = MAX ? umax64(v, y) : v + y;
      }
      remote_store(remote(&sm->xch[parity][which][rank], to), v);
    }
    cluster_sync();
    return sm->xch[parity];
  }
  __device__ __forceinline__ void sums2(u64& a, u64& b) {
    const auto x = tell<false>(a, b);
    a = b = 0;
    for (int r = 0; r < size; ++r) {
      a += x[0][r];
      b += x[1][r];
    }
  }
  // The calling thread (one of the cluster) writes two words to every CTA; all
  // then call heard(), which returns them.
  __device__ __forceinline__ void say(u64 a, u64 b) {
    for (int r = 0; r < size; ++r) {
      remote_store(remote(&sm->word[parity ^ 1][0], r), a);
      remote_store(remote(&sm->word[parity ^ 1][1], r), b);
    }
  }
  __device__ __forceinline__ const u64* heard() {
    parity ^= 1;
    cluster_sync();
    return sm->word[parity];
  }
};

// f(vector, its index) over the CTA's slice, each(): f(logit, id).
template <typename T, int BATCH = kSmpBatch, typename F>
__device__ __forceinline__ void each_vec(const RowSlice<T>& sl, F&& f) {
  for (int v0 = threadIdx.x; v0 < sl.nvec; v0 += kSmpThreads * BATCH) {
    uint4 u[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int v = v0 + i * kSmpThreads;
      u[i] = v < sl.nvec ? sl.get(v) : Elem<T>::neg_inf_vec();
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int v = v0 + i * kSmpThreads;
      if (v >= sl.nvec) break;
      f(u[i], v);
    }
  }
}
template <typename T, typename F>
__device__ __forceinline__ void each(const RowSlice<T>& sl, F&& f) {
  constexpr int E = Elem<T>::kPerVec;
  each_vec<T>(sl, [&](const uint4& u, int v) {
    float x[E];
    Elem<T>::unpack(u, x);
    const int id = sl.first + v * E;
#pragma unroll
    for (int e = 0; e < E; ++e) f(x[e], id + e);
  });
}

// All threads of one CTA: the smallest id of its slice whose cumulative g(x, id)
// (a non-negative integer) exceeds thr, thr < the slice's total: the thread with
// that token calls hit(id, x).  A warp takes up to 512 neighbouring vectors at a
// time (no barrier in between); those that hold thr are split over the warps
// again, down to 64 or less, which one warp's lanes share.
template <typename T, typename G, typename H>
__device__ __forceinline__ void select_local(SmpShared& sm, const RowSlice<T>& sl, u64 thr, G&& g, H&& hit) {
  constexpr int E = Elem<T>::kPerVec;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto vec_sum = [&](const uint4& u, int v) {
    float y[E];
    Elem<T>::unpack(u, y);
    u64 s = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) s += g(y[e], sl.first + v * E + e);
    return s;
  };
  constexpr int kBatch = 4;
  auto region_sum = [&](int v0, int count) {  // of the warp, count a multiple of 32
    u64 s = 0;
    for (int i = 0; i < count; i += 32 * kBatch) {
      uint4 u[kBatch];
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        const int v = v0 + i + q * 32 + lane;
        u[q] = v < sl.nvec && i + q * 32 < count ? sl.get(v) : Elem<T>::neg_inf_vec();
      }
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        const int v = v0 + i + q * 32 + lane;
        if (v < sl.nvec && i + q * 32 < count) s += vec_sum(u[q], v);
      }
    }
    return warp_sum_u64(s);
  };
  // the part of list[0..8) that holds thr (kSmpWarps: none); base becomes what lies before it
  u64 base = 0;
  auto part_of = [&](const u64* parts) {
    int at = kSmpWarps;
    u64 run = base;
#pragma unroll
    for (int w = 0; w < kSmpWarps; ++w) {
      const u64 y = parts[w];
      if (at == kSmpWarps && thr < run + y) {
        at = w;
        base = run;
      }
      run += y;
    }
    if (at == kSmpWarps) base = run;
    return at;
  };
  u64* parts = sm.list;
  int v0 = -1, owner = 0;
  int region = sl.nvec <= kSmpWarps * 32 ? 32 : (sl.nvec <= kSmpWarps * 64 ? 64 : (sl.nvec <= kSmpWarps * 256 ? 256 : 512));
  for (int b = 0; b < sl.nvec; b += kSmpWarps * region) {
    const u64 s = b + warp * region < sl.nvec ? region_sum(b + warp * region, region) : 0;
    if (lane == 0) parts[warp] = s;
    __syncthreads();
    const int at = part_of(parts);
    __syncthreads();
    if (at < kSmpWarps) {
      v0 = b + at * region;
      owner = at;
      break;
    }
  }
  if (v0 < 0) return;  // (thr is below the total)
  if (region > 64) {
    region /= kSmpWarps;
    const u64 s = region_sum(v0 + warp * region, region);
    if (lane == 0) parts[warp] = s;
    __syncthreads();
    const int at = part_of(parts);
    __syncthreads();
    v0 += at * region;
    owner = at;
  }
  if (owner != warp) return;
  for (int i = 0; i < region; i += 32) {
    const int v = v0 + i + lane;
    const uint4 u = v < sl.nvec ? sl.get(v) : Elem<T>::neg_inf_vec();
    const u64 c = v < sl.nvec ? vec_sum(u, v) : 0;
    const u64 inc = warp_scan_u64(c);
    u64 cum = base + inc - c;
    if (thr >= cum && thr < cum + c) {
      float y[E];
      Elem<T>::unpack(u, y);
      bool done = false;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        cum += g(y[e], sl.first + v * E + e);
        if (!done && thr < cum) {
          done = true;
          hit(sl.first + v * E + e, y[e]);
        }
      }
    }
    base += __shfl_sync(kFull, inc, 31);
  }
}

// The CTA whose part of `x[rank]` holds thr, and what lies before it (size: none).
__device__ __forceinline__ int owner_of(const u64* x, int size, u64 thr, u64& before) {
  before = 0;
  for (int r = 0; r < size; ++r) {
    if (thr < before + x[r]) return r;
    before += x[r];
  }
  return size;
}

// select_local over the cluster: every CTA sums g over its slice first.
template <typename T, typename G, typename H>
__device__ __forceinline__ void select(Team& tm, const RowSlice<T>& sl, u64 thr, G&& g, H&& hit) {
  u64 mine = 0, before;
  each<T>(sl, [&](float x, int id) { mine += g(x, id); });
  const auto x = tm.tell<false>(mine, 0);
  if (owner_of(x[0], tm.size, thr, before) == tm.rank) select_local<T>(*tm.sm, sl, thr - before, g, hit);
}

// ------------------------------------------------------------ a row's cut
constexpr int kTieUnknown = -2;

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

// What is asked of a row: k > 0: the first k tokens; by_p: top-p of those.
struct RowAsk {
  long long k;
  bool by_p;
  float p;
  float floor;  // min-p as a value: kept tokens are at or above it
};

__device__ __forceinline__ u64 share_of(float p, u64 Z) {  // ceil(p Z), within [1, Z]
  const u64 need = (u64)ceil((double)p * (double)Z);
  return need < 1 ? 1 : (need > Z ? Z : need);
}

// Row constants once M is known.
__device__ __forceinline__ RowAsk row_ask(const RowParams& pr, int V, RowStat& s) {
  RowAsk q;
  const bool greedy = !(pr.temperature > 0.f);
  const double T_ = greedy ? 1.0 : fmax((double)pr.temperature, 0x1p-100);
  s.c32 = 32.0 * 1.4426950408889634 / T_;
  s.c = (float)(s.c32 / 32.0);
  q.by_p = !greedy && pr.top_p < 1.f;  // (NaN: off)
  q.p = pr.top_p;
  q.k = greedy || (q.by_p && !(pr.top_p > 0.f)) ? 1 : (pr.top_k > 0 && pr.top_k < V ? pr.top_k : 0);
  if (q.k == 1) q.by_p = false;  // one token is its own share
  q.floor = -INFINITY;
  if (!greedy && pr.min_p > 0.f && T_ < INFINITY) {  // (T infinite: every e is 1)
    // e >= min_p where x >= M + T ln(min_p): the smallest float at or above it
    const double at = pr.min_p >= 1.f ? (double)s.top : (double)s.top + T_ * log((double)pr.min_p);
    q.floor = __double2float_ru(at);
  }
  return q;
}

// Cuts by halving the ordered bit patterns, a pass over the row per step; any
// values, any ties.  Leaves s.vcut, s.idcut and each CTA's kept weight.
template <typename T>
__device__ __forceinline__ void cut_by_halving(Team& tm, const RowSlice<T>& sl, const RowParams& pr, int V, RowStat& s) {
  SmpShared& sm = *tm.sm;
  s.infinite = s.merged = false;
  s.bin0 = s.bin1 = -1;
  s.total = 0;
  {
    float m = -INFINITY;
    each<T>(sl, [&](float x, int) { m = fmaxf(m, canon<T>(s, x)); });
    const auto x = tm.tell<true>(order_bits(m), 0);
    u64 t = 0;
    for (int r = 0; r < tm.size; ++r) t = umax64(t, x[0][r]);
    s.top = order_value((uint32_t)t);
    if (s.top == INFINITY) {
      s.infinite = true;
      s.top = 0.f;
    }
    if (s.top == -INFINITY) return;  // nothing to draw
  }
  s.vcut = s.floor = -INFINITY;
  s.idcut = 0x7fffffff;
  const RowAsk ask = row_ask(pr, V, s);
  auto measure = [&](float cut, bool strict, bool mass) {
    u64 n = 0, unused = 0;
    each<T>(sl, [&](float y, int id) {
      const float x = canon<T>(s, y);
      if (kept(s, x, id) && (strict ? x > cut : x >= cut)) n += mass ? weight(s, sm.tab, x) : 1ull;
    });
    tm.sums2(n, unused);
    return n;
  };
  // the largest v with measure(x >= v) >= need; then how many of the tokens
  // equal to v belong, by id
  auto cut_at = [&](u64 need, bool mass) {
    uint32_t lo = order_bits(-INFINITY) + 1, hi = order_bits(s.top);  // lo always holds enough
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo + 1) / 2;
      if (measure(order_value(mid), false, mass) >= need) lo = mid;
      else hi = mid - 1;
    }
    const float v = order_value(lo);
    const u64 above = measure(v, true, mass);
    const u64 one = mass ? weight(s, sm.tab, v) : 1ull;
    const u64 ties = (need - above + one - 1) / one;  // >= 1 of them
    select<T>(tm, sl, ties - 1, [&](float y, int id) {
                const float x = canon<T>(s, y);
                return (u64)(x == v && kept(s, x, id));
              }, [&](int id, float) { tm.say((u64)id, 0); });
    const u64* w = tm.heard();
    s.vcut = v;
    s.idcut = (int)w[0];
  };
  if (ask.k > 0 && measure(-INFINITY, true, false) > (u64)ask.k) cut_at((u64)ask.k, false);
  if (ask.by_p) cut_at(share_of(ask.p, measure(-INFINITY, true, true)), true);
  s.floor = ask.floor;
  u64 mine = 0;
  each<T>(sl, [&](float y, int id) {
    const float x = canon<T>(s, y);
    if (kept(s, x, id)) mine += weight(s, sm.tab, x);
  });
  const auto x = tm.tell<false>(mine, 0);
  s.total = 0;
  for (int r = 0; r < tm.size; ++r) s.total += x[0][r];
  if (threadIdx.x < tm.size) sm.cta_mass[threadIdx.x] = x[0][threadIdx.x];
  __syncthreads();
}

// Sum of `mine` over the threads of the CTA before this one, and over all of them.
__device__ __forceinline__ u64 cta_exclusive(SmpShared& sm, u64 mine, u64* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const u64 own = warp_sum_u64(mine);
  __syncthreads();
  if (lane == 0) sm.warp_part[0][warp] = own;
  __syncthreads();
  u64 before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kSmpWarps; ++w) {
    const u64 y = sm.warp_part[0][w];
    if (w < warp) before += y;
    total += y;
  }
  __syncthreads();
  if (all) *all = total;
  return before + warp_scan_u64(mine) - mine;
}

// The first bin (in descending order of value) at which the running measure of
// the cluster reaches `need`; per bin `of(j)`, per CTA the measure `seg` of its
// segment, `mine` this thread's part of it.  A warp's bins are [j0, j1), its lanes
// take them in turn.  1 <= need <= the total, so that exactly one thread of the
// cluster calls found(bin, measure before it): what it says is what all hear next.
template <typename O, typename F>
__device__ __forceinline__ void find_bin(Team& tm, const u64* seg, u64 need, u64 mine, int j0, int j1, O&& of,
                                         F&& found) {
  u64 before;
  if (owner_of(seg, tm.size, need - 1, before) != tm.rank) return;
  SmpShared& sm = *tm.sm;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const u64 own = warp_sum_u64(mine);
  __syncthreads();
  if (lane == 0) sm.warp_part[0][warp] = own;
  __syncthreads();
  u64 at = before;
#pragma unroll
  for (int w = 0; w < kSmpWarps; ++w) {
    const u64 y = sm.warp_part[0][w];
    if (w < warp) at += y;
  }
  __syncthreads();
  if (need <= at || need > at + own) return;  // the same in every lane
  for (int j = j0 + lane; j - lane < j1; j += 32) {
    const u64 m = j < j1 ? of(j) : 0;
    if (!__any_sync(kFull, m != 0)) continue;
    const u64 inc = warp_scan_u64(m);
    const unsigned hit = __ballot_sync(kFull, need <= at + inc);
    if (hit) {
      if (lane == __ffs(hit) - 1) found(j, at + inc - m);
      return;
    }
    at += __shfl_sync(kFull, inc, 31);
  }
}

// Sort n <= kListCap keys of shared memory in descending order (whole CTA).
__device__ __forceinline__ void sort_list(u64* a, int n) {
  int size = 1;
  while (size < n) size <<= 1;
  for (int i = n + threadIdx.x; i < size; i += kSmpThreads) a[i] = 0;
  __syncthreads();
  for (int k = 2; k <= size; k <<= 1) {
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int t = threadIdx.x; t < size / 2; t += kSmpThreads) {
        const int i = (t / j) * 2 * j + t % j, p = i + j;
        const u64 x = a[i], y = a[p];
        const bool desc = (i & k) == 0;
        if (desc ? x < y : x > y) {
          a[i] = y;
          a[p] = x;
        }
      }
      __syncthreads();
    }
  }
}

// The row's maximum, cut, total and each CTA's share of it, by way of the bins;
// false (in every CTA) for a row that they do not settle.  s.idcut is right for
// the CTA's own slice (GLOBAL: for every token).
template <typename T, bool GLOBAL>
__device__ __forceinline__ bool cut_by_bins(Team& tm, const RowSlice<T>& sl, const RowParams& pr, int V, RowStat& s) {
  SmpShared& sm = *tm.sm;
  const int tid = threadIdx.x;
  constexpr bool kExact = sizeof(T) == 2;  // a bin is one value
  s.infinite = false;
  s.merged = kExact;
  s.bin0 = s.bin1 = -1;
  s.ties = ~0ull;
  s.vcut = s.floor = -INFINITY;
  s.idcut = 0x7fffffff;
  s.total = 0;
  // ---- counts by value
  // (fp32 needs the places inside a bin only to estimate weights)
  const bool placed = !kExact && pr.temperature > 0.f && pr.top_p < 1.f;
  for (int i = tid; i < kBinWords / 4; i += kSmpThreads) reinterpret_cast<uint4*>(tm.bins)[i] = make_uint4(0, 0, 0, 0);
  if (placed)
    for (int i = tid; i < kNegative / 4; i += kSmpThreads) reinterpret_cast<uint4*>(tm.lows)[i] = make_uint4(0, 0, 0, 0);
  if (tid == 0) {
    sm.list_n = 0;
    sm.pick_entry = 0;
  }
  __syncthreads();
  float m = -INFINITY;
  const uint32_t bins_at = (uint32_t)__cvta_generic_to_shared(tm.bins);
  each_vec<T, 2 * kSmpBatch>(sl, [&](const uint4& u, int) {
    const uint32_t word[4] = {u.x, u.y, u.z, u.w};
    if constexpr (kExact) {
      // two logits at a time: magnitudes clamped to the bins' range, their
      // distances from its low end, the sign as the slots' upper half, as the
      // lower halves of shared-memory addresses (the upper half names the CTA)
      constexpr uint32_t kLow2 = (kPatLow - 1) * 0x10001u, kHigh2 = kPatHigh * 0x10001u;
      const uint32_t base2 = (bins_at & 0xffffu) * 0x10001u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w = word[i];
        const uint32_t t = __vminu2(__vmaxu2(w & 0x7fff7fffu, kLow2), kHigh2) - kLow2;
        const uint32_t a = ((t | ((w >> 3) & (kNegative * 0x10001u))) << 2) + base2;
        count_at(__byte_perm(a, bins_at, 0x7610));
        count_at(__byte_perm(a, bins_at, 0x7632));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w = word[i];
        const int t = min(max((int)((w >> 16) & 0x7fffu), kPatLow - 1), kPatHigh) - (kPatLow - 1);
        count_at(bins_at + 4u * ((uint32_t)t | ((w >> 19) & kNegative)));
        m = fmaxf(m, __uint_as_float(w));
        // (negative logits are only ever estimated roughly)
        if (placed && !(w >> 31)) atomicAdd(tm.lows + t, (w & 0xffffu) >> 4);
      }
    }
  });
  __syncthreads();
  if (tid == 0) tm.bins[0] += tm.bins[kNegative];  // both zeros
  // (padding reads as -inf: it only adds to the last bin, which is never used)
  cluster_sync();
  // ---- this CTA's segment of the bins, summed over the cluster
  const int seg = (kBins + tm.size - 1) / tm.size, seg0 = tm.rank * seg, seg1 = min(kBins, seg0 + seg);
  // (a warp takes neighbouring bins, 32 at a time: the values that occur lie close together)
  const int lane = tid & 31, warp = tid >> 5;
  const int per_warp = (seg + 32 * kSmpWarps - 1) / (32 * kSmpWarps) * 32;
  const int j0 = min(seg1, seg0 + warp * per_warp), j1 = min(seg1, j0 + per_warp);
  u64 first = 0;  // order bits of the largest value counted
  for (int j = j0 + lane; j < j1; j += 32) {
    uint32_t c = 0;
    const int at = slot_of(j);
    if (tm.size == 1) {
      c = tm.bins[at];
    } else {
      uint32_t part[kSmpMaxCluster];
#pragma unroll
      for (int r = 0; r < kSmpMaxCluster; ++r) part[r] = r < tm.size ? remote_load32(remote(tm.bins + at, r)) : 0;
#pragma unroll
      for (int r = 0; r < kSmpMaxCluster; ++r) c += part[r];
      tm.sums[j - seg0] = c;
      if (placed && c && j < kZeroBin) {
        uint32_t l = 0;
#pragma unroll
        for (int r = 0; r < kSmpMaxCluster; ++r) part[r] = r < tm.size ? remote_load32(remote(tm.lows + at, r)) : 0;
#pragma unroll
        for (int r = 0; r < kSmpMaxCluster; ++r) l += part[r];
        tm.lows[kNegative + j - seg0] = l;
      }
    }
    if (c && !first && j < kLastBin) first = order_bits(j == 0 ? INFINITY : bin_value(j, 0));
  }
  {
    const auto x = tm.tell<true>(first, kExact ? 0 : order_bits(m));
    u64 a = 0, b = 0;
    for (int r = 0; r < tm.size; ++r) {
      a = umax64(a, x[0][r]);
      b = umax64(b, x[1][r]);
    }
    // nothing but -512 and below, or 512 and above: not for the bins
    const float lead = a ? order_value((uint32_t)a) : -INFINITY;
    if (lead == -INFINITY || lead == INFINITY) {
      return false;
    }
    s.top = kExact ? lead : order_value((uint32_t)b);
  }
  auto sum_at = [&](int j) { return tm.size == 1 ? tm.bins[slot_of(j)] : tm.sums[j - seg0]; };
  const RowAsk ask = row_ask(pr, V, s);
  if (!((s.top + 512.f) * s.c >= 45.5f)) {  // tokens of the last bin would weigh something
    u64 n = 0, unused = 0;
    each<T>(sl, [&](float x, int) { n += x <= -512.f && x > -INFINITY; });
    tm.sums2(n, unused);
    if (n) {
      return false;
    }
  }
  // ---- bf16: everything from the counts
  if constexpr (kExact) {
    auto mass_of = [&](int j, uint32_t c) { return c && j < kLastBin ? c * weight(s, sm.tab, bin_value(j, 0)) : 0ull; };
    auto count_of = [&](int j, uint32_t c) { return j < kLastBin ? (u64)c : 0ull; };
    u64 n = 0, w = 0;
    for (int j = j0 + lane; j < j1; j += 32) {
      const uint32_t c = sum_at(j);
      n += count_of(j, c);
      if (ask.by_p) w += mass_of(j, c);
    }
    u64 ties = ~0ull;  // of the tokens equal to s.vcut
    int cut_bin = kLastBin;
    u64 zero_in = 0;  // a sum that the zero bin took part in
    if (ask.k > 0 || ask.by_p) {
      const auto x = tm.tell<false>(n, w);
      u64 N = 0, Z = 0;
      for (int r = 0; r < tm.size; ++r) {
        N += x[0][r];
        Z += x[1][r];
      }
      if (ask.k > 0 && N > (u64)ask.k) {
        find_bin(tm, x[0], (u64)ask.k, n, j0, j1, [&](int j) { return count_of(j, sum_at(j)); }, [&](int j, u64 at) {
          // the tokens above the bin, and how many of it
          tm.say((u64)j, (u64)ask.k - at);
        });
        const u64* h = tm.heard();
        cut_bin = (int)h[0];
        ties = h[1];
        if (ask.by_p) {
          // Z: the weight above the bin, and the ties'
          u64 above = 0, unused = 0;
          for (int j = j0 + lane; j < min(j1, cut_bin); j += 32) above += mass_of(j, sum_at(j));
          tm.sums2(above, unused);
          Z = above + ties * weight(s, sm.tab, bin_value(cut_bin, 0));
        }
      }
      if (ask.by_p) {
        if (cut_bin >= kZeroBin) zero_in = Z;  // the zero bin is part of Z
        const u64 need = share_of(ask.p, Z);
        const auto y = tm.tell<false>(n, w);
        find_bin(tm, y[1], need, w, j0, j1, [&](int j) { return mass_of(j, sum_at(j)); }, [&](int j, u64 at) {
          const u64 one = weight(s, sm.tab, bin_value(j, 0));
          tm.say((u64)j, (need - at + one - 1) / one);
        });
        const u64* h = tm.heard();
        cut_bin = (int)h[0];
        ties = h[1];
      }
      if (cut_bin < kLastBin) s.vcut = bin_value(cut_bin, 0);
    }
    s.floor = ask.floor;
    // ---- each CTA's kept weight, from its own counts
    {
      u64 mine = 0;
      const int from = bin_of(__float_as_uint(s.top) >> 16);
      int last = from;  // the last bin kept
      for (int j = from + tid; j < cut_bin; j += kSmpThreads) {
        const uint32_t c = tm.bins[slot_of(j)];
        const float v = bin_value(j, 0);
        if (v < s.floor || !((s.top - v) * s.c < 45.5f)) break;
        last = j;
        if (c) mine += c * weight(s, sm.tab, v);
      }
      last = __reduce_max_sync(kFull, last);
      if ((tid & 31) == 0) atomicMax(&sm.pick_entry, last);  // (set to 0 above)
      const u64 a = tid == 0 && cut_bin < kLastBin ? (u64)tm.bins[slot_of(cut_bin)] : 0ull;
      const auto x = tm.tell<false>(mine, a);
      const bool at_floor = cut_bin < kLastBin && s.vcut >= s.floor;  // the tokens equal to the cut are kept
      const u64 one = at_floor ? weight(s, sm.tab, s.vcut) : 0ull;
      u64 seen = 0, my_ties = 0, before_me = 0;
      s.total = 0;
      for (int r = 0; r < tm.size; ++r) {
        const u64 eq = x[1][r];
        const u64 take = ties > seen ? (ties - seen < eq ? ties - seen : eq) : 0;
        if (r == tm.rank) {
          my_ties = take;
          before_me = seen;
        }
        const u64 mass = x[0][r] + take * one;
        if (tid == 0) sm.cta_mass[r] = mass;
        s.total += mass;
        seen += eq;
      }
      __syncthreads();
      s.bin0 = from;
      s.bin1 = at_floor ? cut_bin : sm.pick_entry;
      s.ties = my_ties;
      // Values below 2^-16 are read as 0, off by at most 2^-16 c of their weight:
      // that must not show in a sum (2^-32 of it), nor in what is kept: no cut or
      // floor among them, and the top, which min-p and an argmax go by, not one of them
      if (cut_bin > kZeroBin && s.floor <= 0.f && (zero_in == 0 || s.total < zero_in)) zero_in = s.total;
      const bool among = cut_bin == kZeroBin || (cut_bin > kZeroBin && (fabsf(s.floor) < 0x1p-16f || s.top == 0.f));
      if (zero_in || among) {
        u64 tiny = 0, unused = 0;
        if (tm.bins[0])
          each<T>(sl, [&](float y, int) { tiny += y != 0.f && fabsf(y) < 0x1p-16f; });
        tm.sums2(tiny, unused);
        if (tiny && (among ||
                     !((double)tiny * (double)weight(s, sm.tab, 0.f) * (double)s.c * 0x1p-16 <= (double)zero_in * 0x1p-32)))
          return false;
      }
      if (cut_bin < kLastBin && ties < seen) {
        // some of the tokens equal to the cut: by id, so all in the CTAs before
        // one, none in those after it
        const u64 eq = tm.bins[slot_of(cut_bin)];
        auto is_tie = [&](float x2, int) { return (u64)(canon<T>(s, x2) == s.vcut); };
        if constexpr (GLOBAL) {
          // the CTA that holds the last tie taken finds its id for all
          if (my_ties > 0 && (my_ties < eq || ties == before_me + eq))
            select_local<T>(sm, sl, my_ties - 1, is_tie, [&](int id, float) { tm.say((u64)id, 0); });
          s.idcut = (int)tm.heard()[0];
        } else if (my_ties == 0) {
          s.idcut = -1;
        } else if (my_ties < eq) {
          s.idcut = kTieUnknown;  // looked up by the CTA that the draw falls into, see draw_kept
        }
      }
    }
    return true;
  } else {
    // ---- fp32: exact sums and a list around the cut, in a second pass
    auto count_of = [&](int j, uint32_t c) { return j < kLastBin ? (u64)c : 0ull; };
    // a bin's weight, estimated: its tokens at their mean place, and what their
    // spread adds to the mean of an exponential (variance width^2 / 12); the top's
    // bin at least the top's own weight, so that no T makes the total 0
    const int top_bin = bin_of(__float_as_uint(s.top) >> 16);
    auto guess_of = [&](int j, uint32_t c) {
      if (!c || j == 0 || j >= kLastBin) return 0ull;
      const uint32_t mean = j < kZeroBin ? min(0xffffu, (tm.size == 1 ? tm.lows[slot_of(j)] : tm.lows[kNegative + j - seg0]) / c * 16 + 8) : 0x8000u;
      const float v = bin_value(j, mean);
      const u64 w1 = weight(s, sm.tab, v < s.top ? v : s.top);
      const float wide = (bin_value(j, 0xffffu) - bin_value(j, 0)) * (s.c * (float)kLn2);
      const u64 w = (u64)((double)c * (double)w1 * (c > 1 ? 1.0 + (double)fminf(wide * wide, 1.f) / 24.0 : 1.0));
      return j == top_bin ? umax64(w, 1ull << kWeightBits) : w;
    };
    u64 n = 0, w = 0;
    for (int j = j0 + lane; j < j1; j += 32) {
      const uint32_t c = sum_at(j);
      n += count_of(j, c);
      if (ask.by_p) w += guess_of(j, c);
    }
    int lo_bin = 0, hi_bin = -1;  // bins whose tokens are listed
    bool by_k = false, window = false, slow = false;
    if (ask.k > 0 || ask.by_p) {
      const auto x = tm.tell<false>(n, w);
      u64 N = 0, Zg = 0;
      for (int r = 0; r < tm.size; ++r) {
        N += x[0][r];
        Zg += x[1][r];
      }
      by_k = ask.k > 0 && N > (u64)ask.k;
      window = ask.by_p && !by_k;
      if (by_k) {
        find_bin(tm, x[0], (u64)ask.k, n, j0, j1, [&](int j) { return count_of(j, sum_at(j)); },
                 [&](int j, u64 at) { tm.say((u64)j, at + sum_at(j)); });
        const u64* h = tm.heard();
        hi_bin = (int)h[0];
        slow = h[1] > (u64)kListCap;
      } else if (window) {
        // the bins where the estimated share may be reached, the estimate taken
        // to be within 1 part in 128 of what remains on either side
        const u64 need = share_of(ask.p, Zg), rest = Zg - need;
        const u64 slack = (need < rest ? need : rest) / 128;
        const u64 lo = need > slack ? need - slack : 1, hi = need + slack;
        find_bin(tm, x[1], lo, w, j0, j1, [&](int j) { return guess_of(j, sum_at(j)); }, [&](int j, u64) { tm.say((u64)j, 0); });
        lo_bin = (int)tm.heard()[0];
        const auto y = tm.tell<false>(n, w);
        find_bin(tm, y[1], hi, w, j0, j1, [&](int j) { return guess_of(j, sum_at(j)); }, [&](int j, u64) { tm.say((u64)j, 0); });
        hi_bin = (int)tm.heard()[0];
        // few tokens up to there: list them all, so that nothing depends on the estimate's lower end
        u64 upto = 0, unused = 0;
        for (int j = j0 + lane; j < min(j1, hi_bin + 1); j += 32) upto += sum_at(j);
        tm.sums2(upto, unused);
        if (upto <= (u64)kListCap) lo_bin = 0;
      }
    }
    if (slow) {
      return false;
    }
    const bool listed = hi_bin >= 0;
    // above: tokens before the listed bins; Z: all
    u64 Z = 0, above = 0, kept_above = 0;
    const uint32_t list_n = remote(&sm.list_n, 0), list = remote(sm.list, 0);  // CTA 0's
    // the listed bins as values: from the least of hi_bin to the largest of lo_bin
    const float list_lo = !listed ? INFINITY : (hi_bin < kZeroBin ? bin_value(hi_bin, 0) : (hi_bin == kZeroBin ? -0x1p-16f : bin_value(hi_bin, 0xffffu)));
    const float list_hi = !listed ? -INFINITY : (lo_bin < kZeroBin ? bin_value(lo_bin, 0xffffu) : (lo_bin == kZeroBin ? 0x1p-16f : bin_value(lo_bin, 0)));
    each<T>(sl, [&](float x, int id) {
      const bool before = x > list_hi;
      const bool in = x >= list_lo && !before;
      if (window || before) {
        const u64 y = weight(s, sm.tab, x);
        Z += y;
        if (before) above += y;
        if (before && x >= ask.floor) kept_above += y;
      }
      if (in) {
        const int at = remote_add(list_n, 1);
        if (at < kListCap) remote_store(list + 8 * at, make_key(x, id));
      }
    });
    s.floor = ask.floor;
    if (!listed) {
      const auto x = tm.tell<false>(kept_above, 0);
      for (int r = 0; r < tm.size; ++r) {
        s.total += x[0][r];
        if (tid == 0) sm.cta_mass[r] = x[0][r];
      }
      __syncthreads();
      return true;
    }
    tm.sums2(Z, above);
    // ---- CTA 0 sorts the list and cuts it
    if (tm.rank == 0) {
      const int cnt = sm.list_n;
      if (cnt == 0 || cnt > kListCap) {
        if (tid == 0) tm.say(0, 1);
      } else {
        sort_list(sm.list, cnt);
        const int kk = by_k ? (int)ask.k : cnt;  // tokens of the list that top-k leaves
        // this thread's run of the list and its weight
        const int run = (cnt + kSmpThreads - 1) / kSmpThreads, i0 = min(cnt, tid * run), i1 = min(cnt, i0 + run);
        u64 mine = 0;
        for (int i = i0; i < i1; ++i)
          if (i < kk) mine += weight(s, sm.tab, key_value(sm.list[i]));
        u64 all;
        const u64 at = cta_exclusive(sm, mine, &all);
        if (ask.by_p) {
          const u64 total = by_k ? all : Z;
          const u64 need = share_of(ask.p, total);
          if (need <= above || need > above + all) {
            if (tid == 0) tm.say(0, 1);  // the estimate missed
          } else if (need - above > at && need - above <= at + mine) {
            u64 c = at;
            for (int i = i0; i < i1; ++i) {
              c += i < kk ? weight(s, sm.tab, key_value(sm.list[i])) : 0;
              if (c >= need - above) {
                tm.say(sm.list[i], 0);
                break;
              }
            }
          }
        } else if (tid == 0) {
          tm.say(sm.list[kk - 1], 0);
        }
      }
    }
    const u64* h = tm.heard();
    if (h[1]) {
      return false;
    }
    const u64 key = h[0];
    s.vcut = key_value(key);
    s.idcut = key_index(key);
    // ---- each CTA's kept weight: what lies above the list, and its own part of it
    const int cnt = (int)remote_load32(list_n);
    const int id0 = sl.first, id1 = sl.first + sl.nvec * Elem<T>::kPerVec;
    for (int i = tid; i < cnt; i += kSmpThreads) {
      const u64 y = remote_load(list + 8 * i);
      const int id = key_index(y);
      if (y < key) break;  // sorted, descending
      if (id >= id0 && id < id1 && key_value(y) >= s.floor) kept_above += weight(s, sm.tab, key_value(y));
    }
    const auto x = tm.tell<false>(kept_above, 0);
    for (int r = 0; r < tm.size; ++r) {
      s.total += x[0][r];
      if (tid == 0) sm.cta_mass[r] = x[0][r];
    }
    __syncthreads();
    return true;
  }
}

template <typename T, bool GLOBAL>
__device__ __forceinline__ void filter_row(Team& tm, const RowSlice<T>& sl, const RowParams& pr, int V, RowStat& s) {
  if (!cut_by_bins<T, GLOBAL>(tm, sl, pr, V, s)) cut_by_halving<T>(tm, sl, pr, V, s);
}

// u as the draws read it: NaN and negative as 0, 1 and above as the largest float below 1
__device__ __forceinline__ double draw_u(float u) { return u >= 0.f ? (double)fminf(u, 0x1.fffffep-1f) : 0.0; }

__device__ __forceinline__ void team_init(Team& tm, SmpShared& sm, unsigned char* dyn) {
  tm.sm = &sm;
  tm.rank = (int)tm.cl.block_rank();
  tm.size = (int)tm.cl.num_blocks();
  tm.parity = 0;
  tm.bins = reinterpret_cast<uint32_t*>(dyn);
  // one CTA per row: its counts are the cluster's
  const int seg = tm.size > 1 ? ((kBins + tm.size - 1) / tm.size + 3) / 4 * 4 : 0;
  tm.sums = tm.bins + kBinWords;
  tm.lows = tm.bins + kBinWords + seg;
  if (threadIdx.x < 32) sm.tab[threadIdx.x] = exp2((double)kWeightBits - threadIdx.x / 32.0);
}

// Where few values are kept (bf16, all positive), the CTA first counts them by
// sub-slice: counts again make exact weights, one per value instead of one per
// token, and the draw reads only one sub-slice token by token (1056 rows
// of 128256 tokens, p = 0.9: 256 us against 470 with a weight per token kept).  Below
// four sub-slices of 64 vectors, two per lane, there is nothing to narrow.  Narrows
// sl, thr and s.ties to it.
template <typename T>
__device__ __forceinline__ void narrow(Team& tm, RowSlice<T>& sl, RowStat& s, u64& thr) {
  SmpShared& sm = *tm.sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nb = s.bin1 - s.bin0 + 1;
  constexpr int kSubs = 64;  // at most; their weights and the values' share sm.list
  const int subs = min(min(kSubs, kBinWords / nb), sl.nvec / 64);
  if (subs < 4 || nb > kListCap - kSubs || s.bin1 >= kZeroBin) return;
  const int vps = (sl.nvec + subs - 1) / subs;  // vectors per sub-slice
  __syncthreads();
  for (int i = tid; i < subs * nb; i += kSmpThreads) tm.bins[i] = 0;
  u64* wt = sm.list + kSubs;
  for (int i = tid; i < nb; i += kSmpThreads) wt[i] = weight(s, sm.tab, bin_value(s.bin1 - i, 0));
  __syncthreads();
  // a kept logit's pattern, as a signed 16-bit number, is at least the last kept bin's
  const int low = (int)(__float_as_uint(bin_value(s.bin1, 0)) >> 16);
  for (int q = warp; q < subs; q += kSmpWarps) {
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(tm.bins + q * nb);
    const int end = min((q + 1) * vps, sl.nvec);
    for (int v0 = q * vps + lane; v0 < end; v0 += 32 * kSmpBatch) {
      uint4 u[kSmpBatch];
#pragma unroll
      for (int i = 0; i < kSmpBatch; ++i) u[i] = v0 + 32 * i < end ? sl.get(v0 + 32 * i) : Elem<T>::neg_inf_vec();
#pragma unroll
      for (int i = 0; i < kSmpBatch; ++i) {
        const uint32_t word[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int a = ((int)(word[k] << 16) >> 16) - low, b = ((int)word[k] >> 16) - low;
          if (a >= 0) count_at(base + 4u * a);
          if (b >= 0) count_at(base + 4u * b);
        }
      }
    }
  }
  __syncthreads();
  const bool cut = bin_value(s.bin1, 0) == s.vcut;  // then the first count is of ties
  for (int q = warp; q < subs; q += kSmpWarps) {
    u64 m = 0;
    for (int i = lane + (cut ? 1 : 0); i < nb; i += 32) m += tm.bins[q * nb + i] * wt[i];
    m = warp_sum_u64(m);
    if (lane == 0) sm.list[q] = m;
  }
  __syncthreads();
  u64 run = 0, ties = s.ties;
  int at = subs - 1;
  for (int q = 0; q < subs; ++q) {
    const u64 eq = cut ? tm.bins[q * nb] : 0ull;
    const u64 take = ties < eq ? ties : eq;
    const u64 m = sm.list[q] + take * (cut ? wt[0] : 0ull);
    if (thr < run + m) {
      at = q;
      if (s.idcut == kTieUnknown) s.idcut = take == eq ? 0x7fffffff : (take == 0 ? -1 : kTieUnknown);
      s.ties = take;
      break;
    }
    run += m;
    ties -= take;
  }
  thr -= run;
  sl.first += at * vps * Elem<T>::kPerVec;
  sl.nvec = min(vps, sl.nvec - at * vps);
  __syncthreads();
}

// Draw from the kept tokens of the row: the CTA that the draw falls into finds the token.
template <typename T, typename H>
__device__ __forceinline__ void draw_kept(Team& tm, RowSlice<T> sl, RowStat s, double u, H&& hit) {
  SmpShared& sm = *tm.sm;
  u64 thr = (u64)(u * (double)s.total);
  u64 before;
  if (owner_of(sm.cta_mass, tm.size, thr, before) != tm.rank) return;
  thr -= before;
  if constexpr (sizeof(T) == 2) {
    if (s.bin0 >= 0) narrow<T>(tm, sl, s, thr);
  }
  if (s.idcut == kTieUnknown) {  // the first s.ties ties of this slice: find the last one's id
    select_local<T>(sm, sl, s.ties - 1, [&](float x, int) { return (u64)(canon<T>(s, x) == s.vcut); },
                    [&](int id, float) { sm.pick_id = id; });
    __syncthreads();
    s.idcut = sm.pick_id;
  }
  select_local<T>(sm, sl, thr, [&](float y, int id) {
                    const float x = canon<T>(s, y);
                    return kept(s, x, id) ? weight(s, sm.tab, x) : 0ull;
                  }, [&](int id, float y) { hit(id, own(s, y)); });
}

// bf16: four CTAs per SM (64 registers): the passes wait on memory and shared
// atomics in turn, so more rows in flight count for more than registers (1056 rows
// of 128256, p = 0.9: 258 us against 293 at three).  fp32: three, as many as shared
// memory holds (58 KB each with the places inside the bins); 64 registers would
// spill for nothing.
template <typename T>
__global__ void __launch_bounds__(kSmpThreads, sizeof(T) == 2 ? 4 : 3)
sample_kernel(const T* __restrict__ logits, int V, long long stride, eagle_sampling_t params,
              const float* __restrict__ uniforms, int32_t* __restrict__ tokens, float* __restrict__ logprob, int per) {
  __shared__ SmpShared sm;
  extern __shared__ __align__(16) unsigned char dyn[];
  griddep_wait();
  griddep_launch_dependents();
  Team tm{cg::this_cluster(), &sm, nullptr, nullptr, nullptr, 0, 0, 0};
  team_init(tm, sm, dyn);
  const long long row = blockIdx.x / tm.size;
  RowSlice<T> sl;
  place_slice<T>(sl, logits + row * stride, V, per, tm.rank);
  const RowParams pr = row_params(params, row);
  const float u = uniforms[row];
  RowStat s;
  filter_row<T, false>(tm, sl, pr, V, s);
  if (s.total == 0) {
    if (tm.rank == 0 && threadIdx.x == 0) {
      tokens[row] = -1;
      if (logprob) logprob[row] = -INFINITY;
    }
  } else {
    draw_kept<T>(tm, sl, s, draw_u(u), [&](int id, float x) {
      tokens[row] = id;
      if (logprob) {
        // log of the kept probability: (x - M) / T - ln(S / 2^44)
        const double z = ((double)x - (double)s.top) * (s.c32 * (kLn2 / 32.0));
        logprob[row] = (float)(z - log(ldexp((double)s.total, -kWeightBits)));
      }
    });
  }
  cluster_sync();  // no CTA leaves while another may still use its shared memory
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
    remote_store(remote(&ws.xd[tm.parity][tm.rank], threadIdx.x), (u64)__double_as_longlong(a));
  }
  cluster_sync();
  double a = 0.0;
  for (int r = 0; r < tm.size; ++r) a += ws.xd[tm.parity][r];
  return a;
}

template <typename T>
__global__ void __launch_bounds__(kSmpThreads, 2)
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
  Team tm{cg::this_cluster(), &sm, nullptr, nullptr, nullptr, 0, 0, 0};
  team_init(tm, sm, dyn);
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
  RowSlice<T> sl;
  __syncthreads();

  int j = 0, len = 0;
  RowStat s;
  while (true) {
    const T* trow = tgt + (trow0 + j) * (size_t)V;
    const int r = ws.drow[j];
    const T* drow = r >= 0 ? dft + ((size_t)b * R + r) * (size_t)V : nullptr;
    const double lse = r >= 0 ? dlse[(size_t)b * R + r] : 0.0;
    place_slice<T>(sl, trow, V, per, tm.rank);
    filter_row<T, true>(tm, sl, pr, V, s);
    const double inv_S = s.total ? 1.0 / (double)s.total : 0.0;
    // p and q of every child's token (0 for a token outside the vocabulary)
    if (tid < n && ws.par[tid] == j) {
      const int x = ws.tok[tid];
      double p = 0.0, q = 0.0;
      if (x >= 0 && x < V && r >= 0) {
        const float xt = own(s, (float)trow[x]);
        if (kept(s, xt, x)) p = (double)weight(s, sm.tab, xt) * inv_S;
        q = exp((double)(float)drow[x] - lse);
      }
      ws.px[tid + 1] = p;
      ws.qx[tid + 1] = q;
    }
    __syncthreads();
    double t = 0.0, F = 1.0, Q = 1.0;  // Q: draft mass not yet rejected at j (1 with replacement)
    bool rejected = false, spent = false;
    int moved = 0;
    // max(0, p - t q) of a token
    auto residual = [&](float y, int id) {
      const float x = own(s, y);
      if (!kept(s, x, id)) return 0.0;
      const u64 w = weight(s, sm.tab, x);
      if (w == 0) return 0.0;
      return fmax(0.0, fma(-t, exp((double)(float)drow[id] - lse), __dmul_rn((double)w, inv_S)));  // (see weight)
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
        draw_kept<T>(tm, sl, s, u, [&](int id, float) { bonus[b] = id; });
        drawn = true;
      } else {
        // integer weights of the residual, of a total F(t) <= 1 as 2^60
        auto g = [&](float x, int id) { return (u64)(residual(x, id) * 1152921504606846976.0); };
        u64 mine = 0, W = 0, before;
        each<T>(sl, [&](float x, int id) { mine += g(x, id); });
        const auto x = tm.tell<false>(mine, 0);
        for (int r2 = 0; r2 < tm.size; ++r2) W += x[0][r2];
        if (W) {
          const u64 thr = (u64)(u * (double)W);
          if (owner_of(x[0], tm.size, thr, before) == tm.rank)
            select_local<T>(sm, sl, thr - before, g, [&](int id, float) { bonus[b] = id; });
          drawn = true;
        }
      }
    }
    if (!drawn) {
      // nothing left to draw from: the target's argmax (-1 in a row without a finite logit)
      if (s.top == -INFINITY) {
        if (leader) bonus[b] = -1;
      } else {
        select<T>(tm, sl, 0ull, [&](float x, int) { return (u64)(canon<T>(s, x) == s.top); },
                  [&](int id, float) { bonus[b] = id; });
      }
    }
    break;
  }
  cluster_sync();  // no CTA leaves while another may still write to its shared memory
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
  int cl = 1;
  // Few rows: more CTAs each, as long as all fit at two per SM.  A wider cluster
  // shortens the passes and pays for every exchange.  Measured over filters of
  // all kinds, V = 128256, fp32 / bf16 (us): 1 row, 16 CTAs 26-42 / 23-34, eight
  // 38-57 / 26-34, one 106-241 / 48-114; 32 rows, nine CTAs 40-77 / 27-38, 16 (two
  // waves) 51-105 / 44-68, four 52-104 / 33-53; 1056 rows, one 568-938 / 175-404, two
  // 636-1148 / 207-376.  Between, two CTAs would gain on rows this wide (211 rows,
  // one 192-344 / 59-155, two 165-310 / 54-116) and lose on narrower ones (32003
  // tokens: one 56-124 / 36-58, two 79-159 / 36-49; 300 rows of them: one 64-131 /
  // 42-67, two 116-204 / 58-80).
  const long long want = 2LL * device_sm_count() / rows;
  if (cl < want) cl = (int)(want < kSmpMaxCluster ? want : kSmpMaxCluster);
  if (cl > (all + kSmpThreads - 1) / kSmpThreads) cl = (all + kSmpThreads - 1) / kSmpThreads;  // a vector per thread at least
  return {cl, (all + cl - 1) / cl};
}
// The counts and the cluster's counts of one CTA's segment; for fp32 the places too.
size_t bins_bytes(int cluster, int elem_bytes) {
  const size_t seg = cluster > 1 ? align_up((kBins + cluster - 1) / cluster, 4) : 0;
  return (kBinWords + seg + (elem_bytes == 4 ? kNegative + seg : 0)) * sizeof(uint32_t);
}

template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), long long grid, int cluster, size_t smem, bool pdl, cudaStream_t s,
                           Args... args) {
  // (the limit without opting in counts the static shared memory too, at most 16 KB here)
  cudaError_t e = ensure_smem_limit((const void*)kernel, smem + 16 * 1024);
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
  const size_t smem = bins_bytes(pl.cluster, dtype_bytes(dtype));
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
  const size_t smem = bins_bytes(pl.cluster, dtype_bytes(dtype));
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
