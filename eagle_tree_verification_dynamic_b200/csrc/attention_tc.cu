// Tree-masked split-KV attention on the 5th-generation tensor cores
// ("Tree Attention" verification of the EAGLE notes, "3.Verify"; mask
// semantics of "Технический анализ EAGLE-4", section "Деревья проверки
// EAGLE-4 и утилита управления").
//
// Work decomposition.  A unit is (sequence b, KV head g, group rg of 128 query
// rows); the rows are the (node, head-in-group) pairs of head g, so every K/V
// tile staged in shared memory serves all tree queries of the GQA group.  A
// unit's keys are cut into tiles of 64: its visible prefix range first, then
// its n tree keys.  All tiles of all units form one list (unit-major) that is
// cut into C equal contiguous ranges, one per CTA, with C <= the SM count and
// one CTA per SM: every CTA streams the same amount of KV whatever the prefix
// lengths of a ragged batch.  Each CTA derives the list from prefix_len itself.
// A unit that lies inside one CTA's range is finished there (bf16 output); a
// unit cut by range boundaries leaves one normalised partial (O rows and
// log-sum-exp) per piece, merged by attn_combine_kernel.
//
// Roles inside a CTA (320 threads):
//   warp 0      producer: Q of each unit (TMA box, or a gather when G does not
//               divide 128) into one of two Q buffers; K and V tiles into a
//               ring of stages (128-byte swizzle, no multicast); TMEM owner
//   warp 1      one thread issues tcgen05.mma: S = Q K^T into one of three TMEM
//               S buffers, at most two tiles ahead of PV; O += P V into TMEM,
//               each tile's keys 0..31 into O_A and keys 32..63 into O_B
//   warps 2-9   softmax, two warps per TMEM lane quarter: thread r owns query
//               row r, one warp the first 32 keys of every tile (and O_A), the
//               other the last 32 (and O_B).  Each applies the prefix range /
//               window / tree bitmask, keeps its own running reference max
//               (re-based only when it grows by > 8 in log2 units, then its O
//               and row sum are rescaled in TMEM) and writes P = 2^(x - m) as
//               bf16 over the S it has read (the type of V: one product takes
//               one type; a rounding of up to 2^-8 per weight, which averages
//               out over the keys, beside the output's own; the row sum adds
//               the fp32 values).  At the end of a unit's piece the
//               pair exchanges (max, sum) through shared memory, merges O_A and
//               O_B, and writes the output or partial
// Over a shared prefix (wide units, 352 threads) a unit has 256 rows, the two
// softmax warps of a quarter each have a row block of 128 to themselves, with all
// keys, Q buffer and O, and warp 10 issues the O products while warp 1 issues the
// S ones.
//
// Every mbarrier wait is bounded (about 2 s of wall time); a timeout sets an
// abort flag that ends all roles, records a per-CTA status word and still
// frees the TMEM columns.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "eagle_internal.h"
#include "sm100_ptx.cuh"

namespace eagle {

using namespace sm100;

constexpr int kTcThreads = 320;   // 10 warps: producer, MMA, 8 softmax
constexpr int kWideThreads = 352;  // wide units: a second MMA warp (the last)
constexpr int kBN = kAttnKeysPerTile;
constexpr int kRowsPerCta = kAttnRowsPerUnit;  // rows of one MMA
constexpr int kMaxStages = 12;
constexpr int kSmemOptIn = 232448;  // largest dynamic shared memory a block may opt into on sm_100
constexpr int kCombineThreads = 128;

// Shared memory from the (1024-byte aligned) dynamic base: a 3 KB header
// (barriers, then each row's (max, sum) exchange between the two softmax
// warps of a lane quarter), two Q buffers, the K/V ring (P lives in TMEM).
// WIDE: what the two softmax warps of a lane quarter do.  Narrow: a unit has 128
// rows and they share each tile's keys (32 per thread), three S buffers; the
// shortest way from a tile to its product, for CTAs with a handful of tiles.
// Wide: a unit has 256 rows, two blocks of 128 (each with a Q buffer, O_A and
// O_B), and a warp has a row of its block per thread and all 64 keys: every K/V
// tile staged serves twice the rows, and two S buffers per block let one block's
// softmax run beside the other's products.
template <int D, bool WIDE = false>
struct TcLayout {
  static constexpr int kAtoms = D / 64;               // 128-byte column atoms along D
  static constexpr int kQBytes = kAtoms * 128 * 128;  // 128 rows
  static constexpr int kKVAtomBytes = kBN * 128;      // 64 keys x 128 B
  static constexpr int kKBytes = kAtoms * kKVAtomBytes;
  static constexpr int kStageBytes = 2 * kKBytes;     // K + V
  static constexpr int kHdrBytes = 3072;
  static constexpr int kBarOff = 0;
  static constexpr int kXchOff = 512;                 // float2 [2 halves][128 rows]
  static constexpr int kQOff = kHdrBytes;             // two Q buffers
  static constexpr int kStageOff = kQOff + 2 * kQBytes;
  static constexpr int kStagesFit = (kSmemOptIn - kStageOff) / kStageBytes;
  static constexpr int kStages = kStagesFit > kMaxStages ? kMaxStages : kStagesFit;
  static constexpr int kSmemBytes = kStageOff + kStages * kStageBytes;
  // TMEM: three S buffers (64 columns each: QK^T may run two tiles ahead of
  // PV, so the softmax warps find the next S ready), then O over each tile's
  // keys 0..31 (O_A) and over keys 32..63 (O_B): the two softmax warps of a
  // lane quarter keep independent running maxima and are merged once per piece.
  // P (bf16, two keys per column) overwrites the S it came from: keys 0..31
  // at the buffer's columns 0..15, keys 32..63 at columns 32..47, each inside
  // the columns of S its own warp has already read.
  static constexpr uint32_t kTmemCols = 512;
  static constexpr int kSBufs = WIDE ? 4 : 3;
  static constexpr uint32_t kColS = 0;  // S buffer i at column 64 * i
  static constexpr uint32_t kColOA = kSBufs * 64;
  static constexpr uint32_t kColOB = kSBufs * 64 + D;
  static_assert(kStages >= 2, "at least a double-buffered K/V ring");
  static_assert(kSmemBytes <= kSmemOptIn, "shared memory");
  static_assert(kXchOff + 2 * 128 * 8 <= kHdrBytes, "header");
  static_assert(kColOB + D <= kTmemCols, "TMEM");
  static_assert(!WIDE || kSBufs % 2 == 0, "a buffer always the same block's");
};

struct TcBars {
  uint64_t q_full[2];
  uint64_t q_empty[2];
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t s_full[4];
  uint64_t p_full[4][2];  // per S buffer, per half of the tile's keys (the four warps writing that half; wide: [0])
  uint64_t pv_done[4];
  uint64_t mma_idle;
  uint64_t s_idle;   // wide: the S warp's
  uint64_t pair[4];  // per lane quarter: both softmax warps wrote their (max, sum)
  uint64_t never;    // nothing arrives here: the wait probe's barrier
  uint32_t tmem_base;
  int abort;
  int bad_page;  // a key inside the sequence sat on a page id outside the pool
  // this CTA's tile range [t0, t1) of the global list, and where it starts
  int n_tiles;  // t1 - t0
  int b0, hr0, off0;
};
static_assert(sizeof(TcBars) <= 512, "barrier block");  // kXchOff

// ----------------------------------------------------------- tile schedule
// The visible prefix keys of a unit come in one of three forms:
//   kModePlain   one range: the whole prefix, or the window's part of it
//   kModeSinks   a window and the first `sinks` keys: two ranges (one, when
//                they meet), each cut into tiles of 64 from its own start
//   kModeShared  the prefix is `shared` keys that every sequence of the batch
//                has in common, then the sequence's own: the shared keys get
//                units of their own, whose rows are (node, head) pairs of
//                the whole batch, so they are read once per 256 rows of the
//                batch instead of once per sequence.  Every unit leaves
//                partials there and the combine joins a row's two units.
// In kModeShared "sequence" 0 of the schedule is the shared range and 1..B the
// batch; in the other modes sequence b of the schedule is sequence b.
enum AttnMode { kModePlain = 0, kModeSinks = 1, kModeShared = 2 };

// Wide units (256 rows) over a shared prefix: there a CTA streams a hundred tiles
// and more, and with 128 rows each the loads alone took 1040 of 1190 us (16
// sequences over 32763 keys, 80-node trees; 5.5 GB, in part past L2).  256 rows:
// 850-1000 us; 32 sequences over 4096 keys 197 -> 153, 4 over 2048 with a KV head per
// query head 48 -> 38, 16 over 2048 with 80-node trees 133 -> 114.  A batch of few
// rows a head leaves half a unit empty and loses a little: 1 of 128 rows over
// 32768 keys 75 -> 79, 8 of 32 rows over 8192 keys 35 -> 41.  With sinks every unit
// has one sequence's rows only: narrow.
template <int MODE>
constexpr bool kWideTiles = MODE == kModeShared;
template <int MODE>
constexpr int unit_rows = kWideTiles<MODE> ? kAttnRowsShared : kAttnRowsPerUnit;

struct AttnGeom {
  const int32_t* plen;
  int B, Hkv, RG, n, Lmax, window, C;
  int lo_align;  // the first prefix tile starts at a multiple of this (64 for a paged cache, else 1)
  int sinks;                   // kModeSinks
  const int32_t* shared_len;   // kModeShared: device int, clamped to [0, Lshared]
  int Lshared;
  int RGs;                     // kModeShared: row groups of the whole batch's rows
};

// sequences of the schedule; their row groups, nodes and first node
template <int MODE>
__device__ __forceinline__ int geom_seqs(const AttnGeom& a) { return MODE == kModeShared ? a.B + 1 : a.B; }
template <int MODE>
__device__ __forceinline__ int geom_rg(const AttnGeom& a, int b) { return MODE == kModeShared && b == 0 ? a.RGs : a.RG; }
template <int MODE>
__device__ __forceinline__ int geom_nodes(const AttnGeom& a, int b) {
  return MODE == kModeShared && b == 0 ? a.B * a.n : a.n;
}
template <int MODE>
__device__ __forceinline__ int geom_node0(const AttnGeom& a, int b) {
  return MODE == kModeShared ? (b == 0 ? 0 : (b - 1) * a.n) : b * a.n;
}
// index of unit (b, hr) among all units
template <int MODE>
__device__ __forceinline__ int geom_unit(const AttnGeom& a, int b, int hr) {
  if (MODE == kModeShared) return b == 0 ? hr : a.Hkv * a.RGs + (b - 1) * a.Hkv * a.RG + hr;
  return b * a.Hkv * a.RG + hr;
}

template <int MODE>
__device__ __forceinline__ int geom_len(const AttnGeom& a, int b) {
  if (MODE == kModeShared) {
    if (b == 0) return min(max(__ldg(a.shared_len), 0), a.Lshared);
    --b;
  }
  return min(max(__ldg(a.plen + b), 0), a.Lmax);
}
// first key of the window range of a sequence of length L (the window of the
// shallowest tree node, depth 1, at position L), and kModeSinks' sink tiles
// before it (0 when the two ranges meet: then the window range starts at 0)
template <int MODE>
__device__ __forceinline__ int geom_lo(const AttnGeom& a, int L) {
  if (MODE == kModeShared) return 0;
  const int lo = a.window > 0 ? max(0, L - a.window + 1) : 0;
  const int at = lo - lo % a.lo_align;  // keys below the window start are masked row by row
  if (MODE == kModeSinks && at <= (min(a.sinks, L) + kBN - 1) / kBN * kBN) return 0;
  return at;
}
template <int MODE>
__device__ __forceinline__ int geom_sink_tiles(const AttnGeom& a, int L, int lo) {
  return MODE == kModeSinks && lo > 0 ? (a.sinks + kBN - 1) / kBN : 0;
}
template <int MODE>
__device__ __forceinline__ int geom_ptiles(const AttnGeom& a, int L) {
  const int lo = geom_lo<MODE>(a, L);
  return geom_sink_tiles<MODE>(a, L, lo) + (L - lo + kBN - 1) / kBN;
}
template <int MODE>
__device__ __forceinline__ int geom_tiles(const AttnGeom& a, int b) {
  const int pt = geom_ptiles<MODE>(a, geom_len<MODE>(a, b));
  return MODE == kModeShared && b == 0 ? pt : pt + (a.n + kBN - 1) / kBN;
}

// Whole warp: total tiles of all units of the schedule's sequences below b_end.
template <int MODE>
__device__ __forceinline__ long long geom_prefix(const AttnGeom& a, int b_end, int lane) {
  long long acc = 0;
  for (int b = lane; b < b_end; b += 32) acc += (long long)(a.Hkv * geom_rg<MODE>(a, b)) * geom_tiles<MODE>(a, b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(kFull, acc, o);
  return acc;
}

// Whole warp: the unit (b, hr) holding global tile t and t's offset in it.
template <int MODE>
__device__ __forceinline__ void geom_locate(const AttnGeom& a, long long t, int lane, int& b_out, int& hr_out,
                                            int& off_out) {
  const int nb = geom_seqs<MODE>(a);
  long long base = 0;
  for (int bc = 0; bc < nb; bc += 32) {
    const int b = bc + lane;
    const int tb = b < nb ? geom_tiles<MODE>(a, b) : 0;
    const long long v = (long long)(a.Hkv * geom_rg<MODE>(a, b)) * tb;
    long long inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(kFull, inc, o);
      if (lane >= o) inc += y;
    }
    const long long exc = inc - v;
    const bool hit = b < nb && base + exc <= t && t < base + inc;
    const unsigned m = __ballot_sync(kFull, hit);
    if (m) {
      const int src = __ffs(m) - 1;
      int bb = 0, hr = 0, off = 0;
      if (lane == src) {
        const long long within = t - (base + exc);
        bb = b;
        hr = (int)(within / tb);
        off = (int)(within % tb);
      }
      b_out = __shfl_sync(kFull, bb, src);
      hr_out = __shfl_sync(kFull, hr, src);
      off_out = __shfl_sync(kFull, off, src);
      return;
    }
    base += __shfl_sync(kFull, inc, 31);
  }
  b_out = nb;
  hr_out = 0;
  off_out = 0;
}

// CTA c holds tiles [c*T/C, (c+1)*T/C); this is the CTA holding tile t.
__device__ __forceinline__ int cta_of_tile(long long t, long long T, int C) {
  if (T * C < 0xffffffffLL) return (int)(((uint32_t)(t + 1) * (uint32_t)C - 1u) / (uint32_t)T);
  return (int)(((t + 1) * C - 1) / T);
}
// With fewer tiles than CTAs (a ragged batch far below Lmax) some ranges are empty.
__device__ __forceinline__ bool cta_nonempty(int c, long long T, int C) {
  return (long long)(c + 1) * T / C > (long long)c * T / C;
}

// One contiguous piece of a unit inside one CTA's range.
struct Piece {
  int b, hr;    // sequence of the schedule and (head, row group) of the unit
  int tb, te;   // tiles [tb, te) of the unit
  int ptiles;   // the unit's prefix tiles (tiles >= ptiles are tree tiles)
  int L, lo;    // prefix length and first key of its window range
  int st;       // kModeSinks: sink tiles before the window range
  bool whole;   // the piece is the entire unit and its result final
};
// first key of prefix tile t
template <int MODE>
__device__ __forceinline__ int piece_key0(const Piece& pc, int t) {
  if (MODE == kModeSinks) return t < pc.st ? t * kBN : pc.lo + (t - pc.st) * kBN;
  return pc.lo + t * kBN;
}

template <int MODE>
struct PieceCursor {
  int b, hr, off, left;
  __device__ __forceinline__ void init(int b0, int hr0, int off0, int n_tiles) {
    b = b0;
    hr = hr0;
    off = off0;
    left = n_tiles;
  }
  __device__ __forceinline__ void init(const TcBars* s) { init(s->b0, s->hr0, s->off0, s->n_tiles); }
  __device__ __forceinline__ bool next(const AttnGeom& a, Piece& pc) {
    if (left <= 0) return false;
    pc.b = b;
    pc.hr = hr;
    pc.L = geom_len<MODE>(a, b);
    pc.lo = geom_lo<MODE>(a, pc.L);
    pc.st = geom_sink_tiles<MODE>(a, pc.L, pc.lo);
    pc.ptiles = geom_ptiles<MODE>(a, pc.L);
    const int tiles = MODE == kModeShared && b == 0 ? pc.ptiles : pc.ptiles + (a.n + kBN - 1) / kBN;
    const int nt = min(tiles - off, left);
    pc.tb = off;
    pc.te = off + nt;
    pc.whole = MODE != kModeShared && off == 0 && nt == tiles;
    left -= nt;
    off = 0;
    if (++hr == a.Hkv * geom_rg<MODE>(a, b)) {
      hr = 0;
      ++b;
    }
    return true;
  }
};

struct TcParams {
  const __nv_bfloat16* q;
  const uint64_t* mask;
  const int32_t* pos;
  __nv_bfloat16* out;
  float* part_o;    // [C + U][unit_rows][D] normalised partial outputs
  float* part_lse;  // [C + U][unit_rows]
  int* cta_status;  // [C]
  AttnGeom geo;
  int Hq;
  int q_by_tma;      // 1: Q rows arrive by TMA (G divides 128), 0: gathered by the producer warp
  float scale_log2;  // softmax scale * log2(e)
  // paged prefix cache (block_table != null): pools [num_pages][Hkv][page_size][D],
  // block_table [B][pages_per_seq] page ids
  const int32_t* block_table;
  int page_size, pages_per_seq, num_pages;
  const int32_t* shared_table;  // kModeShared, paged: the shared keys' page ids [shared_pages]
  int shared_pages;
  // > 0: every softmax warp first waits this long (ns) on a barrier nothing
  // completes, so the CTA takes its abort path (eagle_debug_attention_wait_probe)
  unsigned long long probe_ns;
  // 1: everything but mask and pos was written before the previous kernel on
  // the stream started (the fused step, where that kernel is the expansion),
  // so Q, the prefix and tree K/V and prefix_len are read at once and only the
  // softmax warps wait for the previous kernel (for mask and pos)
  int early;
};

// Loads issued now and consumed later: the K/V stream keeps HBM saturated, so
// a demand load waits behind it for microseconds; the per-row inputs of a
// piece are therefore requested a whole piece ahead (the first piece's before
// the stream starts).
__device__ __forceinline__ uint64_t ld_early_u64(const uint64_t* p) {
  uint64_t v;
  asm volatile("ld.global.nc.u64 %0, [%1];" : "=l"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ int ld_early_s32(const int32_t* p) {
  int v;
  asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

// What a softmax thread reads besides S for one piece.
struct RowCtx {
  uint64_t mw0, mw1;  // ancestor-or-self bitmask of this row's node (pieces with tree tiles)
  int qpos;           // this row's position (window only)
  int tpos[4];        // positions of tree keys lane, 32+lane, 64+lane, 96+lane (window and tree tiles)
};

template <int MODE>
__device__ __forceinline__ void row_issue(RowCtx& rc, const Piece& pc, const TcParams& p, int r_unit, int lane,
                                          int G) {
  const AttnGeom& a = p.geo;
  const int r_glob = (pc.hr % geom_rg<MODE>(a, pc.b)) * unit_rows<MODE> + r_unit;
  const bool row_ok = r_glob < geom_nodes<MODE>(a, pc.b) * G;
  const int qi = row_ok ? r_glob / G : 0;
  const size_t nb = (size_t)geom_node0<MODE>(a, pc.b);
  const bool has_tree = pc.te > pc.ptiles;
  rc.mw0 = rc.mw1 = 0;
  rc.qpos = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) rc.tpos[i] = 0;
  if (row_ok && has_tree) {
    rc.mw0 = ld_early_u64(p.mask + (nb + qi) * 2);
    rc.mw1 = ld_early_u64(p.mask + (nb + qi) * 2 + 1);
  }
  if (MODE != kModeShared && a.window > 0) {
    if (row_ok) rc.qpos = ld_early_s32(p.pos + nb + qi);
    if (has_tree) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (32 * i + lane < a.n) rc.tpos[i] = ld_early_s32(p.pos + nb + 32 * i + lane);
    }
  }
}

// Block-table entry idx of a sequence (-1 past the table's width).
__device__ __forceinline__ int table_entry(const int32_t* bt, int idx, int width) {
  return idx < width ? ld_early_s32(bt + idx) : -1;
}

// Producer for a paged prefix cache: the K/V tiles of one piece.  A prefix
// tile's 64 keys (starting at a multiple of 64) arrive as boxes of
// min(page_size, 64) keys, each from the page the sequence's block table
// names.  The whole warp walks the tiles (lane 0 waits and issues) and reads
// the table 32 entries per coalesced load; the next 32 are requested as soon
// as the current ones are first used, so only a piece's first lookup waits on
// memory.  A page id outside the pool turns into a box past the end, which
// reads zeros; if a key inside the sequence sat there, the CTA reports it.
// (kModeSinks only reports pages that hold a key some row sees: a page between
// the sinks and the window may have been given back.)
// Returns false when a wait gave up.
template <int D, int MODE>
__device__ bool produce_paged(const TcParams& p, const AttnGeom& a, const Piece& pc, int g, uint32_t s_base,
                              TcBars* bars, volatile int* abort, const CUtensorMap* tm_k, const CUtensorMap* tm_v,
                              const CUtensorMap* tm_kt, const CUtensorMap* tm_vt, int lane, int& jg) {
  using Lay = TcLayout<D, kWideTiles<MODE>>;
  constexpr int S = Lay::kStages;
  const int ps = p.page_size;
  const int sub = ps < kBN ? ps : kBN;  // keys per box
  const int nsub = kBN / sub;           // boxes per tile: 1, 2 or 4
  const bool in_shared = MODE == kModeShared && pc.b == 0;
  const int width = in_shared ? p.shared_pages : p.pages_per_seq;
  const int seq = MODE == kModeShared ? pc.b - 1 : pc.b;
  const int32_t* bt = in_shared ? p.shared_table : p.block_table + (size_t)seq * p.pages_per_seq;
  const int past_end = p.num_pages * a.Hkv * ps;  // first row past the pools (the host keeps it in int range)
  int c0 = -64, cur = -1, nxt = -1;               // table chunk [c0, c0 + 32): lane l holds entry c0 + l
  for (int t = pc.tb; t < pc.te; ++t) {
    const int st = jg % S;
    bool w = true;
    if (lane == 0 && jg >= S) w = mbar_wait(smem_u32(&bars->empty[st]), ((jg / S) - 1) & 1, abort);
    if (!__shfl_sync(kFull, w, 0)) return false;
    const uint32_t fb = smem_u32(&bars->full[st]);
    const uint32_t kdst = s_base + Lay::kStageOff + st * Lay::kStageBytes;
    const uint32_t vdst = kdst + Lay::kKBytes;
    if (t < pc.ptiles) {
      const int key0 = piece_key0<MODE>(pc, t);
      const int e0 = key0 / ps;  // the tile's first entry; its nsub entries share e0's chunk
      const int base = e0 & ~31;
      if (base != c0) {  // warp-uniform
        cur = base == c0 + 32 ? nxt : table_entry(bt, base + lane, width);
        c0 = base;
        nxt = table_entry(bt, c0 + 32 + lane, width);
      }
      int row[4];
      bool bad = false;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int page = __shfl_sync(kFull, cur, (e0 - c0 + j) & 31);  // every lane takes part
        const int kj = key0 + j * sub;
        const bool valid = page >= 0 && page < p.num_pages;
        bool needed = kj < pc.L;
        if (MODE == kModeSinks) needed = needed && (kj < a.sinks || kj + sub > pc.L - a.window + 1);
        if (j < nsub && !valid && needed) bad = true;
        row[j] = valid ? (page * a.Hkv + g) * ps + kj % ps : past_end;
      }
      if (lane == 0) {
        if (bad) bars->bad_page = 1;
        mbar_arrive_expect_tx(fb, Lay::kStageBytes);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j < nsub) {
            for (int at = 0; at < Lay::kAtoms; ++at) {
              tma_load_2d(kdst + at * Lay::kKVAtomBytes + j * sub * 128, tm_k, at * 64, row[j], fb);
              tma_load_2d(vdst + at * Lay::kKVAtomBytes + j * sub * 128, tm_v, at * 64, row[j], fb);
            }
          }
        }
      }
    } else if (lane == 0) {
      mbar_arrive_expect_tx(fb, Lay::kStageBytes);
      const int z = geom_node0<MODE>(a, pc.b) + (t - pc.ptiles) * kBN;
      for (int at = 0; at < Lay::kAtoms; ++at) {
        tma_load_3d(kdst + at * Lay::kKVAtomBytes, tm_kt, at * 64, g, z, fb);
        tma_load_3d(vdst + at * Lay::kKVAtomBytes, tm_vt, at * 64, g, z, fb);
      }
    }
    ++jg;
  }
  return true;
}

// The lowest `count` of 32 bits (none below 0, all from 32 on).
__device__ __forceinline__ uint32_t low_bits(int count) {
  return count >= 32 ? 0xffffffffu : (count > 0 ? (1u << count) - 1u : 0u);
}

// How long a waiting softmax warp or producer lane may sleep per poll (ns):
// the MMA warp shares a scheduler with two softmax warps, and a warp that
// polls in a tight loop takes issue slots from it.
constexpr uint32_t kSoftmaxSleepNs = 300u;
constexpr uint32_t kProducerSleepNs = 500u;

// The MMA warps over wide units: one issues S = Q K^T, the other O += P V.  Each
// goes through its schedule with all lanes and only the issue itself is one
// lane's, so that addresses and descriptors stay in uniform registers, where the
// instruction wants them.  A tile costs such a warp some 500 cycles of waits,
// elections and commits, as much as the tensor pipe needs for it, so one warp
// doing both was the bound (with no MMA, no softmax and no load at all the tiles
// still took 0.55 us each).  They count products: j is row block j & 1 over tile
// j / 2.  S(j) goes where P(j - NB) was, once its PV is done.
template <int D, int MODE>
__device__ __forceinline__ void mma_scores(const AttnGeom& a, TcBars* bars, uint32_t s_base, uint32_t tmem,
                                           volatile int* abort) {
  using Lay = TcLayout<D, true>;
  constexpr int S = Lay::kStages, NB = Lay::kSBufs;
  constexpr uint32_t id_qk = idesc_bf16_f32(128, kBN, 0, 0);
  const int total = __shfl_sync(kFull, bars->n_tiles, 0);
  const uint64_t q_desc = smem_desc(s_base + Lay::kQOff, 16, 1024, kSwizzle128B);
  const uint64_t k_desc = smem_desc(s_base + Lay::kStageOff, 16, 1024, kSwizzle128B);
  PieceCursor<MODE> cur;
  cur.init(bars);
  Piece pc;
  int si = -1, rem = 0, st = 0, ph = 0;  // piece, tiles left in it, stage and its parity
  bool ok = true;
  for (int j = 0; ok && j < 2 * total; ++j) {
    const int blk = j & 1;
    if (blk == 0) {
      if (rem == 0) {
        cur.next(a, pc);
        ++si;
        rem = __shfl_sync(kFull, pc.te - pc.tb, 0);
        ok = __all_sync(kFull, mbar_wait(smem_u32(&bars->q_full[0]), si & 1, abort));
        if (!ok) break;
      }
      --rem;
      ok = __all_sync(kFull, mbar_wait(smem_u32(&bars->full[st]), ph, abort));
      if (!ok) break;
    }
    const int jb = j - NB;
    if (jb >= 0) ok = __all_sync(kFull, mbar_wait(smem_u32(&bars->pv_done[j % NB]), (uint32_t)(jb / NB) & 1u, abort));
    if (!ok) break;
    tc_fence_after();
    const uint64_t da = q_desc + (uint64_t)(blk * (Lay::kQBytes >> 4));
    const uint64_t db = k_desc + (uint64_t)(st * (Lay::kStageBytes >> 4));
    const uint32_t t_s = tmem + Lay::kColS + (uint32_t)((j % NB) * kBN);
    if (elect_one()) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        mma_bf16_ss(t_s, da + ((kk / 4) * 16384 + (kk % 4) * 32) / 16,
                    db + ((kk / 4) * Lay::kKVAtomBytes + (kk % 4) * 32) / 16, id_qk, kk > 0);
      mma_commit(smem_u32(&bars->s_full[j % NB]));
      if (rem == 0 && blk == 1) mma_commit(smem_u32(&bars->q_empty[0]));
    }
    __syncwarp();
    if (blk == 1 && ++st == S) {
      st = 0;
      ph ^= 1;
    }
  }
  // every MMA has finished before TMEM is released
  if (elect_one()) mma_commit(smem_u32(&bars->s_idle));
  __syncwarp();
  mbar_wait_drain(smem_u32(&bars->s_idle), 0, 200000000ull);
}

template <int D, int MODE>
__device__ __forceinline__ void mma_outputs(const AttnGeom& a, TcBars* bars, uint32_t s_base, uint32_t tmem,
                                            volatile int* abort) {
  using Lay = TcLayout<D, true>;
  constexpr int S = Lay::kStages, NB = Lay::kSBufs;
  constexpr uint32_t id_pv = idesc_bf16_f32(128, D, 0, 1);
  const int total = __shfl_sync(kFull, bars->n_tiles, 0);
  const uint64_t v_desc = smem_desc(s_base + Lay::kStageOff + Lay::kKBytes, Lay::kKVAtomBytes, 1024, kSwizzle128B);
  PieceCursor<MODE> cur;
  cur.init(bars);
  Piece pc;
  int rem = 0, st = 0;  // tiles left in the piece, stage
  bool first = true;    // of the piece: an accumulator starts there
  for (int j = 0; j < 2 * total; ++j) {
    if ((j & 1) == 0) {
      first = rem == 0;
      if (first) {
        cur.next(a, pc);
        rem = __shfl_sync(kFull, pc.te - pc.tb, 0);
      }
      --rem;
    }
    // (P(j) is there, so S(j) and with it this stage's copies have landed)
    if (!__all_sync(kFull, mbar_wait(smem_u32(&bars->p_full[j % NB][0]), (uint32_t)(j / NB) & 1u, abort))) break;
    tc_fence_after();
    const uint64_t db = v_desc + (uint64_t)(st * (Lay::kStageBytes >> 4));
    const uint32_t t_p = tmem + Lay::kColS + (uint32_t)((j % NB) * kBN);
    const uint32_t t_o = tmem + ((j & 1) ? Lay::kColOB : Lay::kColOA);
    const uint32_t more = first ? 0u : 1u;
    if (elect_one()) {
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) mma_bf16_ts(t_o, t_p + (uint32_t)(kk * 8), db + kk * 2048 / 16, id_pv, kk ? 1u : more);
      if (j & 1) mma_commit(smem_u32(&bars->empty[st]));
      mma_commit(smem_u32(&bars->pv_done[j % NB]));
    }
    __syncwarp();
    if ((j & 1) && ++st == S) st = 0;
  }
  if (elect_one()) mma_commit(smem_u32(&bars->mma_idle));
  __syncwarp();
  mbar_wait_drain(smem_u32(&bars->mma_idle), 0, 200000000ull);
}

template <int D, int MODE>
__global__ void __launch_bounds__(kWideTiles<MODE> ? kWideThreads : kTcThreads, 1)
attn_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
               const __grid_constant__ CUtensorMap tm_kt, const __grid_constant__ CUtensorMap tm_vt,
               const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_ks,
               const __grid_constant__ CUtensorMap tm_vs, const TcParams p) {
  constexpr bool kWide = kWideTiles<MODE>;
  using Lay = TcLayout<D, kWide>;
  constexpr int S = Lay::kStages;
  constexpr int NB = Lay::kSBufs;
  extern __shared__ __align__(1024) unsigned char smem[];
  const AttnGeom& a = p.geo;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = blockIdx.x;
  // The layout fills the opt-in maximum and the swizzled tiles need a
  // 1024-byte aligned base: with any other base the CTA does nothing and
  // reports status 2 (the whole CTA leaves here, before any barrier).
  if ((smem_u32(smem) & 1023u) != 0u) {
    if (tid == 0) p.cta_status[c] = 2;
    griddep_wait();
    griddep_launch_dependents();
    return;
  }
  TcBars* bars = reinterpret_cast<TcBars*>(smem + Lay::kBarOff);
  const uint32_t s_base = smem_u32(smem);
  const int G = p.Hq / a.Hkv;
  volatile int* abort = &bars->abort;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars->q_full[i]), 1);
      mbar_init(smem_u32(&bars->q_empty[i]), 1);
    }
    for (int i = 0; i < NB; ++i) {
      mbar_init(smem_u32(&bars->s_full[i]), 1);
      // every softmax thread of a half (4 warps) arrives for every tile, rows
      // or not; S(j) is written only after PV(j - NB) was issued, so a phase
      // completes before the next one on the same barrier begins
      mbar_init(smem_u32(&bars->p_full[i][0]), kWide ? 4 : 128);  // (wide: one arrival per warp)
      mbar_init(smem_u32(&bars->p_full[i][1]), 128);
      mbar_init(smem_u32(&bars->pv_done[i]), 1);
    }
    for (int i = 0; i < S; ++i) {
      mbar_init(smem_u32(&bars->full[i]), 1);
      mbar_init(smem_u32(&bars->empty[i]), 1);
    }
    mbar_init(smem_u32(&bars->mma_idle), 1);
    mbar_init(smem_u32(&bars->s_idle), 1);
    for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&bars->pair[i]), 64);
    mbar_init(smem_u32(&bars->never), 1);
    bars->abort = 0;
    bars->bad_page = 0;
    fence_mbar_init();
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
    prefetch_tmap(&tm_kt);
    prefetch_tmap(&tm_vt);
    if (p.q_by_tma) prefetch_tmap(&tm_q);
    if (MODE == kModeShared) {
      prefetch_tmap(&tm_ks);
      prefetch_tmap(&tm_vs);
    }
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(&bars->tmem_base), Lay::kTmemCols);
    tmem_relinquish();
  }
  // inputs may come from the previous kernel on the stream (with p.early only
  // mask and pos do, and the softmax warps wait for them after the barrier)
  if (!p.early) griddep_wait();
  // softmax warps: cursor and the first piece's row inputs, requested before
  // the K/V stream starts
  PieceCursor<MODE> scur;
  Piece spc;
  RowCtx src;
  bool s_have = false;
  const int quad = warp & 3;
  const int half = (warp - 2) >> 2;      // softmax: half of a tile's keys (wide: row block)
  const int r_local = quad * 32 + lane;  // softmax: TMEM lane = row within the block's 128
  const int r_unit = r_local + (kWide ? half * kRowsPerCta : 0);
  if (warp >= 1) {
    const long long T = geom_prefix<MODE>(a, geom_seqs<MODE>(a), lane);
    const long long t0 = (long long)c * T / a.C, t1 = (long long)(c + 1) * T / a.C;
    int b0 = geom_seqs<MODE>(a), hr0 = 0, off0 = 0;
    if (t1 > t0) geom_locate<MODE>(a, t0, lane, b0, hr0, off0);
    if (warp == 1 && lane == 0) {
      bars->n_tiles = (int)(t1 - t0);
      bars->b0 = b0;
      bars->hr0 = hr0;
      bars->off0 = off0;
    }
    if (warp >= 2 && warp < kTcThreads / 32) {
      scur.init(b0, hr0, off0, (int)(t1 - t0));
      s_have = scur.next(a, spc);
      // issued before the block barrier, so ahead of the first K/V copies,
      // and consumed only at the piece's first tile: the producer does not
      // wait for them (a load issued behind the K/V stream waits microseconds)
      if (s_have && !p.early) row_issue<MODE>(src, spc, p, r_unit, lane, G);
    }
  }
  // a thread lets the next kernel start only after its own griddep_wait, so
  // that kernel's early reads never see work older than this kernel's
  // predecessor unfinished
  if (!p.early) griddep_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    PieceCursor<MODE> cur;
    cur.init(bars);
    Piece pc;
    int si = 0, jg = 0;  // pieces whose Q was loaded; tiles issued
    bool ok = true;
    while (ok && cur.next(a, pc)) {
      // narrow: two Q buffers in turn; wide: both hold the piece's 256 rows
      const int qb = kWide ? 0 : si & 1, qround = kWide ? si : si >> 1;
      const int RG = geom_rg<MODE>(a, pc.b);
      const int g = pc.hr / RG, rg = pc.hr % RG;
      const int node0 = geom_node0<MODE>(a, pc.b), rows = geom_nodes<MODE>(a, pc.b) * G;
      // Q buffer qb was last read by the QK^T of piece si - 2 (wide: si - 1)
      if (qround >= 1 && !__all_sync(kFull, mbar_wait(smem_u32(&bars->q_empty[qb]), (qround - 1) & 1, abort))) {
        ok = false;
        break;
      }
      const uint32_t qdst = s_base + Lay::kQOff + qb * Lay::kQBytes;
      const uint32_t qbar = smem_u32(&bars->q_full[qb]);
      if (p.q_by_tma) {
        // 128 rows = (node, head-in-group) pairs: a box of {64 dims, G
        // heads, 128/G nodes} of q viewed as [B*n][Hq][D]
        if (lane == 0) {
          constexpr int kBlocks = unit_rows<MODE> / kRowsPerCta;
          mbar_arrive_expect_tx(qbar, kBlocks * Lay::kQBytes);
          const int rows_i = kRowsPerCta / G;
          for (int blk = 0; blk < kBlocks; ++blk)
            for (int at = 0; at < Lay::kAtoms; ++at)
              tma_load_3d(qdst + blk * Lay::kQBytes + at * 16384, &tm_q, at * 64, g * G,
                          node0 + (rg * kBlocks + blk) * rows_i, qbar);
        }
      } else {
        // gather: 16-byte pieces of the unit's rows into the swizzled K-major tiles
        constexpr int kVec = unit_rows<MODE> * Lay::kAtoms * 8;
        constexpr int kBatch = 8;
        for (int e0 = lane; e0 < kVec; e0 += 32 * kBatch) {
          uint4 v[kBatch];
#pragma unroll
          for (int u = 0; u < kBatch; ++u) {
            const int e = e0 + u * 32;
            v[u] = make_uint4(0, 0, 0, 0);
            if (e < kVec) {
              const int r = e / (Lay::kAtoms * 8), at = (e / 8) % Lay::kAtoms, cc = e % 8;
              const int rr = rg * unit_rows<MODE> + r;
              if (rr < rows) {
                const int i = rr / G, h = g * G + rr % G;
                v[u] = *reinterpret_cast<const uint4*>(p.q + (((size_t)node0 + i) * p.Hq + h) * D + at * 64 +
                                                       cc * 8);
              }
            }
          }
#pragma unroll
          for (int u = 0; u < kBatch; ++u) {
            const int e = e0 + u * 32;
            if (e < kVec) {
              const int r = e / (Lay::kAtoms * 8), at = (e / 8) % Lay::kAtoms, cc = e % 8;
              *reinterpret_cast<uint4*>(smem + Lay::kQOff + (qb + r / kRowsPerCta) * Lay::kQBytes + at * 16384 +
                                        (r % kRowsPerCta) * 128 + ((cc ^ (r & 7)) << 4)) = v[u];
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(qbar);
      }
      ++si;
      if (p.block_table != nullptr) {
        ok = produce_paged<D, MODE>(p, a, pc, g, s_base, bars, abort, &tm_k, &tm_v, &tm_kt, &tm_vt, lane, jg);
      } else if (lane == 0) {
        for (int t = pc.tb; t < pc.te; ++t) {
          const int st = jg % S;
          if (jg >= S && !mbar_wait(smem_u32(&bars->empty[st]), ((jg / S) - 1) & 1, abort, 2000000000ull,
                                    kProducerSleepNs)) {
            ok = false;
            break;
          }
          const uint32_t fb = smem_u32(&bars->full[st]);
          mbar_arrive_expect_tx(fb, Lay::kStageBytes);
          const uint32_t kdst = s_base + Lay::kStageOff + st * Lay::kStageBytes;
          const uint32_t vdst = kdst + Lay::kKBytes;
          if (t < pc.ptiles) {
            const bool in_shared = MODE == kModeShared && pc.b == 0;
            const int seq = MODE == kModeShared ? pc.b - 1 : pc.b;
            const int y = (in_shared ? g * a.Lshared : (seq * a.Hkv + g) * a.Lmax) + piece_key0<MODE>(pc, t);
            const CUtensorMap* mk = in_shared ? &tm_ks : &tm_k;
            const CUtensorMap* mv = in_shared ? &tm_vs : &tm_v;
            for (int at = 0; at < Lay::kAtoms; ++at) {
              tma_load_2d(kdst + at * Lay::kKVAtomBytes, mk, at * 64, y, fb);
              tma_load_2d(vdst + at * Lay::kKVAtomBytes, mv, at * 64, y, fb);
            }
          } else {
            const int z = node0 + (t - pc.ptiles) * kBN;
            for (int at = 0; at < Lay::kAtoms; ++at) {
              tma_load_3d(kdst + at * Lay::kKVAtomBytes, &tm_kt, at * 64, g, z, fb);
              tma_load_3d(vdst + at * Lay::kKVAtomBytes, &tm_vt, at * 64, g, z, fb);
            }
          }
          ++jg;
        }
      }
      ok = __shfl_sync(kFull, ok, 0);
      jg = __shfl_sync(kFull, jg, 0);
    }
    if (p.early) {
      griddep_wait();
      griddep_launch_dependents();
    }
    // drain: every issued copy lands before the CTA may exit
    if (lane == 0) {
      for (int j = (jg > S ? jg - S : 0); j < jg; ++j)
        mbar_wait_drain(smem_u32(&bars->full[j % S]), (j / S) & 1, 200000000ull);
      constexpr int kQs = kWide ? 1 : 2;  // Q loads that may be in flight
      for (int s2 = (si > kQs ? si - kQs : 0); s2 < si; ++s2)
        mbar_wait_drain(smem_u32(&bars->q_full[s2 % kQs]), (s2 / kQs) & 1, 200000000ull);
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------------- MMA
    if (p.early) {
      griddep_wait();
      griddep_launch_dependents();
    }
    if constexpr (kWide) {
      mma_scores<D, MODE>(a, bars, __shfl_sync(kFull, s_base, 0), __shfl_sync(kFull, tmem, 0), abort);
    } else if (lane == 0) {
      const uint32_t id_qk = idesc_bf16_f32(128, kBN, 0, 0);
      const uint32_t id_pv = idesc_bf16_f32(128, D, 0, 1);
      const uint32_t t_oa = tmem + Lay::kColOA, t_ob = tmem + Lay::kColOB;
      const int total = bars->n_tiles;
      // one throw-away MMA while the first tiles are in flight (the first
      // MMA of a CTA was measured to take ~3 us longer than the next ones):
      // it reads the second Q buffer and the last K/V stage, whatever they
      // hold, into the third S buffer, which QK^T(2) overwrites (in order)
      if (total > 0) {
        const uint64_t da = smem_desc(s_base + Lay::kQOff + Lay::kQBytes, 16, 1024, kSwizzle128B);
        const uint64_t db = smem_desc(s_base + Lay::kStageOff + (S - 1) * Lay::kStageBytes, 16, 1024, kSwizzle128B);
        mma_bf16_ss(tmem + Lay::kColS + 2u * kBN, da, db, id_qk, 0u);
      }
      PieceCursor<MODE> qc, pcur;
      qc.init(bars);
      pcur.init(bars);
      Piece qp, pp;
      int q_si = -1, q_rem = 0, jq = 0;  // QK^T cursor: piece, tiles left in it, next tile
      int p_rem = 0, p_len = 0;          // PV cursor: tiles left in its piece, piece length
      bool ok = true;
      for (int jp = 0; jp < total && ok; ++jp) {
        if (p_rem == 0) {
          pcur.next(a, pp);
          p_len = p_rem = pp.te - pp.tb;
        }
        const bool first = p_rem == p_len;  // O restarts at the first tile of a piece
        // issue whatever is ready: the next QK^T (its Q and K landed; at most
        // two tiles ahead), and this tile's PV per half of its keys (that
        // half's P is written)
        const int pbuf = jp % NB;
        const uint32_t ppar = (uint32_t)(jp / NB) & 1u;
        const int st = jp % S;
        const uint32_t p_tmem = tmem + Lay::kColS + (uint32_t)(pbuf * kBN);
        const uint32_t v_addr = s_base + Lay::kStageOff + st * Lay::kStageBytes + Lay::kKBytes;
        bool done_h[2] = {false, false};
        uint64_t tw = 0;
        for (uint32_t it = 0;; ++it) {
          if (jq < total && jq <= jp + NB - 1) {
            if (q_rem == 0) {
              qc.next(a, qp);
              ++q_si;
              q_rem = qp.te - qp.tb;
            }
            const int qb = q_si & 1;
            if (mbar_test_wait(smem_u32(&bars->q_full[qb]), (q_si >> 1) & 1) &&
                mbar_test_wait(smem_u32(&bars->full[jq % S]), (jq / S) & 1)) {
              tc_fence_after();
              const uint32_t q_addr = s_base + Lay::kQOff + qb * Lay::kQBytes;
              const uint32_t k_addr = s_base + Lay::kStageOff + (jq % S) * Lay::kStageBytes;
              const uint32_t t_s = tmem + Lay::kColS + (uint32_t)((jq % NB) * kBN);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = (kk % 4) * 32;
                const uint64_t da = smem_desc(q_addr + (kk / 4) * 16384 + off, 16, 1024, kSwizzle128B);
                const uint64_t db = smem_desc(k_addr + (kk / 4) * Lay::kKVAtomBytes + off, 16, 1024, kSwizzle128B);
                mma_bf16_ss(t_s, da, db, id_qk, kk > 0);
              }
              mma_commit(smem_u32(&bars->s_full[jq % NB]));
              if (--q_rem == 0) mma_commit(smem_u32(&bars->q_empty[qb]));
              ++jq;
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // the first half still missing is waited for with a short sleep
            // (the MMA warp shares its scheduler with two softmax warps, whose
            // issue slots a spinning poll would take); the other is only tested
            const uint32_t pbar = smem_u32(&bars->p_full[pbuf][h]);
            const bool waited = (h == 0 || done_h[0]) ? mbar_try_wait_hint(pbar, ppar, 200u) : mbar_test_wait(pbar, ppar);
            if (!done_h[h] && waited) {
              tc_fence_after();
              // keys 32h..32h+31 of the tile into O_A (h = 0) or O_B (h = 1); P
              // from TMEM, 16 keys = 8 columns per MMA
#pragma unroll
              for (int kk = 2 * h; kk < 2 * h + 2; ++kk) {
                const uint32_t a_col = (uint32_t)((kk >> 1) * 32 + (kk & 1) * 8);
                const uint64_t db = smem_desc(v_addr + kk * 2048, Lay::kKVAtomBytes, 1024, kSwizzle128B);
                mma_bf16_ts(h ? t_ob : t_oa, p_tmem + a_col, db, id_pv, (!first || (kk & 1)) ? 1u : 0u);
              }
              done_h[h] = true;
            }
          }
          if (done_h[0] && done_h[1]) break;
          if ((it & 15u) == 15u) {
            if (*abort) { ok = false; break; }
            const uint64_t now = globaltimer();
            if (tw == 0) tw = now;
            else if (now - tw > 2000000000ull) { *abort = 1; ok = false; break; }
          }
        }
        if (!ok) break;
        mma_commit(smem_u32(&bars->empty[st]));
        mma_commit(smem_u32(&bars->pv_done[pbuf]));
        --p_rem;
      }
      // every MMA this thread issued has finished before TMEM is released
      mma_commit(smem_u32(&bars->mma_idle));
      mbar_wait_drain(smem_u32(&bars->mma_idle), 0, 200000000ull);
    }
  } else if (kWide && warp == kWideThreads / 32 - 1) {
    if (p.early) {
      griddep_wait();
      griddep_launch_dependents();
    }
    mma_outputs<D, MODE>(a, bars, __shfl_sync(kFull, s_base, 0), __shfl_sync(kFull, tmem, 0), abort);
  } else {
    // ------------------------------------------------------------- softmax
    // warps 2..9: quad = TMEM lane quarter (32 query rows); half = which 32
    // keys of every tile, and which O accumulator, this warp owns.  The two
    // halves keep independent running maxima and sums and are merged once
    // per piece.
    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
    constexpr int KW = kWide ? 64 : 32;  // keys per thread and tile
    const uint32_t t_s = tmem + lane_base + Lay::kColS + (uint32_t)(kWide ? 0 : half * 32);
    const uint32_t t_own = tmem + lane_base + (half ? Lay::kColOB : Lay::kColOA);
    const uint32_t t_oa = tmem + lane_base + Lay::kColOA, t_ob = tmem + lane_base + Lay::kColOB;
    float2* xch = reinterpret_cast<float2*>(smem + Lay::kXchOff);  // [half][row]
    const float sl2 = p.scale_log2;
    if (p.early) {
      griddep_wait();  // mask and pos come from the previous kernel
      griddep_launch_dependents();
      if (s_have) row_issue<MODE>(src, spc, p, r_unit, lane, G);
    }
    Piece pc = spc;
    RowCtx rc = src;
    bool have = s_have;
    int jg = 0, n_epi = 0;
    bool ok = true;
    // the wait probe: a bounded wait that runs out, then the same abort path as
    // any wait that gives up (the other roles see the flag and drain)
    if (p.probe_ns != 0ull && !__all_sync(kFull, mbar_wait(smem_u32(&bars->never), 0, abort, p.probe_ns))) ok = false;
    while (ok && have) {
      Piece pn;
      RowCtx rn;
      const bool have_next = scur.next(a, pn);
      if (have_next) row_issue<MODE>(rn, pn, p, r_unit, lane, G);  // in flight during this piece
      const int RG = geom_rg<MODE>(a, pc.b);
      const int g = pc.hr / RG, rg = pc.hr % RG;
      const int rows = geom_nodes<MODE>(a, pc.b) * G;
      const int row0 = rg * unit_rows<MODE> + (kWide ? half * kRowsPerCta : 0);
      const int r_glob = row0 + r_local;
      const bool row_ok = r_glob < rows;
      const bool warp_live = row0 + quad * 32 < rows;  // a warp of padding rows only keeps the protocol
      const int qi = row_ok ? r_glob / G : 0;
      const int qh = row_ok ? g * G + r_glob % G : 0;
      const int win_lo = rc.qpos - a.window + 1;
      float m_used = -INFINITY, l = 0.f;  // reference max (scaled, log2) and row sum of this half
      for (int t = pc.tb; t < pc.te; ++t, ++jg) {
        // jp counts products: wide, two of them (row blocks) per tile.  (An even
        // number of S buffers: a buffer is always the same warps', which so wait for
        // each phase of its barrier in turn; a parity wait that skips a phase would
        // pass too early.)
        const int jp = kWide ? 2 * jg + half : jg;
        const int sbuf = jp % NB;
        if (!__all_sync(kFull, mbar_wait(smem_u32(&bars->s_full[sbuf]), (uint32_t)(jp / NB) & 1u, abort, 2000000000ull,
                                         kSoftmaxSleepNs))) {
          ok = false;
          break;
        }
        // (wide units have no window: all but a range's last tile and the tree's are seen whole by every row)
        const bool whole_tile = kWide && t < pc.ptiles && piece_key0<MODE>(pc, t) + kBN <= pc.L;
        if (MODE != kModePlain && !whole_tile) {
          // Values of keys that no row sees (past the prefix, between sinks and
          // window, another sequence's tree) may be anything, NaN included, and
          // 0 x NaN is NaN: this half's such rows of V are zeroed before P says
          // that PV may read them.  Only a range's first or last tile has any.
          const bool tree = t >= pc.ptiles;
          const int key0 = (tree ? (t - pc.ptiles) * kBN : piece_key0<MODE>(pc, t)) + (kWide ? 0 : half * 32);
#pragma unroll
          for (int hh = 0; hh < KW / 32; ++hh) {
            const int k0 = key0 + hh * 32;
            uint32_t seen = low_bits((tree ? a.n : pc.L) - k0);
            if (MODE == kModeSinks && !tree) seen &= ~low_bits(pc.L - a.window + 1 - k0) | low_bits(a.sinks - k0);
            if (seen != 0xffffffffu) {  // the same in every warp of the half
              unsigned char* v = smem + Lay::kStageOff + (jg % S) * Lay::kStageBytes + Lay::kKBytes +
                                 (kWide ? hh : half) * 32 * 128;
              for (int e = r_local; e < 32 * Lay::kAtoms * 8; e += 128) {
                const int key = e / (Lay::kAtoms * 8), piece = e % (Lay::kAtoms * 8);
                if (!((seen >> key) & 1u))
                  *reinterpret_cast<uint4*>(v + (piece / 8) * Lay::kKVAtomBytes + key * 128 + (piece % 8) * 16) =
                      make_uint4(0, 0, 0, 0);
              }
              fence_proxy_async_smem();
            }
          }
        }
        if (warp_live) {
          tc_fence_after();
          float x[KW];
#pragma unroll
          for (int hh = 0; hh < KW / 32; ++hh)
            tmem_ld32(t_s + (uint32_t)(sbuf * kBN + hh * 32), x + hh * 32);
          tmem_wait_ld();
          const bool tree = t >= pc.ptiles;
          float mx = -INFINITY;
#pragma unroll
          for (int hh = 0; hh < KW / 32; ++hh) {
            float* xh = x + hh * 32;
            if (!whole_tile) {
              const int key0 = (tree ? (t - pc.ptiles) * kBN : piece_key0<MODE>(pc, t)) + (kWide ? hh : half) * 32;
              const int k1 = tree ? a.n : pc.L;
              // visibility of 32 keys as one bit mask, built the same way on every
              // tile (so the code stays hot in the instruction cache): keys below
              // the piece's end, then the ancestor bits (tree keys) or the window's
              // lower bound (prefix keys)
              const int lim = k1 - key0;
              uint32_t vm = low_bits(lim);
              const uint64_t mw = key0 >= 64 ? rc.mw1 : rc.mw0;
              const uint32_t tree_bits = (uint32_t)(mw >> (key0 & 63));
              const int lo_cut = win_lo - key0;  // prefix keys below it are outside the window
              uint32_t win_bits =
                  (MODE == kModeShared || a.window == 0 || lo_cut <= 0) ? 0xffffffffu : (lo_cut >= 32 ? 0u : ~((1u << lo_cut) - 1u));
              if (MODE == kModeSinks) win_bits |= low_bits(a.sinks - key0);
              vm &= tree ? tree_bits : win_bits;
              if (!row_ok) vm = 0u;
              if (MODE != kModeShared && tree && a.window > 0) {  // the window on tree keys' positions (rare; warp-uniform)
                const int grp = key0 >> 5;
                const int tsel = grp == 0 ? rc.tpos[0] : grp == 1 ? rc.tpos[1] : grp == 2 ? rc.tpos[2] : rc.tpos[3];
#pragma unroll
                for (int cc = 0; cc < 32; ++cc) {
                  const int kpos = __shfl_sync(kFull, tsel, cc);  // every lane takes part
                  if (kpos < win_lo && !(MODE == kModeSinks && kpos < a.sinks)) vm &= ~(1u << cc);
                }
              }
              if (__any_sync(kFull, vm != 0xffffffffu)) {  // most prefix tiles see every key
#pragma unroll
                for (int cc = 0; cc < 32; ++cc) xh[cc] = ((vm >> cc) & 1u) ? xh[cc] : -INFINITY;
              }
            }
            float m4[4] = {fmax3(xh[0], xh[1], xh[2]), fmax3(xh[3], xh[4], xh[5]), fmax3(xh[6], xh[7], xh[8]),
                           fmax3(xh[9], xh[10], xh[11])};
#pragma unroll
            for (int cc = 12; cc < 28; cc += 8) {
              m4[0] = fmax3(m4[0], xh[cc], xh[cc + 1]);
              m4[1] = fmax3(m4[1], xh[cc + 2], xh[cc + 3]);
              m4[2] = fmax3(m4[2], xh[cc + 4], xh[cc + 5]);
              m4[3] = fmax3(m4[3], xh[cc + 6], xh[cc + 7]);
            }
            const float mh = fmax3(fmax3(m4[0], m4[1], m4[2]), fmax3(m4[3], xh[28], xh[29]), fmaxf(xh[30], xh[31]));
            mx = hh ? fmaxf(mx, mh) : mh;
          }
          mx *= sl2;  // scale > 0 keeps the order
          // (P of this tile replaces S(jg) in TMEM: PV(jg - NB), the last reader of
          // those columns, completed before QK^T(jg), whose commit s_full waited on)
          const bool rebase = mx > m_used + 8.f;
          if (__any_sync(kFull, rebase && t > pc.tb && l > 0.f)) {
            // these warps' O may only be rescaled once the PV before has finished
            // accumulating into it
            const int jb = jp - (kWide ? 2 : 1);
            if (!__all_sync(kFull, mbar_wait(smem_u32(&bars->pv_done[jb % NB]), (uint32_t)(jb / NB) & 1u, abort))) {
              ok = false;
              break;
            }
            tc_fence_after();
            const float f = (rebase && l > 0.f) ? ex2(m_used - mx) : 1.f;
            for (int c0 = 0; c0 < D; c0 += 16) {
              float o[16];
              tmem_ld16(t_own + c0, o);
              tmem_wait_ld();
#pragma unroll
              for (int u = 0; u < 16; ++u) o[u] *= f;
              tmem_st16(t_own + c0, o);
            }
            tmem_wait_st();
            l *= f;
          }
          if (rebase) m_used = mx;
          const float neg_m = m_used > -INFINITY ? -m_used : 0.f;  // no visible key yet: every x is -inf
          float2 s2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          uint32_t packed[KW / 2];
          const float2 sl2x2 = make_float2(sl2, sl2), nm2 = make_float2(neg_m, neg_m);
#pragma unroll
          for (int c2 = 0; c2 < KW / 2; ++c2) {
            const float2 z = ffma2(make_float2(x[2 * c2], x[2 * c2 + 1]), sl2x2, nm2);
            const float2 e = make_float2(ex2(z.x), ex2(z.y));
            s2[c2 & 1] = fadd2(s2[c2 & 1], e);
            const __nv_bfloat162 h2 = __floats2bfloat162_rn(e.x, e.y);
            packed[c2] = *reinterpret_cast<const uint32_t*>(&h2);
          }
          const float2 st2 = fadd2(s2[0], s2[1]);
          l += st2.x + st2.y;
          // P over the first columns of the S it came from (two keys per column)
#pragma unroll
          for (int hh = 0; hh < KW / 32; ++hh)
            tmem_st16u(t_s + (uint32_t)(sbuf * kBN + hh * 16), packed + hh * 16);
          tmem_wait_st();
        }
        tc_fence_before();
        if constexpr (kWide) {
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bars->p_full[sbuf][0]));
        } else {
          mbar_arrive(smem_u32(&bars->p_full[sbuf][half]));
        }
      }
      if (!ok) break;
      // ---- end of the piece: merge the two halves' (max, sum), normalise,
      // write bf16 output or the partial + log-sum-exp.  Each warp of the pair
      // writes its half of the output columns from both accumulators.
      if (kWide) {
        // The block's rows are these warps' alone, and their next P only follows
        // the last read here: no exchange.
        if (warp_live) {
          const int jl = 2 * (jg - 1) + half;
          if (!__all_sync(kFull, mbar_wait(smem_u32(&bars->pv_done[jl % NB]), (uint32_t)(jl / NB) & 1u, abort))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const float inv = l > 0.f ? 1.f / l : 0.f;
          const size_t row = ((size_t)c + (size_t)geom_unit<MODE>(a, pc.b, pc.hr)) * unit_rows<MODE> + r_unit;
          for (int c0 = 0; c0 < D; c0 += 16) {
            float o[16];
            tmem_ld16(t_own + c0, o);
            tmem_wait_ld();
            if (!row_ok) continue;
#pragma unroll
            for (int u = 0; u < 16; ++u) o[u] = inv > 0.f ? o[u] * inv : 0.f;  // (a row that saw nothing: zeros)
            // (whole 32-byte sectors: every piece comes this way)
            st_global_32(p.part_o + row * D + c0, o);
            st_global_32(p.part_o + row * D + c0 + 8, o + 8);
          }
          if (row_ok) p.part_lse[row] = l > 0.f ? (m_used + __log2f(l)) * (float)kLn2 : -INFINITY;
          tc_fence_before();
        }
      } else if (warp_live) {
        const int jl = jg - 1;
        if (!__all_sync(kFull, mbar_wait(smem_u32(&bars->pv_done[jl % NB]), (uint32_t)(jl / NB) & 1u, abort))) {
          ok = false;
          break;
        }
        tc_fence_after();
        xch[half * kRowsPerCta + r_local] = make_float2(m_used, l);
        mbar_arrive(smem_u32(&bars->pair[quad]));
        if (!__all_sync(kFull, mbar_wait(smem_u32(&bars->pair[quad]), n_epi & 1, abort))) {
          ok = false;
          break;
        }
        ++n_epi;
        const float2 other = xch[(half ^ 1) * kRowsPerCta + r_local];
        const float ma = half ? other.x : m_used, la = half ? other.y : l;
        const float mb = half ? m_used : other.x, lb = half ? l : other.y;
        const float M = fmaxf(ma, mb);
        const float wa = la > 0.f ? ex2(ma - M) : 0.f;
        const float wb = lb > 0.f ? ex2(mb - M) : 0.f;
        const float Ltot = la * wa + lb * wb;
        const float inv = Ltot > 0.f ? 1.f / Ltot : 0.f;
        const float fa = wa * inv, fb = wb * inv;
        const size_t slot = (size_t)c + (size_t)geom_unit<MODE>(a, pc.b, pc.hr);
        for (int c0 = half * (D / 2); c0 < (half + 1) * (D / 2); c0 += 16) {  // 16 columns at a time
          float oa[16], ob[16];
          tmem_ld16(t_oa + c0, oa);
          tmem_ld16(t_ob + c0, ob);
          tmem_wait_ld();
          if (!row_ok) continue;
#pragma unroll
          for (int u = 0; u < 16; ++u) oa[u] = fmaf(oa[u], fa, ob[u] * fb);
          if (pc.whole) {
            __nv_bfloat16* dst = p.out + (((size_t)geom_node0<MODE>(a, pc.b) + qi) * p.Hq + qh) * D + c0;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              uint32_t w[4];
#pragma unroll
              for (int v = 0; v < 4; ++v) {
                const __nv_bfloat162 h2 = __floats2bfloat162_rn(oa[u * 8 + 2 * v], oa[u * 8 + 2 * v + 1]);
                w[v] = *reinterpret_cast<const uint32_t*>(&h2);
              }
              *reinterpret_cast<uint4*>(dst + u * 8) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
            float* dst = p.part_o + (slot * kRowsPerCta + r_local) * D + c0;
#pragma unroll
            for (int u = 0; u < 4; ++u)
              *reinterpret_cast<float4*>(dst + 4 * u) = make_float4(oa[4 * u], oa[4 * u + 1], oa[4 * u + 2], oa[4 * u + 3]);
          }
        }
        if (row_ok && !pc.whole && half == 0)
          p.part_lse[slot * kRowsPerCta + r_local] = Ltot > 0.f ? (M + __log2f(Ltot)) * (float)kLn2 : -INFINITY;
        tc_fence_before();
        if (have_next) {
          // the other warp of the pair has read O too before either lets the next
          // piece's first P.V write it
          mbar_arrive(smem_u32(&bars->pair[quad]));
          if (!__all_sync(kFull, mbar_wait(smem_u32(&bars->pair[quad]), n_epi & 1, abort))) {
            ok = false;
            break;
          }
          ++n_epi;
        }
      }
      pc = pn;
      rc = rn;
      have = have_next;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, Lay::kTmemCols);
  if (tid == 0) p.cta_status[c] = bars->abort ? 1 : (bars->bad_page ? 3 : 0);
}

// Merge the pieces of every unit cut by CTA range boundaries:
//   out = sum_s e^{lse_s - M} O_s / sum_s e^{lse_s - M}
// One warp per query row (blockIdx.x = unit, blockIdx.y = group of 4 rows);
// each lane loads its D/32 dims of every piece's partial in one round of
// independent L2 reads, up to eight pieces at a time, merged online (the modes with
// sinks or a shared prefix: two rows, four pieces of each).
// A unit finished inside one CTA is skipped.  Block (0, 0) also folds the
// per-CTA status words into the workspace header.  In kModeShared the units
// are the sequences' own, every one left partials, and a row also takes the
// pieces of the shared unit that holds it.
constexpr int kCombineWarps = kCombineThreads / 32;
// Rows a warp merges, one after another: over a shared prefix every row has
// pieces to merge, and the schedule's divisions before them are paid per block
// (2, 4, 8 rows a warp, two at a time: 48, 46, 52 us at 4 sequences, 198, 194,
// 192 at 32).  With sinks only cut units do: one row, for latency (1, 2, 4: 30.7,
// 31.7, 34 us at one long sequence; 87, 87, 83 at 32).
template <int MODE>
constexpr int combine_rows = MODE == kModeShared ? 4 : 1;

struct CombParams {
  const float* part_o;
  const float* part_lse;
  const int* cta_status;
  int* status;
  __nv_bfloat16* out;
  AttnGeom geo;
  int Hq;
};

// Where a row's partials are: its pieces in CTAs c_shared.. (n_shared of them, of
// row r_shared of a shared unit), then those of its own unit in CTAs c_own.., row
// r_own, `count` in all.  A unit's slots start at its first CTA + its number.
struct RowPieces {
  int n_shared, count, c_shared, c_own, r_shared, r_own;
  size_t slot_shared, slot_own;
};

// Merge ROWS rows' pieces, up to CHUNK of each per round of loads.
template <int D, int UNIT, int ROWS, int CHUNK>
__device__ __forceinline__ void combine_pieces(const CombParams& p, long long T, const RowPieces (&w)[ROWS], int lane,
                                               float (&wsum)[ROWS], float (&acc)[ROWS][D / 32]) {
  constexpr int DPL = D / 32;  // output dims per lane
  const int C = p.geo.C;
  const bool all_live = T >= C;  // with at least one tile per CTA no range is empty
  float M[ROWS];
  int most = 0;
#pragma unroll
  for (int q = 0; q < ROWS; ++q) {
    M[q] = -INFINITY;
    wsum[q] = 0.f;
#pragma unroll
    for (int t = 0; t < DPL; ++t) acc[q][t] = 0.f;
    most = max(most, w[q].count);
  }
  for (int s0 = 0; s0 < most; s0 += CHUNK) {
    float ls[ROWS][CHUNK];
    float v[ROWS][CHUNK][DPL];
#pragma unroll
    for (int q = 0; q < ROWS; ++q) {
#pragma unroll
      for (int j = 0; j < CHUNK; ++j) {
        const int s = s0 + j;
        const bool sh = s < w[q].n_shared;
        const int at = sh ? s : s - w[q].n_shared;
        // (a CTA with an empty range wrote no partial)
        const bool live = s < w[q].count && (all_live || cta_nonempty((sh ? w[q].c_shared : w[q].c_own) + at, T, C));
        ls[q][j] = -INFINITY;
#pragma unroll
        for (int t = 0; t < DPL; ++t) v[q][j][t] = 0.f;
        if (!live) continue;
        const size_t sl = ((sh ? w[q].slot_shared : w[q].slot_own) + at) * UNIT + (sh ? w[q].r_shared : w[q].r_own);
        ls[q][j] = __ldcg(p.part_lse + sl);
        const float* src = p.part_o + sl * D + lane * DPL;
        if constexpr (DPL == 4) {
          const float4 f = __ldcg(reinterpret_cast<const float4*>(src));
          v[q][j][0] = f.x; v[q][j][1] = f.y; v[q][j][2] = f.z; v[q][j][3] = f.w;
        } else {
          const float2 f = __ldcg(reinterpret_cast<const float2*>(src));
          v[q][j][0] = f.x; v[q][j][1] = f.y;
        }
      }
    }
#pragma unroll
    for (int q = 0; q < ROWS; ++q) {
      float mc = M[q];
#pragma unroll
      for (int j = 0; j < CHUNK; ++j) mc = fmaxf(mc, ls[q][j]);
      if (mc == -INFINITY) continue;
      const float f = M[q] > -INFINITY ? __expf(M[q] - mc) : 0.f;
      wsum[q] *= f;
#pragma unroll
      for (int t = 0; t < DPL; ++t) acc[q][t] *= f;
#pragma unroll
      for (int j = 0; j < CHUNK; ++j) {
        const float e = ls[q][j] > -INFINITY ? __expf(ls[q][j] - mc) : 0.f;
        wsum[q] += e;
#pragma unroll
        for (int t = 0; t < DPL; ++t) acc[q][t] = fmaf(e, v[q][j][t], acc[q][t]);
      }
      M[q] = mc;
    }
  }
}

template <int D, int MODE>
__global__ void __launch_bounds__(kCombineThreads)
attn_combine_kernel(const CombParams p) {
  const AttnGeom& a = p.geo;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int HR = a.Hkv * a.RG;
  const int u = blockIdx.x, b = u / HR, hr = u % HR;
  const int sb = MODE == kModeShared ? b + 1 : b;  // the schedule's sequence
  const int g = hr / a.RG, rg = hr % a.RG;
  const int G = p.Hq / a.Hkv;
  constexpr int kUnit = unit_rows<MODE>;
  const int row0 = rg * kUnit, valid = min(kUnit, a.n * G - row0);
  constexpr int kRows = combine_rows<MODE>;        // per warp,
  constexpr int kAtOnce = MODE == kModeShared ? 2 : 1;  // as many at a time,
  constexpr int kChunk = MODE == kModePlain ? 8 : 4;   // so many pieces of each
  constexpr int kBlockRows = kRows * kCombineWarps;
  static_assert(kBlockRows <= 32 && kRows % kAtOnce == 0, "a lane per row of the block");
  __shared__ long long s_T;
  __shared__ int s_cfirst, s_clast, s_stat[kCombineWarps];
  __shared__ int3 s_shared[kBlockRows];  // kModeShared: each row's shared unit, its first and its last CTA
  if (warp == 0) {  // the schedule depends only on prefix_len, not on the attention kernel
    const int nb = geom_seqs<MODE>(a);
    long long T = 0, cum = 0;
    for (int s = lane; s < nb; s += 32) {
      const long long v = (long long)(a.Hkv * geom_rg<MODE>(a, s)) * geom_tiles<MODE>(a, s);
      T += v;
      if (s < sb) cum += v;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      T += __shfl_xor_sync(kFull, T, o);
      cum += __shfl_xor_sync(kFull, cum, o);
    }
    if (lane == 0) {  // (divisions: done before the wait, while the attention runs)
      const int tiles = geom_tiles<MODE>(a, sb);
      const long long start = cum + (long long)hr * tiles;
      s_T = T;
      s_cfirst = cta_of_tile(start, T, a.C);
      s_clast = cta_of_tile(start + tiles - 1, T, a.C);
    }
    if (MODE == kModeShared && lane < kBlockRows) {
      const int tiles = geom_tiles<MODE>(a, 0);
      const int us = g * a.RGs + (b * a.n * G + row0 + (int)blockIdx.y * kBlockRows + lane) / kUnit;
      s_shared[lane] = tiles > 0 ? make_int3(us, cta_of_tile((long long)us * tiles, T, a.C),
                                             cta_of_tile((long long)us * tiles + tiles - 1, T, a.C))
                                 : make_int3(us, 0, -1);
    }
  }
  __syncthreads();
  const long long T = s_T;
  const int c_first = s_cfirst, c_last = s_clast;
  griddep_wait();
  griddep_launch_dependents();  // the next kernel's prologue may overlap this one
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    int st = 0;
    for (int i = tid; i < a.C; i += kCombineThreads) st = max(st, p.cta_status[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) st = max(st, __shfl_xor_sync(kFull, st, o));
    if (lane == 0) s_stat[warp] = st;
    __syncthreads();
    if (tid == 0) {
      for (int w = 0; w < kCombineWarps; ++w) st = max(st, s_stat[w]);
      *p.status = st;
    }
  }
  if (MODE != kModeShared && c_first == c_last) return;
  constexpr int DPL = D / 32;  // output dims per lane
  for (int q0 = 0; q0 < kRows; q0 += kAtOnce) {
    const int first = (blockIdx.y * kRows + q0) * kCombineWarps + warp;  // rows first, first + kCombineWarps, ...
    if (first >= valid) return;
    RowPieces w[kAtOnce];
    float wsum[kAtOnce], acc[kAtOnce][DPL];
#pragma unroll
    for (int q = 0; q < kAtOnce; ++q) {
      const int r = first + q * kCombineWarps;
      w[q].n_shared = 0;
      w[q].c_shared = w[q].r_shared = 0;
      w[q].slot_shared = 0;
      if (MODE == kModeShared) {
        const int3 sh = s_shared[(q0 + q) * kCombineWarps + warp];
        w[q].n_shared = sh.z - sh.y + 1;
        w[q].c_shared = sh.y;
        w[q].r_shared = (b * a.n * G + row0 + r) % kUnit;
        w[q].slot_shared = (size_t)sh.y + sh.x;
      }
      w[q].c_own = c_first;
      w[q].r_own = r;
      w[q].slot_own = (size_t)c_first + geom_unit<MODE>(a, sb, hr);
      w[q].count = r < valid ? w[q].n_shared + c_last - c_first + 1 : 0;
    }
    combine_pieces<D, unit_rows<MODE>, kAtOnce, kChunk>(p, T, w, lane, wsum, acc);
#pragma unroll
    for (int q = 0; q < kAtOnce; ++q) {
      const int r = first + q * kCombineWarps;
      if (r >= valid) break;
      const int row = row0 + r, i = row / G, h = g * G + row % G;
      __nv_bfloat16* dst = p.out + (((size_t)b * a.n + i) * p.Hq + h) * D + lane * DPL;
      const float inv = wsum[q] > 0.f ? 1.f / wsum[q] : 0.f;
#pragma unroll
      for (int t = 0; t < DPL; t += 2)
        *reinterpret_cast<__nv_bfloat162*>(dst + t) = __floats2bfloat162_rn(acc[q][t] * inv, acc[q][t + 1] * inv);
    }
  }
}

// ------------------------------------------------------------------- host
namespace {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// bf16 tensor map with 128-byte swizzle (box given by the caller).
bool make_map(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides_bytes,
              const cuuint32_t* box) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides_bytes, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

}  // namespace

template <int D, int MODE>
static cudaError_t launch_tc(const AttnCall& k, cudaStream_t s) {
  const PagedKV* pg = k.pg;
  const int B = k.B, n = k.n, Hq = k.Hq, Hkv = k.Hkv;
  CUtensorMap mk, mv, mkt, mvt, mks, mvs;
  const bool paged = pg != nullptr && pg->block_table != nullptr;
  const int Lmax = paged ? pg->pages_per_seq * pg->page_size : k.Lmax;  // a sequence's capacity
  const int Lrows = Lmax > 0 ? Lmax : 1;
  const void* kbase = Lmax > 0 ? k.kc : k.kt;  // any valid address when the cache is empty
  const void* vbase = Lmax > 0 ? k.vc : k.vt;
  if (paged) {
    // pools [num_pages][Hkv][page_size][D] as rows of D; a box is min(page_size, 64) keys
    const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)pg->num_pages * Hkv * pg->page_size};
    const cuuint64_t str[1] = {(cuuint64_t)D * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)(pg->page_size < kBN ? pg->page_size : kBN)};
    if (!make_map(&mk, k.kc, 2, dims, str, box) || !make_map(&mv, k.vc, 2, dims, str, box)) return cudaErrorInvalidValue;
  } else {
    const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)B * Hkv * Lrows};
    const cuuint64_t str[1] = {(cuuint64_t)D * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)kBN};
    const cuuint64_t dims0[2] = {(cuuint64_t)D, (cuuint64_t)(Lmax > 0 ? (cuuint64_t)B * Hkv * Lrows : 1)};
    if (!make_map(&mk, kbase, 2, Lmax > 0 ? dims : dims0, str, box) ||
        !make_map(&mv, vbase, 2, Lmax > 0 ? dims : dims0, str, box))
      return cudaErrorInvalidValue;
  }
  {
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)Hkv, (cuuint64_t)B * n};
    const cuuint64_t str[2] = {(cuuint64_t)D * 2, (cuuint64_t)Hkv * D * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)kBN};
    if (!make_map(&mkt, k.kt, 3, dims, str, box) || !make_map(&mvt, k.vt, 3, dims, str, box))
      return cudaErrorInvalidValue;
  }
  mks = mk;
  mvs = mv;
  if (MODE == kModeShared && !paged && k.Lshared > 0) {
    const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)Hkv * k.Lshared};
    const cuuint64_t str[1] = {(cuuint64_t)D * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)kBN};
    if (!make_map(&mks, k.ks, 2, dims, str, box) || !make_map(&mvs, k.vs, 2, dims, str, box)) return cudaErrorInvalidValue;
  }
  const int G = Hq / Hkv;
  CUtensorMap mq;
  const bool q_tma = (kRowsPerCta % G) == 0;
  {
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)Hq, (cuuint64_t)B * n};
    const cuuint64_t str[2] = {(cuuint64_t)D * 2, (cuuint64_t)Hq * D * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)(q_tma ? G : 1), (cuuint32_t)(q_tma ? kRowsPerCta / G : 1)};
    if (!make_map(&mq, k.q, 3, dims, str, box)) return cudaErrorInvalidValue;
  }
  const AttnShape shape = {B, n, Hq, Hkv, D, Lmax, k.window, k.sinks, k.Lshared, MODE == kModeShared};
  const AttnWorkspace wl = attention_ws_layout(shape);
  unsigned char* wsb = static_cast<unsigned char*>(k.ws);
  TcParams p;
  p.q = static_cast<const __nv_bfloat16*>(k.q);
  p.mask = k.mask;
  p.pos = k.pos;
  p.out = static_cast<__nv_bfloat16*>(k.out);
  p.part_o = reinterpret_cast<float*>(wsb + wl.part_o_off);
  p.part_lse = reinterpret_cast<float*>(wsb + wl.part_lse_off);
  p.cta_status = reinterpret_cast<int*>(wsb + wl.cta_status_off);
  p.geo.plen = k.plen;
  p.geo.B = B;
  p.geo.Hkv = Hkv;
  p.geo.RG = attention_row_groups(shape);
  p.geo.n = n;
  p.geo.Lmax = Lmax;
  p.geo.window = k.window;
  p.geo.C = attention_ctas(shape);
  p.geo.lo_align = paged ? kBN : 1;
  p.geo.sinks = k.sinks;
  p.geo.shared_len = k.shared_len;
  p.geo.Lshared = k.Lshared;
  p.geo.RGs = MODE == kModeShared ? attention_shared_row_groups(shape) : 0;
  p.Hq = Hq;
  p.block_table = paged ? pg->block_table : nullptr;
  p.page_size = paged ? pg->page_size : 0;
  p.pages_per_seq = paged ? pg->pages_per_seq : 0;
  p.num_pages = paged ? pg->num_pages : 0;
  p.shared_table = k.shared_table;
  p.shared_pages = k.shared_pages;
  p.q_by_tma = q_tma ? 1 : 0;
  p.scale_log2 = k.scale * 1.4426950408889634f;
  p.probe_ns = attention_wait_probe_ns();
  p.early = k.early ? 1 : 0;
  const size_t smem = TcLayout<D, kWideTiles<MODE>>::kSmemBytes;
  cudaError_t e = ensure_smem_limit((const void*)attn_tc_kernel<D, MODE>, smem);
  if (e != cudaSuccess) return e;

  // both kernels may start while their predecessor drains (programmatic
  // dependent launch); each waits in griddep_wait before reading its inputs
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.geo.C);
  cfg.blockDim = dim3(kWideTiles<MODE> ? kWideThreads : kTcThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, attn_tc_kernel<D, MODE>, mk, mv, mkt, mvt, mq, mks, mvs, p);
  if (e != cudaSuccess) return e;

  CombParams cp;
  cp.part_o = p.part_o;
  cp.part_lse = p.part_lse;
  cp.cta_status = p.cta_status;
  cp.status = reinterpret_cast<int*>(wsb + wl.status_off);
  cp.out = p.out;
  cp.geo = p.geo;
  cp.Hq = Hq;
  cudaLaunchConfig_t cfg2 = {};
  // (over a shared prefix, whose units are often half empty, no blocks for rows that no unit has)
  constexpr int kPerBlock = kCombineWarps * combine_rows<MODE>;
  const int rows = MODE == kModeShared && n * G < unit_rows<MODE> ? n * G : unit_rows<MODE>;
  cfg2.gridDim = dim3((unsigned)((size_t)B * Hkv * p.geo.RG), (rows + kPerBlock - 1) / kPerBlock);
  cfg2.blockDim = dim3(kCombineThreads);
  cfg2.dynamicSmemBytes = 0;
  cfg2.stream = s;
  cfg2.attrs = attr;
  cfg2.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg2, attn_combine_kernel<D, MODE>, cp);
}

cudaError_t launch_tree_attention(const AttnCall& k, cudaStream_t s) {
  if (k.shared_len != nullptr) return k.D == 128 ? launch_tc<128, kModeShared>(k, s) : launch_tc<64, kModeShared>(k, s);
  // without a window every key is visible and the sinks change nothing
  if (k.sinks > 0 && k.window > 0)
    return k.D == 128 ? launch_tc<128, kModeSinks>(k, s) : launch_tc<64, kModeSinks>(k, s);
  return k.D == 128 ? launch_tc<128, kModePlain>(k, s) : launch_tc<64, kModePlain>(k, s);
}

}  // namespace eagle
