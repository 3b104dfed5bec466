// jf_shared.cu -- tree-causal paged attention for sequences that share a long prefix.
//
// The sequences of a group have their first S keys in common (the same pages: a prompt's beams
// after a fork, requests behind one system prompt).  A softmax over a set of keys is the merge
// of softmaxes over its parts: with (O_x, l_x) the output and log-sum-exp over part x,
//     l = log sum_x exp(l_x),   O = sum_x exp(l_x - l) O_x.
// So each group's shared keys are attended to once by the rows of all its sequences together
// (they lie one after the other in q, so they are one long list of nodes), and each sequence's
// own keys (from S on, its tree included) by its own rows; the parts merge at the end.  Shared
// K/V are read once per row tile group of the group instead of once per sequence, and rows fill
// the 128-row tensor-core tile that a single sequence's G rows leave nearly empty.
//
// Work.  A unit is a group's shared part or a sequence's own part; an item is a unit, a
// kv-head and a row tile.  Items lie end to end, T key tiles plus X::SW for the change of item,
// and are cut into equal ranges: lengths and group sizes are data, so every CTA forms the same
// schedule from them (about 3 us, a chain of barriers and of shared-memory reads) and walks its ranges.
// Every piece leaves normalised fp32 rows and their log-sum-exp: whole items in the rows' own
// slots (shared and own part apart), items that a range boundary cuts in the range's slots 0 (cut
// at its start) and 1; the first piece of an item tells each of its rows where its pieces are.
// The merge kernel reads that and adds up.
//
// Two kernels walk ranges; where both run, the one after the other.  (Alternatives' times in this file stand beside
// the chosen one's of the same run: device times in captured graphs.  Where a step is told as from .. to .., it is
// the step's own before and after.)
//   shared_attention_kernel: 256 rows (two tiles of 128) an item, tcgen05 products, one range per SM,
//     with the pipeline of the stream-K attention kernel (see jf_attention.cu: producer, MMA issuer,
//     vouchers, softmax warpgroups, all counters running over the range's tiles as one sequence).
//     A step of 128 keys takes 1.7 us, 78% of the tensor rate while it lasts: packed trees of 16
//     sequences over 8K shared keys, 106 GFLOP, take 120 us in all (0.89 PFLOP/s; rows that fill their
//     last tile in part, the prologue and the merge are the rest).
//   shared_rows_kernel (below): 16 to 64 rows an item, bound by the K/V stream: 256 beams in 32
//     groups over 4K keys take 87 us, 4.7 TB/s.
// jf_tree_attention on the same inputs reads a prefix once per sequence and takes 566 us for the
// beams, 695 us for 64 sequences over 32K shared keys (here 80).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "jf_attention.cuh"
#include "jf_common.cuh"
#include "jf_sm100.cuh"
#include "jf_tensormap.cuh"

namespace jf {
namespace {

// How a kernel cuts its units: row tiles of R rows, key tiles of KT keys, what a change of item
// costs, in key tiles, and the least that a range is cut for (small calls leave ranges empty).
template <int R_, int KT_, int SW_, int LEAST_>
struct Cut {
  static constexpr int R = R_, KT = KT_, SW = SW_, LEAST = LEAST_;
};
constexpr int kSharedMaxB = 4096;   // the schedule is formed in shared memory

struct SharedParams {
  const int32_t *block_table, *prefix_len, *tree_len, *cu, *group_start, *shared_pages;
  const uint64_t* mask;
  uint16_t* out;
  float* lse;
  float* ws_o;       // [2 * rows + 2 * ranges * R][D]: shared parts, own parts, cut pieces
  float* ws_lse;     // the same rows' log-sum-exp (log2 domain)
  int4* ws_desc;     // [2][rows]: first piece's row, pieces, second piece's row, rows from there to the next
  int32_t* dev_err;
  long long T;       // packed nodes
  const uint16_t* q;
  int B, N, Hq, Hkv, G, W, max_pages, num_pages, n_groups;
  int rows;          // (node, query head) rows
  int kinds;         // units of this launch: kShared, kOwn or both
  int ranges;        // of this launch
  int cut0;          // first workspace row of its cut pieces
  float scale_log2;
};
constexpr int kShared = 1, kOwn = 2;

// Time limit of the kernels' waits on their own pipeline, and the test hook that makes one run out (see
// jf_debug_set_wait_limit_ns): non-zero withholds what says that data or a piece is there.
__constant__ uint64_t c_wait_limit_ns = kWaitLimitNs;
__constant__ int c_withhold = 0;

// ------------------------------------------------------------------------ the schedule

// Keys that a group's sequences share, of its shared_pages entry: none when it has one sequence
// (nothing to share).  The block table alone bounds them: how many nodes follow is each
// sequence's own matter, and most have fewer than N.
__device__ __forceinline__ int group_keys(const SharedParams& p, int pages, int b0, int b1) {
  if (b1 - b0 < 2) return 0;
  return max(0, min(pages, p.max_pages)) * kPage;
}

// One unit: rows f0 .. f0 + nr - 1 of q's nodes attend to keys key0 .. L - 1 of block-table row
// bt, T tiles; mpc row-tile groups.  Keys below P are visible to every row.
struct Unit {
  int f0, nr, key0, P, L, T, mpc, bt;
};

template <typename X>
__device__ __forceinline__ void cut_unit(const SharedParams& p, Unit& t) {
  t.mpc = static_cast<int>((static_cast<long long>(t.nr) * p.G + X::R - 1) / X::R);
  t.T = t.nr > 0 ? (t.L - t.key0 + X::KT - 1) / X::KT : 0;
}
template <typename X>
__device__ __forceinline__ Unit shared_unit(const SharedParams& p, int b0, int b1, int S, const int32_t* cu) {
  Unit t;
  t.bt = b0;
  t.key0 = 0;
  t.P = t.L = S;
  if (p.cu == nullptr) {
    t.f0 = b0 * p.N;
    t.nr = (b1 - b0) * p.N;
  } else {
    const long long r0 = cu[b0], r1 = cu[b1];
    const bool ok = r0 >= 0 && r1 <= p.T && r1 >= r0;
    t.f0 = ok ? static_cast<int>(r0) : 0;
    t.nr = ok ? static_cast<int>(r1 - r0) : 0;
  }
  cut_unit<X>(p, t);
  return t;
}
template <typename X>
__device__ __forceinline__ Unit own_unit(const SharedParams& p, int b, int S, int prefix, int row0, int n) {
  Unit t;
  t.bt = b;
  // (A sequence whose nodes have no room behind S is malformed, its P < S or its keys past the table: it
  // starts where they do have room.)
  const int last = p.max_pages * kPage - n;
  t.key0 = min(S, last & -kPage);
  t.P = max(t.key0, min(prefix, last));
  t.L = t.P + n;
  t.f0 = row0;
  t.nr = n;
  cut_unit<X>(p, t);
  return t;
}

struct Schedule {
  int lo, hi;        // this range, in positions
  int q, rem;        // range v starts at v * q + min(v, rem)
  int tiles;         // key tiles in the range
  int u, b, off;     // the unit at lo (b < 0: shared) and lo's offset in it
  __device__ int range_of(int x) const {
    const int big = rem * (q + 1);
    return x < big ? x / (q + 1) : rem + (x - big) / q;
  }
};

// The ranges v0, v0 + vstep, .. (TEAMS of them) of the launch.  Every thread of the block calls it and
// then waits for the block; scratch: schedule_bytes().  Unit order: group by group, its shared part
// (if any), then its sequences.  Units of kinds that the launch does not do cost nothing.
constexpr int schedule_bytes(int B, int n_groups) { return 4 * (4 * n_groups + 5 * B + 4); }

template <typename X, int TEAMS>
__device__ __forceinline__ void make_schedule(const SharedParams& p, int v0, int vstep, int32_t* err, int* scratch,
                                              Schedule* out) {
  const int ng = p.n_groups, B = p.B, U = ng + B, tid = threadIdx.x, nth = blockDim.x;
  int* gs = scratch;                 // [ng + 1]
  int* sp = gs + ng + 1;             // [ng]
  int* pl = sp + ng;                 // [B] prefix lengths
  int* nn = pl + B;                  // [B] nodes, with kClamped where a span or length is malformed
  int* cost = nn + B;                // [U + 1] positions of the unit, then before it
  int* items = cost + U + 1;         // [U + 1]
  int* cs = items + U + 1;           // [B + 1] packed spans
  constexpr int kClamped = 1 << 30;
  __shared__ int s_scan[32];
  __shared__ int s_items[32];
  // (Nothing here is unrolled: it runs once, and what it costs is mostly the instructions' own trip
  // from memory and the barriers.)  One trip for all the data that the schedule depends on.
  bool bad = false, down = false;    // group_start is not a partition; cu descends
#pragma unroll 1
  for (int u = tid; u < ng; u += nth) {
    const int g0 = p.group_start[u], g1 = p.group_start[u + 1];
    gs[u] = g0;
    sp[u] = p.shared_pages[u];
    bad = bad || g0 > g1 || (u == 0 && g0 != 0) || (u == ng - 1 && g1 != B);
    if (u == ng - 1) gs[ng] = g1;
  }
#pragma unroll 1
  for (int b = tid; b < B; b += nth) {
    pl[b] = p.prefix_len[b];
    const SeqSpan span = seq_span(p.cu, p.tree_len, b, p.N, p.T);
    nn[b] = span.n | (span.ok ? 0 : kClamped);
    if (p.cu != nullptr) {
      const int r0 = p.cu[b], r1 = p.cu[b + 1];
      cs[b] = r0;
      if (b == B - 1) cs[B] = r1;
      down = down || r0 > r1;        // (spans that overlap could add up to more positions than 32 bits hold)
    }
  }
  if (tid < TEAMS) out[tid].tiles = out[tid].lo = out[tid].hi = 0;
  if (err != nullptr && (bad || down)) report(err, (bad ? JF_DEVERR_BAD_GROUP : 0) | (down ? JF_DEVERR_BAD_TREE_LEN : 0));
  if (__syncthreads_or(bad || down)) return;       // no work at all
  auto group_of = [&](int e) {       // of unit e: unit u + gs[u] is group u's shared part
    int u = 0, hi = ng;
#pragma unroll 1
    while (hi - u > 1) {
      const int mid = (u + hi) >> 1;
      if (mid + gs[mid] <= e) u = mid; else hi = mid;
    }
    return u;
  };
  const int cap = p.max_pages * kPage;
  // A thread's units are consecutive, so that sums run over threads.
  const int chunk = (U + nth - 1) / nth;
  const int e0 = min(U, tid * chunk), e1 = min(U, e0 + chunk);
  int mine = 0, mine_items = 0;      // positions are 32-bit (a limit of the call)
#pragma unroll 1
  for (int e = e0; e < e1; ++e) {
    const int u = group_of(e), b0 = gs[u], b1 = gs[u + 1];
    const int b = e - u - 1;
    const int S = group_keys(p, sp[u], b0, b1);
    const bool shared = e == u + b0;
    const int n_b = shared ? 0 : nn[b] & ~kClamped;
    if (err != nullptr) {
      int bits = 0;
      if (shared) {
        if (sp[u] < 0 || (b1 - b0 >= 2 && S / kPage != sp[u])) bits |= JF_DEVERR_BAD_GROUP;
      } else {
        if (nn[b] & kClamped) bits |= JF_DEVERR_BAD_TREE_LEN;
        if (pl[b] < S || pl[b] > cap - n_b) bits |= JF_DEVERR_BAD_PREFIX;
      }
      if (bits) report(err, bits);
    }
    int n = 0, c = 0;
    if (shared ? S > 0 && (p.kinds & kShared) : (p.kinds & kOwn) != 0) {
      const Unit t = shared ? shared_unit<X>(p, b0, b1, S, cs) : own_unit<X>(p, b, S, pl[b], 0, n_b);
      n = t.T == 0 ? 0 : p.Hkv * t.mpc;
      c = n * (t.T + X::SW);
    }
    cost[e] = c;
    items[e] = n;
    mine += c;
    mine_items += n;
  }
  // What lies before a thread's units: sums over its warp's lanes, then over the warps before it.
  int upto = mine, upto_items = mine_items;
  const int lane = tid & 31, warp = tid >> 5;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, upto, o);
    const int z = __shfl_up_sync(0xffffffffu, upto_items, o);
    if (lane >= o) upto += y, upto_items += z;
  }
  if (lane == 31) s_scan[warp] = upto, s_items[warp] = upto_items;
  __syncthreads();
  const int warps = (nth + 31) / 32;
  const int all = lane < warps ? s_scan[lane] : 0, all_items = lane < warps ? s_items[lane] : 0;
  const int total = __reduce_add_sync(0xffffffffu, all);
  const int total_items = __reduce_add_sync(0xffffffffu, all_items);
  int first = upto - mine + __reduce_add_sync(0xffffffffu, lane < warp ? all : 0);
  int first_items = upto_items - mine_items + __reduce_add_sync(0xffffffffu, lane < warp ? all_items : 0);
#pragma unroll 1
  for (int e = e0; e < e1; ++e) {
    const int c = cost[e], n = items[e];
    cost[e] = first;
    items[e] = first_items;
    first += c;
    first_items += n;
  }
  if (tid == 0) cost[U] = total, items[U] = total_items;
  __syncthreads();
  // Starts (even lanes) and ends of the teams' ranges: the unit that holds each, then the item.
  if (warp == 0) {
    const int used = max(1, min(p.ranges, total / X::LEAST));
    const int q = total / used, rem = total - q * used;
    const int k = min(lane, 2 * TEAMS - 1);
    const int v = min(v0 + (k >> 1) * vstep + (k & 1), used), x = v * q + min(v, rem);
    int before = total - X::SW * total_items;      // tiles before x: the position less SW per item completed
    int e = 0, off = 0;
    if (x < total) {
      int hi = U;                    // (units without positions share theirs with the next one that has some)
#pragma unroll 1
      while (hi - e > 1) {
        const int mid = (e + hi) >> 1;
        if (cost[mid] <= x) e = mid; else hi = mid;
      }
      off = x - cost[e];
      const int per = (cost[e + 1] - cost[e]) / (items[e + 1] - items[e]);     // T + SW
      const int item = off / per, in = off - item * per;
      before = x - X::SW * (items[e] + item) - max(0, in - (per - X::SW));
    }
    const int x1 = __shfl_down_sync(0xffffffffu, x, 1), before1 = __shfl_down_sync(0xffffffffu, before, 1);
    if (lane < 2 * TEAMS && (lane & 1) == 0) {
      const int u = group_of(e);
      Schedule& o = out[lane >> 1];
      o.u = u;
      o.b = e == u + gs[u] ? -1 : e - u - 1;
      o.off = off;
      o.lo = v < used ? x : total;
      o.hi = v < used ? x1 : total;
      o.q = q;
      o.rem = rem;
      o.tiles = o.lo < o.hi ? before1 - before : 0;
    }
  }
}

// One piece as the CTA's roles need it.  The producer, which runs ahead of the others, walks the
// range and posts its pieces in a ring in shared memory; s_posted counts them.
struct Piece {
  int T;                   // key tiles
  int first, P, L;         // the first key; keys below P are seen by every row, keys from L on by none
  int node0, nrows;        // first node, and rows from it on (the item's row tiles hold fewer or as many)
  int g, b;                // kv-head; sequence, -1 for a shared part
  int slots;               // workspace row of a cut item's row 0
  bool whole, direct, opens, alone;   // uncut; nothing to merge with; the item's first piece; no shared part
  int n, second;           // a cut item's pieces, and workspace row of row 0 of the second
};
// A piece's slot is written once the S MMAs of the last tile of the piece before it are done: every
// role has then left the pieces up to the third before it.
constexpr int kPieces = 4;
// A change of item costs the tcgen05 kernel some tiles' time: the next item's Q and K arrive, the rows leave TMEM.
// No one count is best for all: 16 trees of up to 64 nodes 3 129 us, 4 117, 5 118, 6 120, 8 124, 10 129; of up to 256
// 346, 320, 303, 302, 310, 313; 128 beams in two groups over 16K keys (own parts in the row kernel) 73.3, 75.8,
// 71.7, 71.5, 69.0, 68.8; 64 requests over 32K keys 82.3, 81.3, 79.6, 80.2, 78.7, 78.1.  6 is within 4% of each one's best.
constexpr int kTileSwitch = 6;
template <int NT>
using TileCut = Cut<NT * kRowTile, kKeyTile, kTileSwitch, 1>;

__device__ __forceinline__ void store_sector(float* p, const float (&y)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(y[0]), "f"(y[1]), "f"(y[2]),
               "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7])
               : "memory");
}

// What a piece leaves beside a row's output: its log-sum-exp and, from the item's first piece, where
// the row's pieces are (stride: workspace rows from the second piece to the third, and so on).
__device__ __forceinline__ void write_row_facts(const SharedParams& p, const Piece& c, int row, int prow, int r,
                                                float lse2, int stride) {
  if (c.direct) {
    if (p.lse != nullptr) {
      const int node = row / p.Hq, h = row - node * p.Hq;
      p.lse[p.cu != nullptr ? static_cast<size_t>(h * p.T + node)
                            : (static_cast<size_t>(c.b) * p.Hq + h) * p.N + (node - c.b * p.N)] =
          lse2 * 0.69314718055994531f;
    }
  } else {
    p.ws_lse[prow] = lse2;
  }
  if (c.opens) {
    p.ws_desc[(c.b < 0 ? 0 : p.rows) + row] = make_int4(prow, c.n, c.second + r, stride);
    if (c.alone) p.ws_desc[row] = make_int4(0, 0, 0, 0);
  }
}

// The pieces of a range, one after the other.
template <typename X>
struct Walk {
  const SharedParams& p;
  int lo, hi;
  int u, b, b0, b1, S;     // group, sequence (-1: shared part), the group's sequences, shared keys
  int g, mp, x;            // kv-head, row-tile group, the item's position
  int k0, k1;              // the piece: key tiles k0 .. k1 - 1 of the item
  Unit t;

  __device__ __forceinline__ Walk(const SharedParams& p_, const Schedule& s) : p(p_), lo(s.lo), hi(s.hi) {
    u = s.u;
    b = s.b;
    b0 = p.group_start[u];
    b1 = p.group_start[u + 1];
    S = group_keys(p, p.shared_pages[u], b0, b1);
    load_unit();
    const int per = t.T + X::SW, item = s.off / per;
    g = item / t.mpc;
    mp = item - g * t.mpc;
    x = lo - (s.off - item * per);
    settle(false);
  }
  __device__ __forceinline__ bool live() const { return x < hi; }
  __device__ __forceinline__ void next() { settle(true); }
  __device__ __forceinline__ Piece piece(const Schedule& s, int v) const {
    constexpr int R = X::R;
    Piece c;
    c.T = k1 - k0;
    c.first = t.key0 + k0 * X::KT;
    c.P = t.P;
    c.L = t.L;
    c.node0 = t.f0 + mp * R / p.G;
    c.nrows = t.nr * p.G - mp * R;
    c.g = g;
    c.b = b;
    c.whole = k0 == 0 && k1 == t.T;
    c.alone = b >= 0 && S == 0;
    c.direct = c.whole && c.alone;
    c.opens = k0 == 0;
    const int slot = x + k0 == lo ? 0 : 1;
    c.slots = p.cut0 + (2 * v + slot) * R;
    c.n = c.direct ? 0 : 1;
    c.second = 0;
    if (!c.whole && c.opens) {
      const int va = s.range_of(x), vb = s.range_of(x + t.T - 1);
      c.n = vb - va + 1;
      c.second = p.cut0 + 2 * (va + 1) * R;
    }
    return c;
  }

 private:
  // The first piece at or after the current item, or after it (a range may start or end in an item's
  // switch).
  __device__ __forceinline__ void settle(bool move) {
    for (;; move = true) {
      if (move) {
        x += t.T + X::SW;
        if (++mp >= t.mpc) {
          mp = 0;
          if (++g >= p.Hkv) {
            g = 0;
            if (x < hi) next_unit();
          }
        }
      }
      if (x >= hi) return;
      k0 = max(lo - x, 0);
      k1 = min(hi - x, t.T);
      if (k0 < k1) return;
    }
  }
  __device__ __forceinline__ void next_unit() {
    do {
      b = b < 0 ? b0 : b + 1;
      if (!(p.kinds & kOwn)) b = b1;     // shared parts alone: on to the next group
      while (b >= b1) {
        if (++u >= p.n_groups) {
          x = INT_MAX;
          return;
        }
        b0 = b1;
        b1 = p.group_start[u + 1];
        S = group_keys(p, p.shared_pages[u], b0, b1);
        b = S > 0 && (p.kinds & kShared) ? -1 : ((p.kinds & kOwn) ? b0 : b1);
      }
      load_unit();
    } while (t.T == 0);
  }
  __device__ __forceinline__ void load_unit() {
    if (b < 0) {
      t = shared_unit<X>(p, b0, b1, S, p.cu);
    } else {
      const int prefix = p.prefix_len[b];
      const SeqSpan sp = seq_span(p.cu, p.tree_len, b, p.N, p.T);
      t = own_unit<X>(p, b, S, prefix, static_cast<int>(sp.row0), sp.n);
    }
  }
};

__device__ __forceinline__ void shared_count_add(int* c) {
  asm volatile("red.release.cta.shared::cta.add.s32 [%0], 1;" ::"r"(smem_u32(c)) : "memory");
}
__device__ __forceinline__ int shared_count(int* c) {
  int v;
  asm volatile("ld.acquire.cta.shared::cta.s32 %0, [%1];" : "=r"(v) : "r"(smem_u32(c)) : "memory");
  return v;
}
__device__ __forceinline__ bool wait_shared_count(int* c, int target, volatile int* abort, uint64_t wlim) {
  if (shared_count(c) > target) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (shared_count(c) > target) return true;
    if ((it & 255u) == 0u && (*abort || global_timer_ns() - t0 > wlim)) return false;
  }
}

// ------------------------------------------------------------------------ the parts

template <int NT, int D>
__global__ void __launch_bounds__(Cfg<NT, D>::kThreads, 1)
    shared_attention_kernel(const __grid_constant__ CUtensorMap qmap,
                            const __grid_constant__ CUtensorMap kmap,
                            const __grid_constant__ CUtensorMap vmap,
                            const __grid_constant__ CUtensorMap kmap_run,
                            const __grid_constant__ CUtensorMap vmap_run,
                            const __grid_constant__ SharedParams p) {
  using C = Cfg<NT, D>;
  constexpr int SK = C::kKStages;
  constexpr int SV = C::kVStages;
  const uint64_t wlim = c_wait_limit_ns;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  __shared__ uint64_t q_full, o_full, fin;
  __shared__ uint64_t k_full[SK], v_full[SV], step_done[kStepRing];
  __shared__ uint64_t s_full[NT], p_full[NT];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ Piece s_piece[kPieces];
  __shared__ int s_posted;                   // pieces posted
  __shared__ int s_tails;                    // pieces whose V tail is ready
  __shared__ int s_lo[NT];                   // current key tile of row tile t stores P in two parts
  __shared__ Schedule s_sch;
  volatile int* abort = &abort_flag;
  uint8_t* q_s = sm + C::kQOff;
  uint8_t* k_s = sm + C::kKOff;
  uint8_t* v_s = sm + C::kVOff;
  const int v = blockIdx.x;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(&q_full, 1);
    mbar_init(&o_full, 1);
    mbar_init(&fin, 1);
    for (int st = 0; st < SK; ++st) mbar_init(&k_full[st], 1);
    for (int st = 0; st < SV; ++st) mbar_init(&v_full[st], 1);
    for (int st = 0; st < kStepRing; ++st) mbar_init(&step_done[st], 1);
    for (int t = 0; t < NT; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], 128 + 1);   // the softmax warpgroup + its data voucher
    }
    s_posted = 0;
    s_tails = 0;
    abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&qmap);
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
    tma_prefetch_desc(&kmap_run);
    tma_prefetch_desc(&vmap_run);
  }
  grid_dependency_wait();
  grid_dependents_launch();             // whatever follows waits for all of this one before it reads or writes
  make_schedule<TileCut<NT>, 1>(p, v, 1, v == 0 ? p.dev_err : nullptr, reinterpret_cast<int*>(sm), &s_sch);
  fence_proxy_async_smem();             // the scratch becomes the target of TMA copies
  if (warp == 1) {
    tmem_alloc(&tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const int Wc = s_sch.tiles;
  if (Wc <= 0) {                        // fewer tiles than ranges (or nothing to do)
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
    return;
  }

  if (warp < 4) {
  if constexpr (NT == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
  if (warp == 0) {
    // ================================================================ TMA producer
    constexpr int kLookahead = 4;
    int k_issued = 0, v_issued = 0, q_issued = 0, bad = 0;
    bool ok = true;
    auto issue = [&](uint8_t* ring, const CUtensorMap* map, const CUtensorMap* map_run,
                     uint64_t* full, int st, int page, int page0, int g, bool run) {
      if (run) {
        if (lane < C::kHalves)
          tma_load_3d(ring + st * C::kTileBytes + lane * C::kHalfBytes, map_run, full, lane * 64, g,
                      page0 * kPage);
      } else if (lane < kPagesPerTile * C::kHalves) {
        const int q = lane % kPagesPerTile, hh = lane / kPagesPerTile;
        tma_load_3d(ring + st * C::kTileBytes + hh * C::kHalfBytes + q * (kPage * 128), map, full,
                    hh * 64, g, page * kPage);
      }
    };
    int jg0 = 0;
    Walk<TileCut<NT>> w(p, s_sch);
    for (int s = 0; w.live() && ok; ++s, w.next()) {
      const int T = w.k1 - w.k0, L = w.t.L;
      const int page0_of = w.t.key0 / kPage + w.k0 * kPagesPerTile;     // the piece's first page
      const int32_t* bt = p.block_table + static_cast<size_t>(w.t.bt) * p.max_pages;
      // this piece's Q, once the previous piece's S MMAs no longer read the buffer
      int okq = 1;
      if (lane == 0) {
        const int rq = jg0 - 1;   // S of the previous piece's last tile: step record rq
        if (s > 0 && !mbar_wait(&step_done[rq % kStepRing], static_cast<uint32_t>(rq / kStepRing) & 1u,
                                abort, wlim)) {
          okq = 0;
        } else {
          s_piece[s % kPieces] = w.piece(s_sch, v);
          shared_count_add(&s_posted);
          mbar_arrive_expect_tx(&q_full, NT * C::kTileBytes);
          for (int t = 0; t < NT; ++t) {
            const int node0 = w.t.f0 + ((w.mp * NT + t) * kRowTile) / p.G;
            for (int hh = 0; hh < C::kHalves; ++hh)
              tma_load_3d(q_s + t * C::kTileBytes + hh * C::kHalfBytes, &qmap, &q_full, hh * 64,
                          w.g * p.G, node0);
          }
        }
      }
      if (!__shfl_sync(0xffffffffu, okq, 0)) { ok = false; break; }
      q_issued = s + 1;
      auto load_pid = [&](int j) -> int {
        const int pl = page0_of + j * kPagesPerTile + lane;
        if (lane >= kPagesPerTile || j >= T || pl * kPage >= L) return p.num_pages;
        return __ldg(bt + pl);
      };
      int pid[kLookahead];
#pragma unroll
      for (int u = 0; u < kLookahead; ++u) pid[u] = load_pid(u);
      for (int j = 0; j < T; ++j) {
        const int jg = jg0 + j;
        int mine = pid[0];
        if (mine < 0 || mine > p.num_pages) { bad = 1; mine = p.num_pages; }
        else if (mine == p.num_pages && lane < kPagesPerTile &&
                 (page0_of + j * kPagesPerTile + lane) * kPage < L) bad = 1;
        const int page = __shfl_sync(0xffffffffu, mine, lane % kPagesPerTile);
        const int page0 = __shfl_sync(0xffffffffu, mine, 0);
        const bool run = __all_sync(0xffffffffu, page == page0 + lane % kPagesPerTile);
#pragma unroll
        for (int u = 0; u < kLookahead - 1; ++u) pid[u] = pid[u + 1];
        pid[kLookahead - 1] = load_pid(j + kLookahead);
        const int sk = jg % SK, sv = jg % SV;
        const int rec = jg - C::kStageLag;
        int okl = 1;
        if (lane == 0) {
          if (rec >= 0 && !mbar_wait(&step_done[rec % kStepRing],
                                     static_cast<uint32_t>(rec / kStepRing) & 1u, abort, wlim)) {
            okl = 0;
          } else {
            mbar_arrive_expect_tx(&k_full[sk], C::kTileBytes);
            mbar_arrive_expect_tx(&v_full[sv], C::kTileBytes);
          }
        }
        if (!__shfl_sync(0xffffffffu, okl, 0)) { ok = false; break; }
        issue(k_s, &kmap, &kmap_run, &k_full[sk], sk, page, page0, w.g, run);
        k_issued = jg + 1;
        issue(v_s, &vmap, &vmap_run, &v_full[sv], sv, page, page0, w.g, run);
        v_issued = jg + 1;
      }
      if (!ok) break;
      // V rows past the part's end in its last tile meet a zero probability: make them zero,
      // then release the tile to the MMA issuer's voucher (every piece).
      const int jl = jg0 + T - 1;
      const int last_key0 = w.t.key0 + (w.k1 - 1) * kKeyTile;
      if (last_key0 + kKeyTile > L) {
        if (!wait_warp(&v_full[jl % SV], static_cast<uint32_t>(jl / SV) & 1u, abort, wlim)) { ok = false; break; }
        const int r0 = L - last_key0;
        uint8_t* vt = v_s + (jl % SV) * C::kTileBytes;
        const int per_half = (-r0 & (kPage - 1)) * 8;     // to the page's end: later pages came as zeros
        for (int c = lane; c < per_half * C::kHalves; c += 32) {
          const int hh = c / per_half, rem = c % per_half;
          *reinterpret_cast<uint4*>(vt + hh * C::kHalfBytes + (r0 + rem / 8) * 128 + (rem % 8) * 16) =
              make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (lane == 0) shared_count_add(&s_tails);
      jg0 += T;
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) report(p.dev_err, JF_DEVERR_BAD_PAGE);
    if (!ok && lane == 0) set_abort(abort, p.dev_err);
    __syncwarp();
    if (lane == 0) {                   // no copy may still be landing when the CTA exits
      int zero = 0;
      if (q_issued > 0) mbar_wait(&q_full, static_cast<uint32_t>(q_issued - 1) & 1u, &zero);
      for (int j = max(0, k_issued - SK); j < k_issued; ++j)
        mbar_wait(&k_full[j % SK], static_cast<uint32_t>(j / SK) & 1u, &zero);
      for (int j = max(0, v_issued - SV); j < v_issued; ++j)
        mbar_wait(&v_full[j % SV], static_cast<uint32_t>(j / SV) & 1u, &zero);
    }
  } else if (warp == 1) {
    // ================================================================ MMA issuer
    constexpr uint32_t idS = idesc_bf16(kRowTile, kKeyTile, false, false);
    constexpr uint32_t idO = idesc_bf16(kRowTile, D, false, true);
    const uint64_t dq = desc_sw128(smem_u32(q_s), 16, 1024);
    const uint64_t dk = desc_sw128(smem_u32(k_s), 16, 1024);
    const uint64_t dv = desc_sw128(smem_u32(v_s), C::kHalfBytes, 1024);
    auto issue_s = [&](int t, int st) {
      const uint64_t da = dq + static_cast<uint64_t>((t * C::kTileBytes) >> 4);
      const uint64_t db = dk + static_cast<uint64_t>((st * C::kTileBytes) >> 4);
      const uint32_t d_tmem = tmem + C::kTmemS + t * 128;
      mma_ss_tile<D / 16>(d_tmem, da, db, idS);
    };
    auto issue_pv = [&](int t, int st, bool acc, bool lo) {
      const uint64_t db = dv + static_cast<uint64_t>((st * C::kTileBytes) >> 4);
      const uint32_t d_tmem = tmem + C::kTmemO + t * 128;
      const uint32_t a_tmem = tmem + C::kTmemS + t * 128;
      mma_ts_tile(d_tmem, a_tmem, db, idO, acc);
      if (lo) issue_pv_lo(d_tmem, a_tmem, db, idO);
    };
    bool ok = wait_warp(&q_full, 0, abort, wlim) && wait_warp(&k_full[0], 0, abort, wlim);
    if (ok) {
      // The whole warp runs this loop; the MMA and commit wrappers issue from one elected lane.
      tc_fence_after();
      for (int t = 0; t < NT; ++t) {
        issue_s(t, 0);
        mma_commit(&s_full[t]);
      }
      mma_commit(&step_done[0]);
      int jn[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) jn[t] = 0;
      int left = NT * Wc;
      uint32_t idle = 0;
      uint64_t idle_since = 0;
      while (left > 0) {
        bool progressed = false;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const int j = jn[t];
          if (j >= Wc) continue;
          if (__shfl_sync(0xffffffffu, mbar_try_wait(&p_full[t], static_cast<uint32_t>(j) & 1u) ? 1 : 0, 0) == 0)
            continue;
          bool last = true;
#pragma unroll
          for (int u = 0; u < NT; ++u)
            if (u != t && jn[u] <= j) last = false;
          tc_fence_after();
          // s_lo[t] was written before the softmax's arrival on p_full[t]: lane 0 reads it
          const bool lo = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&s_lo[t]), 0) != 0;
          issue_pv(t, j % SV, j > 0, lo);
          if (j + 1 < Wc) {
            issue_s(t, (j + 1) % SK);
            mma_commit(&s_full[t]);
          }
          if (last) mma_commit(&step_done[(j + 1) % kStepRing]);
          jn[t] = j + 1;
          --left;
          progressed = true;
        }
        if (progressed) {
          idle = 0;
        } else {
          if (idle == 0) idle_since = global_timer_ns();
          if ((++idle & 255u) == 0u &&
              __shfl_sync(0xffffffffu, (*abort || global_timer_ns() - idle_since > wlim) ? 1 : 0, 0) != 0) {
            ok = false;
            break;
          }
        }
      }
    }
    if (!ok && lane == 0) set_abort(abort, p.dev_err);
    if (ok) mma_commit(&o_full);   // the range's last PV
    mma_commit(&fin);   // all MMAs done before TMEM is released
    {
      int zero = 0;
      wait_warp(&fin, 0, &zero, kWaitLimitNs);
    }
  } else if (warp >= 2 && warp < 2 + NT) {
    // ================================================================ data vouchers
    // The last arrival on p_full[t] for tile j: V tile j and K tile j + 1 have landed and, at a
    // piece's last tile, its V tail and the next piece's Q.
    const int t = warp - 2;
    if (lane == 0 && c_withhold == 0) {
      bool ready = wait_shared_count(&s_posted, 0, abort, wlim);
      int s = 0, e = ready ? s_piece[0].T : 0;
      for (int j = 0; j < Wc && ready; ++j) {
        const bool last_of_piece = j + 1 == e;
        ready = (j == 0 || mbar_wait(&p_full[t], static_cast<uint32_t>(j - 1) & 1u, abort, wlim)) &&
                mbar_wait(&v_full[j % SV], static_cast<uint32_t>(j / SV) & 1u, abort, wlim) &&
                (j + 1 >= Wc ||
                 mbar_wait(&k_full[(j + 1) % SK], static_cast<uint32_t>((j + 1) / SK) & 1u, abort, wlim)) &&
                (!last_of_piece || wait_shared_count(&s_tails, s, abort, wlim)) &&
                (!last_of_piece || j + 1 >= Wc ||
                 mbar_wait(&q_full, static_cast<uint32_t>(s + 1) & 1u, abort, wlim));
        if (!ready) break;
        mbar_arrive(&p_full[t]);
        if (last_of_piece && j + 1 < Wc) {
          ++s;
          ready = wait_shared_count(&s_posted, s, abort, wlim);
          if (ready) e += *reinterpret_cast<volatile int*>(&s_piece[s % kPieces].T);
        }
      }
      if (!ready) set_abort(abort, p.dev_err);
    }
    __syncwarp();
  }
  } else {
    if constexpr (NT == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    // ================================================================ softmax / epilogue
    const int t = (warp >> 2) - 1;
    const int wq = warp & 3;
    const int rl = wq * 32 + lane;                       // row within the tile = TMEM lane
    const int W = p.W;
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem + C::kTmemS + t * 128 + lane_off;
    const uint32_t tO = tmem + C::kTmemO + t * 128 + lane_off;
    const float sl2 = p.scale_log2;
    bool ok = true;
    int jg0 = 0;
    for (int s = 0; jg0 < Wc && ok; ++s) {
      int posted = 1;
      if (lane == 0) posted = wait_shared_count(&s_posted, s, abort, wlim) ? 1 : 0;
      posted = __shfl_sync(0xffffffffu, posted, 0);      // and what the lane acquired is the warp's
      __syncwarp();
      // (The piece is read where it is needed: registers belong to the scores.)
      const volatile Piece& c = s_piece[s % kPieces];
      const int T = posted ? c.T : 0;
      const int r = t * kRowTile + rl;                   // row of the item
      float m_run = -INFINITY;
      float l = 0.f;
      ok = posted != 0;
      {
        const int P = c.P, L = c.L, first = c.first;
        const bool valid = r < c.nrows, tree = valid && c.b >= 0;
        const uint64_t* mrow = p.mask + (static_cast<size_t>(c.node0) + (valid ? r / p.G : 0)) * W;
        // Key tiles before jm hold keys that every row sees and nothing else.
        const int jm = min(max((P - first) / kKeyTile, 0), T);
        volatile int* lo_flag = &s_lo[t];
        for (int j = 0; j < jm && ok; ++j)
          ok = softmax_tile<false, false, D>(&s_full[t], static_cast<uint32_t>(jg0 + j) & 1u, abort, &p_full[t],
                                             tS, tO, mrow, tree, W, first + j * kKeyTile, P, L, sl2, j > 0,
                                             lo_flag, rl == 0, m_run, l, wlim);
        // Rows with fewer than kSplitPrefix keys that all of them see: P in two bf16 parts.  (A
        // shared part has no tree keys: its ancestor words are not read.)
        if (P < kSplitPrefix) {
          for (int j = jm; j < T && ok; ++j)
            ok = softmax_tile<true, true, D>(&s_full[t], static_cast<uint32_t>(jg0 + j) & 1u, abort,
                                             &p_full[t], tS, tO, mrow, tree, W, first + j * kKeyTile,
                                             P, L, sl2, j > 0, lo_flag, rl == 0, m_run, l, wlim);
        } else {
          for (int j = jm; j < T && ok; ++j)
            ok = softmax_tile<true, false, D>(&s_full[t], static_cast<uint32_t>(jg0 + j) & 1u, abort,
                                              &p_full[t], tS, tO, mrow, tree, W, first + j * kKeyTile,
                                              P, L, sl2, j > 0, lo_flag, rl == 0, m_run, l, wlim);
        }
      }
      // A failed wait still reaches the warpgroup vote below (every warp must enter it).
      if (!ok && lane == 0) set_abort(abort, p.dev_err);
      // ---- the piece's rows, once its last PV is done: S of the next tile (committed after it)
      // or, for the range's last piece, o_full.
      const int je = jg0 + T;
      const bool pv_done = ok && (je < Wc ? wait_warp(&s_full[t], static_cast<uint32_t>(je) & 1u, abort, wlim)
                                          : wait_warp(&o_full, 0u, abort, wlim));
      if (!named_bar_and(1 + t, 128, pv_done)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const float lse2 = l == 0.f ? -INFINITY : m_run + __log2f(l);
      const bool valid = r < c.nrows, direct = c.direct;
      const int row = (c.node0 + (valid ? r / p.G : 0)) * p.Hq + c.g * p.G + r % p.G;    // (node, head)
      const int prow = c.whole ? (c.b < 0 ? 0 : p.rows) + row : c.slots + r;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        uint32_t o[32];
        tmem_ld32(tO + k * 32, o);
        tmem_ld_wait(o);
        if (!valid) continue;
        if (direct) {
          uint4* dst = reinterpret_cast<uint4*>(p.out + static_cast<size_t>(row) * D + k * 32);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint4 y;
            y.x = pack_bf16x2(__uint_as_float(o[8 * q + 0]) * inv, __uint_as_float(o[8 * q + 1]) * inv);
            y.y = pack_bf16x2(__uint_as_float(o[8 * q + 2]) * inv, __uint_as_float(o[8 * q + 3]) * inv);
            y.z = pack_bf16x2(__uint_as_float(o[8 * q + 4]) * inv, __uint_as_float(o[8 * q + 5]) * inv);
            y.w = pack_bf16x2(__uint_as_float(o[8 * q + 6]) * inv, __uint_as_float(o[8 * q + 7]) * inv);
            dst[q] = y;
          }
        } else {
          // A lane's row is its own, so a store instruction touches 32 lines whatever its width: the
          // widest one, a whole sector a lane.
          float* dst = p.ws_o + static_cast<size_t>(prow) * D + k * 32;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = __uint_as_float(o[8 * q + e]) * inv;
            store_sector(dst + 8 * q, y);
          }
        }
      }
      if (valid) write_row_facts(p, const_cast<const Piece&>(s_piece[s % kPieces]), row, prow, r, lse2, 2 * NT * kRowTile);
      if (je < Wc) {                   // the next piece's first PV accumulates onto zero
        uint32_t z[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) z[e] = 0u;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) tmem_st32(tO + c * 32, z);
      }
      jg0 += T;
    }
    if (!ok) set_abort(abort, p.dev_err);
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
  grid_dependents_launch();
}

// ------------------------------------------------------------------------ few rows

// Units of few rows (a decode step's G rows of a sequence, the beams of a prompt) are bound by the K/V
// stream and by the latency of an item, not by matrix products.  A team of MT warps, 16 rows each,
// takes a range of its own; a producer warp per team walks the range ahead of it, through item
// changes too, and keeps a ring of key pages (K and V of 16 keys, by TMA) in flight: 24 pages of
// 8 KB per SM at D = 128, some 190 KB, where the HBM rate needs about 40.
//   Scores: m16n8k16 products.  A thread's 16-byte chunks 2 (lane % 4) + {0, 1} of a K row (key lane / 4 of
//   eight) are two k-steps' B fragments if Q's chunks are cut the same way: the order of the
//   contraction is free.  (Under the 128-byte swizzle the eight lanes of a phase then hit all banks; with
//   chunks lane % 4 + 4 i two rows collide, 186 us for four groups of 64 rows over 32K keys against 181.)
//   Output: V's fragments come transposed from shared memory (ldmatrix), two n-tiles at a time.
// Its time is the latency of a page's chain (products, maximum, exponentials, products) at two warps a
// scheduler: issue slots 43% busy, HBM 69%.  Two pages a step (103 us for 256 beams), four accumulators for the
// scores (93) and V's fragments kept for the second product (92) gained nothing on the 91 us of the time.
// A change of item, in pages: what it costs is the same for both head dimensions, a page at D = 64 half
// (256 beams in 32 groups, D = 128: 2 95.3 us, 3 86.8, 4 89.0, 8 98.1, in 16 groups 107, 106, 111, 130; D = 64: 3 72.5,
// 4 66.9, 5 63.6, in 16 groups 76.5, 72.8, 75.5).
template <int D>
constexpr int kRowSwitch = D == 128 ? 3 : 4;
constexpr int kRowLeast = 4;            // pages (4 beams over 2K keys: 1 15.3 us, 2 13.2, 4 12.8, 8 15.3)
constexpr int kRowWarps = 8;            // and as many producer warps, of which one per team works
template <int D, int MT>
using RowCut = Cut<16 * MT, kPage, kRowSwitch<D>, kRowLeast>;

template <int D, int MT>
struct RowCfg {
  static constexpr int kTeams = kRowWarps / MT;
  static constexpr int kHalves = D / 64;                      // 128-byte swizzle atoms per row
  static constexpr int kHalfBytes = kPage * 128;              // one 64-column half of a page
  static constexpr int kStageBytes = 2 * kHalves * kHalfBytes;     // K, then V
  static constexpr int kStages = 24 * 8192 / kStageBytes / kTeams;
  static constexpr int kPosts = 32;                           // piece slots: kStages + 2 at least
  static_assert(kPosts >= kStages + 2, "a piece is read until its last step's successor ring is full");
  static constexpr int kSmemBytes = kTeams * kStages * kStageBytes + 1024;
};

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr)
               : "memory");
}

template <int D, int MT>
__global__ void __launch_bounds__(64 * kRowWarps, 1)
    shared_rows_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                       const __grid_constant__ SharedParams p) {
  using X = RowCut<D, MT>;
  using C = RowCfg<D, MT>;
  constexpr int kTeams = C::kTeams, kS = C::kStages;
  constexpr int kI = D / 32;            // 16-byte chunks of a row per thread (scores)
  constexpr int kH = C::kHalves;
  const uint64_t wlim = c_wait_limit_ns;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  __shared__ Schedule s_sch[kTeams];
  __shared__ Piece s_post[kTeams][C::kPosts];
  __shared__ uint64_t s_full[kTeams][kS], s_empty[kTeams][kS];
  __shared__ int s_posted[kTeams];
  __shared__ int abort_flag;
  volatile int* abort = &abort_flag;
  if (threadIdx.x == 0) {
    for (int t = 0; t < kTeams; ++t) {
      for (int st = 0; st < kS; ++st) {
        mbar_init(&s_full[t][st], 1);
        mbar_init(&s_empty[t][st], MT);
      }
      s_posted[t] = c_withhold == 0 ? 0 : INT_MIN / 2;      // (withheld: no piece is ever there)
    }
    abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  grid_dependency_wait();               // (of own parts alone too: behind the shared parts' kernel)
  grid_dependents_launch();
  // (Consecutive ranges lie on different SMs: small calls reach them all.)
  make_schedule<X, kTeams>(p, blockIdx.x, gridDim.x, blockIdx.x == 0 && p.kinds == (kShared | kOwn) ? p.dev_err : nullptr,
                           reinterpret_cast<int*>(sm), s_sch);
  fence_proxy_async_smem();             // the scratch becomes the target of TMA copies
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // 512 threads x 128 registers at launch: 56 * 256 + 200 * 256 = 128 * 512.
  if (warp >= kRowWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    // ================================================================ producers
    const int team = warp - kRowWarps;
    if (team < kTeams && s_sch[team].tiles > 0) {
      const Schedule& sch = s_sch[team];
      uint8_t* ring = sm + team * kS * C::kStageBytes;
      int it = 0, posted = 0, bad = 0;
      bool ok = true;
      auto free_stage = [&] {           // lane 0: the stage of step `it` has been read by the whole team
        return it < kS || mbar_wait(&s_empty[team][it % kS], static_cast<uint32_t>(it / kS - 1) & 1u, abort, wlim);
      };
      for (Walk<X> w(p, sch); w.live() && ok; w.next()) {
        const int first = w.t.key0 + w.k0 * X::KT, end = min(w.t.L, w.t.key0 + w.k1 * X::KT);
        const int steps = (end - first + kPage - 1) / kPage;
        const int32_t* bt = p.block_table + static_cast<size_t>(w.t.bt) * p.max_pages + first / kPage;
        int ids = p.num_pages;          // lane l: the page of step 32 * k + l
        if (lane < steps) ids = __ldg(bt + lane);
        if (lane == 0) {                // its rows' Q can be read while its first page is under way
          s_post[team][posted % C::kPosts] = w.piece(sch, blockIdx.x + team * gridDim.x);
          shared_count_add(&s_posted[team]);
        }
        for (int s = 0; s < steps; ++s) {
          if ((s & 31) == 0 && s + lane < steps) {
            if (s > 0) ids = __ldg(bt + s + lane);
            if (ids < 0 || ids >= p.num_pages) {
              ids = p.num_pages;        // out of bounds: TMA fills zeros
              bad = 1;
            }
          }
          const int page = __shfl_sync(0xffffffffu, ids, s & 31);
          int go = 1;
          if (lane == 0) {
            go = free_stage() ? 1 : 0;
            if (go) mbar_arrive_expect_tx(&s_full[team][it % kS], C::kStageBytes);
          }
          if (!__shfl_sync(0xffffffffu, go, 0)) {
            ok = false;
            break;
          }
          if (lane < 2 * kH) {          // K halves, then V halves
            const int h = lane % kH;
            tma_load_3d(ring + (it % kS) * C::kStageBytes + lane * C::kHalfBytes, lane < kH ? &kmap : &vmap,
                        &s_full[team][it % kS], h * 64, w.g, page * kPage);
          }
          ++it;
        }
        ++posted;
      }
      if (__any_sync(0xffffffffu, bad) && lane == 0) report(p.dev_err, JF_DEVERR_BAD_PAGE);
      if (lane == 0) {
        s_post[team][posted % C::kPosts].T = 0;          // the end
        shared_count_add(&s_posted[team]);
        int zero = 0;                   // no copy may still be landing when the block exits
        for (int j = max(0, it - kS); j < it; ++j)
          ok = mbar_wait(&s_full[team][j % kS], static_cast<uint32_t>(j / kS) & 1u, &zero) && ok;
        if (!ok) set_abort(abort, p.dev_err);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    // ================================================================ the teams
    const int team = warp / MT, tw = warp % MT;
    const int q4 = lane & 3, r8 = lane >> 2;
    const uint8_t* ring = sm + team * kS * C::kStageBytes;
    bool ok = s_sch[team].tiles > 0;
    int st = 0;                          // the ring's next stage, and the phase of its barrier
    uint32_t phase = 0;
    for (int post = 0; ok; ++post) {
      int there = 1;
      if (lane == 0) there = wait_shared_count(&s_posted[team], post, abort, wlim) ? 1 : 0;
      there = __shfl_sync(0xffffffffu, there, 0);
      __syncwarp();                     // what the lane acquired is the warp's
      if (!there) {
        ok = false;
        break;
      }
      const Piece& c = s_post[team][post % C::kPosts];
      const int T = c.T;
      if (T == 0) break;
      const int first = c.first, P = c.P, end = min(c.L, first + T * X::KT);
      const int steps = (end - first + kPage - 1) / kPage;
      const int ra = tw * 16 + r8, rb = ra + 8;      // the thread's rows of the item
      const bool va = ra < c.nrows, vb = rb < c.nrows, some = tw * 16 < c.nrows;
      const int na = c.node0 + (va ? ra / p.G : 0), nb = c.node0 + (vb ? rb / p.G : 0);
      uint4 qa[kI], qb[kI];
#pragma unroll
      for (int i = 0; i < kI; ++i) {
        const int ch = 2 * q4 + (i & 1) + 8 * (i >> 1);
        const size_t rowa = static_cast<size_t>(na) * p.Hq + c.g * p.G + ra % p.G;
        const size_t rowb = static_cast<size_t>(nb) * p.Hq + c.g * p.G + rb % p.G;
        qa[i] = va ? reinterpret_cast<const uint4*>(p.q + rowa * D)[ch] : make_uint4(0u, 0u, 0u, 0u);
        qb[i] = vb ? reinterpret_cast<const uint4*>(p.q + rowb * D)[ch] : make_uint4(0u, 0u, 0u, 0u);
      }
      // Probabilities in two bf16 parts: for rows with few keys (see jf_attention.cuh), and in one-warp
      // teams, where the K/V stream leaves time for it, always: rounding them to bf16 alone costs the
      // output as much precision as its own rounding.
      const bool split = MT == 1 || P < kSplitPrefix;
      float o[8 * kH][4];
#pragma unroll
      for (int j = 0; j < 8 * kH; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
      float ma = -INFINITY, mb = -INFINITY, la = 0.f, lb = 0.f;
      for (int s = 0; s < steps; ++s) {
        if (!wait_lanes(&s_full[team][st], phase, abort, wlim)) {
          ok = false;
          break;
        }
        const uint8_t* kt = ring + st * C::kStageBytes;
        const uint8_t* vt = kt + kH * C::kHalfBytes;
        const int key0 = first + s * kPage;
        if (some) {                                  // warp-uniform
          float x[2][4];
#pragma unroll
          for (int t = 0; t < 2; ++t) x[t][0] = x[t][1] = x[t][2] = x[t][3] = 0.f;
#pragma unroll
          for (int i = 0; i < kI; ++i) {
            const int ch = 2 * q4 + (i & 1) + 8 * (i >> 1);
            uint4 kr[2];
#pragma unroll
            for (int t = 0; t < 2; ++t)
              kr[t] = *reinterpret_cast<const uint4*>(kt + (ch >> 3) * C::kHalfBytes + (8 * t + r8) * 128 +
                                                      (((ch & 7) ^ r8) << 4));
            mma_16816(x[0], qa[i].x, qb[i].x, qa[i].y, qb[i].y, kr[0].x, kr[0].y);
            mma_16816(x[1], qa[i].x, qb[i].x, qa[i].y, qb[i].y, kr[1].x, kr[1].y);
            mma_16816(x[0], qa[i].z, qb[i].z, qa[i].w, qb[i].w, kr[0].z, kr[0].w);
            mma_16816(x[1], qa[i].z, qb[i].z, qa[i].w, qb[i].w, kr[1].z, kr[1].w);
          }
          if (key0 + kPage > P) {                    // tree keys, or keys past the end
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int key = key0 + 8 * t + 2 * q4 + e, j = key - P;
                bool sa = key < end, sb = sa;
                if (sa && j >= 0) {
                  sa = va && c.b >= 0 && ((p.mask[static_cast<size_t>(na) * p.W + (j >> 6)] >> (j & 63)) & 1ull);
                  sb = vb && c.b >= 0 && ((p.mask[static_cast<size_t>(nb) * p.W + (j >> 6)] >> (j & 63)) & 1ull);
                }
                if (!sa) x[t][e] = -INFINITY;
                if (!sb) x[t][2 + e] = -INFINITY;
              }
          }
          // The running maximum rises only by more than 2^8 (see jf_attention.cu): O is rescaled rarely, and
          // most pages need no maximum across the row's four lanes, only that no lane passes it.
          const float ta = fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[1][0], x[1][1])) * p.scale_log2;
          const float tb = fmaxf(fmaxf(x[0][2], x[0][3]), fmaxf(x[1][2], x[1][3])) * p.scale_log2;
          if (__any_sync(0xffffffffu, ta > ma + kRescaleThreshold || tb > mb + kRescaleThreshold)) {
            float ra2 = ta, rb2 = tb;
#pragma unroll
            for (int k = 1; k < 4; k <<= 1) {
              ra2 = fmaxf(ra2, __shfl_xor_sync(0xffffffffu, ra2, k));
              rb2 = fmaxf(rb2, __shfl_xor_sync(0xffffffffu, rb2, k));
            }
            const bool ua = ra2 > ma + kRescaleThreshold, ub = rb2 > mb + kRescaleThreshold;
            const float fa = ua ? fast_exp2(ma - ra2) : 1.f, fb = ub ? fast_exp2(mb - rb2) : 1.f;
            if (ua) ma = ra2;
            if (ub) mb = rb2;
            la *= fa;
            lb *= fb;
#pragma unroll
            for (int j = 0; j < 8 * kH; ++j) {
              o[j][0] *= fa; o[j][1] *= fa;
              o[j][2] *= fb; o[j][3] *= fb;
            }
          }
          const float oa = ma == -INFINITY ? 0.f : -ma, ob = mb == -INFINITY ? 0.f : -mb;
          uint32_t pa[4];                            // the A fragment of the probabilities
#pragma unroll
          for (int t = 0; t < 2; ++t) {              // which replace the scores
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              x[t][e] = fast_exp2(fmaf(x[t][e], p.scale_log2, oa));
              x[t][2 + e] = fast_exp2(fmaf(x[t][2 + e], p.scale_log2, ob));
            }
            la += x[t][0] + x[t][1];
            lb += x[t][2] + x[t][3];
            pa[2 * t] = pack_bf16x2(x[t][0], x[t][1]);
            pa[2 * t + 1] = pack_bf16x2(x[t][2], x[t][3]);
          }
          const bool tail = key0 + kPage > end;
          uint32_t keep0 = 0xFFFFFFFFu, keep1 = keep0;
          if (tail) {
            const int left = end - key0 - 2 * q4;    // of the thread's keys 2 q4, 2 q4 + 1, and eight further on
            keep0 = left >= 2 ? 0xFFFFFFFFu : (left == 1 ? 0xFFFFu : 0u);
            keep1 = left >= 10 ? 0xFFFFFFFFu : (left == 9 ? 0xFFFFu : 0u);
          }
          // Lane l's row of the four 8 x 8 blocks: key l % 16, the first (l < 16) or second d-tile of two.
          const uint32_t vaddr = smem_u32(vt) + (lane & 15) * 128;
          const int vx = (lane & 7) ^ (lane >> 4);   // chunk j + lane / 16, swizzled by the key
          auto pv = [&](const uint32_t (&a)[4]) {
#pragma unroll
            for (int h = 0; h < kH; ++h) {
#pragma unroll
              for (int j = 0; j < 8; j += 2) {       // n-tiles 8 h + j and the next: d from 8 (8 h + j) on
                uint32_t b0, b1, c0, c1;             // keys 0 .. 7 and 8 .. 15 of either
                ldmatrix_x4_trans(b0, b1, c0, c1, vaddr + h * C::kHalfBytes + ((j ^ vx) << 4));
                if (tail) {                          // keys past the end: zero (their probability is, too)
                  b0 &= keep0; b1 &= keep1; c0 &= keep0; c1 &= keep1;
                }
                mma_16816(o[8 * h + j], a[0], a[1], a[2], a[3], b0, b1);
                mma_16816(o[8 * h + j + 1], a[0], a[1], a[2], a[3], c0, c1);
              }
            }
          };
          pv(pa);
          if (split) {                               // and of what their rounding dropped
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const uint32_t u0 = pa[2 * t], u1 = pa[2 * t + 1];
              pa[2 * t] = pack_bf16x2(x[t][0] - __uint_as_float(u0 << 16), x[t][1] - __uint_as_float(u0 & 0xFFFF0000u));
              pa[2 * t + 1] = pack_bf16x2(x[t][2] - __uint_as_float(u1 << 16), x[t][3] - __uint_as_float(u1 & 0xFFFF0000u));
            }
            pv(pa);
          }
        }
        __syncwarp();                                // every lane has read the stage
        if (lane == 0) mbar_arrive(&s_empty[team][st]);
        if (++st == kS) st = 0, phase ^= 1u;
      }
      if (!ok) break;
#pragma unroll
      for (int k = 1; k < 4; k <<= 1) {
        la += __shfl_xor_sync(0xffffffffu, la, k);
        lb += __shfl_xor_sync(0xffffffffu, lb, k);
      }
      // ---- the piece's rows
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const bool mine = half == 0 ? va : vb;
        const int r = half == 0 ? ra : rb;
        const int row = (half == 0 ? na : nb) * p.Hq + c.g * p.G + r % p.G;
        const float l = half == 0 ? la : lb, m = half == 0 ? ma : mb;
        if (!mine) continue;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const float lse2 = l == 0.f ? -INFINITY : m + __log2f(l);
        const int prow = c.whole ? (c.b < 0 ? 0 : p.rows) + row : c.slots + r;
#pragma unroll
        for (int j = 0; j < 8 * kH; ++j) {           // four lanes write a sector of the row
          const float y0 = o[j][2 * half] * inv, y1 = o[j][2 * half + 1] * inv;
          const int d0 = 8 * j + 2 * q4;
          if (c.direct) *reinterpret_cast<uint32_t*>(p.out + static_cast<size_t>(row) * D + d0) = pack_bf16x2(y0, y1);
          else *reinterpret_cast<float2*>(p.ws_o + static_cast<size_t>(prow) * D + d0) = make_float2(y0, y1);
        }
        if (q4 == 0) write_row_facts(p, c, row, prow, r, lse2, 2 * X::R);
      }
    }
    if (!ok && s_sch[team].tiles > 0 && lane == 0) set_abort(abort, p.dev_err);
  }
}

// ------------------------------------------------------------------------ the merge

// The pieces of a (node, query head) row's shared and own parts, listed by ws_desc, merged by
// log-sum-exp.  ROWS > 1: a warp merges ROWS rows, whose reads overlap (four rows for two: 131 -> 144 us
// for 16 trees); ROWS == 1, for few rows: a block merges one, its warps sharing out the pieces.
// A piece that saw a NaN or an infinite score has a NaN log-sum-exp and makes its row NaN; one whose keys were
// all hidden has -inf and is passed over.  Rows behind the last sequence keep what they hold.  What ws_desc
// says is checked against the workspace and against the pieces an item can have (`most_pieces`): a malformed
// group_start or span, or a wait that gave up, leaves it unwritten, with whatever the memory held.
template <int D, int ROWS, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) shared_merge_kernel(const __grid_constant__ SharedParams p, int total, int most_pieces) {
  constexpr int E = D / 32;
  constexpr int kWarps = WARPS;
  constexpr int kStep = ROWS == 1 ? kWarps : 1;       // pieces a warp skips
  constexpr int kBatch = ROWS == 1 ? 6 : 2;           // pieces of a row whose reads overlap
  using Vec = typename std::conditional<E == 4, float4, float2>::type;
  __shared__ float s_part[ROWS == 1 ? kWarps : 1][D + 2];
  grid_dependency_wait();
  grid_dependents_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long r0 = ROWS == 1 ? blockIdx.x : (static_cast<long long>(blockIdx.x) * kWarps + warp) * ROWS;
  int row[ROWS], n[ROWS];
  int4 da[ROWS], db[ROWS];
  bool live[ROWS];                 // of a sequence (its span or length is read beside the descriptors)
  const int behind = p.cu != nullptr ? p.cu[p.B] : 0;
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    const long long rr = r0 + k;
    live[k] = rr < p.rows;
    row[k] = live[k] ? static_cast<int>(rr) : 0;
    da[k] = p.ws_desc[row[k]];
    db[k] = p.ws_desc[p.rows + row[k]];
    const int node = row[k] / p.Hq;
    if (p.cu != nullptr) live[k] = live[k] && node < behind;
    else if (p.tree_len != nullptr) live[k] = live[k] && node % p.N < seq_span(nullptr, p.tree_len, node / p.N, p.N, p.T).n;
  }
  auto bad = [&](const int4& d) {
    return d.y < 0 || d.y > most_pieces || (d.y > 0 && (d.x < 0 || d.x >= total)) ||
           (d.y > 1 && (d.z < 0 || d.w < 0 || d.z + static_cast<long long>(d.y - 2) * d.w >= total));
  };
  auto piece = [&](const int4& a, const int4& b, int k) {      // workspace row of piece k
    const int at = k < a.y ? k : k - a.y;
    const int x = k < a.y ? a.x : b.x, z = k < a.y ? a.z : b.z, w = k < a.y ? a.w : b.w;
    return at == 0 ? x : z + (at - 1) * w;
  };
  float acc[ROWS][E], m[ROWS], sum[ROWS];
  int most = 0;
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    // db.y == 0: written by its only piece
    n[k] = live[k] && db[k].y != 0 && !bad(da[k]) && !bad(db[k]) ? da[k].y + db[k].y : 0;
    most = max(most, n[k]);
    m[k] = -INFINITY;
    sum[k] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[k][e] = 0.f;
  }
  for (int j0 = ROWS == 1 ? warp : 0; j0 < most; j0 += kBatch * kStep) {
    float l[ROWS][kBatch];
    Vec x[ROWS][kBatch];
#pragma unroll
    for (int k = 0; k < ROWS; ++k)
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        l[k][j] = -INFINITY;
        if (j0 + j * kStep < n[k]) {
          const int at = piece(da[k], db[k], j0 + j * kStep);
          l[k][j] = p.ws_lse[at];
          x[k][j] = *reinterpret_cast<const Vec*>(p.ws_o + static_cast<size_t>(at) * D + lane * E);
        }
      }
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      float top = m[k];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) top = fmaxf(top, l[k][j]);      // (passes a NaN by: its weight is one)
      const float f0 = m[k] == -INFINITY ? 0.f : exp2f(m[k] - top);
      m[k] = top;
      sum[k] *= f0;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[k][e] *= f0;
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (l[k][j] == -INFINITY) continue;
        const float f = exp2f(l[k][j] - top);
        const float* xs = reinterpret_cast<const float*>(&x[k][j]);
        sum[k] += f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[k][e] = fmaf(f, xs[e], acc[k][e]);
      }
    }
  }
  if constexpr (ROWS == 1) {
    if (n[0] == 0) return;                       // block-uniform
#pragma unroll
    for (int e = 0; e < E; ++e) s_part[warp][lane * E + e] = acc[0][e];
    if (lane == 0) s_part[warp][D] = m[0], s_part[warp][D + 1] = sum[0];
    __syncthreads();
    if (warp != 0) return;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_part[w][D]);
    m[0] = top;
    sum[0] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[0][e] = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (s_part[w][D + 1] == 0.f) continue;     // nothing that saw a key
      const float f = exp2f(s_part[w][D] - top);
      sum[0] = fmaf(f, s_part[w][D + 1], sum[0]);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[0][e] = fmaf(f, s_part[w][lane * E + e], acc[0][e]);
    }
  }
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    if (n[k] == 0) continue;
    const float inv = sum[k] == 0.f ? 0.f : 1.f / sum[k];
    uint32_t y[E / 2];
#pragma unroll
    for (int e = 0; e < E; e += 2) y[e / 2] = pack_bf16x2(acc[k][e] * inv, acc[k][e + 1] * inv);
    uint16_t* dst = p.out + static_cast<size_t>(row[k]) * D + lane * E;
    if constexpr (E == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(y[0], y[1]);
    else *reinterpret_cast<uint32_t*>(dst) = y[0];
    if (p.lse != nullptr && lane == 0) {
      const int node = row[k] / p.Hq, h = row[k] - node * p.Hq, b = node / p.N;
      p.lse[p.cu != nullptr ? static_cast<size_t>(h) * p.T + node
                            : (static_cast<size_t>(b) * p.Hq + h) * p.N + (node - b * p.N)] =
          (sum[k] == 0.f ? -INFINITY : m[k] + __log2f(sum[k])) * 0.69314718055994531f;
    }
  }
}

// ------------------------------------------------------------------------ host side

struct SharedPlan {
  int tile_nt;             // row tiles per CTA of the tcgen05 kernel, 0: it is not used
  int tile_kinds, tile_ranges, tile_cut0;
  int row_mt;              // warps per team of the row kernel, 0: it is not used
  int row_kinds, row_ranges, row_cut0;
  long long rows, total;   // (node, head) rows; workspace rows
  size_t ws_bytes;
};

constexpr int kMaxRanges = 1024;   // SMs that the 32-bit limits allow for
constexpr int kRowKernelRows = 64; // rows of a unit up to which the row kernel takes it

// nodes: B * N padded, T packed.
bool shared_sizes(long long nodes, int B, int N, int n_groups, int Hq, int Hkv, int D, int max_pages,
                  int page_size) {
  if (B < 1 || B > kSharedMaxB || N < 1 || N > JF_MAX_NODES || nodes < 1 || Hq < 1 || Hkv < 1 || max_pages < 1) return false;
  if (n_groups < 1 || n_groups > B || (D != 64 && D != 128) || page_size != kPage || Hq % Hkv != 0) return false;
  const int G = Hq / Hkv;
  if (G > kRowTile || (G & (G - 1)) != 0) return false;
  if (static_cast<long long>(max_pages) * kPage < N || static_cast<long long>(max_pages) * kPage > (1ll << 30)) return false;
  // workspace rows are 32-bit
  return 2 * nodes * Hq + 8 * kMaxRanges * kRowTile < INT_MAX;
}

// Which kernel takes which units, by the average rows of a group: the groups' own sizes are device data.  Up to 64
// rows the row kernel takes both parts, in teams by the rows (32 rows fill two warps: 256 beams 86.8 us, 126 with one
// warp twice).  Groups of more rows have their shared parts on the tcgen05 kernel, two row tiles per CTA (each key
// tile loaded feeds both) once they fill more than one, and so have own parts of more than 64 rows.
//   33 to 64 rows: the row kernel is ahead while the keys are few (one group of 64 rows over 32K keys 52 us, four over
// 2K 27; with the shared parts on the tcgen05 kernel 53 and 34), behind where they are many (four over 32K 174 and
// 121).  How many there are is device data too, of which the host knows the table's width alone.
//   Uneven groups: one much larger than the average has its shared keys read once per 16 to 64 of its rows (33
// sequences behind 32K keys beside 31 that share nothing, 8 rows a sequence: 458 us; the group alone 58, the others 316.
// 900 sequences behind 4K keys beside 63: 566; alone 126 and 108).
SharedPlan plan_shared(long long nodes, int N, int n_groups, int Hq, int Hkv, int D, int sms) {
  SharedPlan pl = {};
  const long long G = Hq / Hkv, group_rows = (nodes * G + n_groups - 1) / n_groups, own_rows = N * G;
  sms = std::min(sms, kMaxRanges);
  pl.rows = nodes * Hq;
  auto team = [](long long rows) { return rows <= 16 ? 1 : (rows <= 32 ? 2 : 4); };
  if (group_rows <= kRowKernelRows) {
    pl.row_mt = team(group_rows);
    pl.row_kinds = kShared | kOwn;
  } else {
    pl.tile_nt = group_rows > kRowTile ? 2 : 1;
    pl.tile_kinds = kShared;
    if (own_rows <= kRowKernelRows) {
      pl.row_mt = team(own_rows);
      pl.row_kinds = kOwn;
    } else {
      pl.tile_kinds |= kOwn;
    }
  }
  pl.total = 2 * pl.rows;
  if (pl.tile_nt > 0) {
    pl.tile_ranges = sms;
    pl.tile_cut0 = static_cast<int>(pl.total);
    pl.total += 2ll * pl.tile_ranges * pl.tile_nt * kRowTile;
  }
  if (pl.row_mt > 0) {
    pl.row_ranges = sms * (kRowWarps / pl.row_mt);
    pl.row_cut0 = static_cast<int>(pl.total);
    pl.total += 2ll * pl.row_ranges * pl.row_mt * 16;
  }
  pl.ws_bytes = static_cast<size_t>(pl.total) * (D + 1) * sizeof(float) +
                static_cast<size_t>(2 * pl.rows) * sizeof(int4) + 128;
  return pl;
}

// Whether the schedule's positions fit in 32 bits in each kernel of the plan: every item counts as many key
// tiles as the block table holds and a change of item, and a unit's last item may be part empty.
bool positions_fit(const SharedPlan& pl, long long nodes, int B, int n_groups, int Hq, int Hkv, int D, int max_pages) {
  auto fit = [&](int kinds, long long R, long long KT, int change) {
    const long long filled = nodes * (Hq / Hkv) / R;
    const long long items = (kinds & kShared ? filled + n_groups : 0) + (kinds & kOwn ? filled + B : 0);
    return items <= INT_MAX / (((max_pages * kPage + KT - 1) / KT + change) * Hkv);
  };
  return (pl.tile_nt == 0 || fit(pl.tile_kinds, pl.tile_nt * kRowTile, kKeyTile, kTileSwitch)) &&
         (pl.row_mt == 0 || fit(pl.row_kinds, pl.row_mt * 16, kPage, D == 128 ? kRowSwitch<128> : kRowSwitch<64>));
}

// The plan of a call on a device of so many SMs, if its sizes are supported.
bool shared_supported(long long nodes, int B, int N, int n_groups, int Hq, int Hkv, int D, int max_pages,
                      int page_size, int sms, SharedPlan* pl) {
  if (!shared_sizes(nodes, B, N, n_groups, Hq, Hkv, D, max_pages, page_size)) return false;
  *pl = plan_shared(nodes, N, n_groups, Hq, Hkv, D, sms);
  return positions_fit(*pl, nodes, B, n_groups, Hq, Hkv, D, max_pages);
}

template <int NT, int D>
jf_status launch_tiles(const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm, const CUtensorMap& kr,
                       const CUtensorMap& vr, const SharedParams& prm, cudaStream_t s) {
  using C = Cfg<NT, D>;
  static_assert(C::kSmemBytes >= schedule_bytes(kSharedMaxB, kSharedMaxB) + 1024, "the schedule's scratch fits");
  static SmemAttr attr;
  if (!attr.ensure(shared_attention_kernel<NT, D>, C::kSmemBytes)) return JF_ERR_CUDA;
  return launch_pdl(shared_attention_kernel<NT, D>, dim3(static_cast<unsigned>(prm.ranges)), dim3(C::kThreads),
                    C::kSmemBytes, s, qm, km, vm, kr, vr, prm) == cudaSuccess
             ? JF_OK
             : JF_ERR_CUDA;
}

template <int D, int MT>
jf_status launch_rows(const CUtensorMap& km, const CUtensorMap& vm, const SharedParams& prm, cudaStream_t s) {
  using C = RowCfg<D, MT>;
  static_assert(C::kSmemBytes >= schedule_bytes(kSharedMaxB, kSharedMaxB) + 1024, "the schedule's scratch fits");
  static SmemAttr attr;
  if (!attr.ensure(shared_rows_kernel<D, MT>, C::kSmemBytes)) return JF_ERR_CUDA;
  return launch_pdl(shared_rows_kernel<D, MT>, dim3(static_cast<unsigned>(prm.ranges / C::kTeams)),
                    dim3(64 * kRowWarps), C::kSmemBytes, s, km, vm, prm) == cudaSuccess
             ? JF_OK
             : JF_ERR_CUDA;
}

template <int D>
jf_status launch_merge(const SharedParams& prm, int total, int most, int sms, cudaStream_t s) {
  // A block a row while that keeps the SMs at most 32 blocks deep (its warps share a long list of
  // pieces: 64 requests 80.2 us, with two rows a warp 91.6), of eight warps while all blocks are resident
  // (4 beams 12.8, with four 14.3), else of four (64 requests 80.2, with eight 82.3); beyond that two rows a
  // warp (16 trees 120 us, with a block a row 145; 256 beams 86.8 and 94.8).
  const long long rows = prm.rows;
  const dim3 each(static_cast<unsigned>(rows)), half(static_cast<unsigned>((rows + 15) / 16));
  const cudaError_t e = rows <= 4ll * sms    ? launch_pdl(shared_merge_kernel<D, 1, 8>, each, dim3(256), 0, s, prm, total, most)
                        : rows <= 32ll * sms ? launch_pdl(shared_merge_kernel<D, 1, 4>, each, dim3(128), 0, s, prm, total, most)
                                             : launch_pdl(shared_merge_kernel<D, 2, 8>, half, dim3(256), 0, s, prm, total, most);
  return e == cudaSuccess ? JF_OK : JF_ERR_CUDA;
}

jf_status shared_call(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                      const int32_t* prefix_len, const int32_t* tree_len, const int32_t* cu, const uint64_t* mask,
                      const int32_t* group_start, const int32_t* shared_pages, int32_t n_groups, int32_t B, int32_t N,
                      int32_t T, int32_t Hq, int32_t Hkv, int32_t D, int32_t page_size, int32_t max_pages,
                      int32_t num_pages, float scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                      int32_t* dev_err, jf_stream_t stream) {
  if (q == nullptr || k_cache == nullptr || v_cache == nullptr || block_table == nullptr || prefix_len == nullptr ||
      mask == nullptr || group_start == nullptr || shared_pages == nullptr || out == nullptr)
    return JF_ERR_INVALID_ARGUMENT;
  if (B < 1 || N < 1 || Hq < 1 || Hkv < 1 || D < 1 || page_size < 1 || max_pages < 1 || num_pages < 1 ||
      n_groups < 1 || n_groups > B || (cu != nullptr && T < 1) || !(scale > 0.f) || !std::isfinite(scale))
    return JF_ERR_INVALID_ARGUMENT;
  if (cu != nullptr && static_cast<long long>(T) + N >= (1ll << 31)) return JF_ERR_UNSUPPORTED;
  if (static_cast<long long>(num_pages) * kPage >= (1ll << 31)) return JF_ERR_UNSUPPORTED;
  const long long nodes = cu != nullptr ? T : static_cast<long long>(B) * N;
  const int sms = current_sm_count();
  SharedPlan pl;
  if (!shared_supported(nodes, B, N, n_groups, Hq, Hkv, D, max_pages, page_size, sms, &pl)) return JF_ERR_UNSUPPORTED;
  if (!aligned_to(q, 16) || !aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) || !aligned_to(out, 16) ||
      !aligned_to(mask, 8))
    return JF_ERR_MISALIGNED;
  // What is written shares no byte with what is read or with another output.
  const size_t qb = static_cast<size_t>(nodes) * Hq * D * 2, cb = static_cast<size_t>(num_pages) * kPage * Hkv * D * 2;
  const size_t lb = static_cast<size_t>(nodes) * Hq * 4, seqs = static_cast<size_t>(B), gb = static_cast<size_t>(n_groups) * 4;
  auto over_inputs = [&](const void* to, size_t bytes) {
    return overlaps_any(to, bytes, {{q, qb}, {k_cache, cb}, {v_cache, cb}, {block_table, seqs * max_pages * 4},
                                    {prefix_len, seqs * 4}, {tree_len, seqs * 4}, {cu, (seqs + 1) * 4},
                                    {mask, static_cast<size_t>(nodes) * ((N + 63) / 64) * 8}, {group_start, gb + 4},
                                    {shared_pages, gb}});
  };
  if (over_inputs(out, qb) || (lse != nullptr && (over_inputs(lse, lb) || overlap(lse, lb, out, qb))))
    return JF_ERR_INVALID_ARGUMENT;
  const size_t wb = std::min(workspace_bytes, pl.ws_bytes);       // what of the workspace would be used
  if (workspace != nullptr && (over_inputs(workspace, wb) || overlaps_any(workspace, wb, {{out, qb}, {lse, lb}})))
    return JF_ERR_INVALID_ARGUMENT;
  if (sms <= 0) return JF_ERR_CUDA;
  if (workspace == nullptr || workspace_bytes < pl.ws_bytes) return JF_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned_to(workspace, 16)) return JF_ERR_MISALIGNED;
  const int G = Hq / Hkv;
  CUtensorMap qm, km, vm, kr, vr;
  {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(Hkv),
                                static_cast<cuuint64_t>(num_pages) * kPage};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(Hkv) * D * 2};
    const cuuint32_t box[3] = {64, 1, kPage}, box_run[3] = {64, 1, kKeyTile};
    if (!encode(&km, k_cache, 3, dims, strides, box) || !encode(&vm, v_cache, 3, dims, strides, box)) return JF_ERR_CUDA;
    if (pl.tile_nt > 0 &&
        (!encode(&kr, k_cache, 3, dims, strides, box_run) || !encode(&vr, v_cache, 3, dims, strides, box_run)))
      return JF_ERR_CUDA;
  }
  if (pl.tile_nt > 0) {
    // q as one list of nodes: sequences of a group follow each other
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(Hq), static_cast<cuuint64_t>(nodes)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(Hq) * D * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(kRowTile / G)};
    if (!encode(&qm, q, 3, dims, strides, box)) return JF_ERR_CUDA;
  }
  SharedParams prm = {};
  prm.block_table = block_table; prm.prefix_len = prefix_len; prm.tree_len = tree_len; prm.cu = cu;
  prm.group_start = group_start; prm.shared_pages = shared_pages; prm.mask = mask;
  prm.out = static_cast<uint16_t*>(out);
  prm.lse = lse;
  // partial rows first, from a 128-byte boundary on
  prm.ws_o = reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(workspace) + 127) & ~static_cast<uintptr_t>(127));
  prm.ws_desc = reinterpret_cast<int4*>(prm.ws_o + static_cast<size_t>(pl.total) * D);
  prm.ws_lse = reinterpret_cast<float*>(prm.ws_desc + 2 * pl.rows);
  prm.dev_err = dev_err;
  prm.T = cu != nullptr ? T : 0;
  prm.B = B; prm.N = N; prm.Hq = Hq; prm.Hkv = Hkv; prm.G = G; prm.W = (N + 63) / 64;
  prm.max_pages = max_pages; prm.num_pages = num_pages; prm.n_groups = n_groups;
  prm.q = static_cast<const uint16_t*>(q);
  prm.rows = static_cast<int>(pl.rows);
  prm.scale_log2 = scale * 1.4426950408889634f;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  jf_status st = JF_OK;
  if (pl.tile_nt > 0) {
    prm.kinds = pl.tile_kinds;
    prm.ranges = pl.tile_ranges;
    prm.cut0 = pl.tile_cut0;
    if (D == 128)
      st = pl.tile_nt == 2 ? launch_tiles<2, 128>(qm, km, vm, kr, vr, prm, s) : launch_tiles<1, 128>(qm, km, vm, kr, vr, prm, s);
    else
      st = pl.tile_nt == 2 ? launch_tiles<2, 64>(qm, km, vm, kr, vr, prm, s) : launch_tiles<1, 64>(qm, km, vm, kr, vr, prm, s);
    if (st != JF_OK) return st;
  }
  if (pl.row_mt > 0) {
    prm.kinds = pl.row_kinds;
    prm.ranges = pl.row_ranges;
    prm.cut0 = pl.row_cut0;
    if (D == 128)
      st = pl.row_mt == 1 ? launch_rows<128, 1>(km, vm, prm, s) : (pl.row_mt == 2 ? launch_rows<128, 2>(km, vm, prm, s) : launch_rows<128, 4>(km, vm, prm, s));
    else
      st = pl.row_mt == 1 ? launch_rows<64, 1>(km, vm, prm, s) : (pl.row_mt == 2 ? launch_rows<64, 2>(km, vm, prm, s) : launch_rows<64, 4>(km, vm, prm, s));
    if (st != JF_OK) return st;
  }
  const int total = static_cast<int>(pl.total), pieces = std::max(pl.tile_ranges, pl.row_ranges);    // one a range
  return D == 128 ? launch_merge<128>(prm, total, pieces, sms, s) : launch_merge<64>(prm, total, pieces, sms, s);
}

}  // namespace

bool set_shared_wait_limit(uint64_t limit_ns, int withhold) {
  return cudaMemcpyToSymbol(c_wait_limit_ns, &limit_ns, sizeof(limit_ns)) == cudaSuccess &&
         cudaMemcpyToSymbol(c_withhold, &withhold, sizeof(withhold)) == cudaSuccess;
}

}  // namespace jf

extern "C" size_t jf_tree_attention_shared_workspace_size(int32_t B, int32_t N, int32_t T, int32_t n_groups,
                                                          int32_t Hq, int32_t Hkv, int32_t D, int32_t max_pages,
                                                          int32_t page_size) {
  const long long nodes = T > 0 ? T : static_cast<long long>(B) * N;
  const int sms = jf::current_sm_count();
  jf::SharedPlan pl;
  const bool ok = jf::shared_supported(nodes, B, N, n_groups, Hq, Hkv, D, max_pages, page_size, sms, &pl);
  return ok && sms > 0 ? pl.ws_bytes : static_cast<size_t>(-1);
}

extern "C" jf_status jf_tree_attention_shared(const void* q, const void* k_cache, const void* v_cache,
                                              const int32_t* block_table, const int32_t* prefix_len,
                                              const int32_t* tree_len, const uint64_t* mask,
                                              const int32_t* group_start, const int32_t* shared_pages,
                                              int32_t n_groups, int32_t B, int32_t N, int32_t Hq, int32_t Hkv,
                                              int32_t D, int32_t page_size, int32_t max_pages, int32_t num_pages,
                                              float scale, void* out, float* lse, void* workspace,
                                              size_t workspace_bytes, int32_t* dev_err, jf_stream_t stream) {
  return jf::shared_call(q, k_cache, v_cache, block_table, prefix_len, tree_len, nullptr, mask, group_start,
                         shared_pages, n_groups, B, N, 0, Hq, Hkv, D, page_size, max_pages, num_pages, scale, out,
                         lse, workspace, workspace_bytes, dev_err, stream);
}

extern "C" jf_status jf_tree_attention_shared_packed(
    const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table, const int32_t* prefix_len,
    const int32_t* cu_seqlens, const uint64_t* mask, const int32_t* group_start, const int32_t* shared_pages,
    int32_t n_groups, int32_t B, int32_t N_max, int32_t T, int32_t Hq, int32_t Hkv, int32_t D, int32_t page_size,
    int32_t max_pages, int32_t num_pages, float scale, void* out, float* lse, void* workspace,
    size_t workspace_bytes, int32_t* dev_err, jf_stream_t stream) {
  if (cu_seqlens == nullptr) return JF_ERR_INVALID_ARGUMENT;
  return jf::shared_call(q, k_cache, v_cache, block_table, prefix_len, nullptr, cu_seqlens, mask, group_start,
                         shared_pages, n_groups, B, N_max, T, Hq, Hkv, D, page_size, max_pages, num_pages, scale,
                         out, lse, workspace, workspace_bytes, dev_err, stream);
}
