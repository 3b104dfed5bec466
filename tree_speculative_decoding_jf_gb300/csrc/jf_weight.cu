// jf_weight.cu -- accumulated attention weight of every cached key.
//
// For sequence b, kv-head g and cache position t the call adds the softmax probabilities
// that the step's query rows gave the key:
//     sum_{k < R_b} sum_{h in group g} [t <= P_b + k] exp(scale q_kh . K_t - lse_kh),
// where lse is what the attention call left, so no softmax statistics are formed here and
// every key is independent: no reduction crosses keys.
//
// The scores are taken transposed, S^T = K Q^T: a 128-key tile is the A operand, a block of
// query rows the B operand (whole nodes of G rows, at most 128 rows; row = k * G + head in
// group), and a TMEM lane is a key.  So the thread that owns a lane owns its key: it adds
// its probabilities in registers over all row blocks and writes the key's weight once.  K
// is read once, nothing is merged between CTAs, and the order of every sum is fixed.
//
// Work: the key tiles of all sequences lie end to end, a tile weighted by its row blocks,
// and are cut into (SMs / kv-heads) equal ranges; the CTAs of a range (one per kv-head, side
// by side) walk the same tokens together, so the 256-byte rows that they read lie next to
// each other.  (Rounded down: of 152 SMs, 32 kv-heads use 128, 40 use 120 and 80 use 80, and
// more than 152 kv-heads take a second round.)  Up to four consecutive tiles of a sequence form a group that shares every
// row block loaded; with one row block (a verified path) it stays in shared memory for the
// whole run of the sequence.
//
// Roles (768 threads):
//   warps 0, 1     issue the MMAs of the even and the odd tiles (warp 0 allocates TMEM): one
//                  warp's waits and bookkeeping, some 500 cycles a tile, pass while the
//                  other's eight MMAs run.
//   warps 2, 3     query rows, one warp per stage: a full block of a chain as one TMA box
//                  per 64-column half, else one box per (node, half), and the rows' lse.
//                  (Gathered with 16-byte asynchronous copies instead, a block took 13,000
//                  cycles to issue beside the polling warps.)
//   warps 4..19    four warpgroups, one per TMEM slot (128 columns): tile c of the CTA goes
//                  to slot c % 4.  (Two warpgroups with two slots each leave a scheduler
//                  with two such warps and their latencies: 136 us against 122 on a 512-row
//                  window over 2 x 16K keys.)
//   warps 20..23   K tiles by TMA into a ring, a quarter of every tile's pages each (issued
//                  from 16 lanes of one warp, a tile's boxes took 1400 cycles to go out,
//                  more than its share of the HBM bandwidth); page ids four to eight tiles
//                  ahead; pages past the end and malformed ids load as zeros.
// What bounds it: HBM with few rows (54 us for 8 x 32K keys, 32/4 heads, whose bytes take 41);
// with many, the instructions of the probabilities: the window took 124 us, whose products
// take 71, and still 114 without the MMAs, or without MMAs and TMEM loads, but 87 when the
// reads of -lse went as well (103 without the exponentials, 79 with the TMEM loads and the
// waits alone).
// Slots past a block's rows and rows whose lse is -inf get zero queries and lse = +inf, so
// they add exp(-inf) = 0.  Only with an infinity or a NaN in the key is such a score not zero
// but NaN (0 * inf): one such column of the block tells, and its warp then leaves them all out
// (122 against 119 us on the window, nothing on the others; testing every column of a block
// that has any, 82 against 57 us on a window of three heads a group).
// Keys past the sequence's end are lanes whose sum is dropped: whatever their page slots hold
// stays in their lane.
// All waits are bounded; on a timeout the CTA records JF_DEVERR_TIMEOUT, drains its copies
// and MMAs, frees TMEM and returns.
#include <algorithm>
#include <cmath>

#include "jf_common.cuh"
#include "jf_sm100.cuh"
#include "jf_tensormap.cuh"

namespace jf {
namespace {

constexpr int kPage = 16;
constexpr int kKeyTile = 128;
constexpr int kPagesPerTile = kKeyTile / kPage;
constexpr int kRowBlock = 128;
constexpr int kSlots = 4;                 // TMEM slots = epilogue warpgroups
constexpr int kGroup = kSlots;            // key tiles that share a loaded row block
constexpr int kThreads = 768;
constexpr int kQWarp = 2, kEpiWarp = 4, kKWarp = 20;   // first warps of the roles
constexpr int kKWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kTileBytes = kKeyTile * D * 2;
  static constexpr int kHalfBytes = kKeyTile * 128;
  // 160 KB of K in flight, far above the ~45 KB an SM needs to cover the latency of HBM at
  // its share of the bandwidth, and a group's four tiles plus the next one for D = 128.
  static constexpr int kKStages = D == 128 ? 5 : 10;
  // Barriers of the ring: twice the stages, so that every barrier belongs to tiles of one
  // parity and thus to one MMA warp.  (With one a stage, a warp may come to wait for the
  // phase after one that the other warp's tile has not completed, and a parity wait takes
  // the phase before that for its own.)
  static constexpr int kKBars = 2 * kKStages;
  static constexpr int kQStages = 2;          // one producer warp each
  static constexpr int kLseStages = 3;        // held until the probabilities are added
  static constexpr int kQOff = kKStages * kTileBytes;
  static constexpr int kSmemBytes = kQOff + kQStages * kTileBytes + 1024;
};

struct WeightParams {
  const int32_t* block_table;
  const int32_t* prefix_len;
  const int32_t* path;        // or null: row k is node k
  const int32_t* accept_len;  // or null: every node is a row
  const int32_t* cu;          // packed calls, else null
  const float* lse;
  const float* weight;        // or null: from zero
  float* weight_out;
  int32_t* dev_err;
  long long T;
  int B, N, Hq, Hkv, G, max_pages, num_pages;
  int nodes;                  // nodes of a full row block: 128 / G
  float scale_log2;
};

struct SeqInfo {
  long long row0;             // first row of the sequence in q
  int n, P, R, L;             // nodes, prefix, query rows, keys
  int tiles, blocks, unit;    // key tiles and row blocks of a kv-head, cost of a tile
  int bits;
};

__device__ __forceinline__ SeqInfo seq_info(const WeightParams& p, int b) {
  SeqInfo s;
  const int cap = p.max_pages * kPage;
  const SeqSpan sp = seq_span(p.cu, nullptr, b, p.N, p.T);
  s.bits = sp.ok ? 0 : JF_DEVERR_BAD_TREE_LEN;
  s.row0 = sp.row0;
  s.n = sp.n;
  int R = sp.n;
  if (p.accept_len != nullptr) {
    const int a = p.accept_len[b];
    R = a < -1 ? 0 : (a >= sp.n ? sp.n : a + 1);
    if (sp.ok && (a < -1 || a >= sp.n)) s.bits |= JF_DEVERR_BAD_PATH;
  }
  int P = p.prefix_len[b];
  if (P < 0 || P > cap - R) {
    s.bits |= JF_DEVERR_BAD_PREFIX;
    P = max(0, min(P, cap));
    R = min(R, cap - P);
  }
  s.P = P;
  s.R = R;
  s.L = P + R;
  s.tiles = (s.L + kKeyTile - 1) / kKeyTile;
  s.blocks = (R + p.nodes - 1) / p.nodes;
  // A tile with one or two row blocks costs its 32 KB from HBM, one with more its blocks.
  s.unit = s.blocks == 0 ? 1 : max(2, s.blocks);
  return s;
}

// This CTA's range [x0, x1) of the total cost, and the sequence where it starts.
struct Range {
  long long x0, x1, base;
  int b;
};

// Calls f(b, first tile, tiles, info) for every sequence's run of tiles in the range, in
// order, until f returns false.
template <typename F>
__device__ __forceinline__ void for_each_run(const WeightParams& p, const Range& r, F f) {
  long long base = r.base;
  for (int b = r.b; b < p.B && base < r.x1; ++b) {
    const SeqInfo s = seq_info(p, b);
    const long long lo = r.x0 - base, hi = r.x1 - base;
    int i = lo <= 0 ? 0 : static_cast<int>((lo + s.unit - 1) / s.unit);
    const long long last = (hi + s.unit - 1) / s.unit;
    const int end = last < s.tiles ? static_cast<int>(last) : s.tiles;
    if (i < end && !f(b, i, end - i, s)) return;
    base += static_cast<long long>(s.tiles) * s.unit;
  }
}

// Rows of earlier positions than the group's first key do not see it: the first row block
// that does.
__device__ __forceinline__ int first_block(const SeqInfo& s, int tile, int nodes) {
  return max(0, tile * kKeyTile - s.P) / nodes;
}

// Columns (rows of Q) that block qb's MMAs compute: a multiple of 32.
__device__ __forceinline__ int block_cols(const SeqInfo& s, int qb, int nodes, int G) {
  return (min(nodes, s.R - qb * nodes) * G + 31) & ~31;
}

// Adds 16 columns' probabilities 2^(s * c + nlse) to acc; MASKED: only columns j >= j_min of
// rows that add something (nlse above -inf), whatever the others' scores are.
// (One instantiation with the test inside has a branch every four columns, which keeps the
// compiler from overlapping them: 237 cycles for each four instead of about 20.)
template <bool MASKED>
__device__ __forceinline__ void add16(const uint32_t (&sv)[16], const float* nlse, int j_min, uint64_t c2,
                                      uint64_t (&acc)[2]) {
  const float4* nl = reinterpret_cast<const float4*>(nlse);
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const float4 l = nl[v];
    float x0, x1, x2, x3;
    f2_split(ffma2(f2(__uint_as_float(sv[4 * v]), __uint_as_float(sv[4 * v + 1])), c2, f2(l.x, l.y)), x0, x1);
    f2_split(ffma2(f2(__uint_as_float(sv[4 * v + 2]), __uint_as_float(sv[4 * v + 3])), c2, f2(l.z, l.w)), x2, x3);
    if constexpr (MASKED) {
      x0 = 4 * v + 0 < j_min || l.x == -INFINITY ? -INFINITY : x0;
      x1 = 4 * v + 1 < j_min || l.y == -INFINITY ? -INFINITY : x1;
      x2 = 4 * v + 2 < j_min || l.z == -INFINITY ? -INFINITY : x2;
      x3 = 4 * v + 3 < j_min || l.w == -INFINITY ? -INFINITY : x3;
    }
    acc[0] = fadd2(acc[0], f2(fast_exp2(x0), fast_exp2(x1)));
    acc[1] = fadd2(acc[1], f2(fast_exp2(x2), fast_exp2(x3)));
  }
}

// All columns of a slot (a multiple of 32); the next 16 travel from TMEM while 16 are
// worked on.
template <bool MASKED>
__device__ __forceinline__ void add_columns(uint32_t addr, const float* nlse, int cols, int j_min, uint64_t c2,
                                            uint64_t (&acc)[2]) {
  uint32_t sa[16], sb[16];
  tmem_ld16(addr, sa);
#pragma unroll 1
  for (int c = 0; c < cols; c += 32) {
    tmem_ld_wait16(sa);
    tmem_ld16(addr + c + 16, sb);
    add16<MASKED>(sa, nlse + c, j_min - c, c2, acc);
    tmem_ld_wait16(sb);
    tmem_ld16(addr + min(c + 32, cols - 32), sa);   // (the last one is not used)
    add16<MASKED>(sb, nlse + c + 16, j_min - c - 16, c2, acc);
  }
  tmem_ld_wait16(sa);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    weight_kernel(const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap qmap_node,
                  const WeightParams p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  uint8_t* k_s = sm;
  uint8_t* q_s = sm + C::kQOff;
  __shared__ uint64_t k_full[C::kKBars], k_empty[C::kKBars];
  __shared__ uint64_t q_full[C::kQStages], q_empty[C::kQStages], q_raw[C::kQStages];
  __shared__ uint64_t l_full[C::kLseStages], l_empty[C::kLseStages];
  __shared__ uint64_t s_full[kSlots], s_empty[kSlots], fin;
  __shared__ __align__(16) float s_nlse[C::kLseStages][kRowBlock];   // -lse in log2 units
  __shared__ int s_idle[C::kLseStages];       // a column of the block that adds nothing; kRowBlock: none
  __shared__ Range s_range;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  volatile int* abort = &abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < C::kKBars; ++i) {
      mbar_init(&k_full[i], kKWarps);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < C::kQStages; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 2);
      mbar_init(&q_raw[i], 1);
    }
    for (int i = 0; i < C::kLseStages; ++i) {
      mbar_init(&l_full[i], 32);
      mbar_init(&l_empty[i], 4 * kSlots);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 4);
    }
    mbar_init(&fin, 2);
    abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&qmap);
    tma_prefetch_desc(&qmap_node);
  }
  grid_dependency_wait();

  // ---- this CTA's range: the block scans the sequences' costs, kThreads at a time.
  auto cost_of = [&](int b) -> long long {
    if (b >= p.B) return 0;
    const SeqInfo s = seq_info(p, b);
    if (s.bits && blockIdx.x == 0) report(p.dev_err, s.bits);
    return static_cast<long long>(s.tiles) * s.unit;
  };
  long long* s_scan = reinterpret_cast<long long*>(&s_nlse[0][0]);   // not in use yet
  auto scan = [&](long long mine, long long* excl) -> long long {   // returns the block's sum
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    __syncthreads();
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    long long before = 0, all = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += s_scan[w];
      all += s_scan[w];
    }
    *excl = before + incl - mine;
    return all;
  };
  long long total = 0, excl = 0, mine = 0;
  for (int b0 = 0; b0 < p.B; b0 += kThreads) {
    mine = cost_of(b0 + tid);
    total += scan(mine, &excl);
  }
  const int g = blockIdx.x % p.Hkv, part = blockIdx.x / p.Hkv, parts = gridDim.x / p.Hkv;
  const long long x0 = total * part / parts, x1 = total * (part + 1) / parts;
  if (x0 == x1) {
    grid_dependents_launch();
    return;
  }
  long long run = 0;
  for (int b0 = 0; b0 < p.B && run <= x0; b0 += kThreads) {
    if (p.B > kThreads) mine = cost_of(b0 + tid);
    const long long all = p.B > kThreads ? scan(mine, &excl) : total;
    if (run + excl <= x0 && x0 < run + excl + mine) s_range = Range{x0, x1, run + excl, b0 + tid};
    run += all;
  }
  if (warp == 0) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const Range range = s_range;
  const uint32_t tmem = tmem_slot;
  const uint64_t wlim = kWaitLimitNs;
  const int G = p.G, nodes = p.nodes;

  if (warp >= kKWarp) {
    // ================================================================ K producers
    constexpr int kMine = kPagesPerTile / kKWarps;          // pages of a tile for this warp
    const int quarter = warp - kKWarp;
    int issued = 0, bits = 0;
    for_each_run(p, range, [&](int b, int t0, int n, const SeqInfo& s) -> bool {
      if (s.blocks == 0) return true;
      const int32_t* bt = p.block_table + static_cast<size_t>(b) * p.max_pages;
      // Lane l holds page l % 8 of tile l / 8 of a batch of four tiles; the next batch is
      // asked for when a batch's first tile is issued.  num_pages: loads as zeros.
      auto pages_of = [&](int tile4) -> int {
        const int pl = tile4 * kPagesPerTile + lane;
        if (tile4 + lane / kPagesPerTile >= t0 + n || pl * kPage >= s.L) return p.num_pages;
        return __ldg(bt + pl);
      };
      int now = 0, next = pages_of(t0);
      for (int tile = t0; tile < t0 + n; ++tile) {
        const int sub = (tile - t0) % 4;
        if (sub == 0) {
          now = next;
          next = pages_of(tile + 4);
          if (now < 0 || now > p.num_pages) {
            bits |= JF_DEVERR_BAD_PAGE;
            now = p.num_pages;
          } else if (now == p.num_pages && tile + lane / kPagesPerTile < t0 + n &&
                     (tile * kPagesPerTile + lane) * kPage < s.L) {
            bits |= JF_DEVERR_BAD_PAGE;
          }
        }
        const int st = issued % C::kKStages, before = issued - C::kKStages;   // the stage's last tile
        if (before >= 0 && !wait_lanes(&k_empty[before % C::kKBars], static_cast<uint32_t>(before / C::kKBars) & 1u,
                                       abort, wlim)) {
          if (lane == 0) set_abort(abort, p.dev_err);
          return false;
        }
        uint64_t* full = &k_full[issued % C::kKBars];
        uint8_t* dst = k_s + st * C::kTileBytes + quarter * kMine * (kPage * 128);
        elect_arrive_expect_tx(full, C::kTileBytes / kKWarps);
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          const int page = __shfl_sync(0xffffffffu, now, sub * kPagesPerTile + quarter * kMine + i);
#pragma unroll
          for (int hh = 0; hh < C::kHalves; ++hh)
            elect_tma_load_3d(dst + hh * C::kHalfBytes + i * (kPage * 128), &kmap, full, hh * 64, g,
                              page * kPage);
        }
        ++issued;
      }
      return true;
    });
    if (bits) report(p.dev_err, bits);
    __syncwarp();
    if (lane == 0) {                          // no copy is still landing when the CTA exits
      int zero = 0;
      for (int i = max(0, issued - C::kKStages); i < issued; ++i)
        mbar_wait(&k_full[i % C::kKBars], static_cast<uint32_t>(i / C::kKBars) & 1u, &zero);
    }
  } else if (warp < kQWarp) {
    // ================================================================ MMA issuer
    const uint64_t dk = desc_sw128(smem_u32(k_s), 16, 1024);
    const uint64_t dq = desc_sw128(smem_u32(q_s), 16, 1024);
    int tile_no = 0, q_no = 0;                // tiles and row blocks so far
    uint32_t free_phase = (1u << kSlots) - 1u;  // parity to wait for on s_empty, per slot
    auto fail = [&]() -> bool {
      if (lane == 0) set_abort(abort, p.dev_err);
      return false;
    };
    // S^T of K stage k_at and row block q_at into a slot.
    auto issue = [&](int k_at, int q_at, int slot, int cols) -> bool {
      if (!wait_lanes(&s_empty[slot], (free_phase >> slot) & 1u, abort, wlim)) return false;
      free_phase ^= 1u << slot;
      tc_fence_after();
      mma_ss_tile<D / 16>(tmem + slot * kRowBlock,
                          dk + static_cast<uint64_t>((k_at * C::kTileBytes) >> 4),
                          dq + static_cast<uint64_t>((q_at * C::kTileBytes) >> 4),
                          idesc_bf16(kKeyTile, cols, false, false));
      mma_commit(&s_full[slot]);
      return true;
    };
    for_each_run(p, range, [&](int b, int t0, int n, const SeqInfo& s) -> bool {
      if (s.blocks == 0) return true;
      const bool one = s.blocks == 1;         // its block stays for the whole run
      for (int i0 = 0; i0 < n; i0 += kGroup) {
        const int m = min(kGroup, n - i0), ia = (tile_no ^ warp) & 1;
        const int na = tile_no + ia, nb = na + 2;           // this warp's tiles of the group
        const int ka = na % C::kKBars, kb = nb % C::kKBars;
        const uint32_t pa = static_cast<uint32_t>(na / C::kKBars) & 1u;
        const uint32_t pb = static_cast<uint32_t>(nb / C::kKBars) & 1u;
        const int sa = na % kSlots, sb = nb % kSlots;
        const int qb0 = first_block(s, t0 + i0, nodes);
        for (int qb = qb0; qb < s.blocks; ++qb) {
          const bool last = qb == s.blocks - 1;
          const int cols = block_cols(s, qb, nodes, G);
          const int qs = q_no % C::kQStages;
          if ((!one || i0 == 0) &&
              !wait_lanes(&q_full[qs], static_cast<uint32_t>(q_no / C::kQStages) & 1u, abort, wlim))
            return fail();
          if (ia < m) {
            if (qb == qb0 && !wait_lanes(&k_full[ka], pa, abort, wlim)) return fail();
            if (!issue(na % C::kKStages, qs, sa, cols)) return fail();
            if (last) mma_commit(&k_empty[ka]);
          }
          if (ia + 2 < m) {
            if (qb == qb0 && !wait_lanes(&k_full[kb], pb, abort, wlim)) return fail();
            if (!issue(nb % C::kKStages, qs, sb, cols)) return fail();
            if (last) mma_commit(&k_empty[kb]);
          }
          if (one && i0 + kGroup < n) break;
          mma_commit(&q_empty[qs]);
          ++q_no;
        }
        tile_no += m;
      }
      return true;
    });
    mma_commit(&fin);                         // all MMAs are done before TMEM is released
    if (lane == 0) {
      int zero = 0;
      mbar_wait(&fin, 0, &zero);
    }
    __syncwarp();
  } else if (warp >= kQWarp && warp < kEpiWarp) {
    // ================================================================ query rows
    constexpr int kVecs = 8;                  // 16-byte vectors of a row's half
    const int stage = warp - kQWarp;
    int q_no = 0, mine = 0, raw_no = 0, bits = 0;
    uint8_t* dst = q_s + stage * C::kTileBytes;
    auto zero_row = [&](int r, int c) {       // vector c of row r, all halves
      for (int hh = 0; hh < C::kHalves; ++hh)
        *reinterpret_cast<uint4*>(dst + hh * C::kHalfBytes + r * 128 + (c << 4)) = make_uint4(0u, 0u, 0u, 0u);
    };
    // Loads block qb of sequence b if it is this warp's turn.
    auto load = [&](int b, const SeqInfo& s, int qb) -> bool {
      const int no = q_no++;
      if (no % C::kQStages != stage) return true;
      const int n0 = qb * nodes, nb = min(nodes, s.R - n0), rows = nb * G, cols = block_cols(s, qb, nodes, G);
      auto node_at = [&](int k) -> int {      // -1: malformed
        const int node = p.path == nullptr ? k : __ldg(p.path + static_cast<size_t>(b) * p.N + k);
        if (node >= 0 && node < s.n) return node;
        bits |= JF_DEVERR_BAD_PATH;
        return -1;
      };
      // Four rows a lane: their lse, asked for before the stage is free.
      float nl[kRowBlock / 32];
      int dead = kRowBlock;                   // a row that adds nothing
#pragma unroll
      for (int u = 0; u < kRowBlock / 32; ++u) {
        const int r = u * 32 + lane, k = r / G, h = g * G + r - k * G;
        nl[u] = -INFINITY;
        if (r >= rows) continue;
        const int node = node_at(n0 + k);
        if (node >= 0) {
          const float lse = p.cu != nullptr ? __ldg(p.lse + static_cast<size_t>(h) * p.T + s.row0 + node)
                                            : __ldg(p.lse + (static_cast<size_t>(b) * p.Hq + h) * p.N + node);
          if (lse != -INFINITY) nl[u] = -lse * kLog2e;
        }
        if (nl[u] == -INFINITY) dead = r;     // (lse = +inf as well: it adds nothing)
      }
      const int ls = no % C::kLseStages;
      if (!wait_lanes(&q_empty[stage], (static_cast<uint32_t>(no / C::kQStages) & 1u) ^ 1u, abort, wlim) ||
          !wait_lanes(&l_empty[ls], (static_cast<uint32_t>(no / C::kLseStages) & 1u) ^ 1u, abort, wlim)) {
        if (lane == 0) set_abort(abort, p.dev_err);
        return false;
      }
      ++mine;
#pragma unroll
      for (int u = 0; u < kRowBlock / 32; ++u) s_nlse[ls][u * 32 + lane] = nl[u];
      const int idle = __reduce_min_sync(0xffffffffu, dead);
      const bool rare = idle < kRowBlock;
      if (lane == 0) s_idle[ls] = rows < cols ? rows : idle;
      for (int i = lane; i < (cols - rows) * kVecs; i += 32) zero_row(rows + i / kVecs, i % kVecs);
      fence_proxy_async_smem();
      // A block with rows that add nothing lands on a barrier of its own: those rows are
      // zeroed before the MMA warp hears of it, whatever their queries hold.
      uint64_t* bar = rare ? &q_raw[stage] : &q_full[stage];
      const bool whole = p.path == nullptr && nb == nodes;
      int boxes = nb;
      if (p.path != nullptr) {
        boxes = 0;
        for (int v = 0; v < nb; v += 32)
          boxes += __popc(__ballot_sync(0xffffffffu, v + lane < nb && node_at(n0 + v + lane) >= 0));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(boxes * G * 128 * C::kHalves));
      __syncwarp();
      const int c3 = p.cu != nullptr ? 0 : b, base = p.cu != nullptr ? static_cast<int>(s.row0) : 0;
      if (whole) {
        if (lane < C::kHalves)
          tma_load_4d(dst + lane * C::kHalfBytes, &qmap, bar, lane * 64, g * G, base + n0, c3);
      } else {
        for (int v = lane; v < nb; v += 32) {
          const int node = node_at(n0 + v);
          if (node < 0) continue;
          for (int hh = 0; hh < C::kHalves; ++hh)
            tma_load_4d(dst + hh * C::kHalfBytes + v * G * 128, &qmap_node, bar, hh * 64, g * G, base + node, c3);
        }
      }
      mbar_arrive(&l_full[ls]);
      if (rare) {
        const bool ok = wait_lanes(bar, static_cast<uint32_t>(raw_no++) & 1u, abort, wlim);
        if (!ok) {
          if (lane == 0) set_abort(abort, p.dev_err);
          return false;
        }
#pragma unroll
        for (int u = 0; u < kRowBlock / 32; ++u)
          if (u * 32 + lane < rows && nl[u] == -INFINITY)
            for (int c = 0; c < kVecs; ++c) zero_row(u * 32 + lane, c);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[stage]);
      }
      return true;
    };
    for_each_run(p, range, [&](int b, int t0, int n, const SeqInfo& s) -> bool {
      if (s.blocks == 1) return load(b, s, 0);
      for (int i0 = 0; i0 < n; i0 += kGroup)
        for (int qb = first_block(s, t0 + i0, nodes); qb < s.blocks; ++qb)
          if (!load(b, s, qb)) return false;
      return true;
    });
    if (bits) report(p.dev_err, bits);
    __syncwarp();
    if (lane == 0 && mine > 0) {              // the last copies have landed before the CTA exits
      int zero = 0;
      mbar_wait(&q_full[stage], static_cast<uint32_t>(mine - 1) & 1u, &zero);
    }
  } else if (warp >= kEpiWarp && warp < kKWarp) {
    // ================================================================ probabilities
    const int slot = (warp - kEpiWarp) / 4;   // this warpgroup's
    const int key = (warp & 3) * 32 + lane;   // TMEM lane = key of the tile
    const uint32_t t_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint64_t c2 = f2(p.scale_log2, p.scale_log2);
    int tile_no = 0, q_no = 0;
    uint32_t phase = 0;                       // parity to wait for on s_full
    auto fail = [&]() -> bool {
      if (lane == 0) set_abort(abort, p.dev_err);
      return false;
    };
    // Adds the block's probabilities to acc; row j of the block counts if j >= j_min.
    auto add_block = [&](int ls, int cols, int j_min, uint64_t (&acc)[2]) -> bool {
      const int idle = s_idle[ls];            // (the same in every lane; so is the branch, as the load wants it)
      if (!wait_lanes(&s_full[slot], phase, abort, wlim)) return false;
      phase ^= 1u;
      tc_fence_after();
      uint32_t zero = 0u;
      if (idle < kRowBlock) zero = tmem_ld1(t_addr + slot * kRowBlock + idle);
      if (__all_sync(0xffffffffu, j_min <= 0 & __uint_as_float(zero) == 0.f))
        add_columns<false>(t_addr + slot * kRowBlock, s_nlse[ls], cols, j_min, c2, acc);
      else
        add_columns<true>(t_addr + slot * kRowBlock, s_nlse[ls], cols, j_min, c2, acc);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_empty[slot]);
      return true;
    };
    auto old_weight = [&](int b, int t, const SeqInfo& s) -> float {
      const size_t at = (static_cast<size_t>(b) * p.Hkv + g) * (static_cast<size_t>(p.max_pages) * kPage) + t;
      return t < s.P && p.weight != nullptr ? p.weight[at] : 0.f;
    };
    auto write = [&](int b, int t, const SeqInfo& s, float old, const uint64_t (&acc)[2]) {
      float a, c, d, e;
      f2_split(acc[0], a, c);
      f2_split(acc[1], d, e);
      const size_t at = (static_cast<size_t>(b) * p.Hkv + g) * (static_cast<size_t>(p.max_pages) * kPage) + t;
      if (t < s.L) p.weight_out[at] = old + ((a + c) + (d + e));
    };
    for_each_run(p, range, [&](int b, int t0, int n, const SeqInfo& s) -> bool {
      if (s.blocks == 0) {                    // no rows: the old weights, nothing from the tensor cores
        for (int i = slot; i < n; i += kSlots) {
          const int t = (t0 + i) * kKeyTile + key;
          const uint64_t none[2] = {0ull, 0ull};
          write(b, t, s, old_weight(b, t, s), none);
        }
        return true;
      }
      // With one row block its lse stays for the whole run.
      const bool one = s.blocks == 1;
      for (int i0 = 0; i0 < n; i0 += kGroup) {
        const int m = min(kGroup, n - i0);
        const int i = (slot - tile_no) & (kSlots - 1);      // this warpgroup's tile of the group
        const int t = (t0 + i0 + i) * kKeyTile + key;
        float old = 0.f;
        if (i < m) old = old_weight(b, t, s);
        uint64_t acc[2] = {0ull, 0ull};
        for (int qb = first_block(s, t0 + i0, nodes); qb < s.blocks; ++qb) {
          const int ls = q_no % C::kLseStages;
          if ((!one || i0 == 0) &&
              !wait_lanes(&l_full[ls], static_cast<uint32_t>(q_no / C::kLseStages) & 1u, abort, wlim))
            return fail();
          const int cols = block_cols(s, qb, nodes, G);
          if (i < m && !add_block(ls, cols, (max(t - s.P, 0) - qb * nodes) * G, acc)) return fail();
          if (one && i0 + kGroup < n) break;
          __syncwarp();
          if (lane == 0) mbar_arrive(&l_empty[ls]);
          ++q_no;
        }
        if (i < m) write(b, t, s, old, acc);
        tile_no += m;
      }
      return true;
    });
  }
  tc_fence_before();
  __syncthreads();
  grid_dependents_launch();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

template <int D>
jf_status launch_weight(const CUtensorMap& km, const CUtensorMap& qm, const CUtensorMap& qn,
                        const WeightParams& p, int sms, cudaStream_t s) {
  static SmemAttr attr;
  if (!attr.ensure(weight_kernel<D>, Cfg<D>::kSmemBytes)) return JF_ERR_CUDA;
  const int ranges = std::max(1, sms / p.Hkv);
  const cudaError_t e = launch_pdl(weight_kernel<D>, dim3(static_cast<unsigned>(ranges * p.Hkv)), dim3(kThreads),
                                   Cfg<D>::kSmemBytes, s, km, qm, qn, p);
  return e == cudaSuccess ? JF_OK : JF_ERR_CUDA;
}

jf_status attention_weight_call(const void* q, const void* k_cache, const int32_t* block_table,
                                const int32_t* prefix_len, const int32_t* cu,
                                const int32_t* path, const int32_t* accept_len,
                                const float* lse, const float* weight, int32_t B, int32_t N,
                                int32_t T, int32_t Hq, int32_t Hkv, int32_t D,
                                int32_t page_size, int32_t max_pages, int32_t num_pages,
                                float scale, float* weight_out, int32_t* dev_err,
                                jf_stream_t stream) {
  if (q == nullptr || k_cache == nullptr || block_table == nullptr || prefix_len == nullptr ||
      lse == nullptr || weight_out == nullptr)
    return JF_ERR_INVALID_ARGUMENT;
  if (path != nullptr && accept_len == nullptr) return JF_ERR_INVALID_ARGUMENT;
  if (B < 1 || N < 1 || Hq < 1 || Hkv < 1 || max_pages < 1 || num_pages < 1 ||
      !(scale > 0.f) || !std::isfinite(scale))
    return JF_ERR_INVALID_ARGUMENT;
  if (N > JF_MAX_NODES || (D != 64 && D != 128) || page_size != kPage || Hq % Hkv != 0)
    return JF_ERR_UNSUPPORTED;
  if (B > 65535 || Hkv > 65535 || Hq / Hkv > 128 ||
      static_cast<long long>(max_pages) * kPage >= (1ll << 30) ||
      static_cast<long long>(num_pages) * kPage >= (1ll << 31) ||
      static_cast<long long>(N) * (Hq / Hkv) >= (1ll << 30))
    return JF_ERR_UNSUPPORTED;
  if (cu != nullptr && T < 1) return JF_ERR_INVALID_ARGUMENT;
  if (cu != nullptr && static_cast<long long>(T) + N >= (1ll << 31)) return JF_ERR_UNSUPPORTED;
  const size_t weight_bytes = sizeof(float) * static_cast<size_t>(B) * Hkv * max_pages * kPage;
  if (weight != nullptr && weight != weight_out && overlap(weight, weight_bytes, weight_out, weight_bytes))
    return JF_ERR_INVALID_ARGUMENT;
  if (!aligned_to(q, 16) || !aligned_to(k_cache, 16)) return JF_ERR_MISALIGNED;
  const int sms = current_sm_count();
  if (sms <= 0) return JF_ERR_CUDA;
  WeightParams p;
  p.block_table = block_table;
  p.prefix_len = prefix_len;
  p.path = path;
  p.accept_len = accept_len;
  p.cu = cu;
  p.lse = lse;
  p.weight = weight;
  p.weight_out = weight_out;
  p.dev_err = dev_err;
  p.T = cu != nullptr ? T : 0;
  p.B = B;
  p.N = N;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.nodes = kRowBlock / p.G;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  p.scale_log2 = scale * kLog2e;
  CUtensorMap km;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(Hkv),
                              static_cast<cuuint64_t>(num_pages) * kPage};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(Hkv) * D * 2};
  const cuuint32_t box[3] = {64, 1, kPage};
  if (!encode(&km, k_cache, 3, dims, strides, box)) return JF_ERR_CUDA;
  CUtensorMap qm, qn;
  const cuuint64_t rows = cu != nullptr ? static_cast<cuuint64_t>(T) : static_cast<cuuint64_t>(N);
  const cuuint64_t qdims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(Hq), rows,
                               cu != nullptr ? 1u : static_cast<cuuint64_t>(B)};
  const cuuint64_t qstrides[3] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(Hq) * D * 2,
                                  rows * Hq * D * 2};
  const cuuint32_t qbox[4] = {64, static_cast<cuuint32_t>(p.G), static_cast<cuuint32_t>(p.nodes), 1};
  const cuuint32_t qbox_node[4] = {64, static_cast<cuuint32_t>(p.G), 1, 1};
  if (!encode(&qm, q, 4, qdims, qstrides, qbox) || !encode(&qn, q, 4, qdims, qstrides, qbox_node)) return JF_ERR_CUDA;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return D == 128 ? launch_weight<128>(km, qm, qn, p, sms, s) : launch_weight<64>(km, qm, qn, p, sms, s);
}

}  // namespace
}  // namespace jf

extern "C" jf_status jf_attention_weight(
    const void* q, const void* k_cache, const int32_t* block_table, const int32_t* prefix_len,
    const int32_t* path, const int32_t* accept_len, const float* lse, const float* weight,
    int32_t B, int32_t N, int32_t Hq, int32_t Hkv, int32_t D, int32_t page_size,
    int32_t max_pages, int32_t num_pages, float scale, float* weight_out, int32_t* dev_err,
    jf_stream_t stream) {
  return jf::attention_weight_call(q, k_cache, block_table, prefix_len, nullptr, path, accept_len,
                                   lse, weight, B, N, 0, Hq, Hkv, D, page_size, max_pages,
                                   num_pages, scale, weight_out, dev_err, stream);
}

extern "C" jf_status jf_attention_weight_packed(
    const void* q, const void* k_cache, const int32_t* block_table, const int32_t* prefix_len,
    const int32_t* cu_seqlens, const int32_t* path, const int32_t* accept_len, const float* lse,
    const float* weight, int32_t B, int32_t N_max, int32_t T, int32_t Hq, int32_t Hkv, int32_t D,
    int32_t page_size, int32_t max_pages, int32_t num_pages, float scale, float* weight_out,
    int32_t* dev_err, jf_stream_t stream) {
  if (cu_seqlens == nullptr) return JF_ERR_INVALID_ARGUMENT;
  return jf::attention_weight_call(q, k_cache, block_table, prefix_len, cu_seqlens, path,
                                   accept_len, lse, weight, B, N_max, T, Hq, Hkv, D, page_size,
                                   max_pages, num_pages, scale, weight_out, dev_err, stream);
}
