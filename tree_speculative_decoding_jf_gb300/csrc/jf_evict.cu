// jf_evict.cu -- bounding the paged cache: which keys stay (by accumulated attention
// weight), and the move of their K/V rows to the front.
#include <algorithm>
#include <cmath>

#include "jf_common.cuh"
#include "jf_sm100.cuh"

namespace jf {
namespace {

constexpr int kPage = 16;

// ------------------------------------------------------------------------ selection

// One thread-block cluster per (sequence, kv-head) row; its CTAs take equal slices of the
// row and keep them on chip as 32-bit keys that order as the weights do, so the weights are
// read once.  The smallest kept key is found by counting: the keys' range is cut into 1024
// steps (2048 with 1024 threads), and the step that holds the wanted rank usually holds few
// enough keys to list and rank directly; otherwise it becomes the next range, down to one
// value (2^32 in four counts), of which the first by position stay.  (A count of a row of
// 32K takes 5,500 cycles; ranking a list goes with its square, 50,000 cycles at 1000 keys.)
// Then one pass makes a bit a key, and a thread a 32-key word puts the kept offsets together
// on chip, from where they are written side by side.
//
// What bounds the call is not the 8 bytes a key but, for a row of 32K in one CTA, in cycles:
// the load 10,800, the counts 4,700, the bits 4,000, the list 1,700, the positions 4,300;
// for few rows, the barriers between the steps.  256 rows of 32K: 30 us, of which the 256
// CTAs on 152 SMs take two rounds; 8 rows of 2304: 5.8 us, one call after the other.  (With a second pass of ballots for the positions, 1024
// steps and lists of 1024: 40 us, and 87 us where a step held 700 keys.)
// Keys that stay whatever they are (the first `sink`, the last `recent`) become kForced,
// above every weight, and the padding 0, below every one, so no pass tests positions.
constexpr int kSelShort = 8192;           // keys of a row that 512 threads take alone, ..
constexpr int kSelTwo = 20480;            // .. where two such CTAs share an SM, ..
constexpr int kSelRow = 32768;            // .. that 1024 threads take alone
constexpr int kSelMost = 192 * 1024 / 4;  // keys that fit on chip; longer slices are read again
constexpr int kSelPad = 128;              // a slice fills whole 128-key runs of a warp
constexpr int kSelList = 256;             // listed keys of a row
constexpr int kMaxCluster = 8;
constexpr uint32_t kForced = 0xffffffffu; // above every weight's key
constexpr uint32_t kNone = 0u;            // below every weight's key

__device__ __forceinline__ uint32_t weight_key(float w) {
  uint32_t u = __float_as_uint(w);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 1u;           // NaN: below every number
  if (u == 0x80000000u) u = 0u;                             // -0 == +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ uint32_t dsmem_ld_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// ONE: a cluster of one CTA; RESIDENT: the slices fit on chip.
template <int THREADS, bool ONE, bool RESIDENT>
__global__ void __launch_bounds__(THREADS, THREADS == 512 ? 3 : 1)
    select_kernel(const float* __restrict__ weight, const int32_t* __restrict__ seq_len, int Hkv,
                  int cap, int sink, int recent, int budget, int C, int32_t* __restrict__ keep,
                  int32_t* __restrict__ kept_len, int32_t* dev_err) {
  constexpr int kWarps = THREADS / 32, kMine = 2, kBins = kMine * THREADS;   // steps of a count
  constexpr int kBinBits = THREADS == 512 ? 10 : 11;
  static_assert(kBins == 1 << kBinBits, "a step each");
  extern __shared__ uint4 s_keys[];                         // this CTA's slice, four keys each
  __shared__ uint32_t s_hist[2][kBins];                     // this CTA's counts (two rounds' in turn)
  __shared__ uint32_t s_range[2];                           // min, max of this CTA
  __shared__ uint32_t s_count[4];                           // this CTA's: above the step, in it, listed; listed before it that stay
  __shared__ uint32_t s_warp[2][kWarps];
  __shared__ uint32_t s_bin[3];                             // the step, keys above it, keys in it
  __shared__ uint64_t s_list[kSelList];                     // key << 32 | ~position, this CTA's
  __shared__ uint64_t s_all[kSelList];                      // the row's
  __shared__ __align__(16) uint32_t s_in[RESIDENT ? kSelMost / 32 : 1];  // a bit a key: in the step
  __shared__ uint64_t s_cut;
  __shared__ __align__(16) uint32_t s_mask[RESIDENT ? kSelMost / 32 : 1];   // a bit a key: it stays
  __shared__ uint32_t s_scan[kWarps];
  grid_dependency_wait();
  const int rank = ONE ? 0 : static_cast<int>(cluster_ctarank());
  const int row = blockIdx.x / C, b = row / Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto row_sync = [&]() {
    if constexpr (ONE) __syncthreads();
    else cluster_sync();
  };
  // The word in every CTA of the row (`none` past the last), all on their way at once.
  uint32_t from[kMaxCluster];
  auto peers = [&](const uint32_t* local, uint32_t none) {
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      from[r] = none;
      if constexpr (ONE) {
        if (r == 0) from[r] = *local;
      } else {
        if (r < C) from[r] = dsmem_ld_u32(dsmem_addr(local, r));
      }
    }
  };
  int L = seq_len[b];
  if (L < 0 || L > cap) {
    if (tid == 0 && rank == 0 && row % Hkv == 0) report(dev_err, JF_DEVERR_BAD_PREFIX);
    L = max(0, min(L, cap));
  }
  int32_t* out = keep + static_cast<size_t>(row) * budget;
  if (tid == 0 && rank == 0 && row % Hkv == 0) kept_len[b] = min(L, budget);
  if (L <= budget) {                      // everything stays
    for (int j = rank * THREADS + tid; j < budget; j += C * THREADS) out[j] = j < L ? j : -1;
    grid_dependents_launch();
    return;
  }
  const uint32_t want = static_cast<uint32_t>(budget - sink - recent);   // of the keys that compete
  const int per = ((L + C - 1) / C + kSelPad - 1) / kSelPad * kSelPad;   // slice of this CTA
  const int t_lo = min(L, rank * per), n_slice = min(L, t_lo + per) - t_lo;
  const int c_lo = sink - t_lo, c_hi = L - recent - t_lo;   // its competing part, as offsets
  const float* ws = weight + static_cast<size_t>(row) * cap + t_lo;
  auto load_key = [&](int e) -> uint32_t {
    if (e >= n_slice) return kNone;
    return e >= c_lo && e < c_hi ? weight_key(ws[e]) : kForced;
  };
  auto load4 = [&](int i) -> uint4 {
    return make_uint4(load_key(4 * i), load_key(4 * i + 1), load_key(4 * i + 2), load_key(4 * i + 3));
  };
  auto keys4 = [&](int i) -> uint4 {
    if constexpr (RESIDENT) return s_keys[i];
    else return load4(i);
  };
  // Runs of 128 keys, which the warps take in order.
  const int runs = (n_slice + kSelPad - 1) / kSelPad, vecs = runs * (kSelPad / 4);

  // ---- the slice, and the range of the competing keys
  if (tid < 2) s_range[tid] = tid == 0 ? 0xffffffffu : 0u;
  uint32_t kmin = 0xffffffffu, kmax = 0u;
  // Vectors [va, vb) hold competing keys alone: four loads a thread on their way at once (a
  // test inside the loop kept them apart: 13,700 cycles a row of 32K; eight at once gain
  // nothing).
  const bool wide = (reinterpret_cast<uintptr_t>(ws) & 15u) == 0;
  const int va = wide ? min(vecs, (max(c_lo, 0) + 3) / 4) : 0;
  const int vb = wide ? max(va, max(min(c_hi, n_slice), 0) / 4) : 0;
  for (int j = tid; j < va + vecs - vb; j += THREADS) {     // the others, first: their latency passes under the bulk
    const int i = j < va ? j : j - va + vb;
    const uint4 k = load4(i);
    const uint32_t e[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (e[c] != kForced && e[c] != kNone) {
        kmin = min(kmin, e[c]);
        kmax = max(kmax, e[c]);
      }
    if constexpr (RESIDENT) s_keys[i] = k;
  }
  for (int i0 = va + tid; i0 < vb; i0 += THREADS * 4) {
    float4 f[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i0 + u * THREADS < vb) f[u] = __ldg(reinterpret_cast<const float4*>(ws) + i0 + u * THREADS);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i0 + u * THREADS < vb) {
        const uint4 k = make_uint4(weight_key(f[u].x), weight_key(f[u].y), weight_key(f[u].z), weight_key(f[u].w));
        kmin = min(min(kmin, min(k.x, k.y)), min(k.z, k.w));
        kmax = max(max(kmax, max(k.x, k.y)), max(k.z, k.w));
        if constexpr (RESIDENT) s_keys[i0 + u * THREADS] = k;
      }
  }
  for (int i = tid; i < kBins; i += THREADS) s_hist[0][i] = 0u;
  kmin = __reduce_min_sync(0xffffffffu, kmin);
  kmax = __reduce_max_sync(0xffffffffu, kmax);
  __syncthreads();
  if (lane == 0) {
    atomicMin(&s_range[0], kmin);
    atomicMax(&s_range[1], kmax);
  }
  row_sync();
  peers(&s_range[0], 0xffffffffu);
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r) kmin = min(kmin, from[r]);
  peers(&s_range[1], 0u);
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r) kmax = max(kmax, from[r]);

  // ---- kept: keys above lo + last; of the keys lo .. lo + last (the step), `need`
  uint32_t lo = kmin, last = kmax - kmin, need = want;
  int shift = max(0, 32 - __clz(last) - kBinBits);
  bool listed = false;
  if (want == 0u) {                       // nothing that competes stays: the step is empty
    lo = kForced - 1u;
    last = 0u;
  }
  for (int round = 0; want > 0u; ++round) {
    uint32_t* hist = s_hist[round & 1];
    auto tally = [&](uint32_t k) {
      const uint32_t d = k - lo;
      if (d <= last) atomicAdd(&hist[d >> shift], 1u);
    };
#pragma unroll 2
    for (int i = tid; i < vecs; i += THREADS) {
      const uint4 k = keys4(i);
      tally(k.x);
      tally(k.y);
      tally(k.z);
      tally(k.w);
    }
    row_sync();
    // The step where the count from above reaches `need`: kMine steps a thread, thread 0 the
    // highest.
    const int top = kBins - 1 - kMine * tid;
    uint32_t c[kMine], mine = 0u;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      c[i] = 0u;
      peers(&hist[top - i], 0u);
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) c[i] += from[r];
      mine += c[i];
    }
    for (int i = tid; i < kBins; i += THREADS) s_hist[(round & 1) ^ 1][i] = 0u;   // (read by nobody now)
    uint32_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) s_warp[0][warp] = incl;
    __syncthreads();
    uint32_t above = incl - mine;
    above += __reduce_add_sync(0xffffffffu, lane < warp ? s_warp[0][lane] : 0u);
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      if (above < need && above + c[i] >= need) {
        s_bin[0] = top - i;
        s_bin[1] = above;
        s_bin[2] = c[i];
      }
      above += c[i];
    }
    __syncthreads();
    need -= s_bin[1];
    lo += s_bin[0] << shift;
    last = min(last - (s_bin[0] << shift), (1u << shift) - 1u);
    listed = s_bin[2] <= kSelList;
    if (listed || shift == 0) break;
    shift = max(0, shift - kBinBits);
  }

  // Every CTA's listed keys into s_all; returns their number.
  auto gather_lists = [&]() -> uint32_t {
    peers(&s_count[2], 0u);
    uint32_t all = 0u;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      for (uint32_t i = tid; i < from[r]; i += THREADS) {
        const uint32_t* e = reinterpret_cast<const uint32_t*>(&s_list[i]);
        const uint32_t a = dsmem_ld_u32(dsmem_addr(e, r)), c = dsmem_ld_u32(dsmem_addr(e + 1, r));
        s_all[all + i] = (static_cast<uint64_t>(c) << 32) | a;
      }
      all += from[r];
    }
    return all;
  };
  const uint32_t hi = lo + last;
  const uint32_t not_first = 0xffffffffu - static_cast<uint32_t>(t_lo);   // ~position of offset 0
  auto entry = [&](uint32_t k, int e) -> uint64_t {   // of offset e in a list
    return (static_cast<uint64_t>(k) << 32) | (not_first - static_cast<uint32_t>(e));
  };
  if (tid == 0) s_count[2] = s_count[3] = 0u;
  __syncthreads();
  if constexpr (RESIDENT) {
    // ---- a bit a key: forced or above the step; keys in the step are listed, or (equal keys
    // without number) get bits of their own.  From here on the keys are not read again.
    uint8_t* up8 = reinterpret_cast<uint8_t*>(s_mask);
    uint32_t n_above = 0u, n_in = 0u;
#pragma unroll 2
    for (int i = tid; i < vecs; i += THREADS) {
      const uint4 k = s_keys[i];
      const uint32_t up = static_cast<uint32_t>(k.x > hi) | (k.y > hi) << 1 | (k.z > hi) << 2 | (k.w > hi) << 3;
      const uint32_t in = static_cast<uint32_t>(k.x - lo <= last) | (k.y - lo <= last) << 1 |
                          (k.z - lo <= last) << 2 | (k.w - lo <= last) << 3;
      const uint32_t up_next = __shfl_down_sync(0xffffffffu, up, 1);
      if ((lane & 1) == 0) up8[i >> 1] = static_cast<uint8_t>(up | up_next << 4);
      if constexpr (!ONE) n_above += __popc(up);
      if (listed) {
        const uint32_t e[4] = {k.x, k.y, k.z, k.w};
        if (in != 0u)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if ((in >> c) & 1u) s_list[atomicAdd(&s_count[2], 1u)] = entry(e[c], 4 * i + c);
      } else {
        const uint32_t in_next = __shfl_down_sync(0xffffffffu, in, 1);
        if ((lane & 1) == 0) reinterpret_cast<uint8_t*>(s_in)[i >> 1] = static_cast<uint8_t>(in | in_next << 4);
        if constexpr (!ONE) n_in += __popc(in);
      }
    }
    uint32_t at = 0u, in_before = 0u;     // kept and in-step keys of earlier CTAs, then threads
    if constexpr (ONE) {
      __syncthreads();
    } else {
      n_above = __reduce_add_sync(0xffffffffu, n_above);
      n_in = __reduce_add_sync(0xffffffffu, n_in);
      if (lane == 0) {
        s_warp[0][warp] = n_above;
        s_warp[1][warp] = n_in;
      }
      __syncthreads();
      if (tid < 2) {
        uint32_t v = 0u;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) v += s_warp[tid][i];
        s_count[tid] = v;
      }
      row_sync();
      peers(&s_count[0], 0u);
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        if (r < rank) at += from[r];
      peers(&s_count[1], 0u);
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        if (r < rank) in_before += from[r];
    }
    if (listed) {                         // of the step's keys, those with fewer than `need` before them stay
      const uint64_t* list = s_list;
      uint32_t all = 0u;
      if constexpr (ONE) {
        all = s_count[2];
      } else {
        list = s_all;
        all = gather_lists();
        __syncthreads();
      }
      for (uint32_t i = warp; i < all; i += kWarps) {
        const uint64_t x = list[i];
        uint32_t before = 0u;
        for (uint32_t j = lane; j < all; j += 32) before += list[j] > x;
        before = __reduce_add_sync(0xffffffffu, before);
        if (before < need && lane == 0) {
          const int e = static_cast<int>(not_first - static_cast<uint32_t>(x));   // offset in this slice
          if (e < 0) atomicAdd(&s_count[3], 1u);
          else if (e < n_slice) atomicOr(&s_mask[e >> 5], 1u << (e & 31));
        }
      }
      __syncthreads();
      at += s_count[3];
    }
    // ---- the kept offsets in order, gathered on chip, and written
    const int words = vecs / 8, mine = (words + THREADS - 1) / THREADS;
    const int w0 = min(words, tid * mine), w1 = min(words, w0 + mine);
    uint32_t sum = 0u;                    // kept keys, and in-step ones << 16 (a slice has fewer than 2^16)
    for (int w = w0; w < w1; ++w) sum += __popc(s_mask[w]) + (listed ? 0u : __popc(s_in[w]) << 16);
    uint32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    const uint32_t of_warp = lane < kWarps ? s_scan[lane] : 0u;
    const uint32_t prior = incl - sum + __reduce_add_sync(0xffffffffu, lane < warp ? of_warp : 0u);
    const uint32_t total = __reduce_add_sync(0xffffffffu, of_warp);
    uint32_t* offs = reinterpret_cast<uint32_t*>(s_keys);
    // Kept keys before in-step ones of rank n: all above, and the first `need` of the step.
    uint32_t n = in_before + (prior >> 16);
    const uint32_t in_kept = min(need, in_before);
    uint32_t to = (prior & 0xffffu) + (listed ? 0u : min(need, n) - in_kept);
    for (int w = w0; w < w1; ++w) {
      uint32_t m = s_mask[w];
      if (!listed) {
        uint32_t q = s_in[w];
        for (; q != 0u && n < need; ++n, q &= q - 1u) m |= q & (0u - q);
      }
      for (; m != 0u; m &= m - 1u) offs[to++] = 32u * w + __ffs(m) - 1u;
    }
    uint32_t kept = total & 0xffffu;
    if (!listed) {
      kept += min(need, in_before + (total >> 16)) - in_kept;
      at += in_kept;
    }
    __syncthreads();
    for (uint32_t i = tid; i < kept; i += THREADS) out[at + i] = t_lo + static_cast<int>(offs[i]);
  } else {
    // ---- longer slices, whose keys are read again.  Counts: forced keys and keys above the
    // step, keys in it; the latter listed
    const int per_warp = (runs + kWarps - 1) / kWarps;
    const int v_lo = min(runs, warp * per_warp) * 32, v_hi = min(runs, (warp + 1) * per_warp) * 32;
    uint32_t n_above = 0u, n_in = 0u;
#pragma unroll 2
    for (int i = v_lo + lane; i < v_hi; i += 32) {
      const uint4 k = keys4(i);
      n_above += (k.x > hi) + (k.y > hi) + (k.z > hi) + (k.w > hi);
      if (k.x - lo <= last || k.y - lo <= last || k.z - lo <= last || k.w - lo <= last) {
        const uint32_t e[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (e[c] - lo <= last) {
            ++n_in;
            if (listed) s_list[atomicAdd(&s_count[2], 1u)] = entry(e[c], 4 * i + c);
          }
      }
    }
    n_above = __reduce_add_sync(0xffffffffu, n_above);
    n_in = __reduce_add_sync(0xffffffffu, n_in);
    if (lane == 0) {
      s_warp[0][warp] = n_above;
      s_warp[1][warp] = n_in;
    }
    __syncthreads();
    if (tid < 2) {
      uint32_t v = 0u;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) v += s_warp[tid][i];
      s_count[tid] = v;
    }
    row_sync();
    uint32_t at = 0u, in_before = 0u;       // kept and in-step keys before this warp's runs
    peers(&s_count[0], 0u);
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      if (r < rank) at += from[r];
    peers(&s_count[1], 0u);
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      if (r < rank) in_before += from[r];
    for (int v = 0; v < warp; ++v) {
      at += s_warp[0][v];
      in_before += s_warp[1][v];
    }
    uint64_t cut = ~0ull;
    if (listed) {                           // the step's keys that stay: `cut` and what ranks before it
      const uint32_t all = gather_lists();
      __syncthreads();
      for (uint32_t i = warp; i < all; i += kWarps) {
        const uint64_t e = s_all[i];
        uint32_t before = 0u;
        for (uint32_t j = lane; j < all; j += 32) before += s_all[j] > e;
        before = __reduce_add_sync(0xffffffffu, before);
        if (before == need - 1u && lane == 0) s_cut = e;
      }
      __syncthreads();
      cut = s_cut;
      uint32_t n = 0u;
      for (uint32_t i = lane; i < all; i += 32) {
        const uint64_t e = s_all[i];
        n += e >= cut && 0xffffffffu - static_cast<uint32_t>(e) < static_cast<uint32_t>(t_lo + 4 * v_lo);
      }
      at += __reduce_add_sync(0xffffffffu, n);
    } else {                                // one value: the first by position stay
      at += min(need, in_before);
    }
    // ---- the kept positions, in order: a lane's four are consecutive
#pragma unroll 2
    for (int i = v_lo + lane; i < v_hi; i += 32) {
      const uint4 k = keys4(i);
      const uint32_t e[4] = {k.x, k.y, k.z, k.w};
      uint32_t stay = 0u, in = 0u;          // a bit a key
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        stay |= static_cast<uint32_t>(e[c] > hi) << c;
        in |= static_cast<uint32_t>(e[c] - lo <= last) << c;
      }
      const uint32_t below = (1u << lane) - 1u;
      if (__any_sync(0xffffffffu, in != 0u)) {
        uint32_t before = 0u, all = 0u;     // in-step keys of earlier lanes, of all
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t m = __ballot_sync(0xffffffffu, (in >> c) & 1u);
          before += __popc(m & below);
          all += __popc(m);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if ((in >> c) & 1u) {
            const uint64_t x = entry(e[c], 4 * i + c);
            if (listed ? x >= cut : in_before + before < need) stay |= 1u << c;
            ++before;
          }
        in_before += all;
      }
      uint32_t to = at, all = 0u;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t m = __ballot_sync(0xffffffffu, (stay >> c) & 1u);
        to += __popc(m & below);
        all += __popc(m);
      }
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if ((stay >> c) & 1u) out[to++] = t_lo + 4 * i + c;
      at += all;
    }
  }
  grid_dependents_launch();
  if constexpr (!ONE) cluster_sync();     // nobody leaves while its lists may be read
}

// ------------------------------------------------------------------------ eviction

constexpr int kEvictHeld = 4;             // 16-byte vectors a thread moves at a time
constexpr int kEvictWeights = 8;          // weights a thread moves at a time

struct EvictParams {
  uint16_t* k_cache;
  uint16_t* v_cache;
  const int32_t* block_table;
  const int32_t* new_table;   // == block_table in place
  const int32_t* seq_len;
  const int32_t* keep;
  const int32_t* kept_len;
  const float* weight;
  float* weight_out;
  int32_t* dev_err;
  int Hkv, D, budget, max_pages, num_pages;
  int kv_in_place, weight_in_place;
};

// One CTA moves one byte slice (VECS 16-byte vectors) of K or V of one kv-head (the last CTA
// of a head: the weights), over its range of kept rows; bound by the bytes, read once and
// written once.
//
// In place the rows go in rising order, in batches, by one CTA a slice (32-byte pieces of
// the rows would spread further, but share the 64-byte accesses of HBM).  keep[j] >= j rises
// strictly, so a row's new place lies below every later row's old one: reading a batch
// whole before any of it is written gives the sequential result, and the next batch may be
// read before this one is written.  Into other pages, whole rows move in any order and the
// rows are split over CTAs.
//
// A row's pool rows (page * 16 + slot) are looked up once, by one thread, two batches ahead.
template <int VECS, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) evict_kernel(const EvictParams p) {
  constexpr int kRows = THREADS / VECS;               // rows a pass of the CTA touches
  constexpr int kBatch = kRows * kEvictHeld;
  static_assert(kBatch <= THREADS, "a thread looks up one row of a batch");
  // Four: a slot is written again only when every thread is done with its last batch.
  __shared__ int s_src[4][kBatch], s_dst[4][kBatch];
  grid_dependency_wait();
  const int slices = p.D / 8 / VECS, parts = 2 * slices + (p.weight_out != nullptr ? 1 : 0);
  const int part = blockIdx.x % parts, row = blockIdx.x / parts;
  const int b = row / p.Hkv, g = row % p.Hkv, tid = threadIdx.x;
  const int cap = p.max_pages * kPage;
  int bits = 0;
  int L = p.seq_len[b], n = p.kept_len[b];
  if (L < 0 || L > cap) bits |= JF_DEVERR_BAD_PREFIX;
  L = max(0, min(L, cap));
  if (n < 0 || n > min(L, p.budget)) bits |= JF_DEVERR_BAD_PATH;
  n = max(0, min(n, min(L, p.budget)));
  const int32_t* keep = p.keep + static_cast<size_t>(row) * p.budget;
  // Ranges of whole batches, so that CTAs differ by at most one.
  const int batches = (n + kBatch - 1) / kBatch, splits = gridDim.y;
  const int j0 = static_cast<int>(static_cast<long long>(batches) * blockIdx.y / splits) * kBatch;
  const int j1 = min(n, static_cast<int>(static_cast<long long>(batches) * (blockIdx.y + 1) / splits) * kBatch);
  auto source = [&](int j) -> int {       // -1: a malformed entry
    const int t = keep[j], before = j > 0 ? keep[j - 1] : -1;
    if (t >= j && t < L && t > before) return t;
    bits |= JF_DEVERR_BAD_PATH;
    return -1;
  };
  if (part == 2 * slices) {
    const float* w = p.weight + static_cast<size_t>(row) * cap;
    float* wo = p.weight_out + static_cast<size_t>(row) * cap;
    // (in place, one CTA goes through all rows in order)
    const int w0 = p.weight_in_place ? 0 : j0, w1 = p.weight_in_place ? (blockIdx.y == 0 ? n : 0) : j1;
    for (int base = w0; base < w1; base += THREADS * kEvictWeights) {
      float v[kEvictWeights];
      int t[kEvictWeights];
#pragma unroll
      for (int u = 0; u < kEvictWeights; ++u) {
        const int j = base + u * THREADS + tid;
        t[u] = j < w1 ? source(j) : -1;
        if (t[u] >= 0) v[u] = w[t[u]];
      }
      if (p.weight_in_place) __syncthreads();
#pragma unroll
      for (int u = 0; u < kEvictWeights; ++u)
        if (t[u] >= 0) wo[base + u * THREADS + tid] = v[u];
      if (p.weight_in_place) __syncthreads();
    }
  } else {
    uint4* cache = reinterpret_cast<uint4*>(part < slices ? p.k_cache : p.v_cache);
    const int32_t* bt = p.block_table + static_cast<size_t>(b) * p.max_pages;
    const int32_t* nt = p.new_table + static_cast<size_t>(b) * p.max_pages;
    const int r = tid / VECS, col = (part % slices) * VECS + tid % VECS;
    const int row_vecs = p.D / 8;
    // Pool rows of row j of a batch into its slot of s_src / s_dst; -1: not moved.
    auto look_up = [&](int base, int slot) {
      if (tid >= kBatch) return;
      const int j = base + tid;
      int from = -1, to = -1;
      if (j < j1) {
        const int t = source(j);
        if (t >= 0 && !(p.kv_in_place && t == j)) {
          const int ps = bt[t / kPage], pd = nt[j / kPage];
          if (ps >= 0 && ps < p.num_pages && pd >= 0 && pd < p.num_pages) {
            from = ps * kPage + t % kPage;
            to = pd * kPage + j % kPage;
          } else {
            bits |= JF_DEVERR_BAD_PAGE;
          }
        }
      }
      s_src[slot][tid] = from;
      s_dst[slot][tid] = to;
    };
    auto vec_at = [&](int pool_row) -> uint4* {
      return cache + (static_cast<size_t>(pool_row) * p.Hkv + g) * row_vecs + col;
    };
    uint4 v[kEvictHeld], next[kEvictHeld];
    auto read = [&](int slot, uint4 (&x)[kEvictHeld]) {
#pragma unroll
      for (int u = 0; u < kEvictHeld; ++u) {
        const int from = s_src[slot][u * kRows + r];
        if (from >= 0) x[u] = *vec_at(from);
      }
    };
    look_up(j0, 0);
    look_up(j0 + kBatch, 1);
    __syncthreads();
    read(0, next);
    int slot = 0;
    for (int base = j0; base < j1; base += kBatch) {
#pragma unroll
      for (int u = 0; u < kEvictHeld; ++u) v[u] = next[u];
      look_up(base + 2 * kBatch, (slot + 2) & 3);
      read((slot + 1) & 3, next);
      __syncthreads();                    // every thread has read this batch, and the one after
#pragma unroll
      for (int u = 0; u < kEvictHeld; ++u) {
        const int to = s_dst[slot][u * kRows + r];
        if (to >= 0) *vec_at(to) = v[u];
      }
      slot = (slot + 1) & 3;
    }
  }
  if (bits) report(p.dev_err, bits);
  grid_dependents_launch();
}

}  // namespace
}  // namespace jf

extern "C" jf_status jf_select_kept(const float* weight, const int32_t* seq_len, int32_t B,
                                    int32_t Hkv, int32_t capacity, int32_t sink, int32_t recent,
                                    int32_t budget, int32_t* keep, int32_t* kept_len,
                                    int32_t* dev_err, jf_stream_t stream) {
  using namespace jf;
  if (weight == nullptr || seq_len == nullptr || keep == nullptr || kept_len == nullptr)
    return JF_ERR_INVALID_ARGUMENT;
  if (B < 1 || Hkv < 1 || capacity < 1 || budget < 1 || sink < 0 || recent < 0 ||
      static_cast<long long>(sink) + recent > budget)
    return JF_ERR_INVALID_ARGUMENT;
  if (capacity > (1 << 30) || budget > (1 << 30) || static_cast<long long>(B) * Hkv > (1ll << 27))
    return JF_ERR_UNSUPPORTED;
  // (every CTA of a sequence reads its length, at a time of its own; CTAs of one cluster that
  // saw different ones would wait for each other)
  const long long rows = static_cast<long long>(B) * Hkv;
  const size_t len_bytes = sizeof(int32_t) * static_cast<size_t>(B);
  if (overlap(kept_len, len_bytes, seq_len, len_bytes) ||
      overlap(keep, sizeof(int32_t) * static_cast<size_t>(rows) * static_cast<size_t>(budget), seq_len, len_bytes))
    return JF_ERR_INVALID_ARGUMENT;
  const int sms = current_sm_count();
  if (sms <= 0) return JF_ERR_CUDA;
  // A row up to kSelRow is one CTA: no exchanges.  Short ones take 512 threads (8 rows of
  // 2304: 5.8 us against 6.2 with 1024 and 9.1 in clusters of two; 256 rows, 7.0 against 11.6),
  // longer ones 1024 (80 rows of 16384: 10.1 against 12.1), unless there are more rows than
  // SMs and two CTAs of 512 fit on each (256 rows of 16384: 16.2 against 19.3; of 20480: 19.8
  // against 21.8).
  // Longer rows are clusters of CTAs of 512 threads, with slices up to kSelTwo (256 rows of
  // 64K: 84 us in fours, 92 in twos, 87 in twos of 1024 threads; 200 rows of 40000: 46 in
  // twos, 56 in fours); of eight where every CTA has an SM of its own (8 rows of 128K: 18 us
  // against 25 in fours of 1024; but 32 rows: 28 against 22 in fours), and past 4 kSelRow keys
  // whatever their number, so that a slice stays within kSelRow as long as it can.
  int C = 1;
  if (capacity > kSelRow)
    while (C < kMaxCluster && (capacity > C * kSelRow || (capacity > C * kSelTwo && (C < 4 || rows * 2 * C <= sms)))) C *= 2;
  const bool wide = C == 1 && capacity > (rows > sms ? kSelTwo : kSelShort);
  const int slice = ((capacity + C - 1) / C + kSelPad - 1) / kSelPad * kSelPad;
  const bool resident = slice <= kSelMost;
  auto* kernel = wide       ? select_kernel<1024, true, true>
                 : C == 1   ? select_kernel<512, true, true>
                 : resident ? select_kernel<512, false, true>
                            : select_kernel<512, false, false>;
  if (resident) {
    static SmemAttr attr[3];
    if (!attr[wide ? 2 : C == 1 ? 1 : 0].ensure(kernel, kSelMost * sizeof(uint32_t))) return JF_ERR_CUDA;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * C));
  cfg.blockDim = dim3(wide ? 1024 : 512);
  cfg.dynamicSmemBytes = resident ? static_cast<size_t>(slice) * sizeof(uint32_t) : 0;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = static_cast<unsigned>(C);
  attrs[1].val.clusterDim.y = 1;
  attrs[1].val.clusterDim.z = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, weight, seq_len, Hkv, capacity, sink, recent,
                                           budget, C, keep, kept_len, dev_err);
  return e == cudaSuccess ? JF_OK : JF_ERR_CUDA;
}

extern "C" jf_status jf_evict_kv(void* k_cache, void* v_cache, const int32_t* block_table,
                                 const int32_t* seq_len, const int32_t* keep,
                                 const int32_t* kept_len, const int32_t* new_block_table,
                                 const float* weight, float* weight_out, int32_t B, int32_t Hkv,
                                 int32_t D, int32_t budget, int32_t page_size, int32_t max_pages,
                                 int32_t num_pages, int32_t* dev_err, jf_stream_t stream) {
  using namespace jf;
  if (k_cache == nullptr || v_cache == nullptr || block_table == nullptr || seq_len == nullptr ||
      keep == nullptr || kept_len == nullptr || (weight == nullptr) != (weight_out == nullptr))
    return JF_ERR_INVALID_ARGUMENT;
  if (B < 1 || Hkv < 1 || budget < 1 || max_pages < 1 || num_pages < 1) return JF_ERR_INVALID_ARGUMENT;
  if (kept_len == seq_len) return JF_ERR_INVALID_ARGUMENT;
  if ((D != 64 && D != 128) || page_size != kPage) return JF_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * Hkv > (1ll << 26) || max_pages > (1 << 26) || budget > (1 << 30) ||
      static_cast<long long>(num_pages) * kPage >= (1ll << 31))
    return JF_ERR_UNSUPPORTED;
  const size_t weight_bytes = sizeof(float) * static_cast<size_t>(B) * Hkv * max_pages * kPage;
  if (weight != nullptr && weight != weight_out && overlap(weight, weight_bytes, weight_out, weight_bytes))
    return JF_ERR_INVALID_ARGUMENT;
  if (!aligned_to(k_cache, 16) || !aligned_to(v_cache, 16)) return JF_ERR_MISALIGNED;
  const int sms = current_sm_count();
  if (sms <= 0) return JF_ERR_CUDA;
  EvictParams p;
  p.k_cache = static_cast<uint16_t*>(k_cache);
  p.v_cache = static_cast<uint16_t*>(v_cache);
  p.block_table = block_table;
  p.kv_in_place = new_block_table == nullptr || new_block_table == block_table;
  p.weight_in_place = weight == weight_out;
  p.new_table = new_block_table == nullptr ? block_table : new_block_table;
  p.seq_len = seq_len;
  p.keep = keep;
  p.kept_len = kept_len;
  p.weight = weight;
  p.weight_out = weight_out;
  p.dev_err = dev_err;
  p.Hkv = Hkv;
  p.D = D;
  p.budget = budget;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  // In place: 64-byte slices, one CTA of 512 threads each (few CTAs, so each holds more on
  // its way: 103 us against 134 us with 256 threads on 16384 of 33024 keys, 8 x 4 heads).
  // Into other pages: whole rows, split so that every SM gets about eight CTAs (two rounds
  // of the four that fit).
  const int vecs = p.kv_in_place ? 4 : D / 8, threads = p.kv_in_place ? 512 : 256;
  const int batch = threads / vecs * kEvictHeld;
  const unsigned parts = 2 * (D / 8 / vecs) + (weight_out != nullptr ? 1 : 0);
  const long long units = static_cast<long long>(B) * Hkv * parts;
  long long splits = 1;
  if (!p.kv_in_place)
    splits = std::max<long long>(1, std::min<long long>((budget + batch - 1) / batch, (8ll * sms + units - 1) / units));
  const dim3 grid(static_cast<unsigned>(units), static_cast<unsigned>(std::min<long long>(splits, 65535)));
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = vecs == 4   ? launch_pdl(evict_kernel<4, 512>, grid, dim3(threads), 0, s, p)
                        : vecs == 8 ? launch_pdl(evict_kernel<8, 256>, grid, dim3(threads), 0, s, p)
                                    : launch_pdl(evict_kernel<16, 256>, grid, dim3(threads), 0, s, p);
  return e == cudaSuccess ? JF_OK : JF_ERR_CUDA;
}
