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
// steps, and the step that holds the wanted rank usually holds few enough keys to list and
// rank directly; otherwise it becomes the next range, down to one value (2^32 in four
// counts), of which the first by position stay.  What bounds the call is the number of such
// row-wide steps and their barriers, not the 8 bytes a key.
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelSlice = 8192;           // keys of a CTA's slice, while a cluster of 8 suffices
constexpr int kSelMost = 200 * 1024 / 4;  // keys that fit on chip; longer slices are read again
constexpr int kBinBits = 10;
constexpr int kBins = 1 << kBinBits;
constexpr int kSelList = 1024;            // listed keys of a row
constexpr int kMaxCluster = 8;
constexpr uint32_t kForced = 0xffffffffu; // above every weight's key

__device__ __forceinline__ uint32_t weight_key(float w) {
  uint32_t u = __float_as_uint(w);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0u;           // NaN: below everything
  if (u == 0x80000000u) u = 0u;                             // -0 == +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ uint32_t dsmem_ld_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

template <bool ONE, bool RESIDENT>   // a cluster of one CTA; slices fit on chip
__global__ void __launch_bounds__(kSelThreads, 3)
    select_kernel(const float* __restrict__ weight, const int32_t* __restrict__ seq_len, int Hkv,
                  int cap, int sink, int recent, int budget, int C,
                  int32_t* __restrict__ keep, int32_t* __restrict__ kept_len, int32_t* dev_err) {
  extern __shared__ uint32_t s_keys[];                      // this CTA's slice
  __shared__ uint32_t s_hist[2][kBins];                     // this CTA's counts (two rounds' in turn)
  __shared__ uint32_t s_range[2];                           // min, max of this CTA
  __shared__ uint32_t s_count[3];                           // above the step, in it, listed (this CTA)
  __shared__ uint32_t s_warp[2][kSelWarps];
  __shared__ uint32_t s_bin[3];                             // the step, keys above it, keys in it
  __shared__ uint64_t s_list[kSelList];                     // key << 32 | ~position, this CTA's
  __shared__ uint64_t s_all[kSelList];                      // the row's
  __shared__ uint64_t s_cut;
  grid_dependency_wait();
  const int rank = ONE ? 0 : static_cast<int>(cluster_ctarank());
  const int row = blockIdx.x / C, b = row / Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto row_sync = [&]() {
    if constexpr (ONE) __syncthreads();
    else cluster_sync();
  };
  // The word in every CTA of the row (0 past the last), all on their way at once.
  auto peers = [&](const uint32_t* local, uint32_t (&v)[kMaxCluster], uint32_t none) {
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      v[r] = none;
      if constexpr (ONE) {
        if (r == 0) v[r] = *local;
      } else {
        if (r < C) v[r] = dsmem_ld_u32(dsmem_addr(local, r));
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
    for (int j = rank * kSelThreads + tid; j < budget; j += C * kSelThreads) out[j] = j < L ? j : -1;
    grid_dependents_launch();
    return;
  }
  const float* w = weight + static_cast<size_t>(row) * cap;
  const uint32_t want = static_cast<uint32_t>(budget - sink - recent);   // of the keys that compete
  const int per = ((L + C - 1) / C + 31) & ~31;             // slice of this CTA
  const int t_lo = min(L, rank * per), t_hi = min(L, t_lo + per);
  const int c_lo = max(t_lo, min(sink, t_hi)), c_hi = max(c_lo, min(t_hi, L - recent));   // its competing part
  // Keys that stay whatever they are (the first `sink`, the last `recent`) count as kForced.
  // Positions below are offsets in the slice.
  const int n_slice = t_hi - t_lo, e_lo = c_lo - t_lo, e_hi = c_hi - t_lo;
  const float* ws = w + t_lo;
  auto key_of = [&](int e) -> uint32_t {
    if constexpr (RESIDENT) return s_keys[e];
    else return e >= e_lo && e < e_hi ? weight_key(ws[e]) : kForced;
  };

  // ---- the slice, and the range of the competing keys
  if (tid < 2) s_range[tid] = tid == 0 ? 0xffffffffu : 0u;
  uint32_t kmin = 0xffffffffu, kmax = 0u;
#pragma unroll 8
  for (int e = tid; e < n_slice; e += kSelThreads) {
    uint32_t k = weight_key(ws[e]);
    const bool in = e >= e_lo && e < e_hi;
    kmin = min(kmin, in ? k : 0xffffffffu);
    kmax = max(kmax, in ? k : 0u);
    if constexpr (RESIDENT) s_keys[e] = in ? k : kForced;
  }
  for (int i = tid; i < kBins; i += kSelThreads) s_hist[0][i] = 0u;
  kmin = __reduce_min_sync(0xffffffffu, kmin);
  kmax = __reduce_max_sync(0xffffffffu, kmax);
  __syncthreads();
  if (lane == 0) {
    atomicMin(&s_range[0], kmin);
    atomicMax(&s_range[1], kmax);
  }
  row_sync();
  uint32_t from[kMaxCluster];
  peers(&s_range[0], from, 0xffffffffu);
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r) kmin = min(kmin, from[r]);
  peers(&s_range[1], from, 0u);
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
#pragma unroll 4
    for (int e = e_lo + tid; e < e_hi; e += kSelThreads) {
      const uint32_t d = key_of(e) - lo;
      if (d <= last) atomicAdd(&hist[d >> shift], 1u);
    }
    row_sync();
    // The step where the count from above reaches `need`: two steps a thread, thread 0 the
    // highest.
    const int top = kBins - 1 - 2 * tid;
    uint32_t c0 = 0u, c1 = 0u;
    peers(&hist[top], from, 0u);
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) c0 += from[r];
    peers(&hist[top - 1], from, 0u);
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) c1 += from[r];
    for (int i = tid; i < kBins; i += kSelThreads) s_hist[(round & 1) ^ 1][i] = 0u;   // (read by nobody now)
    uint32_t incl = c0 + c1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) s_warp[0][warp] = incl;
    __syncthreads();
    uint32_t above = incl - c0 - c1;
    for (int v = 0; v < warp; ++v) above += s_warp[0][v];
    if (above < need && above + c0 >= need) {
      s_bin[0] = top;
      s_bin[1] = above;
      s_bin[2] = c0;
    } else if (above + c0 < need && above + c0 + c1 >= need) {
      s_bin[0] = top - 1;
      s_bin[1] = above + c0;
      s_bin[2] = c1;
    }
    __syncthreads();
    need -= s_bin[1];
    lo += s_bin[0] << shift;
    last = min(last - (s_bin[0] << shift), (1u << shift) - 1u);
    listed = s_bin[2] <= kSelList;
    if (listed || shift == 0) break;
    shift = max(0, shift - kBinBits);
  }

  // ---- counts: forced keys and keys above the step, keys in it; the latter listed
  const int seg = ((n_slice + kSelWarps - 1) / kSelWarps + 31) & ~31;
  const int seg_lo = min(n_slice, warp * seg), seg_hi = min(n_slice, seg_lo + seg);
  const uint32_t hi = lo + last;
  if (tid == 0) s_count[2] = 0u;
  __syncthreads();
  uint32_t n_above = 0u, n_in = 0u;
  const uint32_t not_first = 0xffffffffu - static_cast<uint32_t>(t_lo);   // ~position of offset 0
#pragma unroll 4
  for (int e = seg_lo + lane; e < seg_hi; e += 32) {
    const uint32_t k = key_of(e);
    n_above += k > hi;
    if (k - lo <= last) {
      ++n_in;
      if (listed) s_list[atomicAdd(&s_count[2], 1u)] = (static_cast<uint64_t>(k) << 32) | (not_first - static_cast<uint32_t>(e));
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
    for (int i = 0; i < kSelWarps; ++i) v += s_warp[tid][i];
    s_count[tid] = v;
  }
  row_sync();
  uint32_t at = 0u, in_before = 0u;       // kept and in-step keys before this warp's segment
  peers(&s_count[0], from, 0u);
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r)
    if (r < rank) at += from[r];
  peers(&s_count[1], from, 0u);
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r)
    if (r < rank) in_before += from[r];
  for (int v = 0; v < warp; ++v) {
    at += s_warp[0][v];
    in_before += s_warp[1][v];
  }
  uint64_t cut = ~0ull;
  if (listed) {                           // the step's keys that stay: `cut` and what ranks before it
    uint32_t all = 0u;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      for (uint32_t i = tid; i < from[r]; i += kSelThreads) {
        if constexpr (ONE) {
          s_all[all + i] = s_list[i];
        } else {
          const uint32_t* e = reinterpret_cast<const uint32_t*>(&s_list[i]);
          const uint32_t a = dsmem_ld_u32(dsmem_addr(e, r)), c = dsmem_ld_u32(dsmem_addr(e + 1, r));
          s_all[all + i] = (static_cast<uint64_t>(c) << 32) | a;
        }
      }
      all += from[r];
    }
    __syncthreads();
    for (uint32_t i = warp; i < all; i += kSelWarps) {
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
      n += e >= cut && 0xffffffffu - static_cast<uint32_t>(e) < static_cast<uint32_t>(t_lo + seg_lo);
    }
    at += __reduce_add_sync(0xffffffffu, n);
  } else {                                // one value: the first by position stay
    at += min(need, in_before);
  }
  const uint32_t below = (1u << lane) - 1u;
#pragma unroll 4
  for (int e0 = seg_lo; e0 < seg_hi; e0 += 32) {
    const int e = e0 + lane;
    uint32_t k = 0u;                      // (past the end: below everything that stays)
    bool live = e < seg_hi;
    if (live) k = key_of(e);
    bool stay = live && k > hi;
    const bool in = live && k - lo <= last;
    const uint32_t mi = __ballot_sync(0xffffffffu, in);
    if (mi != 0u) {
      if (listed) stay = stay || (in && ((static_cast<uint64_t>(k) << 32) | (not_first - static_cast<uint32_t>(e))) >= cut);
      else stay = stay || (in && in_before + __popc(mi & below) < need);
      in_before += __popc(mi);
    }
    const uint32_t ms = __ballot_sync(0xffffffffu, stay);
    if (stay) out[at + __popc(ms & below)] = t_lo + e;
    at += __popc(ms);
  }
  grid_dependents_launch();
  if constexpr (!ONE) cluster_sync();     // nobody leaves while its lists may be read
}

// ------------------------------------------------------------------------ eviction

constexpr int kEvictThreads = 256;
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
template <int VECS>
__global__ void __launch_bounds__(kEvictThreads, 4) evict_kernel(const EvictParams p) {
  constexpr int kRows = kEvictThreads / VECS;               // rows a pass of the CTA touches
  constexpr int kBatch = kRows * kEvictHeld;
  static_assert(kBatch <= kEvictThreads, "a thread looks up one row of a batch");
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
    for (int base = w0; base < w1; base += kEvictThreads * kEvictWeights) {
      float v[kEvictWeights];
      int t[kEvictWeights];
#pragma unroll
      for (int u = 0; u < kEvictWeights; ++u) {
        const int j = base + u * kEvictThreads + tid;
        t[u] = j < w1 ? source(j) : -1;
        if (t[u] >= 0) v[u] = w[t[u]];
      }
      if (p.weight_in_place) __syncthreads();
#pragma unroll
      for (int u = 0; u < kEvictWeights; ++u)
        if (t[u] >= 0) wo[base + u * kEvictThreads + tid] = v[u];
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
  const int sms = current_sm_count();
  if (sms <= 0) return JF_ERR_CUDA;
  const long long rows = static_cast<long long>(B) * Hkv;
  // The smallest cluster whose slices stay at kSelSlice keys; with few rows, more CTAs a row
  // while the machine has room for them.
  int C = 1;
  while (C < 8 && (capacity > C * kSelSlice || (rows * C * 2 <= sms && capacity > C * 2048))) C *= 2;
  const int slice = ((capacity + C - 1) / C + 31) & ~31;
  const int resident = slice <= kSelMost;
  const size_t smem = resident ? static_cast<size_t>(slice) * sizeof(uint32_t) : 0;
  // (a slice of a single CTA is at most 8192 keys, so it always fits)
  auto* kernel = C == 1 ? select_kernel<true, true> : resident ? select_kernel<false, true> : select_kernel<false, false>;
  if (resident) {
    static SmemAttr attr1, attr;
    if (!(C == 1 ? attr1 : attr).ensure(kernel, kSelMost * sizeof(uint32_t))) return JF_ERR_CUDA;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * C));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
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
  if (static_cast<long long>(B) * Hkv > (1ll << 26) || max_pages > (1 << 26) || budget > (1 << 30))
    return JF_ERR_UNSUPPORTED;
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
  // In place: 64-byte slices, one CTA each.  Into other pages: whole rows, split so that
  // every SM gets about eight CTAs (two rounds of the four that fit).
  const int vecs = p.kv_in_place ? 4 : D / 8;
  const int batch = kEvictThreads / vecs * kEvictHeld;
  const unsigned parts = 2 * (D / 8 / vecs) + (weight_out != nullptr ? 1 : 0);
  const long long units = static_cast<long long>(B) * Hkv * parts;
  long long splits = 1;
  if (!p.kv_in_place)
    splits = std::max<long long>(1, std::min<long long>((budget + batch - 1) / batch, (8ll * sms + units - 1) / units));
  const dim3 grid(static_cast<unsigned>(units), static_cast<unsigned>(std::min<long long>(splits, 65535)));
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = vecs == 4   ? launch_pdl(evict_kernel<4>, grid, dim3(kEvictThreads), 0, s, p)
                        : vecs == 8 ? launch_pdl(evict_kernel<8>, grid, dim3(kEvictThreads), 0, s, p)
                                    : launch_pdl(evict_kernel<16>, grid, dim3(kEvictThreads), 0, s, p);
  return e == cudaSuccess ? JF_OK : JF_ERR_CUDA;
}
