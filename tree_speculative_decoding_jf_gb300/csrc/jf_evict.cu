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
// row.  Weights become 32-bit keys that order as the weights do.  The budget's smallest
// kept key is found by counting: the keys' range is cut into 2048 equal steps, the step
// that holds the wanted rank becomes the next range, and after at most three counts it is
// one value (2^32 = 2^11 * 2^11 * 2^10).  Equal keys are then taken by position.
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelItems = 16;                               // keys a thread holds
constexpr int kSelTile = kSelThreads * kSelItems;           // keys a CTA holds at once
constexpr int kBins = 2048;
constexpr int kBinBits = 11;

__device__ __forceinline__ uint32_t weight_key(float w) {
  uint32_t u = __float_as_uint(w);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0u;           // NaN: below everything
  if (u == 0x80000000u) u = 0u;                             // -0 == +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ void row_sync(int C) {
  if (C == 1) __syncthreads();
  else cluster_sync();
}

__device__ __forceinline__ uint32_t dsmem_ld_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t peer_u32(const uint32_t* local, int rank, int C) {
  return C == 1 ? *local : dsmem_ld_u32(dsmem_addr(local, rank));
}

__global__ void __launch_bounds__(kSelThreads, 2)
    select_kernel(const float* __restrict__ weight, const int32_t* __restrict__ seq_len, int Hkv,
                  int cap, int sink, int recent, int budget, int C, int32_t* __restrict__ keep,
                  int32_t* __restrict__ kept_len, int32_t* dev_err) {
  __shared__ uint32_t s_hist[kBins];      // this CTA's counts
  __shared__ uint32_t s_tot[kBins];       // the row's counts
  __shared__ uint32_t s_red[4];           // min, max (later kept, equal) of this CTA
  __shared__ uint32_t s_warp[2][kSelWarps];
  __shared__ uint32_t s_bin[3];           // the chosen step, keys above it, keys in it
  grid_dependency_wait();
  const int rank = C == 1 ? 0 : static_cast<int>(cluster_ctarank());
  const int row = blockIdx.x / C, b = row / Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
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
  const int lo_t = sink, hi_t = L - recent;                 // positions that compete
  const int want = budget - sink - recent;                  // >= 0, < hi_t - lo_t
  const int per = ((L + C - 1) / C + 31) & ~31;             // slice of this CTA
  const int t_lo = min(L, rank * per), t_hi = min(L, t_lo + per);
  const int ntiles = (per + kSelTile - 1) / kSelTile;

  uint32_t key[kSelItems];
  int seg_lo = 0, seg_n = 0;              // this warp's run of the tile
  auto load = [&](int tile) {
    const int a = t_lo + tile * kSelTile, n = max(0, min(kSelTile, t_hi - a));
    const int seg = (((n + kSelWarps - 1) / kSelWarps) + 31) & ~31;
    seg_lo = a + min(n, warp * seg);
    seg_n = max(0, min(seg, n - warp * seg));
#pragma unroll
    for (int i = 0; i < kSelItems; ++i) {
      const int e = i * 32 + lane;
      key[i] = e < seg_n ? weight_key(w[seg_lo + e]) : 0u;
    }
  };
  auto competes = [&](int i) -> bool {
    const int e = i * 32 + lane, t = seg_lo + e;
    return e < seg_n && t >= lo_t && t < hi_t;
  };

  uint32_t T = 0xffffffffu, need = 0;     // kept: key > T, and the first `need` keys == T
  if (want > 0) {
    uint32_t kmin = 0xffffffffu, kmax = 0u;
    for (int tile = 0; tile < ntiles; ++tile) {
      load(tile);
#pragma unroll
      for (int i = 0; i < kSelItems; ++i)
        if (competes(i)) {
          kmin = min(kmin, key[i]);
          kmax = max(kmax, key[i]);
        }
    }
    kmin = __reduce_min_sync(0xffffffffu, kmin);
    kmax = __reduce_max_sync(0xffffffffu, kmax);
    if (tid == 0) {
      s_red[0] = 0xffffffffu;
      s_red[1] = 0u;
    }
    __syncthreads();
    if (lane == 0) {
      atomicMin(&s_red[0], kmin);
      atomicMax(&s_red[1], kmax);
    }
    row_sync(C);
    for (int r = 0; r < C; ++r) {
      kmin = min(kmin, peer_u32(&s_red[0], r, C));
      kmax = max(kmax, peer_u32(&s_red[1], r, C));
    }
    const uint32_t range = kmax - kmin;
    uint32_t lo = kmin, last = range;     // keys of the current range: lo .. lo + last
    int s = max(0, 32 - __clz(range) - kBinBits);
    need = static_cast<uint32_t>(want);
    for (;;) {
      for (int i = tid; i < kBins; i += kSelThreads) s_hist[i] = 0u;
      __syncthreads();
      for (int tile = 0; tile < ntiles; ++tile) {
        if (ntiles > 1) load(tile);
#pragma unroll
        for (int i = 0; i < kSelItems; ++i)
          if (competes(i) && key[i] >= lo && key[i] - lo <= last) atomicAdd(&s_hist[(key[i] - lo) >> s], 1u);
      }
      const uint32_t* tot = s_hist;
      row_sync(C);
      if (C > 1) {                        // every CTA forms the row's counts for itself
        for (int i = tid; i < kBins; i += kSelThreads) {
          uint32_t v = 0;
          for (int r = 0; r < C; ++r) v += peer_u32(&s_hist[i], r, C);
          s_tot[i] = v;
        }
        cluster_sync();                   // s_hist is read by nobody any more
        tot = s_tot;
      }
      // Four steps a thread, thread 0 the highest: the step where the count from above
      // reaches `need`.
      uint32_t c[4], mine = 0;
      const int top = kBins - 1 - tid * 4;
#pragma unroll
      for (int i = 0; i < 4; ++i) mine += c[i] = tot[top - i];
      uint32_t incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      if (lane == 31) s_warp[0][warp] = incl;
      __syncthreads();
      uint32_t above = incl - mine;
      for (int v = 0; v < warp; ++v) above += s_warp[0][v];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (above < need && above + c[i] >= need) {
          s_bin[0] = top - i;
          s_bin[1] = above;
          s_bin[2] = c[i];
        }
        above += c[i];
      }
      __syncthreads();
      const uint32_t bin = s_bin[0];
      need -= s_bin[1];
      lo += bin << s;
      if (s == 0) {
        T = lo;
        break;
      }
      if (s_bin[2] == need && lo > 0) {   // the whole step stays
        T = lo - 1;
        need = 0;
        break;
      }
      last = min(last - (bin << s), (1u << s) - 1u);
      s = max(0, s - kBinBits);
    }
  }

  // Kept keys (forced ones among them) and keys equal to T, per CTA.
  auto classify = [&](int i, bool& above, bool& equal) {
    const int e = i * 32 + lane, t = seg_lo + e;
    const bool in = e < seg_n, mid = t >= lo_t && t < hi_t;
    above = in && (!mid || (want > 0 && key[i] > T));
    equal = in && mid && need > 0 && key[i] == T;
  };
  uint32_t n_above = 0, n_equal = 0;
  for (int tile = 0; tile < ntiles; ++tile) {
    if (ntiles > 1 || want == 0) load(tile);
#pragma unroll
    for (int i = 0; i < kSelItems; ++i) {
      bool a, q;
      classify(i, a, q);
      n_above += a;
      n_equal += q;
    }
  }
  n_above = __reduce_add_sync(0xffffffffu, n_above);
  n_equal = __reduce_add_sync(0xffffffffu, n_equal);
  __syncthreads();
  if (lane == 0) {
    s_warp[0][warp] = n_above;
    s_warp[1][warp] = n_equal;
  }
  __syncthreads();
  if (tid < 2) {
    uint32_t v = 0;
    for (int i = 0; i < kSelWarps; ++i) v += s_warp[tid][i];
    s_red[2 + tid] = v;
  }
  row_sync(C);
  uint32_t base_above = 0, base_equal = 0;
  for (int r = 0; r < rank; ++r) {
    base_above += peer_u32(&s_red[2], r, C);
    base_equal += peer_u32(&s_red[3], r, C);
  }
  const uint32_t below = (1u << lane) - 1u;
  for (int tile = 0; tile < ntiles; ++tile) {
    if (ntiles > 1) {
      load(tile);
      n_above = n_equal = 0;
#pragma unroll
      for (int i = 0; i < kSelItems; ++i) {
        bool a, q;
        classify(i, a, q);
        n_above += a;
        n_equal += q;
      }
      n_above = __reduce_add_sync(0xffffffffu, n_above);
      n_equal = __reduce_add_sync(0xffffffffu, n_equal);
      __syncthreads();
      if (lane == 0) {
        s_warp[0][warp] = n_above;
        s_warp[1][warp] = n_equal;
      }
      __syncthreads();
    }
    uint32_t at_above = base_above, at_equal = base_equal;
    for (int v = 0; v < kSelWarps; ++v) {
      if (v < warp) {
        at_above += s_warp[0][v];
        at_equal += s_warp[1][v];
      }
      base_above += s_warp[0][v];
      base_equal += s_warp[1][v];
    }
    uint32_t at = at_above + min(need, at_equal);
#pragma unroll
    for (int i = 0; i < kSelItems; ++i) {
      if (i * 32 >= seg_n) break;
      bool a, q;
      classify(i, a, q);
      const uint32_t mq = __ballot_sync(0xffffffffu, q);
      const bool stay = a || (q && at_equal + __popc(mq & below) < need);
      const uint32_t ms = __ballot_sync(0xffffffffu, stay);
      if (stay) out[at + __popc(ms & below)] = seg_lo + i * 32 + lane;
      at += __popc(ms);
      at_equal += __popc(mq);
    }
  }
  grid_dependents_launch();
  if (C > 1) cluster_sync();              // nobody leaves while its counts may be read
}

// ------------------------------------------------------------------------ eviction

constexpr int kEvictThreads = 256;
constexpr int kEvictRows = 8;             // rows a thread has in flight

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
  int slices, splits;         // byte slices of a row; ranges of rows (1 in place)
  int kv_in_place, weight_in_place;
};

// One CTA moves one byte slice of K or V of one kv-head (the last CTA of a head: the
// weights), over its range of kept rows.  In place the rows go in rising order: because
// keep[j] >= j rises strictly, row j's new place lies below every later row's old one, so
// reading a batch whole before writing it gives the sequential result.
__global__ void __launch_bounds__(kEvictThreads) evict_kernel(const EvictParams p) {
  grid_dependency_wait();
  const int parts = 2 * p.slices + (p.weight_out != nullptr ? 1 : 0);
  const int part = blockIdx.x % parts, row = blockIdx.x / parts;
  const int b = row / p.Hkv, g = row % p.Hkv;
  const int cap = p.max_pages * kPage;
  int bits = 0;
  int L = p.seq_len[b], n = p.kept_len[b];
  if (L < 0 || L > cap) bits |= JF_DEVERR_BAD_PREFIX;
  L = max(0, min(L, cap));
  if (n < 0 || n > min(L, p.budget)) bits |= JF_DEVERR_BAD_PATH;
  n = max(0, min(n, min(L, p.budget)));
  const int32_t* keep = p.keep + static_cast<size_t>(row) * p.budget;
  const int32_t* bt = p.block_table + static_cast<size_t>(b) * p.max_pages;
  const int32_t* nt = p.new_table + static_cast<size_t>(b) * p.max_pages;
  const int span = (n + p.splits - 1) / p.splits;
  const int j0 = min(n, static_cast<int>(blockIdx.y) * span), j1 = min(n, j0 + span);
  auto source = [&](int j) -> int {       // -1: a malformed entry
    const int t = keep[j];
    if (t < j || t >= L || (j > 0 && t <= keep[j - 1])) return -1;
    return t;
  };
  if (part == 2 * p.slices) {
    const float* w = p.weight + static_cast<size_t>(row) * cap;
    float* wo = p.weight_out + static_cast<size_t>(row) * cap;
    for (int base = j0; base < j1; base += kEvictThreads * kEvictRows) {
      float v[kEvictRows];
      int t[kEvictRows];
#pragma unroll
      for (int u = 0; u < kEvictRows; ++u) {
        const int j = base + u * kEvictThreads + threadIdx.x;
        t[u] = j < j1 ? source(j) : -1;
        if (t[u] >= 0) v[u] = w[t[u]];
        else if (j < j1) bits |= JF_DEVERR_BAD_PATH;
      }
      if (p.weight_in_place) __syncthreads();
#pragma unroll
      for (int u = 0; u < kEvictRows; ++u)
        if (t[u] >= 0) wo[base + u * kEvictThreads + threadIdx.x] = v[u];
      if (p.weight_in_place) __syncthreads();
    }
  } else {
    uint16_t* cache = part < p.slices ? p.k_cache : p.v_cache;
    const int vecs = p.D / 8 / p.slices;  // 16-byte vectors of a slice
    const int rows = kEvictThreads / vecs;
    const int r = threadIdx.x / vecs;
    const int col = (part % p.slices) * vecs + threadIdx.x % vecs;
    auto at = [&](int page, int t) -> uint4* {
      return reinterpret_cast<uint4*>(cache + ((static_cast<size_t>(page) * kPage + t % kPage) * p.Hkv + g) * p.D) + col;
    };
    for (int base = j0; base < j1; base += rows * kEvictRows) {
      uint4 v[kEvictRows];
      uint4* to[kEvictRows];
#pragma unroll
      for (int u = 0; u < kEvictRows; ++u) {
        const int j = base + u * rows + r;
        to[u] = nullptr;
        if (j >= j1) continue;
        const int t = source(j);
        if (t < 0) {
          bits |= JF_DEVERR_BAD_PATH;
          continue;
        }
        const int ps = bt[t / kPage], pd = nt[j / kPage];
        if (ps < 0 || ps >= p.num_pages || pd < 0 || pd >= p.num_pages) {
          bits |= JF_DEVERR_BAD_PAGE;
          continue;
        }
        if (p.kv_in_place && t == j) continue;
        to[u] = at(pd, j);
        v[u] = *at(ps, t);
      }
      if (p.kv_in_place) __syncthreads();
#pragma unroll
      for (int u = 0; u < kEvictRows; ++u)
        if (to[u] != nullptr) *to[u] = v[u];
      if (p.kv_in_place) __syncthreads();
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
  int C = 1;
  while (C < 8 && (capacity > C * kSelTile || (rows * C * 2 <= sms && capacity > C * 2048))) C *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * C));
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(C);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, select_kernel, weight, seq_len, Hkv, capacity, sink,
                                           recent, budget, C, keep, kept_len, dev_err);
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
  p.slices = 4;
  p.splits = 1;
  const unsigned parts = 2 * p.slices + (weight_out != nullptr ? 1 : 0);
  const cudaError_t e = launch_pdl(evict_kernel, dim3(static_cast<unsigned>(B) * Hkv * parts, p.splits),
                                   dim3(kEvictThreads), 0, reinterpret_cast<cudaStream_t>(stream), p);
  return e == cudaSuccess ? JF_OK : JF_ERR_CUDA;
}
