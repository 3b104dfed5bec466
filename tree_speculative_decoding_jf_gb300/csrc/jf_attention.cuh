// jf_attention.cuh -- what the paged-attention kernels share: tile sizes, the shared-memory and TMEM
// layout of a CTA, and one key tile of the online softmax.
#pragma once

#include "jf_common.cuh"
#include "jf_sm100.cuh"

namespace jf {
namespace {

constexpr int kKeyTile = 128;     // keys per pipeline stage
constexpr int kRowTile = 128;     // rows per tensor-core tile (TMEM lanes)
constexpr int kPage = 16;
constexpr int kPagesPerTile = kKeyTile / kPage;
constexpr float kRescaleThreshold = 8.0f;               // log2 units
// Sequences with fewer prefix keys than this store P as hi + lo bf16 parts on the key
// tiles that hold tree keys (see row_probs); longer prefixes give every row at least this
// many visible keys, over which the bf16 rounding of P averages out.
constexpr int kSplitPrefix = 128;

// Step records: record i completes once step i - 1 (every row tile's PV of key tile i - 1
// and S of key tile i) has finished on the tensor cores; record 0 marks the first S MMAs.
constexpr int kStepRing = 8;

template <int NT, int D>
struct Cfg {
  static constexpr int kHalves = D / 64;                  // 128-byte swizzle atoms per row
  // V stages are released only when a tile's last PV MMA completes, K stages as soon as
  // the next tile's S MMAs are issued, so V gets the deeper ring.
  static constexpr int kKStages = (D == 64) ? 4 : 2;
  static constexpr int kVStages = (D == 64) ? 6 : 3;
  // K tile j may load after record j - kKStages, V tile j after record j - kVStages + 1;
  // the producer loads both after record j - kStageLag.
  static constexpr int kStageLag = kKStages < kVStages - 1 ? kKStages : kVStages - 1;
  static constexpr int kTileBytes = kRowTile * D * 2;     // one 128-row bf16 tile
  static constexpr int kHalfBytes = kRowTile * 128;       // one 64-column half of a tile
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kQOff + NT * kTileBytes;
  static constexpr int kVOff = kKOff + kKStages * kTileBytes;
  static constexpr int kRingBytes = (kKStages + kVStages) * kTileBytes;
  // After the last MMA the ring holds the epilogue: fp32 rows [NT][128][D], then LSEs.
  static constexpr int kPartLseOff = kKOff + NT * 2 * kTileBytes;
  static_assert(NT * 2 * kTileBytes + NT * kRowTile * 4 <= kRingBytes, "epilogue fits the ring");
  static constexpr int kSmemBytes = kKOff + kRingBytes + 1024;
  static constexpr int kThreads = 128 * (1 + NT);
  static constexpr uint32_t kTmemCols = (NT == 2) ? 512 : 256;
  static constexpr uint32_t kTmemO = 0;                   // O_t at column t*128
  static constexpr uint32_t kTmemS = NT * 128;            // S_t (and P_t) at kTmemS + t*128
};

// Packed calls (cu != null) keep q, out and mask as [T][...] rows, sequence b's nodes at
// rows cu[b] .. cu[b + 1] - 1, and lse as [Hq][T]; the others [B][N][...] and [B][Hq][N].
// row0 is the sequence's first row (b * N when not packed).
__device__ __forceinline__ size_t out_row(long long row0, int i, int Hq, int h) {
  return static_cast<size_t>((row0 + i) * Hq + h);
}
__device__ __forceinline__ size_t lse_index(bool packed, long long row0, long long T, int b,
                                            int h, int i, int Hq, int N) {
  return packed ? static_cast<size_t>(h * T + row0 + i)
                : static_cast<size_t>((static_cast<long long>(b) * Hq + h) * N + i);
}

// Nodes of sequence b's tree: N, or tree_len[b] clamped to [1, N] for ragged calls.  The
// tree's keys are the n positions after the prefix, so the sequence has P_b + n keys.
__device__ __forceinline__ int tree_nodes(const int32_t* tree_len, int b, int N) {
  return tree_len == nullptr ? N : max(1, min(tree_len[b], N));
}

// A 3-input max.
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Bits [rel, rel + 32) of the 192-bit little-endian window w[0..3) (zero outside it).
__device__ __forceinline__ uint32_t window_bits32(const uint64_t (&w)[3], int rel) {
  if (rel <= -32 || rel >= 192) return 0u;
  if (rel < 0) return static_cast<uint32_t>(w[0] << (-rel));
  const int wi = rel >> 6, off = rel & 63;
  const uint64_t lo = wi == 0 ? w[0] : (wi == 1 ? w[1] : w[2]);
  const uint64_t hi = wi == 0 ? w[1] : (wi == 1 ? w[2] : 0ull);
  uint64_t v = lo >> off;
  if (off > 32) v |= hi << (64 - off);
  return static_cast<uint32_t>(v);
}

// Four 32-column TMEM loads followed by one wait that ties all 128 registers.
__device__ __forceinline__ void tmem_ld128(uint32_t taddr, uint32_t (&r)[128]) {
  tmem_ld32(taddr + 0, *reinterpret_cast<uint32_t(*)[32]>(&r[0]));
  tmem_ld32(taddr + 32, *reinterpret_cast<uint32_t(*)[32]>(&r[32]));
  tmem_ld32(taddr + 64, *reinterpret_cast<uint32_t(*)[32]>(&r[64]));
  tmem_ld32(taddr + 96, *reinterpret_cast<uint32_t(*)[32]>(&r[96]));
  tmem_ld_wait(*reinterpret_cast<uint32_t(*)[32]>(&r[0]));
  tmem_ld_wait(*reinterpret_cast<uint32_t(*)[32]>(&r[32]));
  tmem_ld_wait(*reinterpret_cast<uint32_t(*)[32]>(&r[64]));
  tmem_ld_wait(*reinterpret_cast<uint32_t(*)[32]>(&r[96]));
}

// Probabilities of one 128-score row (log2 domain: p = 2^(s * sl2 - m)), written back to
// the row's TMEM S columns as the bf16 A operand of the PV MMA: P in columns 0..63 (two
// keys per 32-bit column).  With SPLIT, P is also stored as a second bf16 part
// lo = bf16(p - bf16(p)) in columns 64..127 and the MMA issuer adds a PV MMA on it, so the
// probabilities that reach the tensor cores carry a relative error of about 2^-17 instead
// of bf16's 2^-9.  That matters on tiles that hold tree keys: a row with only a few
// visible keys gets no averaging of the rounding errors, and the output of such a row can
// be small where its values cancel.  Returns the fp32 row sum.
template <bool SPLIT>
__device__ __forceinline__ float row_probs(const float* sv, float sl2, float neg, uint32_t tS) {
  const uint64_t sl2x2 = f2(sl2, sl2), negx2 = f2(neg, neg);
  uint64_t ls2[2] = {0ull, 0ull};       // paired partial row sums (0ull == {+0, +0})
  if constexpr (SPLIT) {
#pragma unroll
    for (int h = 0; h < 4; ++h) {        // quarters of 32 keys keep few registers live
      uint32_t ph[16], pl[16];
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const int cc = 16 * h + c;
        float x0, x1;
        f2_split(ffma2(f2(sv[2 * cc], sv[2 * cc + 1]), sl2x2, negx2), x0, x1);
        const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
        ls2[c & 1] = fadd2(ls2[c & 1], f2(p0, p1));
        ph[c] = pack_bf16x2(p0, p1);
        pl[c] = pack_bf16x2(p0 - __uint_as_float(ph[c] << 16), p1 - __uint_as_float(ph[c] & 0xFFFF0000u));
      }
      tmem_st16(tS + 16 * h, ph);
      tmem_st16(tS + 64 + 16 * h, pl);
    }
  } else {
    uint32_t pk[64];
#pragma unroll
    for (int c = 0; c < 64; ++c) {
      float x0, x1;
      f2_split(ffma2(f2(sv[2 * c], sv[2 * c + 1]), sl2x2, negx2), x0, x1);
      const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
      ls2[c & 1] = fadd2(ls2[c & 1], f2(p0, p1));
      pk[c] = pack_bf16x2(p0, p1);
    }
    tmem_st32(tS, *reinterpret_cast<uint32_t(*)[32]>(&pk[0]));
    tmem_st32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&pk[32]));
  }
  float la, lb, lc, ld;
  f2_split(ls2[0], la, lb);
  f2_split(ls2[1], lc, ld);
  return (la + lb) + (lc + ld);
}

// One key tile of the online softmax for the calling thread's score row (its TMEM lane):
// waits for the tile's S, applies visibility, raises the running maximum when needed,
// writes P back to TMEM, rescales O when the maximum moved, and arrives on p_full.
// MASKED tiles reach positions >= P (tree keys, possibly keys past the sequence end): the
// node's ancestor words are loaded before the wait.  SPLIT (only on masked tiles of
// sequences with a prefix shorter than kSplitPrefix) stores P as hi + lo parts.  Prefix
// tiles take the MASKED = false instantiation, whose loop carries none of that code.  With
// a non-null lo_flag the writer thread records SPLIT there for the MMA issuer once the
// tile's S has arrived.  Returns false if the wait gave up.
template <bool MASKED, bool SPLIT, int D>
__device__ __forceinline__ bool softmax_tile(uint64_t* s_full_bar, uint32_t parity,
                                             volatile int* abort, uint64_t* p_full_bar,
                                             uint32_t tS, uint32_t tO, const uint64_t* mrow,
                                             bool valid, int W, int key0, int P, int L, float sl2,
                                             bool not_first, volatile int* lo_flag, bool writer,
                                             float& m_run, float& l, uint64_t wlim) {
  uint64_t mw[3] = {0ull, 0ull, 0ull};
  const int w_lo = MASKED ? (max(key0 - P, 0) >> 6) : 0;
  if constexpr (MASKED) {
    if (valid) {
#pragma unroll
      for (int u = 0; u < 3; ++u)
        if (w_lo + u < W) mw[u] = __ldg(reinterpret_cast<const unsigned long long*>(mrow) + w_lo + u);
    }
  }
  if (!wait_warp(s_full_bar, parity, abort, wlim)) return false;
  if (lo_flag != nullptr && writer) *lo_flag = SPLIT ? 1 : 0;
  tc_fence_after();
  uint32_t sr[128];
  tmem_ld128(tS, sr);
  float* sv = reinterpret_cast<float*>(sr);
  if constexpr (MASKED) {
    // Visibility of the tile's 128 keys as four 32-bit words: prefix keys always, tree key
    // j iff bit j of the node's ancestor mask, nothing past the sequence end.
    const int pre = min(max(P - key0, 0), kKeyTile);
    const int end = min(max(L - key0, 0), kKeyTile);
    uint32_t vis[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int c0 = 32 * w;
      uint32_t m = window_bits32(mw, key0 + c0 - P - 64 * w_lo);
      const int np = min(max(pre - c0, 0), 32);
      const int ne = min(max(end - c0, 0), 32);
      m |= np >= 32 ? 0xFFFFFFFFu : ((1u << np) - 1u);
      m &= ne >= 32 ? 0xFFFFFFFFu : ((1u << ne) - 1u);
      vis[w] = m;
    }
#pragma unroll
    for (int c = 0; c < kKeyTile; ++c)
      if (!((vis[c >> 5] >> (c & 31)) & 1u)) sv[c] = -INFINITY;
  }
  float m4[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
  for (int c = 4; c < kKeyTile; c += 2) m4[(c >> 1) & 3] = fmax3(m4[(c >> 1) & 3], sv[c], sv[c + 1]);
  const float mx = fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]);
  const float mt = mx * sl2;
  const bool raise = mt > m_run + kRescaleThreshold;
  const float m_old = m_run;
  if (raise) m_run = mt;
  const float corr = raise ? fast_exp2(m_old - m_run) : 1.f;   // 0 when m_old = -inf
  const float neg = (m_run == -INFINITY) ? 0.f : -m_run;
  l = l * corr + row_probs<SPLIT>(sv, sl2, neg, tS);
  // O holds PV of the earlier tiles (complete: this tile's S was committed after them).
  const bool need = raise && not_first && m_old != -INFINITY;
  if (__any_sync(0xffffffffu, need)) {
    const float f = need ? corr : 1.f;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      uint32_t o[32];
      tmem_ld32(tO + c * 32, o);
      tmem_ld_wait(o);
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
      tmem_st32(tO + c * 32, o);
    }
  }
  tmem_st_wait();
  tc_fence_before();
  mbar_arrive(p_full_bar);
  return true;
}

// O += P_lo V from the second bf16 part of P (columns 64..127 of a row tile's S region).
// Out of line: the MMA issuer's steady-state loop carries none of this code.
__device__ __noinline__ void issue_pv_lo(uint32_t d_tmem, uint32_t a_tmem, uint64_t db, uint32_t idO) {
  mma_ts_tile(d_tmem, a_tmem + 64, db, idO, true);
}

}  // namespace
}  // namespace jf
