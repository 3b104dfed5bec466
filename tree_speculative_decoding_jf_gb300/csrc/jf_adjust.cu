// jf_adjust.cu -- penalties for repeated tokens, biases and grammar masks on the logits of
// draft-tree nodes, and the token counts the penalties read.
//
// For node i of sequence b and token v, with c = times v was generated so far (count[b][v])
// plus the drafted tokens equal to v on i's branch (the root's excluded: it is an emitted
// token and belongs to the counts already), and seen = c > 0 or v is in the prompt:
//     x = logits[b][i][v];   seen: x = x > 0 ? x / repetition : x * repetition
//     c > 0: x -= presence + frequency * c;   x += bias[b][v]
//     v forbidden by the node's grammar row: x = masked.
//
// Bound: bytes (logits read and written once: 2048 rows of 151936 take 189 us at the copy rate; this
// takes 235, 80% of it).  A block owns a slice of 2048 tokens, eight per thread, for a run of up to 16 rows of
// one sequence, and passes over them once.  Few tokens change, so values travel as the words they were
// read in: a thread turns its tokens' counts and biases into marks and addends once for the run,
// takes the marked ones out of the words, computes them and puts them back, and forbids the rest by
// bits; logits of eight tokens that the grammar forbids are not read.  (Computing every value took
// 533 us; a copy and a second kernel over the marked tokens more than this one, for the second
// touch of scattered sectors reaches HBM again.)
// Drafted tokens differ from row to row: they are left out of the marks and done afterwards, one
// (row, token) pair a thread.  A bitmap of the nodes whose token lies in the slice is ANDed with the
// rows' ancestor masks, and only rows with a hit walk theirs.
#include <algorithm>
#include <cmath>

#include "jf_common.cuh"

namespace jf {
namespace {

constexpr int kAdjThreads = 256;
constexpr int kPer = 8;                        // tokens per thread
constexpr int kSlice = kAdjThreads * kPer;
constexpr int kMaxRun = 16;                    // rows per block at most (2048 rows: 8 248 us, 16 235, 32 245)
constexpr int kAdjBlocks = 5;                  // resident blocks per SM (4: 249 us, 5: 235, 6: 232, but 54 odd rows 9.4 -> 10.9)
constexpr int kPromptFlag = JF_COUNT_PROMPT;
constexpr float kMaxBf16 = 3.38953138925153547590e38f;      // 2^128 - 2^120

struct AdjustParams {
  const void* logits;
  void* out;
  const int32_t* count;
  const int32_t* draft;
  const uint64_t* mask;
  const float* bias;
  const uint32_t* allowed;
  const int32_t* allowed_row;
  const float *repetition, *presence, *frequency;
  const int32_t *tree_len, *cu;
  int32_t* dev_err;
  long long T;                                 // packed rows
  int B, N, V, W, words, n_allowed, run, slices, runs;
  float masked;
  bool in_place;
};

template <typename T> __device__ __forceinline__ float load1(const T* p);
template <> __device__ __forceinline__ float load1<float>(const float* p) { return *p; }
template <> __device__ __forceinline__ float load1<uint16_t>(const uint16_t* p) {
  return __uint_as_float(static_cast<uint32_t>(*p) << 16);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }
__device__ __forceinline__ void store1(uint16_t* p, float x) { *p = static_cast<uint16_t>(pack2(x, 0.f) & 0xFFFFu); }

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const uint16_t* p, float (&x)[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(u[e] << 16);
    x[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

// Eight logits of a thread on their way from input to output: bf16 that stays bf16 travels as
// the words it was read in, so values that nothing changes are neither unpacked nor rounded.
template <typename TI, typename TO>
struct Chunk {
  float x[kPer];
  __device__ __forceinline__ void load(const TI* p) { load8(p, x); }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int e = 0; e < kPer; ++e) x[e] = 0.f;
  }
  __device__ __forceinline__ float get(int at) const {
    float y = x[0];
#pragma unroll
    for (int e = 1; e < kPer; ++e) y = at == e ? +x[e] : +y;     // values, not places: x stays in registers
    return y;
  }
  __device__ __forceinline__ void put(int at, float y) {
#pragma unroll
    for (int e = 0; e < kPer; ++e) x[e] = at == e ? +y : +x[e];
  }
  __device__ __forceinline__ void forbid(uint32_t ok, float masked) {
#pragma unroll
    for (int e = 0; e < kPer; ++e) x[e] = (ok >> e) & 1u ? x[e] : masked;
  }
  __device__ __forceinline__ void store(TO* p) const { store8(p, x); }
};
__device__ __forceinline__ uint32_t pick(bool c, uint32_t a, uint32_t b) {   // by value: what it picks from stays in registers
  uint32_t r;
  asm("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %3, 0;\n\tselp.b32 %0, %1, %2, p;\n\t}" : "=r"(r) : "r"(a), "r"(b), "r"(c ? 1u : 0u));
  return r;
}
template <>
struct Chunk<uint16_t, uint16_t> {
  uint32_t w0, w1, w2, w3;
  __device__ __forceinline__ void load(const uint16_t* p) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w0 = v.x; w1 = v.y; w2 = v.z; w3 = v.w;
  }
  __device__ __forceinline__ void zero() { w0 = w1 = w2 = w3 = 0u; }
  __device__ __forceinline__ float get(int at) const {
    const uint32_t v = pick(at & 4, pick(at & 2, w3, w2), pick(at & 2, w1, w0));
    return __uint_as_float(pick(at & 1, v & 0xFFFF0000u, v << 16));
  }
  __device__ __forceinline__ void put(int at, float y) {
    const uint32_t bits = pack2(y, y), half = pick(at & 1, 0xFFFF0000u, 0x0000FFFFu);   // the bits to replace
    const int at2 = at >> 1;
    w0 ^= (w0 ^ bits) & pick(at2 == 0, half, 0u);
    w1 ^= (w1 ^ bits) & pick(at2 == 1, half, 0u);
    w2 ^= (w2 ^ bits) & pick(at2 == 2, half, 0u);
    w3 ^= (w3 ^ bits) & pick(at2 == 3, half, 0u);
  }
  static __device__ __forceinline__ uint32_t under(uint32_t w, uint32_t ok2, uint32_t m) {
    const uint32_t keep = (ok2 & 1u) * 0xFFFFu | ((ok2 >> 1) & 1u) * 0xFFFF0000u;      // where the token is allowed
    return (w & keep) | (m & ~keep);
  }
  __device__ __forceinline__ void forbid(uint32_t ok, float masked) {
    const uint32_t m = pack2(masked, masked);
    w0 = under(w0, ok, m);
    w1 = under(w1, ok >> 2, m);
    w2 = under(w2, ok >> 4, m);
    w3 = under(w3, ok >> 6, m);
  }
  __device__ __forceinline__ void store(uint16_t* p) const {
    *reinterpret_cast<uint4*>(p) = make_uint4(w0, w1, w2, w3);
  }
};

// VEC: a thread's eight tokens are consecutive and every row starts at a 16-byte boundary (V a
// multiple of 8).  Otherwise they lie kAdjThreads apart, so that a warp's accesses of one
// element each still cover whole sectors.
template <typename TI, typename TO, bool VEC>
__global__ void __launch_bounds__(kAdjThreads, kAdjBlocks) adjust_kernel(const AdjustParams p) {
  __shared__ float s_add[kPer][kAdjThreads];   // a token's addend, for its own thread alone
  __shared__ uint32_t s_drafted[kSlice / 32];  // tokens that a node of the tree drafts,
  __shared__ uint16_t s_list[kSlice];          // listed
  __shared__ int s_grammar[kMaxRun];           // the rows' grammar rows, -1: none
  __shared__ uint32_t s_rows;                  // rows with a drafted token of the slice on their branch
  __shared__ int s_any, s_listed;
  extern __shared__ unsigned long long s_dyn[];
  grid_dependency_wait();
  const int tid = threadIdx.x, lane = tid & 31;
  const unsigned per = static_cast<unsigned>(p.slices) * static_cast<unsigned>(p.runs);
  const int b = static_cast<int>(blockIdx.x / per);
  const unsigned rem = blockIdx.x - static_cast<unsigned>(b) * per;
  const int run = static_cast<int>(rem / static_cast<unsigned>(p.slices));
  const int slice = static_cast<int>(rem - static_cast<unsigned>(run) * static_cast<unsigned>(p.slices));
  const SeqSpan sp = seq_span(p.cu, p.tree_len, b, p.N, p.T);
  if (!sp.ok && slice == 0 && run == 0 && tid == 0) report(p.dev_err, JF_DEVERR_BAD_TREE_LEN);
  const int i0 = run * p.run, rows = min(p.run, sp.n - i0);
  if (rows <= 0) return;                       // block-uniform
  const int v0 = slice * kSlice;
  const int vmine = VEC ? v0 + tid * kPer : v0 + tid;        // first token of this thread
  constexpr int kStep = VEC ? 1 : kAdjThreads;               // to its next one
  const size_t base = static_cast<size_t>(b) * p.V;
  const float rep = p.repetition != nullptr ? p.repetition[b] : 1.f;
  const float pres = p.presence != nullptr ? p.presence[b] : 0.f;
  const float freq = p.frequency != nullptr ? p.frequency[b] : 0.f;

  if (p.allowed != nullptr && tid < rows) {
    const long long row = sp.row0 + i0 + tid;
    long long at = p.allowed_row != nullptr ? p.allowed_row[row] : row;
    if (at < 0 || at >= p.n_allowed) {
      if (at != -1 && slice == 0) report(p.dev_err, JF_DEVERR_BAD_PATH);
      at = -1;
    }
    s_grammar[tid] = static_cast<int>(at);
  }
  if (tid < kSlice / 32) s_drafted[tid] = 0;
  if (tid == 0) s_any = 0, s_rows = 0;

  // What the history changes: marked tokens, the seen ones among them, and their addends.
  uint32_t mark = 0, seen = 0;
  if (p.count != nullptr || p.bias != nullptr) {
    int c[kPer];
    float bias[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) c[e] = 0, bias[e] = 0.f;
    if (VEC) {
      if (vmine < p.V) {
        if (p.count != nullptr) {
          const int4 a = *reinterpret_cast<const int4*>(p.count + base + vmine);
          const int4 d = *reinterpret_cast<const int4*>(p.count + base + vmine + 4);
          c[0] = a.x; c[1] = a.y; c[2] = a.z; c[3] = a.w;
          c[4] = d.x; c[5] = d.y; c[6] = d.z; c[7] = d.w;
        }
        if (p.bias != nullptr) load8(p.bias + base + vmine, bias);
      }
    } else {
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const int v = vmine + e * kStep;
        if (v < p.V) {
          if (p.count != nullptr) c[e] = p.count[base + v];
          if (p.bias != nullptr) bias[e] = p.bias[base + v];
        }
      }
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int n = c[e] & (kPromptFlag - 1);
      seen |= (c[e] != 0 ? 1u : 0u) << e;
      mark |= (c[e] != 0 || bias[e] != 0.f ? 1u : 0u) << e;
      s_add[e][tid] = n > 0 ? bias[e] - fmaf(freq, static_cast<float>(n), pres) : bias[e];
    }
  }
  __syncthreads();

  // Nodes whose drafted token lies in this slice, the rows that have one on their branch, and the
  // tokens' list.  Drafted tokens leave the marks: they are done row by row at the end.
  const int words64 = (sp.n + 63) / 64;
  unsigned long long* s_hit = s_dyn;           // [W] the nodes
  unsigned long long* s_branch = s_dyn + p.W;  // [run][W] and the row's ancestors
  uint16_t* s_at = reinterpret_cast<uint16_t*>(s_dyn + static_cast<size_t>(p.W) * (1 + p.run));   // [N] a node's place
  bool any = false;
  if (p.draft != nullptr) {
    int bad = 0;
    const int words32 = (sp.n + 31) / 32;
    for (int w = tid >> 5; w < words32; w += kAdjThreads / 32) {
      const int j = w * 32 + lane;
      bool in = false;
      if (j >= 1 && j < sp.n) {
        const int tok = p.draft[sp.row0 + j];
        if (tok < 0 || tok >= p.V) bad = 1;
        else in = tok >= v0 && tok - v0 < kSlice;
        if (in) {
          const int o = tok - v0;
          s_at[j] = static_cast<uint16_t>(o);
          atomicOr(&s_drafted[o >> 5], 1u << (o & 31));
        }
      }
      const uint32_t m = __ballot_sync(0xffffffffu, in);
      if (lane == 0) {
        reinterpret_cast<uint32_t*>(s_hit)[w] = m;
        if (m != 0) s_any = 1;
      }
    }
    if (tid == 0 && (words32 & 1)) reinterpret_cast<uint32_t*>(s_hit)[words32] = 0;
    if (bad) report(p.dev_err, JF_DEVERR_BAD_TOKEN);
    __syncthreads();
    any = s_any != 0;                          // block-uniform
    if (any) {
      for (int e = tid; e < rows * words64; e += kAdjThreads) {
        const int u = e / words64, w = e % words64;
        unsigned long long m = s_hit[w];
        if (m != 0) m &= p.mask[static_cast<size_t>(sp.row0 + i0 + u) * p.W + w];
        s_branch[u * p.W + w] = m;
        if (m != 0) atomicOr(&s_rows, 1u << u);
      }
      if (tid < 32) {                          // lane l lists tokens 64 l .. 64 l + 63
        unsigned long long d = static_cast<unsigned long long>(s_drafted[2 * lane + 1]) << 32 | s_drafted[2 * lane];
        const int mine = __popcll(d);
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += y;
        }
        if (lane == 31) s_listed = upto;
        for (int at = upto - mine; d != 0; d &= d - 1)
          s_list[at++] = static_cast<uint16_t>(64 * lane + __ffsll(static_cast<long long>(d)) - 1);
      }
      if (VEC) {
        mark &= ~static_cast<uint32_t>(reinterpret_cast<const uint8_t*>(s_drafted)[tid]);
      } else {
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          const int o = e * kAdjThreads + tid;
          mark &= ~(((s_drafted[o >> 5] >> (o & 31)) & 1u) << e);
        }
      }
    }
  }

  // x under a seen token's repetition penalty.
  auto repeated = [&](float x) { return x > 0.f ? x / rep : x * rep; };
  const size_t first = static_cast<size_t>(sp.row0 + i0) * p.V;
  const TI* logits = static_cast<const TI*>(p.logits) + first;     // the run's rows
  TO* out = static_cast<TO*>(p.out) + first;
  if constexpr (VEC) {
    if (vmine < p.V) {
      constexpr int kRows = sizeof(Chunk<TI, TO>) <= 16 ? 4 : 2;     // rows whose reads overlap
      const uint8_t* bits = reinterpret_cast<const uint8_t*>(p.allowed) + (vmine >> 3);
      for (int u0 = 0; u0 < rows; u0 += kRows) {
        uint32_t ok[kRows];
        Chunk<TI, TO> x[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
          ok[k] = u0 + k < rows ? 0xFFu : 0u;
          if (p.allowed != nullptr && u0 + k < rows) {
            const int gr = s_grammar[u0 + k];
            if (gr >= 0) ok[k] = bits[static_cast<size_t>(gr) * p.words * 4];
          }
        }
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
          if (ok[k] != 0) x[k].load(logits + static_cast<size_t>(u0 + k) * p.V + vmine);
          else x[k].zero();                    // logits that the grammar forbids are not read
        }
        for (uint32_t m = mark; m != 0; m &= m - 1) {
          const int e = __ffs(static_cast<int>(m)) - 1;
          const float add = s_add[e][tid];
          const bool again = (seen >> e) & 1u;
#pragma unroll
          for (int k = 0; k < kRows; ++k) {
            if (!((ok[k] >> e) & 1u)) continue;
            float y = x[k].get(e);
            if (again) y = repeated(y);
            x[k].put(e, y + add);
          }
        }
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
          if (u0 + k >= rows || (p.in_place && ok[k] == 0xFFu && mark == 0)) continue;
          if (ok[k] != 0xFFu) x[k].forbid(ok[k], p.masked);
          x[k].store(out + static_cast<size_t>(u0 + k) * p.V + vmine);
        }
      }
    }
  } else {
    for (int u = 0; u < rows; ++u) {
      const int gr = p.allowed != nullptr ? s_grammar[u] : -1;
      const uint32_t* words = p.allowed + static_cast<size_t>(max(gr, 0)) * p.words;
      const size_t at = static_cast<size_t>(u) * p.V;
      uint32_t ok = 0;
      float y[kPer];
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const int v = vmine + e * kStep;
        if (v < p.V) ok |= (gr >= 0 ? (words[v >> 5] >> (v & 31)) & 1u : 1u) << e;
      }
#pragma unroll
      for (int e = 0; e < kPer; ++e) y[e] = (ok >> e) & 1u ? load1<TI>(logits + at + vmine + e * kStep) : p.masked;
      if ((mark & ok) != 0) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          if (!((mark & ok) >> e & 1u)) continue;
          if ((seen >> e) & 1u) y[e] = repeated(y[e]);
          y[e] += s_add[e][tid];
        }
      }
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const int v = vmine + e * kStep;
        if (v < p.V && !(p.in_place && (ok & ~mark) >> e & 1u)) store1(out + at + v, y[e]);
      }
    }
  }
  if (any) {
    // The drafted tokens of the slice, one (row, token) pair a thread.
    __syncthreads();
    const int n = s_listed;
    const uint32_t hit_rows = s_rows;
    for (int q = tid; q < n * rows; q += kAdjThreads) {
      const int u = q / n, o = s_list[q - u * n], v = v0 + o;
      const int gr = p.allowed != nullptr ? s_grammar[u] : -1;
      if (gr >= 0 && !((p.allowed[static_cast<size_t>(gr) * p.words + (v >> 5)] >> (v & 31)) & 1u)) continue;
      const int c = p.count != nullptr ? p.count[base + v] : 0;
      const float bias = p.bias != nullptr ? p.bias[base + v] : 0.f;
      const float x = load1<TI>(logits + static_cast<size_t>(u) * p.V + v);
      int times = c & (kPromptFlag - 1);
      bool again = c != 0;
      if ((hit_rows >> u) & 1u) {              // on this row's branch?
        for (int w = 0; w < words64; ++w) {
          for (unsigned long long m = s_branch[u * p.W + w]; m != 0; m &= m - 1) {
            const bool mine = s_at[w * 64 + __ffsll(static_cast<long long>(m)) - 1] == o;
            times += mine ? 1 : 0;
            again = again || mine;
          }
        }
      }
      if (!again && bias == 0.f) continue;
      const float add = times > 0 ? bias - fmaf(freq, static_cast<float>(times), pres) : bias;
      store1(out + static_cast<size_t>(u) * p.V + v, (again ? repeated(x) : x) + add);
    }
  }
  grid_dependents_launch();
}

jf_status adjust_call(AdjustParams p, int32_t dtype, int32_t out_dtype, bool packed, jf_stream_t stream) {
  if (p.logits == nullptr || p.out == nullptr) return JF_ERR_INVALID_ARGUMENT;
  if ((dtype != JF_DTYPE_BF16 && dtype != JF_DTYPE_F32) ||
      (out_dtype != JF_DTYPE_F32 && out_dtype != dtype))
    return JF_ERR_INVALID_ARGUMENT;
  if (p.B < 1 || p.N < 1 || p.V < 1 || (packed && p.T < 1)) return JF_ERR_INVALID_ARGUMENT;
  if ((p.draft == nullptr) != (p.mask == nullptr)) return JF_ERR_INVALID_ARGUMENT;
  if (p.allowed == nullptr ? p.allowed_row != nullptr : p.n_allowed < 1) return JF_ERR_INVALID_ARGUMENT;
  if (std::isnan(p.masked)) return JF_ERR_INVALID_ARGUMENT;
  if (p.N > JF_MAX_NODES || p.V > 0x7FFFFFFF - kSlice) return JF_ERR_UNSUPPORTED;
  if (packed && p.T + p.N >= (1ll << 31)) return JF_ERR_UNSUPPORTED;
  const size_t isz = dtype == JF_DTYPE_BF16 ? 2 : 4, osz = out_dtype == JF_DTYPE_BF16 ? 2 : 4;
  if (!aligned_to(p.logits, isz) || !aligned_to(p.out, osz) || !aligned_to(p.mask, 8) || !aligned_to(p.allowed, 4))
    return JF_ERR_MISALIGNED;
  const size_t rows = packed ? static_cast<size_t>(p.T) : static_cast<size_t>(p.B) * p.N;
  if (rows > (size_t{1} << 40) / p.V) return JF_ERR_UNSUPPORTED;
  // A finite value stays one: fp32's lowest would round to bf16's -inf.
  if (osz == 2 && std::isfinite(p.masked)) p.masked = std::min(std::max(p.masked, -kMaxBf16), kMaxBf16);
  // The same array, or no shared byte: blocks read and write their own slices only.
  p.in_place = p.out == p.logits && isz == osz;
  if (!p.in_place && overlap(p.out, rows * p.V * osz, p.logits, rows * p.V * isz)) return JF_ERR_INVALID_ARGUMENT;
  p.words = (p.V + 31) / 32;
  p.W = (p.N + 63) / 64;
  const size_t seqs = static_cast<size_t>(p.B), seq = seqs * p.V * 4;
  if (overlaps_any(p.out, rows * p.V * osz,
                   {{p.count, seq}, {p.bias, seq}, {p.draft, rows * 4}, {p.mask, rows * p.W * 8},
                    {p.allowed, static_cast<size_t>(p.n_allowed) * p.words * 4}, {p.allowed_row, rows * 4},
                    {p.repetition, seqs * 4}, {p.presence, seqs * 4}, {p.frequency, seqs * 4},
                    {p.tree_len, seqs * 4}, {p.cu, (seqs + 1) * 4}}))
    return JF_ERR_INVALID_ARGUMENT;
  const int sms = current_sm_count();
  if (sms <= 0) return JF_ERR_CUDA;
  p.slices = (p.V + kSlice - 1) / kSlice;
  if (static_cast<long long>(p.B) * p.N * p.slices > 0x7FFFFFFFll) return JF_ERR_UNSUPPORTED;
  // Rows per block: 16, so that what a block does once weighs little, fewer while the grid would
  // leave SMs short of two blocks (a chain of 16 rows of 151936: 7.4 us; short of one 8.2, of four 9.6).
  p.run = std::min(kMaxRun, p.N);
  while (p.run > 1 && static_cast<long long>(p.B) * p.slices * ((p.N + p.run - 1) / p.run) < 2ll * sms) p.run = (p.run + 1) / 2;
  p.runs = (p.N + p.run - 1) / p.run;
  const bool vec = p.V % 8 == 0 && aligned_to(p.logits, 16) && aligned_to(p.out, 16) && aligned_to(p.count, 16) &&
                   aligned_to(p.bias, 16);
  const dim3 g(static_cast<unsigned>(p.B * p.runs * p.slices)), t(kAdjThreads);
  const size_t smem = p.draft != nullptr ? static_cast<size_t>(p.W) * 8 * (1 + p.run) + static_cast<size_t>(p.N) * 2 : 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == JF_DTYPE_F32)
    e = vec ? launch_pdl(adjust_kernel<float, float, true>, g, t, smem, s, p)
            : launch_pdl(adjust_kernel<float, float, false>, g, t, smem, s, p);
  else if (out_dtype == JF_DTYPE_F32)
    e = vec ? launch_pdl(adjust_kernel<uint16_t, float, true>, g, t, smem, s, p)
            : launch_pdl(adjust_kernel<uint16_t, float, false>, g, t, smem, s, p);
  else
    e = vec ? launch_pdl(adjust_kernel<uint16_t, uint16_t, true>, g, t, smem, s, p)
            : launch_pdl(adjust_kernel<uint16_t, uint16_t, false>, g, t, smem, s, p);
  return e == cudaSuccess ? JF_OK : JF_ERR_CUDA;
}

AdjustParams adjust_params(const void* logits, const int32_t* count, const int32_t* draft, const uint64_t* mask,
                           const float* bias, const uint32_t* allowed, const int32_t* allowed_row,
                           int32_t n_allowed, const float* repetition, const float* presence,
                           const float* frequency, float masked, int32_t B, int32_t N, int32_t V, void* out,
                           int32_t* dev_err) {
  AdjustParams p = {};
  p.logits = logits; p.out = out; p.count = count; p.draft = draft; p.mask = mask; p.bias = bias;
  p.allowed = allowed; p.allowed_row = allowed_row; p.n_allowed = n_allowed;
  p.repetition = repetition; p.presence = presence; p.frequency = frequency;
  p.masked = masked; p.B = B; p.N = N; p.V = V; p.dev_err = dev_err;
  return p;
}

// ------------------------------------------------------------------------ token counts

constexpr int kCountThreads = 256;
constexpr int kCountSlice = 4096;              // tokens of a block's table in shared memory

struct CountParams {
  const int32_t* count;
  const int32_t* row;
  const int32_t* token;
  const int32_t* path;
  const int32_t* length;
  const int32_t* extra;
  int32_t* out;
  int32_t* dev_err;
  int B, N, V, rows_in, prompt;
};

// Calls add(v) for the tokens of sequence b with index first, first + step, ..; `judge`: this
// caller reports what is malformed.
template <typename Add>
__device__ __forceinline__ void each_token(const CountParams& p, int b, int first, int step, bool judge, Add add) {
  const int32_t* tok = p.token + static_cast<size_t>(b) * p.N;
  const int32_t* path = p.path != nullptr ? p.path + static_cast<size_t>(b) * p.N : nullptr;
  // With a path: its entries 1 .. length; else tokens 0 .. length - 1.
  const int most = path != nullptr ? p.N - 1 : p.N;
  int n = p.length != nullptr ? p.length[b] : p.N;
  int bad = 0;
  if (n < 0 || n > most) {
    // accept_len -1 is a verified sequence without rows
    if (!(path != nullptr && n == -1)) bad |= path != nullptr ? JF_DEVERR_BAD_PATH : JF_DEVERR_BAD_TREE_LEN;
    n = max(0, min(n, most));
  }
  for (int k = first; k < n; k += step) {
    int at = k;
    if (path != nullptr) {
      at = path[k + 1];
      if (at < 0 || at >= p.N) { bad |= JF_DEVERR_BAD_PATH; continue; }
    }
    const int v = tok[at];
    if (v < 0 || v >= p.V) { bad |= JF_DEVERR_BAD_TOKEN; continue; }
    add(v);
  }
  if (p.extra != nullptr && first == 0) {
    const int v = p.extra[b];
    if (v >= 0 && v < p.V) add(v);
    else if (v != -1) bad |= JF_DEVERR_BAD_TOKEN;
  }
  if (bad && judge) report(p.dev_err, bad);
}

// out[b] = count[row[b]] with the sequence's tokens added: a block copies one slice and adds
// the tokens that fall in it from a table in shared memory, so every byte moves once.
template <bool VEC>
__global__ void __launch_bounds__(kCountThreads) count_copy_kernel(const CountParams p) {
  __shared__ __align__(16) int s_n[kCountSlice];      // read four at a time
  grid_dependency_wait();
  const int b = blockIdx.y;
  const int v0 = blockIdx.x * kCountSlice;
  for (int e = threadIdx.x; e < kCountSlice; e += kCountThreads) s_n[e] = 0;
  __syncthreads();
  each_token(p, b, threadIdx.x, kCountThreads, blockIdx.x == 0, [&](int v) {
    if (v >= v0 && v - v0 < kCountSlice) {
      if (p.prompt) s_n[v - v0] = kPromptFlag;         // every writer writes the same value
      else atomicAdd(&s_n[v - v0], 1);
    }
  });
  const int src = p.row != nullptr ? p.row[b] : b;
  const bool have = p.count != nullptr && src >= 0 && src < p.rows_in;
  if (p.count != nullptr && !have && blockIdx.x == 0 && threadIdx.x == 0) report(p.dev_err, JF_DEVERR_BAD_PATH);
  __syncthreads();
  const int32_t* in = have ? p.count + static_cast<size_t>(src) * p.V : nullptr;
  int32_t* out = p.out + static_cast<size_t>(b) * p.V;
  const int n = min(kCountSlice, p.V - v0);
  if (VEC) {
#pragma unroll
    for (int u = 0; u < kCountSlice / (4 * kCountThreads); ++u) {
      const int e = 4 * (threadIdx.x + u * kCountThreads);
      if (e >= n) break;
      int4 x = have ? *reinterpret_cast<const int4*>(in + v0 + e) : make_int4(0, 0, 0, 0);
      const int4 a = *reinterpret_cast<const int4*>(s_n + e);
      if (p.prompt) { x.x |= a.x; x.y |= a.y; x.z |= a.z; x.w |= a.w; }
      else { x.x += a.x; x.y += a.y; x.z += a.z; x.w += a.w; }
      *reinterpret_cast<int4*>(out + v0 + e) = x;
    }
  } else {
    for (int e = threadIdx.x; e < n; e += kCountThreads) {
      const int x = have ? in[v0 + e] : 0;
      out[v0 + e] = p.prompt ? x | s_n[e] : x + s_n[e];
    }
  }
  grid_dependents_launch();
}

// In place: only the tokens' own entries are touched.  Integer atomics: the order of equal
// tokens does not show.  A prompt's repeated tokens mostly find their flag set and stop there.
__global__ void __launch_bounds__(kCountThreads) count_in_place_kernel(const CountParams p) {
  grid_dependency_wait();
  const int b = blockIdx.y;
  int32_t* out = p.out + static_cast<size_t>(b) * p.V;
  each_token(p, b, blockIdx.x * kCountThreads + threadIdx.x, gridDim.x * kCountThreads, true, [&](int v) {
    if (!p.prompt) atomicAdd(out + v, 1);
    else if (!(__ldcg(out + v) & kPromptFlag)) atomicOr(out + v, kPromptFlag);
  });
  grid_dependents_launch();
}

}  // namespace
}  // namespace jf

extern "C" jf_status jf_adjust_logits(const void* logits, int32_t dtype, const int32_t* count,
                                      const int32_t* draft, const uint64_t* mask, const float* bias,
                                      const uint32_t* allowed, const int32_t* allowed_row, int32_t n_allowed,
                                      const float* repetition, const float* presence, const float* frequency,
                                      float masked, const int32_t* tree_len, int32_t B, int32_t N, int32_t V,
                                      void* out, int32_t out_dtype, int32_t* dev_err, jf_stream_t stream) {
  jf::AdjustParams p = jf::adjust_params(logits, count, draft, mask, bias, allowed, allowed_row, n_allowed,
                                         repetition, presence, frequency, masked, B, N, V, out, dev_err);
  p.tree_len = tree_len;
  return jf::adjust_call(p, dtype, out_dtype, false, stream);
}

extern "C" jf_status jf_adjust_logits_packed(const void* logits, int32_t dtype, const int32_t* count,
                                             const int32_t* draft, const uint64_t* mask, const float* bias,
                                             const uint32_t* allowed, const int32_t* allowed_row,
                                             int32_t n_allowed, const float* repetition, const float* presence,
                                             const float* frequency, float masked, const int32_t* cu_seqlens,
                                             int32_t B, int32_t N_max, int32_t T, int32_t V, void* out,
                                             int32_t out_dtype, int32_t* dev_err, jf_stream_t stream) {
  if (cu_seqlens == nullptr) return JF_ERR_INVALID_ARGUMENT;
  jf::AdjustParams p = jf::adjust_params(logits, count, draft, mask, bias, allowed, allowed_row, n_allowed,
                                         repetition, presence, frequency, masked, B, N_max, V, out, dev_err);
  p.cu = cu_seqlens;
  p.T = T;
  return jf::adjust_call(p, dtype, out_dtype, true, stream);
}

extern "C" jf_status jf_count_tokens(const int32_t* count, const int32_t* row, int32_t rows_in,
                                     const int32_t* token, const int32_t* path, const int32_t* length,
                                     const int32_t* extra, int32_t prompt, int32_t B, int32_t N, int32_t V,
                                     int32_t* count_out, int32_t* dev_err, jf_stream_t stream) {
  using namespace jf;
  if (token == nullptr || count_out == nullptr) return JF_ERR_INVALID_ARGUMENT;
  if (B < 1 || N < 1 || V < 1) return JF_ERR_INVALID_ARGUMENT;
  if (path != nullptr && length == nullptr) return JF_ERR_INVALID_ARGUMENT;
  if (B > 65535 || N > 0x7FFFFFFF - 65536 * kCountThreads || V > 0x7FFFFFFF - kCountSlice) return JF_ERR_UNSUPPORTED;
  if (count == nullptr ? row != nullptr : rows_in < 1) return JF_ERR_INVALID_ARGUMENT;
  if (count != nullptr && row == nullptr && rows_in < B) return JF_ERR_INVALID_ARGUMENT;
  if (!aligned_to(count, 4) || !aligned_to(count_out, 4)) return JF_ERR_MISALIGNED;
  const bool in_place = count == count_out && row == nullptr;
  const size_t ob = static_cast<size_t>(B) * V * 4;
  const size_t tb = static_cast<size_t>(B) * N * 4;
  if (count != nullptr && !in_place && overlap(count_out, ob, count, static_cast<size_t>(rows_in) * V * 4))
    return JF_ERR_INVALID_ARGUMENT;
  if (overlap(count_out, ob, token, tb) || (path != nullptr && overlap(count_out, ob, path, tb)) ||
      (length != nullptr && overlap(count_out, ob, length, static_cast<size_t>(B) * 4)) ||
      (row != nullptr && overlap(count_out, ob, row, static_cast<size_t>(B) * 4)) ||
      (extra != nullptr && overlap(count_out, ob, extra, static_cast<size_t>(B) * 4)))
    return JF_ERR_INVALID_ARGUMENT;
  CountParams p = {count, row, token, path, length, extra, count_out, dev_err, B, N, V, rows_in, prompt != 0 ? 1 : 0};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (in_place) {
    const int blocks = static_cast<int>(std::min<long long>((static_cast<long long>(N) + kCountThreads - 1) / kCountThreads, 1024));
    e = launch_pdl(count_in_place_kernel, dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(B)),
                   dim3(kCountThreads), 0, s, p);
  } else {
    const dim3 grid(static_cast<unsigned>((V + kCountSlice - 1) / kCountSlice), static_cast<unsigned>(B));
    const bool vec = V % 4 == 0 && aligned_to(count, 16) && aligned_to(count_out, 16);
    e = vec ? launch_pdl(count_copy_kernel<true>, grid, dim3(kCountThreads), 0, s, p)
            : launch_pdl(count_copy_kernel<false>, grid, dim3(kCountThreads), 0, s, p);
  }
  return e == cudaSuccess ? JF_OK : JF_ERR_CUDA;
}
