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
// Bound: bytes (logits read and written once).  A block owns a slice of 2048 tokens, eight per
// thread, for a run of rows of one sequence: what depends on the sequence alone (counts and
// bias, 8 bytes a token) becomes one multiplier choice and one addend per token in registers
// and serves all rows of the run, so a row costs its logits, its output and one grammar bit a
// token.  Logits of eight tokens that the grammar forbids are not read.  A branch's drafted
// tokens are few and fall into few slices: a bitmap of the nodes whose token lies in the slice
// is formed once, ANDed with each row's ancestor mask, and only rows with a hit walk the hits,
// each hit counted by the thread that owns the token (no atomics, no shared table).
#include <algorithm>
#include <cmath>

#include "jf_common.cuh"

namespace jf {
namespace {

constexpr int kAdjThreads = 256;
constexpr int kPer = 8;                        // tokens per thread
constexpr int kSlice = kAdjThreads * kPer;
constexpr int kMaxRun = 16;                    // rows per block at most
constexpr int kPromptFlag = JF_COUNT_PROMPT;

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
__device__ __forceinline__ void store8(uint16_t* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}

// VEC: a thread's eight tokens are consecutive and every row starts at a 16-byte boundary (V a
// multiple of 8).  Otherwise they lie kAdjThreads apart, so that a warp's accesses of one
// element each still cover whole sectors.
template <typename TI, typename TO, bool VEC>
__global__ void __launch_bounds__(kAdjThreads) adjust_kernel(const AdjustParams p) {
  __shared__ unsigned long long s_hit[JF_MAX_NODES / 64];   // nodes whose token lies in the slice
  __shared__ int s_any;
  grid_dependency_wait();
  const int tid = threadIdx.x;
  long long bid = blockIdx.x;
  const int slice = static_cast<int>(bid % p.slices);
  bid /= p.slices;
  const int run = static_cast<int>(bid % p.runs);
  const int b = static_cast<int>(bid / p.runs);
  const SeqSpan sp = seq_span(p.cu, p.tree_len, b, p.N, p.T);
  if (!sp.ok && slice == 0 && run == 0 && tid == 0) report(p.dev_err, JF_DEVERR_BAD_TREE_LEN);
  const int i0 = run * p.run, i1 = min(i0 + p.run, sp.n);
  if (i0 >= i1) return;                        // block-uniform
  const int v0 = slice * kSlice;
  const int vmine = VEC ? v0 + tid * kPer : v0 + tid;        // first token of this thread
  constexpr int kStep = VEC ? 1 : kAdjThreads;               // to its next one

  // What depends on the sequence alone.
  const float rep = p.repetition != nullptr ? p.repetition[b] : 1.f;
  const float pres = p.presence != nullptr ? p.presence[b] : 0.f;
  const float freq = p.frequency != nullptr ? p.frequency[b] : 0.f;
  float add[kPer];                             // bias - presence - frequency * c
  float sub[kPer];                             // bias alone
  int c[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) c[e] = 0, sub[e] = 0.f;
  const size_t base = static_cast<size_t>(b) * p.V;
  if (VEC) {
    if (vmine < p.V) {
      if (p.count != nullptr) {
        const int4 a = *reinterpret_cast<const int4*>(p.count + base + vmine);
        const int4 d = *reinterpret_cast<const int4*>(p.count + base + vmine + 4);
        c[0] = a.x; c[1] = a.y; c[2] = a.z; c[3] = a.w;
        c[4] = d.x; c[5] = d.y; c[6] = d.z; c[7] = d.w;
      }
      if (p.bias != nullptr) load8(p.bias + base + vmine, sub);
    }
  } else {
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int v = vmine + e * kStep;
      if (v < p.V) {
        if (p.count != nullptr) c[e] = p.count[base + v];
        if (p.bias != nullptr) sub[e] = p.bias[base + v];
      }
    }
  }
  uint32_t seen = 0;
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const int n = c[e] & (kPromptFlag - 1);
    seen |= (c[e] != 0 ? 1u : 0u) << e;
    add[e] = n > 0 ? sub[e] - fmaf(freq, static_cast<float>(n), pres) : sub[e];
  }

  // Nodes whose drafted token lies in this slice.
  bool hits = false;
  if (p.draft != nullptr) {
    if (tid == 0) s_any = 0;
    __syncthreads();
    int bad = 0;
    const int words32 = (sp.n + 31) / 32;
    for (int w = tid >> 5; w < words32; w += kAdjThreads / 32) {
      const int j = w * 32 + (tid & 31);
      bool in = false;
      if (j >= 1 && j < sp.n) {
        const int tok = p.draft[sp.row0 + j];
        if (tok < 0 || tok >= p.V) bad = 1;
        else in = tok >= v0 && tok - v0 < kSlice;
      }
      const uint32_t m = __ballot_sync(0xffffffffu, in);
      if ((tid & 31) == 0) {
        reinterpret_cast<uint32_t*>(s_hit)[w] = m;
        if (m != 0) s_any = 1;
      }
    }
    if (tid == 0 && (words32 & 1)) reinterpret_cast<uint32_t*>(s_hit)[words32] = 0;
    if (bad) report(p.dev_err, JF_DEVERR_BAD_TOKEN);
    __syncthreads();
    hits = s_any != 0;
  }

  for (int i = i0; i < i1; ++i) {
    const size_t row = static_cast<size_t>(sp.row0 + i);
    // Grammar bits of the thread's tokens.
    uint32_t ok = 0xFFu;
    if (p.allowed != nullptr) {
      const long long ar = p.allowed_row != nullptr ? p.allowed_row[row] : static_cast<long long>(row);
      if (ar >= 0 && ar < p.n_allowed) {
        const uint32_t* aw = p.allowed + static_cast<size_t>(ar) * p.words;
        if (VEC) {
          if (vmine < p.V) ok = reinterpret_cast<const uint8_t*>(aw)[vmine >> 3];
        } else {
          ok = 0;
#pragma unroll
          for (int e = 0; e < kPer; ++e) {
            const int v = vmine + e * kStep;
            if (v < p.V) ok |= ((aw[v >> 5] >> (v & 31)) & 1u) << e;
          }
        }
      } else if (ar != -1 && tid == 0 && slice == 0) {
        report(p.dev_err, JF_DEVERR_BAD_PATH);
      }
    }
    // Drafted tokens of the branch, counted by their owners.
    float ad[kPer];
    uint32_t sn = seen;
#pragma unroll
    for (int e = 0; e < kPer; ++e) ad[e] = add[e];
    if (hits) {
      int extra[kPer];
      bool any = false;
#pragma unroll
      for (int e = 0; e < kPer; ++e) extra[e] = 0;
      const int words64 = (sp.n + 63) / 64;
      for (int w = 0; w < words64; ++w) {
        unsigned long long m = s_hit[w];
        if (m != 0) m &= p.mask[row * p.W + w];
        while (m != 0) {
          const int j = w * 64 + __ffsll(static_cast<long long>(m)) - 1;
          m &= m - 1;
          const int o = p.draft[sp.row0 + j] - v0;
          if ((VEC ? o / kPer : o % kAdjThreads) == tid) {
            const int at = VEC ? o % kPer : o / kAdjThreads;
            any = true;
#pragma unroll
            for (int e = 0; e < kPer; ++e) extra[e] += at == e ? 1 : 0;
          }
        }
      }
      if (any) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          if (extra[e] > 0) {
            const int n = (c[e] & (kPromptFlag - 1)) + extra[e];
            sn |= 1u << e;
            ad[e] = sub[e] - fmaf(freq, static_cast<float>(n), pres);
          }
        }
      }
    }
    const TI* src = static_cast<const TI*>(p.logits) + row * p.V;
    TO* dst = static_cast<TO*>(p.out) + row * p.V;
    float x[kPer];
    if (VEC) {
      if (vmine >= p.V) continue;
      if (ok != 0) {
        load8(src + vmine, x);
      } else {
#pragma unroll
        for (int e = 0; e < kPer; ++e) x[e] = 0.f;
      }
    } else {
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const int v = vmine + e * kStep;
        x[e] = v < p.V && ((ok >> e) & 1u) ? load1<TI>(src + v) : 0.f;
      }
    }
    bool same = ok == 0xFFu && sn == 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      same = same && ad[e] == 0.f;
      if ((sn >> e) & 1u) x[e] = x[e] > 0.f ? x[e] / rep : x[e] * rep;
      x[e] += ad[e];
      if (!((ok >> e) & 1u)) x[e] = p.masked;
    }
    if (p.in_place && same) continue;          // the eight values stay as they are
    if (VEC) {
      store8(dst + vmine, x);
    } else {
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const int v = vmine + e * kStep;
        if (v < p.V) store1(dst + v, x[e]);
      }
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
  // The same array, or no shared byte: blocks read and write their own slices only.
  p.in_place = p.out == p.logits && isz == osz;
  if (!p.in_place && overlap(p.out, rows * p.V * osz, p.logits, rows * p.V * isz)) return JF_ERR_INVALID_ARGUMENT;
  const size_t seq = static_cast<size_t>(p.B) * p.V * 4;
  p.words = (p.V + 31) / 32;
  const size_t ob = rows * p.V * osz;
  if ((p.count != nullptr && overlap(p.out, ob, p.count, seq)) ||
      (p.bias != nullptr && overlap(p.out, ob, p.bias, seq)) ||
      (p.allowed != nullptr && overlap(p.out, ob, p.allowed, static_cast<size_t>(p.n_allowed) * p.words * 4)))
    return JF_ERR_INVALID_ARGUMENT;
  const int sms = current_sm_count();
  if (sms <= 0) return JF_ERR_CUDA;
  p.W = (p.N + 63) / 64;
  p.slices = (p.V + kSlice - 1) / kSlice;
  // Rows per block: 16, so that counts and bias cost half a byte a logit at most, fewer while
  // the grid would leave SMs short of blocks.
  p.run = kMaxRun < p.N ? kMaxRun : p.N;
  while (p.run > 1 && static_cast<long long>(p.B) * p.slices * ((p.N + p.run - 1) / p.run) < 8ll * sms) p.run = (p.run + 1) / 2;
  p.runs = (p.N + p.run - 1) / p.run;
  const long long grid = static_cast<long long>(p.B) * p.runs * p.slices;
  if (grid > 0x7FFFFFFFll) return JF_ERR_UNSUPPORTED;
  const bool vec = p.V % 8 == 0 && aligned_to(p.logits, 16) && aligned_to(p.out, 16) && aligned_to(p.count, 16) &&
                   aligned_to(p.bias, 16);
  const dim3 g(static_cast<unsigned>(grid)), t(kAdjThreads);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == JF_DTYPE_F32)
    e = vec ? launch_pdl(adjust_kernel<float, float, true>, g, t, 0, s, p)
            : launch_pdl(adjust_kernel<float, float, false>, g, t, 0, s, p);
  else if (out_dtype == JF_DTYPE_F32)
    e = vec ? launch_pdl(adjust_kernel<uint16_t, float, true>, g, t, 0, s, p)
            : launch_pdl(adjust_kernel<uint16_t, float, false>, g, t, 0, s, p);
  else
    e = vec ? launch_pdl(adjust_kernel<uint16_t, uint16_t, true>, g, t, 0, s, p)
            : launch_pdl(adjust_kernel<uint16_t, uint16_t, false>, g, t, 0, s, p);
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
  __shared__ int s_n[kCountSlice];
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
