// jf_rotate.cu -- rotary positions for a step's queries and keys, and the append of its keys
// and values to the paged cache.
//
// For every token: each query and key head is normalised (optional: x / sqrt(mean x^2 + eps) *
// w), its pairs (x, y) are turned by the angle pos * freq[f],
//     (x, y) -> scale * (x cos a - y sin a, y cos a + x sin a),
// and rounded to bf16 once; query heads go to q_out, key and value heads to slot P_b + i of the
// sequence's pages.
//
// Angles.  Only the fraction of a turn matters, and with integer positions it can be formed
// exactly modulo one turn: freq / 2 pi as a 64-bit fixed-point fraction of a turn, multiplied
// by the position in 64-bit integer arithmetic (which wraps at whole turns), is off by at most
// |pos| 2^-64 turns plus the 2^-52 relative rounding of freq / 2 pi (a negative frequency's
// fraction is taken from one, which rounds too: |pos| 2^-54).  The signed fraction is then
// rounded to fp32 once, so a position of a million costs no more error than position 1;
// pos * freq in fp32 would be off by up to 2^-24 * pos radians.
//
// Bound: bytes.  Every head row is read and written once, so a thread owns the two 16-byte
// chunks of a head that a half-split pair needs (chunks t and t + R / 16), D / 16 threads a
// head; the cosines and sines of a token are formed once per block and read from shared memory
// by all its heads.  Prompt chunks of 8 x 4096 tokens, 32 + 2 * 8 heads of 128: 144 us, 5.6 TB/s (82% of
// the copy rate); eight trees of up to 256 nodes 12.6 us, a chain of 16 tokens 2.7 us, where the bound is
// the chain of reads position -> angle and length -> page -> store.
#include <algorithm>
#include <cmath>

#include "jf_common.cuh"

namespace jf {
namespace {

constexpr int kPage = 16;
constexpr int kMaxThreads = 384;
constexpr int kAhead = 1;                   // tokens whose rows are on their way (trees: 1 12.6 us, 2 14.0, 3 15.4: registers)
constexpr int kMaxChunk = 16;               // tokens whose facts a block settles at once
constexpr int kBlocks = 4;                  // blocks per SM, resident or next in line (trees: 4 12.6 us, 8 13.8; prompts alike)

struct RotateParams {
  const uint16_t *q, *k, *v;
  long long q_stride, k_stride, v_stride;   // elements between consecutive tokens
  const int32_t* pos;
  const double* freq;                       // null: nothing is rotated
  const uint16_t *q_norm, *k_norm;          // null: not normalised
  const int32_t *block_table, *prefix_len, *tree_len, *cu;
  uint16_t *q_out, *k_cache, *v_cache;
  int32_t* dev_err;
  long long rows;                           // tokens of the call's arrays (padding included)
  int B, N, Hq, Hkv, R, max_pages, num_pages;
  int chunk;                                // tokens a block takes at a time
  float scale, eps;
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void unpack8(uint4 w, float (&x)[8]) {
  x[0] = bf_lo(w.x); x[1] = bf_hi(w.x); x[2] = bf_lo(w.y); x[3] = bf_hi(w.y);
  x[4] = bf_lo(w.z); x[5] = bf_hi(w.z); x[6] = bf_lo(w.w); x[7] = bf_hi(w.w);
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}

// Where a token belongs: its sequence, the sequence's span and its prefix length.
struct Home {
  int b, P;
  SeqSpan sp;
};

// The sequence whose packed span holds `row`: the last b with cu[b] <= row, found by the whole
// warp, 32 probes a round (one round up to 32 sequences, two up to 1024).  The last round's
// probes bring the spans' ends and the prefix lengths along, so they cost no further trip.
__device__ __forceinline__ Home packed_home(const RotateParams& p, long long row) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = p.B;
  while (len > 32) {
    const int step = (len + 31) / 32;
    const int at = lane * step;
    const bool below = at < len && p.cu[lo + at] <= row;
    const int skip = max(__popc(__ballot_sync(0xffffffffu, below)) - 1, 0) * step;
    lo += skip;
    len = min(step, len - skip);
  }
  const int at = lo + min(lane, len - 1);
  const int r0 = p.cu[at], r1 = p.cu[at + 1], P = p.prefix_len[at];
  const int sel = max(__popc(__ballot_sync(0xffffffffu, lane < len && r0 <= row)) - 1, 0);
  Home h;
  h.b = lo + sel;
  h.P = __shfl_sync(0xffffffffu, P, sel);
  const long long a = __shfl_sync(0xffffffffu, r0, sel), e = __shfl_sync(0xffffffffu, r1, sel);
  h.sp.ok = a >= 0 && e <= p.rows && e - a >= 1 && e - a <= p.N;
  h.sp.row0 = h.sp.ok ? a : 0;
  h.sp.n = h.sp.rows = h.sp.ok ? static_cast<int>(e - a) : 0;
  return h;
}

__device__ __forceinline__ Home padded_home(const RotateParams& p, long long row) {
  Home h;
  h.b = static_cast<int>(row / p.N);
  h.P = p.prefix_len[h.b];
  h.sp = seq_span(nullptr, p.tree_len, h.b, p.N, p.rows);
  return h;
}

// Fraction of a turn per position, as a 64-bit fixed-point number (whole turns dropped).
__device__ __forceinline__ uint64_t fixed_turns(double freq) {
  double t = freq * 0.15915494309189533577;   // 1 / (2 pi)
  t -= floor(t);
  return __double2ull_rn(t * 18446744073709551616.0);
}

// A block takes `chunk` consecutive tokens at a time (blocks stride over the chunks).  It first settles
// the chunk's facts, one chain of dependent reads for all its tokens: where each token's keys and
// values go, and its cosines and sines, both into shared memory; then it streams the tokens' rows,
// a thread for each pair of 16-byte chunks of a token's heads (up to kMaxThreads: more heads take
// more rounds), the next tokens' rows being read while the current one's are turned.  The first
// rows' reads go out before the facts'.  INTER: pairs (2 f, 2 f + 1) instead of (f, f + R / 2).
template <int D, bool INTER>
__global__ void __launch_bounds__(kMaxThreads, 2) rotate_append_kernel(const RotateParams p) {
  constexpr int kLanes = D / 16;            // threads per head row
  __shared__ float2 s_cs[kMaxChunk][D / 2]; // (cos, sin) * scale: number e of thread t at e * kLanes + t
  __shared__ long long s_cache[kMaxChunk];  // cache row of the token, -1: none
  __shared__ int s_live[kMaxChunk];
  grid_dependency_wait();

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int cap = p.max_pages * kPage;
  // Thread t of a head: the rotated chunks t and t + R / 16, or two of the chunks behind R (the first
  // ones of all such threads side by side, then the second ones).
  const int t = threadIdx.x % kLanes;
  const int half = p.freq != nullptr ? p.R / 16 : 0;
  const bool turns = t < half;
  const int c0 = turns ? t : half + t;
  const int c1 = turns ? t + half : c0 + kLanes - half;
  const int heads = p.Hq + 2 * p.Hkv;
  const int slots = blockDim.x / kLanes;
  const bool any_norm = p.q_norm != nullptr || p.k_norm != nullptr;
  const int pairs = p.freq != nullptr ? p.R / 2 : 0;

  if (blockIdx.x == 0) {                    // every sequence's span and length are judged once
    for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
      const SeqSpan sp = seq_span(p.cu, p.tree_len, b, p.N, p.rows);
      if (!sp.ok) report(p.dev_err, JF_DEVERR_BAD_TREE_LEN);
      const int P = p.prefix_len[b];
      if (P < 0 || P > cap - sp.n) report(p.dev_err, JF_DEVERR_BAD_PREFIX);
    }
  }
  for (long long row0 = static_cast<long long>(blockIdx.x) * p.chunk; row0 < p.rows;
       row0 += static_cast<long long>(gridDim.x) * p.chunk) {
    const int tokens = static_cast<int>(min(static_cast<long long>(p.chunk), p.rows - row0));
    for (int h0 = 0; h0 < heads; h0 += slots) {
      const int h = h0 + threadIdx.x / kLanes;
      const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.Hkv;
      const int hh = is_q ? h : (is_v ? h - p.Hq - p.Hkv : h - p.Hq);
      const long long stride = is_q ? p.q_stride : (is_v ? p.v_stride : p.k_stride);
      const uint16_t* src = (is_q ? p.q : (is_v ? p.v : p.k)) + row0 * stride + static_cast<long long>(hh) * D;
      uint4 w0[kAhead], w1[kAhead];
      auto load = [&](int k, int to) {       // padding rows exist too; what they hold is dropped
        if (h < heads && k < tokens) {
          const uint4* s4 = reinterpret_cast<const uint4*>(src + k * stride);
          w0[to] = s4[c0];
          w1[to] = s4[c1];
        }
      };
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        w0[k] = w1[k] = make_uint4(0u, 0u, 0u, 0u);
        load(k, k);
      }
      const uint16_t* norm = is_v || h >= heads ? nullptr : (is_q ? p.q_norm : p.k_norm);
      uint4 n0 = make_uint4(0u, 0u, 0u, 0u), n1 = n0;
      if (norm != nullptr) {
        n0 = reinterpret_cast<const uint4*>(norm)[c0];
        n1 = reinterpret_cast<const uint4*>(norm)[c1];
      }
      if (h0 == 0) {
        __syncthreads();                     // the chunk before has been turned
        for (int k = warps - 1 - warp; k < tokens; k += warps) {      // the last warps: the first ones form angles
          const long long row = row0 + k;
          const Home at_home = p.cu != nullptr ? packed_home(p, row) : padded_home(p, row);
          const long long i = row - at_home.sp.row0;
          const bool live = i >= 0 && i < at_home.sp.n;
          if (lane == 0) {
            long long at = -1;
            if (live && at_home.P >= 0 && at_home.P <= cap - at_home.sp.n) {
              const int pt = at_home.P + static_cast<int>(i);
              const int page = p.block_table[static_cast<size_t>(at_home.b) * p.max_pages + pt / kPage];
              if (page >= 0 && page < p.num_pages)
                at = static_cast<long long>(page) * kPage + pt % kPage;
              else
                report(p.dev_err, JF_DEVERR_BAD_PAGE);
            }
            s_live[k] = live ? 1 : 0;
            s_cache[k] = at;
          }
        }
        for (int e = threadIdx.x; e < tokens * pairs; e += blockDim.x) {
          const int k = e / pairs, f = e - k * pairs;
          const uint64_t turn = static_cast<uint64_t>(static_cast<long long>(p.pos[row0 + k])) * fixed_turns(p.freq[f]);
          // signed fraction of a turn in [-1/2, 1/2), in units of pi: [-1, 1)
          const float x = __ll2float_rn(static_cast<long long>(turn)) * 1.0842021724855044e-19f;   // 2^-63
          float s, c;
          sincospif(x, &s, &c);
          // half: the eight pairs of chunk t; interleaved: four pairs each of chunks t and t + half
          const int chunk = f >> 2;
          const int tt = !INTER ? f >> 3 : (chunk < half ? chunk : chunk - half);
          const int ee = !INTER ? f & 7 : (f & 3) + (chunk < half ? 0 : 4);
          s_cs[k][ee * kLanes + tt] = make_float2(c * p.scale, s * p.scale);
        }
        __syncthreads();
      }
      for (int k = 0; k < tokens; ++k) {
        const uint4 v0 = w0[0], v1 = w1[0];
#pragma unroll
        for (int u = 0; u < kAhead - 1; ++u) w0[u] = w0[u + 1], w1[u] = w1[u + 1];
        load(k + kAhead, kAhead - 1);
        if (!s_live[k]) continue;            // block-uniform
        const long long at = s_cache[k];
        float x[8], y[8];
        unpack8(v0, x);
        unpack8(v1, y);
        if (any_norm) {                      // uniform: the shuffles need every lane
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], fmaf(y[e], y[e], ss));
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          if (norm != nullptr) {
            const float inv = 1.f / sqrtf(ss * (1.f / D) + p.eps);
            float u[8];
            unpack8(n0, u);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= inv * u[e];
            unpack8(n1, u);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] *= inv * u[e];
          }
        }
        if (h >= heads || !(is_q || at >= 0)) continue;
        if (!is_v && turns) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 cs = s_cs[k][e * kLanes + t];
            if (!INTER) {
              const float a = x[e], b = y[e];
              x[e] = a * cs.x - b * cs.y;
              y[e] = b * cs.x + a * cs.y;
            } else {
              float* z = e < 4 ? x + 2 * e : y + 2 * (e - 4);
              const float a = z[0], b = z[1];
              z[0] = a * cs.x - b * cs.y;
              z[1] = b * cs.x + a * cs.y;
            }
          }
        }
        uint16_t* d = is_q ? p.q_out + ((row0 + k) * p.Hq + hh) * D
                           : (is_v ? p.v_cache : p.k_cache) + (at * p.Hkv + hh) * D;
        const bool changed = !is_v && (turns || norm != nullptr);
        reinterpret_cast<uint4*>(d)[c0] = changed ? pack8(x) : v0;
        reinterpret_cast<uint4*>(d)[c1] = changed ? pack8(y) : v1;
      }
    }
  }
  grid_dependents_launch();
}

template <int D>
cudaError_t launch_rotate(const RotateParams& p, bool inter, int sms, cudaStream_t s) {
  const long long chunks = (p.rows + p.chunk - 1) / p.chunk;
  const dim3 grid(static_cast<unsigned>(std::min(chunks, static_cast<long long>(sms) * kBlocks)));
  const int need = (p.Hq + 2 * p.Hkv) * (D / 16);
  const int rounds = (need + kMaxThreads - 1) / kMaxThreads;
  const dim3 block(static_cast<unsigned>(((need + rounds - 1) / rounds + 31) / 32 * 32));
  return inter ? launch_pdl(rotate_append_kernel<D, true>, grid, block, 0, s, p)
               : launch_pdl(rotate_append_kernel<D, false>, grid, block, 0, s, p);
}

jf_status rotate_call(RotateParams p, int D, int page_size, bool inter, bool packed, long long T,
                      jf_stream_t stream) {
  if (p.k == nullptr || p.v == nullptr || p.block_table == nullptr || p.prefix_len == nullptr ||
      p.k_cache == nullptr || p.v_cache == nullptr || (p.q == nullptr) != (p.q_out == nullptr))
    return JF_ERR_INVALID_ARGUMENT;
  if (p.freq != nullptr && p.pos == nullptr) return JF_ERR_INVALID_ARGUMENT;
  if (p.q == nullptr) p.Hq = 0;
  if (p.B < 1 || p.N < 1 || p.Hkv < 1 || (p.q != nullptr && p.Hq < 1) || p.max_pages < 1 ||
      p.num_pages < 1 || !std::isfinite(p.scale) || !(p.eps >= 0.f) || !std::isfinite(p.eps))
    return JF_ERR_INVALID_ARGUMENT;
  if (packed && T < 1) return JF_ERR_INVALID_ARGUMENT;
  if (D != 64 && D != 128) return JF_ERR_UNSUPPORTED;
  if (page_size != kPage) return JF_ERR_UNSUPPORTED;
  if (p.freq != nullptr && (p.R < 16 || p.R > D || p.R % 16 != 0)) return JF_ERR_UNSUPPORTED;
  if (p.Hq > (1 << 20) || p.Hkv > (1 << 20)) return JF_ERR_UNSUPPORTED;
  p.rows = packed ? T : static_cast<long long>(p.B) * p.N;
  if (p.rows + p.N >= (1ll << 31)) return JF_ERR_UNSUPPORTED;
  if (static_cast<long long>(p.max_pages) * kPage > (1ll << 30)) return JF_ERR_UNSUPPORTED;
  if (static_cast<long long>(p.num_pages) * kPage >= (1ll << 31)) return JF_ERR_UNSUPPORTED;
  const long long qw = static_cast<long long>(p.Hq) * D, kw = static_cast<long long>(p.Hkv) * D;
  if (p.k_stride < kw || p.v_stride < kw || (p.q != nullptr && p.q_stride < qw)) return JF_ERR_INVALID_ARGUMENT;
  const long long max_stride = 1ll << 31;     // rows * stride stays far inside 64 bits
  if (p.k_stride > max_stride || p.v_stride > max_stride || (p.q != nullptr && p.q_stride > max_stride))
    return JF_ERR_UNSUPPORTED;
  if (!aligned_to(p.k, 16) || !aligned_to(p.v, 16) || !aligned_to(p.q, 16) || !aligned_to(p.q_out, 16) ||
      !aligned_to(p.k_cache, 16) || !aligned_to(p.v_cache, 16) || !aligned_to(p.q_norm, 16) ||
      !aligned_to(p.k_norm, 16) || !aligned_to(p.freq, 8) || p.k_stride % 8 != 0 || p.v_stride % 8 != 0 ||
      (p.q != nullptr && p.q_stride % 8 != 0))
    return JF_ERR_MISALIGNED;
  // Outputs must not overlap what other blocks still read; q_out may be q itself.
  const size_t rows = static_cast<size_t>(p.rows);
  const size_t kb = ((rows - 1) * p.k_stride + kw) * 2, vb = ((rows - 1) * p.v_stride + kw) * 2;
  const size_t qb = p.q != nullptr ? ((rows - 1) * p.q_stride + qw) * 2 : 0, ob = rows * qw * 2;
  const size_t cb = static_cast<size_t>(p.num_pages) * kPage * kw * 2;
  if (overlap(p.k_cache, cb, p.v_cache, cb)) return JF_ERR_INVALID_ARGUMENT;
  const size_t seqs = static_cast<size_t>(p.B), wb = static_cast<size_t>(D) * 2;
  auto over_inputs = [&](const void* out, size_t bytes) {
    return overlaps_any(out, bytes, {{p.k, kb}, {p.v, vb}, {p.freq != nullptr ? p.pos : nullptr, rows * 4},
                                     {p.freq, static_cast<size_t>(p.R) * 4}, {p.q_norm, wb}, {p.k_norm, wb},
                                     {p.block_table, seqs * p.max_pages * 4}, {p.prefix_len, seqs * 4},
                                     {p.tree_len, seqs * 4}, {p.cu, (seqs + 1) * 4}});
  };
  for (void* out : {static_cast<void*>(p.k_cache), static_cast<void*>(p.v_cache)}) {
    if (over_inputs(out, cb) || overlaps_any(out, cb, {{p.q, qb}, {p.q_out, ob}})) return JF_ERR_INVALID_ARGUMENT;
  }
  if (p.q != nullptr) {
    if (over_inputs(p.q_out, ob)) return JF_ERR_INVALID_ARGUMENT;
    if (overlap(p.q_out, ob, p.q, qb) && !(p.q_out == p.q && p.q_stride == qw)) return JF_ERR_INVALID_ARGUMENT;
  }
  const int sms = current_sm_count();
  if (sms <= 0) return JF_ERR_CUDA;
  // One token a block while that leaves no SM with more than kBlocks, then as many as it takes, up
  // to kMaxChunk.
  p.chunk = static_cast<int>(std::min<long long>(kMaxChunk, (p.rows + kBlocks * sms - 1) / (kBlocks * sms)));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = D == 128 ? launch_rotate<128>(p, inter, sms, s) : launch_rotate<64>(p, inter, sms, s);
  return e == cudaSuccess ? JF_OK : JF_ERR_CUDA;
}

RotateParams rotate_params(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                           int64_t v_stride, const int32_t* pos, const double* freq, int32_t R,
                           float scale, const void* q_norm, const void* k_norm, float eps,
                           const int32_t* block_table, const int32_t* prefix_len, int32_t B, int32_t N,
                           int32_t Hq, int32_t Hkv, int32_t max_pages, int32_t num_pages, void* q_out,
                           void* k_cache, void* v_cache, int32_t* dev_err) {
  RotateParams p = {};
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.q_stride = q_stride; p.k_stride = k_stride; p.v_stride = v_stride;
  p.pos = pos; p.freq = freq; p.R = R; p.scale = scale;
  p.q_norm = static_cast<const uint16_t*>(q_norm);
  p.k_norm = static_cast<const uint16_t*>(k_norm);
  p.eps = eps;
  p.block_table = block_table; p.prefix_len = prefix_len;
  p.B = B; p.N = N; p.Hq = Hq; p.Hkv = Hkv; p.max_pages = max_pages; p.num_pages = num_pages;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_cache = static_cast<uint16_t*>(k_cache);
  p.v_cache = static_cast<uint16_t*>(v_cache);
  p.dev_err = dev_err;
  return p;
}

}  // namespace
}  // namespace jf

extern "C" jf_status jf_rotate_append_kv(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                         const void* v, int64_t v_stride, const int32_t* pos,
                                         const double* freq, int32_t rotary_dim, int32_t interleaved,
                                         float rotary_scale, const void* q_norm, const void* k_norm,
                                         float norm_eps, const int32_t* block_table,
                                         const int32_t* prefix_len, const int32_t* tree_len, int32_t B,
                                         int32_t N, int32_t Hq, int32_t Hkv, int32_t D,
                                         int32_t page_size, int32_t max_pages, int32_t num_pages,
                                         void* q_out, void* k_cache, void* v_cache, int32_t* dev_err,
                                         jf_stream_t stream) {
  jf::RotateParams p = jf::rotate_params(q, q_stride, k, k_stride, v, v_stride, pos, freq, rotary_dim,
                                         rotary_scale, q_norm, k_norm, norm_eps, block_table, prefix_len, B,
                                         N, Hq, Hkv, max_pages, num_pages, q_out, k_cache, v_cache, dev_err);
  p.tree_len = tree_len;
  return jf::rotate_call(p, D, page_size, interleaved != 0, false, 0, stream);
}

extern "C" jf_status jf_rotate_append_kv_packed(
    const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
    const int32_t* pos, const double* freq, int32_t rotary_dim, int32_t interleaved, float rotary_scale,
    const void* q_norm, const void* k_norm, float norm_eps, const int32_t* block_table,
    const int32_t* prefix_len, const int32_t* cu_seqlens, int32_t B, int32_t N_max, int32_t T, int32_t Hq,
    int32_t Hkv, int32_t D, int32_t page_size, int32_t max_pages, int32_t num_pages, void* q_out,
    void* k_cache, void* v_cache, int32_t* dev_err, jf_stream_t stream) {
  if (cu_seqlens == nullptr) return JF_ERR_INVALID_ARGUMENT;
  jf::RotateParams p = jf::rotate_params(q, q_stride, k, k_stride, v, v_stride, pos, freq, rotary_dim,
                                         rotary_scale, q_norm, k_norm, norm_eps, block_table, prefix_len, B,
                                         N_max, Hq, Hkv, max_pages, num_pages, q_out, k_cache, v_cache,
                                         dev_err);
  p.cu = cu_seqlens;
  return jf::rotate_call(p, D, page_size, interleaved != 0, true, T, stream);
}
