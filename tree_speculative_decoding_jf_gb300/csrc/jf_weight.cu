// jf_weight.cu -- accumulated attention weight of every cached key.
//
// For sequence b, kv-head g and cache position t the call adds the softmax probabilities
// that the step's query rows gave the key:
//     sum_{k < R_b} sum_{h in group g} [t <= P_b + k] exp(scale q_kh . K_t - lse_kh),
// where lse is what the attention call left, so no softmax statistics are formed here and
// every key is independent: no reduction crosses keys.
#include <algorithm>
#include <cmath>

#include "jf_common.cuh"

namespace jf {
namespace {

constexpr int kPage = 16;
constexpr int kKeys = 128;             // keys (threads) per CTA
constexpr float kLog2e = 1.4426950408889634f;

struct WeightParams {
  const uint16_t* q;
  const uint16_t* k_cache;
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
  int B, N, Hq, Hkv, max_pages, num_pages;
  float scale_log2;
};

__device__ __forceinline__ float bf16_f32(uint32_t bits16) { return __uint_as_float(bits16 << 16); }

template <int D>
__global__ void __launch_bounds__(kKeys) weight_kernel(const WeightParams p) {
  __shared__ float s_q[D];
  grid_dependency_wait();
  const int b = blockIdx.z, g = blockIdx.y, t0 = blockIdx.x * kKeys, t = t0 + threadIdx.x;
  const int G = p.Hq / p.Hkv, cap = p.max_pages * kPage;
  const SeqSpan sp = seq_span(p.cu, nullptr, b, p.N, p.T);
  int bits = sp.ok ? 0 : JF_DEVERR_BAD_TREE_LEN;
  int R = p.accept_len == nullptr ? sp.n : p.accept_len[b] + 1;
  if (R < 0 || R > sp.n) {
    if (sp.ok) bits |= JF_DEVERR_BAD_PATH;
    R = max(0, min(R, sp.n));
  }
  int P = p.prefix_len[b];
  if (P < 0 || P > cap - R) {
    bits |= JF_DEVERR_BAD_PREFIX;
    P = max(0, min(P, cap));
    R = min(R, cap - P);
  }
  const int L = P + R;
  if (t0 >= L) {
    if (t0 == 0 && threadIdx.x == 0 && bits) report(p.dev_err, bits);
    return;
  }
  float kf[D];
  bool live = t < L;
  if (live) {
    const int page = p.block_table[static_cast<size_t>(b) * p.max_pages + t / kPage];
    if (page < 0 || page >= p.num_pages) {
      bits |= JF_DEVERR_BAD_PAGE;
      live = false;
    } else {
      const uint4* row = reinterpret_cast<const uint4*>(
          p.k_cache + ((static_cast<size_t>(page) * kPage + t % kPage) * p.Hkv + g) * D);
#pragma unroll
      for (int v = 0; v < D / 8; ++v) {
        const uint4 x = row[v];
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          kf[v * 8 + e * 2] = bf16_f32(w[e] & 0xffffu);
          kf[v * 8 + e * 2 + 1] = bf16_f32(w[e] >> 16);
        }
      }
    }
  }
  const size_t wi = (static_cast<size_t>(b) * p.Hkv + g) * cap + t;
  float sum = 0.f;
  for (int r = 0; r < R * G; ++r) {
    const int k = r / G, h = g * G + r % G;
    const int node = p.path == nullptr ? k : p.path[static_cast<size_t>(b) * p.N + k];
    const bool ok = node >= 0 && node < sp.n;
    if (!ok) bits |= JF_DEVERR_BAD_PATH;
    __syncthreads();
    if (ok)
      for (int d = threadIdx.x; d < D; d += kKeys)
        s_q[d] = bf16_f32(p.q[(static_cast<size_t>(sp.row0 + node) * p.Hq + h) * D + d]);
    __syncthreads();
    if (!ok || !live || t > P + k) continue;
    const float lse = p.cu != nullptr ? p.lse[static_cast<size_t>(h) * p.T + sp.row0 + node]
                                      : p.lse[(static_cast<size_t>(b) * p.Hq + h) * p.N + node];
    float s = 0.f;
#pragma unroll
    for (int d = 0; d < D; ++d) s = fmaf(s_q[d], kf[d], s);
    if (lse != -INFINITY) sum += exp2f(fmaf(s, p.scale_log2, -lse * kLog2e));
  }
  if (live) p.weight_out[wi] = (t < P && p.weight != nullptr ? p.weight[wi] : 0.f) + sum;
  if (bits) report(p.dev_err, bits);
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
  if (cu == nullptr && static_cast<long long>(max_pages) * kPage < 1) return JF_ERR_UNSUPPORTED;
  if (cu != nullptr && T < 1) return JF_ERR_INVALID_ARGUMENT;
  if (cu != nullptr && static_cast<long long>(T) + N >= (1ll << 31)) return JF_ERR_UNSUPPORTED;
  if (!aligned_to(q, 16) || !aligned_to(k_cache, 16)) return JF_ERR_MISALIGNED;
  WeightParams p;
  p.q = static_cast<const uint16_t*>(q);
  p.k_cache = static_cast<const uint16_t*>(k_cache);
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
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  p.scale_log2 = scale * kLog2e;
  const dim3 grid(static_cast<unsigned>((max_pages * kPage + kKeys - 1) / kKeys), Hkv, B);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = D == 128 ? launch_pdl(weight_kernel<128>, grid, dim3(kKeys), 0, s, p)
                                 : launch_pdl(weight_kernel<64>, grid, dim3(kKeys), 0, s, p);
  return e == cudaSuccess ? JF_OK : JF_ERR_CUDA;
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
