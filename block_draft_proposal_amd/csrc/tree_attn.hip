// Attention of drafted nodes over a paged cache: one wave per (node, query
// head).  64 keys at a time: each lane scores one key, the wave takes the
// running maximum and sum, and each lane then adds the weighted rows of V at
// its own elements.  All arithmetic in fp32.
#include "kv_cache.h"

namespace dflash {
namespace {

template <int DT>
__device__ __forceinline__ float kv_element(const unsigned char* row, int d, float scale) {
  if constexpr (DT == DFLASH_BF16) return bf16_to_f32(reinterpret_cast<const uint16_t*>(row)[d]);
  else if constexpr (DT == DFLASH_E4M3) return __builtin_amdgcn_cvt_f32_fp8((int)row[d], 0) * scale;
  else return (float)(int8_t)row[d] * scale;
}

template <int DT, int D>
__global__ void __launch_bounds__(64) tree_attention_kernel(TreeArgs a) {
  __shared__ float w[64];
  __shared__ int64_t v_at[64];
  __shared__ float v_scale[64];
  __shared__ float q[D];
  const KvView& c = a.c;
  const int lane = threadIdx.x, node = blockIdx.x, h = blockIdx.y, req = blockIdx.z;
  const int64_t first = c.offsets[req], n = min((int64_t)c.offsets[req + 1] - first, (int64_t)a.max_nodes);
  if (node >= n || first < 0 || first + node >= c.n_rows) return;
  const int64_t start = max(c.start[req], 0), len = start + n;
  const int kvh = h / (a.n_q_heads / c.n_kv_heads);
  const int32_t* table = c.table + req * c.table_stride;
  constexpr int kBytes = DT == DFLASH_BF16 ? 2 : 1, kOwn = D / 64;
  for (int d = lane; d < D; d += 64) q[d] = bf16_to_f32(a.q[(first + node) * a.q_row + h * a.q_head + d]);
  float m = -INFINITY, l = 0.f, o[kOwn] = {};
  bool any = false;
  __syncthreads();
  for (int64_t t0 = 0; t0 < len; t0 += 64) {
    const int64_t t = t0 + lane;
    bool see = t < start;
    if (t >= start && t < len) {
      const int64_t j = t - start;
      see = a.mask ? (a.mask[(first + node) * a.mask_words + j / 64] >> (j % 64)) & 1 : j <= node;
    }
    float s = -INFINITY;
    v_at[lane] = -1;
    if (see) {
      int64_t page;
      int32_t slot;
      if (!kv_locate(c, table, t, page, slot)) {
        s = __builtin_nanf("");
      } else {
        const int64_t row = (int64_t)kvh * c.page_size + slot;
        const unsigned char* kr = c.k + page * c.page_bytes + row * D * kBytes;
        const float ks = DT == DFLASH_BF16 ? 1.f : kv_scale_value(c.k_scale[page * c.scale_page_bytes + row]);
        float dot = 0.f;
        for (int d = 0; d < D; ++d) dot = fmaf(q[d], kv_element<DT>(kr, d, 1.f), dot);
        s = dot * ks * a.scale;
        v_at[lane] = page * c.page_bytes + row * D * kBytes;
        v_scale[lane] = DT == DFLASH_BF16 ? 1.f : kv_scale_value(c.v_scale[page * c.scale_page_bytes + row]);
      }
    }
    any = any || __any(see);
    const float top = fmaxf(m, wave_max_f32(s)), base = top == -INFINITY ? 0.f : top;
    const float p = see ? expf(s - base) : 0.f, keep = m == -INFINITY ? 0.f : expf(m - base);
    m = top;
    float sum = p;
    for (int x = 32; x > 0; x >>= 1) sum += __shfl_xor(sum, x, 64);
    l = l * keep + sum;
    w[lane] = p;
    __syncthreads();
    for (int i = 0; i < kOwn; ++i) {
      o[i] *= keep;
      for (int j = 0; j < 64; ++j)
        if (v_at[j] >= 0) o[i] = fmaf(w[j], kv_element<DT>(c.v + v_at[j], lane + 64 * i, v_scale[j]), o[i]);
    }
    __syncthreads();
  }
  for (int i = 0; i < kOwn; ++i)
    a.out[((first + node) * a.n_q_heads + h) * D + lane + 64 * i] = (uint16_t)f32_to_bf16_rne(any ? o[i] / l : 0.f);
}

template <int DT>
hipError_t launch_dt(const TreeArgs& a, hipStream_t s) {
  const dim3 g((unsigned)a.max_nodes, (unsigned)a.n_q_heads, (unsigned)a.c.n_req);
  if (a.c.head_dim == 64) tree_attention_kernel<DT, 64><<<g, 64, 0, s>>>(a);
  else if (a.c.head_dim == 128) tree_attention_kernel<DT, 128><<<g, 64, 0, s>>>(a);
  else tree_attention_kernel<DT, 256><<<g, 64, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

size_t tree_attention_bytes(const KvView&, int32_t, int32_t, int32_t) { return 0; }

hipError_t launch_tree_attention(const TreeArgs& a, hipStream_t stream) {
  if (a.c.dtype == DFLASH_BF16) return launch_dt<DFLASH_BF16>(a, stream);
  if (a.c.dtype == DFLASH_E4M3) return launch_dt<DFLASH_E4M3>(a, stream);
  return launch_dt<DFLASH_I8>(a, stream);
}

}  // namespace dflash
