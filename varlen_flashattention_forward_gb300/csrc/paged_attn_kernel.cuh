// paged_attn_kernel.cuh -- attention over the paged 8-bit cache.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "paged_index.h"
#include "paged_kv_kernels.cuh"

namespace fa {

struct PagedAttnArgs {
  const uint16_t* q;
  long long q_row, q_head;
  const uint8_t *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  const int *cu, *seq_lens, *page_table;
  int batch, total_q, heads, heads_k, dim, max_pages, num_pages;
  float scale;
  int causal, window;
  uint16_t* out;
  float* lse;
};

// One block per query row and head: 128 keys at a time, one key a thread for
// the scores and one dim a thread for the values.
__global__ void __launch_bounds__(128) paged_attn_rows_kernel(const PagedAttnArgs a) {
  __shared__ float s_q[128], s_p[128], s_red[4];
  __shared__ int s_page[128];
  __shared__ float s_vs[128];
  const FoundUnit u = find_unit(blockIdx.x, a.batch, [&](int b) {
    return row_range(__ldg(a.cu + b), __ldg(a.cu + b + 1), a.total_q).n;
  });
  if (u.seq < 0) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const RowRange r = row_range(__ldg(a.cu + u.seq), __ldg(a.cu + u.seq + 1), a.total_q);
  const long long token = (long long)r.lo + u.at;
  const int h = blockIdx.y, hk = h / (a.heads / a.heads_k);
  const KeyRange kr = key_range(u.at, u.at, r.n, __ldg(a.seq_lens + u.seq),
                                a.max_pages * kPageTokens, a.causal != 0, a.window);
  if (tid < a.dim)
    s_q[tid] = __uint_as_float((uint32_t)a.q[token * a.q_row + h * a.q_head + tid] << 16);
  __syncthreads();
  const float neg_inf = -__int_as_float(0x7f800000);
  float m = neg_inf, l = 0.f, acc = 0.f;
  for (int j0 = kr.lo; j0 < kr.hi; j0 += 128) {
    const int j = j0 + tid;
    int page = -1;
    float s = neg_inf, vs = 0.f;
    if (j < kr.hi)
      page = checked_page(
          __ldg(a.page_table + (size_t)u.seq * a.max_pages + j / kPageTokens), a.num_pages);
    if (page >= 0) {
      const size_t cell = (size_t)page * a.heads_k + hk;
      const uint8_t* row = a.k_cache + (cell * kPageTokens + j % kPageTokens) * a.dim;
      float dot = 0.f;
      for (int c = 0; c < a.dim; c += 4) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(row + c);
        const float2 lo = f16x2_floats(unpack_e4m3x2(w)), hi = f16x2_floats(unpack_e4m3x2(w >> 16));
        dot += lo.x * s_q[c] + lo.y * s_q[c + 1] + hi.x * s_q[c + 2] + hi.y * s_q[c + 3];
      }
      s = dot * a.k_scale[cell] * a.scale;
      vs = a.v_scale[cell];
    }
    float mx = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (lane == 0) s_red[warp] = mx;
    s_page[tid] = page;
    s_vs[tid] = vs;
    __syncthreads();
    mx = fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]));
    const float m_new = fmaxf(m, mx);
    const float p = m_new == neg_inf ? 0.f : expf(s - m_new);
    const float old = m_new == neg_inf ? 1.f : expf(m - m_new);
    m = m_new;
    s_p[tid] = p;
    __syncthreads();
    float sum = 0.f, o = 0.f;
    const int n = imin(128, kr.hi - j0);
    for (int i = 0; i < n; ++i) {
      sum += s_p[i];
      if (tid < a.dim && s_page[i] >= 0) {
        const size_t cell = (size_t)s_page[i] * a.heads_k + hk;
        const uint32_t w =
            a.v_cache[(cell * kPageTokens + (j0 + i) % kPageTokens) * a.dim + tid];
        o += s_p[i] * s_vs[i] * f16x2_floats(unpack_e4m3x2(w)).x;
      }
    }
    l = l * old + sum;
    acc = acc * old + o;
    __syncthreads();
  }
  if (tid < a.dim) {
    const float v = l > 0.f ? acc / l : 0.f;
    a.out[((size_t)token * a.heads + h) * a.dim + tid] = (uint16_t)ptx::pack_bf16x2(v, 0.f);
  }
  if (tid == 0 && a.lse)
    a.lse[(size_t)h * a.total_q + token] = l > 0.f ? m + logf(l) : neg_inf;
}

}  // namespace fa
