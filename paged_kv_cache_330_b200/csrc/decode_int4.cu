// Paged decode attention over the INT4 KV cache (format: kv_int4.cu).
//
// For every sequence b and query head h,
//   out[b][h] = sum_t softmax_t(scale <q[b][h], Kd_b[t][h/G]>) Vd_b[t][h/G],
// with Kd, Vd the rows s * (code + z).  One CTA per (sequence, KV head); 128
// tokens a round: thread = token for the scores, thread = column for PV.

#include <algorithm>

#include "common.cuh"
#include "host_common.h"

PA_DEFINE_ERROR_WORD(pa__err_decode_int4)

namespace {

using namespace pa;

struct Params {
  const void* q;
  void* out;
  float* lse;
  const uint8_t* kc;
  const uint8_t* vc;
  const uint32_t* kp;
  const uint32_t* vp;
  const int32_t* block_tables;
  const int32_t* context_lens;
  int max_blocks_per_seq, batch, num_q_heads, num_kv_heads, block_size, num_blocks;
  float scale_log2;
};

template <int DT, int D>
__global__ void __launch_bounds__(128) decode_int4_kernel(const Params p, int G) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int NG = D / 64;
  __shared__ float qs[16 * D], ps[128 * 16], red[4][16];
  __shared__ int64_t rows[128];
  const int b = blockIdx.y, g = blockIdx.x, tid = threadIdx.x, warp = tid >> 5;
  const int cap = p.max_blocks_per_seq * p.block_size;
  int L = __ldg(p.context_lens + b);
  if (L < 0 || L > cap) {
    if (tid == 0) PA_RECORD_ERROR(PA_ERRBIT_INDEX);
    L = min(max(L, 0), cap);
  }
  using T = typename Elt<DT>::T;
  const T* q = reinterpret_cast<const T*>(p.q) + ((size_t)b * p.num_q_heads + (size_t)g * G) * D;
  for (int i = tid; i < G * D; i += 128) qs[i] = (float)q[i] * p.scale_log2;
  float m[16], l[16], o[16];
  for (int h = 0; h < 16; ++h) m[h] = -INFINITY, l[h] = 0.f, o[h] = 0.f;
  for (int t0 = 0; t0 < L; t0 += 128) {
    __syncthreads();
    const int t = t0 + tid;
    float s[16];
    for (int h = 0; h < 16; ++h) s[h] = -INFINITY;
    if (t < L) {
      int blk = __ldg(p.block_tables + (size_t)b * p.max_blocks_per_seq + t / p.block_size);
      if (blk < 0 || blk >= p.num_blocks) {
        PA_RECORD_ERROR(PA_ERRBIT_INDEX);
        blk = 0;
      }
      const int64_t row = ((int64_t)blk * p.num_kv_heads + g) * p.block_size + t % p.block_size;
      rows[tid] = row;
      for (int h = 0; h < G; ++h) s[h] = 0.f;
      const uint32_t* w = reinterpret_cast<const uint32_t*>(p.kc) + row * (D / 8);
      for (int j = 0; j < D / 8; ++j) {
        const float2 par = Elt<DT>::to_f2(__ldg(p.kp + row * NG + j % NG));
        const uint32_t word = __ldg(w + j);
        const int d = 64 * (j % NG) + 8 * (j / NG);
        for (int e = 0; e < 8; ++e) {
          const float x = par.x * ((float)((word >> (4 * e)) & 15u) + par.y);
          for (int h = 0; h < G; ++h) s[h] = fmaf(x, qs[h * D + d + e], s[h]);
        }
      }
    }
    float mn[16];
    for (int h = 0; h < G; ++h) {
      float v = s[h];
      for (int k = 16; k > 0; k >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, k));
      if ((tid & 31) == 0) red[warp][h] = v;
    }
    __syncthreads();
    for (int h = 0; h < G; ++h) {
      mn[h] = fmaxf(m[h], fmaxf(fmaxf(red[0][h], red[1][h]), fmaxf(red[2][h], red[3][h])));
      ps[tid * 16 + h] = fast_exp2(s[h] - mn[h]);
      const float alpha = fast_exp2(m[h] - mn[h]);
      l[h] *= alpha;
      o[h] *= alpha;
      m[h] = mn[h];
    }
    __syncthreads();
    const int n = min(128, L - t0), d = tid;
    for (int k = 0; k < n; ++k) {
      float x = 0.f;
      if (d < D) {
        const int64_t row = rows[k];
        const int grp = d / 64, word = (d % 64) / 8 * NG + grp;
        const uint32_t c = (__ldg(reinterpret_cast<const uint32_t*>(p.vc) + row * (D / 8) + word) >> (4 * (d % 8))) & 15u;
        const float2 par = Elt<DT>::to_f2(__ldg(p.vp + row * NG + grp));
        x = par.x * ((float)c + par.y);
      }
      for (int h = 0; h < G; ++h) {
        o[h] = fmaf(ps[k * 16 + h], x, o[h]);
        l[h] += ps[k * 16 + h];
      }
    }
  }
  T* out = reinterpret_cast<T*>(p.out) + ((size_t)b * p.num_q_heads + (size_t)g * G) * D;
  for (int h = 0; h < G; ++h) {
    if (tid < D) out[h * D + tid] = Elt<DT>::from_f(L > 0 ? o[h] / l[h] : 0.f);
    if (tid == 0 && p.lse)
      p.lse[(size_t)b * p.num_q_heads + g * G + h] = L > 0 ? (m[h] + __log2f(l[h])) * 0.6931471805599453f : -INFINITY;
  }
}

bool make_plan(int batch, int Hq, int Hkv, int D, int max_context_len, int num_partitions, int* grid, size_t* bytes) {
  if (batch < 0 || Hq <= 0 || Hkv <= 0 || num_partitions < 0 || max_context_len < 0 || Hq % Hkv) return false;
  if (!valid_head_dim(D) || !valid_group(Hq / Hkv)) return false;
  *grid = num_partitions ? num_partitions : sm_count();
  *bytes = 256;
  return true;
}

}  // namespace

extern "C" int pa_decode_int4_plan(int batch, int num_q_heads, int num_kv_heads, int head_dim, int max_context_len,
                                   int num_partitions_or_0, int* grid_out, int* max_pieces_out,
                                   size_t* workspace_bytes_out) {
  int grid;
  size_t bytes;
  if (!make_plan(batch, num_q_heads, num_kv_heads, head_dim, max_context_len, num_partitions_or_0, &grid, &bytes))
    return PA_ERR_INVALID;
  if (grid_out) *grid_out = grid;
  if (max_pieces_out) *max_pieces_out = batch * num_kv_heads + grid;
  if (workspace_bytes_out) *workspace_bytes_out = bytes;
  return PA_OK;
}

extern "C" size_t pa_decode_int4_workspace_size(int batch, int num_q_heads, int num_kv_heads, int head_dim,
                                                int max_context_len, int num_partitions_or_0) {
  int grid;
  size_t bytes;
  return make_plan(batch, num_q_heads, num_kv_heads, head_dim, max_context_len, num_partitions_or_0, &grid, &bytes)
             ? bytes
             : 0;
}

extern "C" int pa_decode_int4(const void* q, const void* k_codes, const void* v_codes, const void* k_params,
                              const void* v_params, const int32_t* block_tables, int max_blocks_per_seq,
                              const int32_t* context_lens, int batch, int num_q_heads, int num_kv_heads, int head_dim,
                              int block_size, int num_blocks, int max_context_len, float scale, int dtype,
                              void* workspace, size_t workspace_bytes, int num_partitions_or_0, void* out,
                              float* lse_out, void* stream) {
  if (batch < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || num_blocks < 0 || max_context_len < 0 ||
      max_blocks_per_seq < 0 || num_partitions_or_0 < 0)
    return PA_ERR_INVALID;
  if (!valid_dtype(dtype) || !valid_head_dim(head_dim) || !valid_block_size(block_size)) return PA_ERR_UNSUPPORTED;
  if (num_q_heads % num_kv_heads != 0) return PA_ERR_INVALID;
  const int G = num_q_heads / num_kv_heads;
  if (!valid_group(G)) return PA_ERR_UNSUPPORTED;
  if (batch == 0) return PA_OK;
  if (!q || !k_codes || !v_codes || !k_params || !v_params || !block_tables || !context_lens || !out)
    return PA_ERR_INVALID;
  if (!aligned16(q) || !aligned16(k_codes) || !aligned16(v_codes) || !aligned16(k_params) || !aligned16(v_params) ||
      !aligned16(out) || (reinterpret_cast<uintptr_t>(block_tables) & 3u) ||
      (reinterpret_cast<uintptr_t>(context_lens) & 3u) || (reinterpret_cast<uintptr_t>(lse_out) & 3u))
    return PA_ERR_ALIGN;
  if ((int64_t)max_blocks_per_seq * block_size < max_context_len) return PA_ERR_INVALID;
  if (num_blocks == 0 && max_context_len > 0) return PA_ERR_INVALID;
  if ((int64_t)num_blocks * block_size >= (1ll << 31)) return PA_ERR_UNSUPPORTED;
  if ((int64_t)max_blocks_per_seq * block_size >= (1ll << 31)) return PA_ERR_UNSUPPORTED;
  int grid;
  size_t bytes;
  if (!make_plan(batch, num_q_heads, num_kv_heads, head_dim, max_context_len, num_partitions_or_0, &grid, &bytes))
    return PA_ERR_INVALID;
  if (!workspace || workspace_bytes < bytes) return PA_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return PA_ERR_ALIGN;
  Params p;
  p.q = q;
  p.out = out;
  p.lse = lse_out;
  p.kc = (const uint8_t*)k_codes;
  p.vc = (const uint8_t*)v_codes;
  p.kp = (const uint32_t*)k_params;
  p.vp = (const uint32_t*)v_params;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.batch = batch;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.block_size = block_size;
  p.num_blocks = num_blocks;
  p.scale_log2 = scale * 1.4426950408889634f;
  auto kern = dtype == PA_BF16 ? (head_dim == 128 ? decode_int4_kernel<PA_BF16, 128> : decode_int4_kernel<PA_BF16, 64>)
                               : (head_dim == 128 ? decode_int4_kernel<PA_F16, 128> : decode_int4_kernel<PA_F16, 64>);
  return launch_programmatic(kern, dim3((unsigned)num_kv_heads, (unsigned)batch), dim3(128), 0, (cudaStream_t)stream, p,
                             G);
}
