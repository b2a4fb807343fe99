// INT4 KV cache: the quantising cache write (alone and behind the rotary
// embedding), the block copy, and the expansion of blocks into a 16-bit cache.
//
// KV-cache compression is among the tuning steps of "Nano-vLLM-Ascend:
// lightweight LLM inference framework for Ascend NPU", section 4.3; the pages
// give no format.  The one built here cuts a row of D values (one token, one
// KV head) into groups of 64; a group holds unsigned 4-bit codes, a scale s and
// a zero point z (both in the 16-bit type of the values) and stands for
// s * (code + z):
//
//   lo = min x;  hi = max x;  s = round16(hi / 15 - lo / 15);  z = round16(lo / s);
//   code = clamp(rint(x * (1 / s) - z), 0, 15)
//
// in fp32, every operation rounded by itself (so another IEEE implementation
// reaches the same codes).  The quotients are subtracted, not the values: hi -
// lo can overflow, the difference of the quotients cannot.  s and z are rounded
// before the codes are taken, so a value inside the range the codes span is off
// by half a step s; the rounding shifts that range by up to u (15 + |z|) steps
// (u half a step of the type, 2^-8 or 2^-11), and values beyond its ends are
// clamped and lose what was shifted.  s < 2^-126 (all values alike, or nearer
// than the type can say; 1 / s would overflow): s = |lo|, z = sign(lo), codes 0.
// One group never spans tokens: appending a token re-quantises nothing.  A NaN
// in a group makes both extremes NaN, and s and z with them; an infinity makes s
// infinite or NaN.  Either way the group stands for nothing finite.
//
// Layout: codes [num_blocks][Hkv][block_size][D/2], parameters
// [num_blocks][Hkv][block_size][D/64][2].  Word j (8 codes) of a row holds
// values 8 * (j div n) .. of group j mod n, n = D/64.
//
// Work split of the write and of the expansion: D/16 threads per row, each with
// 8 values of the first and 8 of the second half of the row.  That pair is what
// a rotate-half embedding turns, a 16-byte vector of the input twice, and (at D
// 128, where the halves are the groups) two neighbouring words of the stored
// row; at D 64 it is words j and j + 4.

#include "common.cuh"
#include "host_common.h"

PA_DEFINE_ERROR_WORD(pa__err_int4)

namespace {

using namespace pa;

__device__ __forceinline__ uint4 ld_plain_v4(const void* p) {  // q and k may be overwritten in place
  uint4 r;
  asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}

template <int DT>
__device__ __forceinline__ void unpack8(uint4 u, float* x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = Elt<DT>::to_f2(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

template <int DT>
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(Elt<DT>::from_f2(x[0], x[1]), Elt<DT>::from_f2(x[2], x[3]), Elt<DT>::from_f2(x[4], x[5]),
                    Elt<DT>::from_f2(x[6], x[7]));
}

// 8 values -> a word of 8 codes, code = clamp(rint(x * inv - shift), 0, 15); HELD: x becomes the values s * (code + z)
// that they stand for (unrounded).  Clamping before rounding gives what rounding first gives (the ends are whole), and
// keeps the sum with 1.5 * 2^23 exact but for its one rounding, to a whole number, half to even; the code is then in
// that sum's low bits.
template <bool HELD>
__device__ __forceinline__ uint32_t encode8(float* x, float s, float z, float inv, float shift) {
  constexpr float kWhole = 12582912.f;
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float m = __fadd_rn(fminf(fmaxf(__fsub_rn(__fmul_rn(x[i], inv), shift), 0.f), 15.f), kWhole);
    word += (__float_as_uint(m) - __float_as_uint(kWhole)) << (4 * i);
    if (HELD) x[i] = __fmul_rn(s, __fadd_rn(__fsub_rn(m, kWhole), z));
  }
  return word;
}

// The smaller and the larger of two, NaN where either is: fminf and fmaxf would drop it, and with it what went wrong in
// the values of a group.
__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float min8(const float* x) {
  return min_nan(min_nan(min_nan(x[0], x[1]), min_nan(x[2], x[3])), min_nan(min_nan(x[4], x[5]), min_nan(x[6], x[7])));
}
__device__ __forceinline__ float max8(const float* x) {
  return max_nan(max_nan(max_nan(x[0], x[1]), max_nan(x[2], x[3])), max_nan(max_nan(x[4], x[5]), max_nan(x[6], x[7])));
}

struct WriteArgs {
  const uint4* q;  // rotary form only
  uint4* q_out;
  const uint4* k;
  const uint4* v;
  const int64_t* positions;
  const float4* cos_t;
  const float4* sin_t;
  const int64_t* slots;
  uint8_t* kc;
  uint8_t* vc;
  uint32_t* kp;
  uint32_t* vp;
  uint4* k_out;  // may be null
  uint4* v_out;
  int64_t num_slots, max_position;
  int total;  // threads' items: tokens * (hq + 2 * hkv) * D / 16
  int hq, hkv, bs_shift;  // block sizes are powers of two
};

// 4096 tokens, 32 + 8 heads of 128 (107 MB): 256 threads a CTA 24.2 us, 128 threads 23.2, 128 with 42 registers (12 CTAs
// an SM: the loads of a row wait for its position's and slot's) 22.5, 4.8 TB/s.  4096 tokens without the embedding (38 MB
// with the rows as held): 9.4 us, 4.1 TB/s, by issue: 72 % of the slots.  128 tokens: 1.7 us in a graph, launch alone.
constexpr int kWriteThreads = 128;
// Items: per token hq rows of q (rotary form), hkv rows of k, hkv rows of v; D/16 neighbouring threads a row.
// Warps run whole iterations (the group extremes come from shuffles), threads past the end idle along.
template <int DT, int D, bool ROPE>
__global__ void __launch_bounds__(kWriteThreads, 12) write_kv_int4_kernel(const WriteArgs a) {
  // a decode launched after this may start its set-up now; it waits for this grid before it reads the cache
  asm volatile("griddepcontrol.launch_dependents;");
  // launched programmatically itself: wait for the preceding grid before reading inputs or writing slots
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int TPR = D / 16, NG = D / 64;
  const int rows = a.hq + 2 * a.hkv;
  {
    const int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
    const bool in = i < a.total;
    const int row = in ? (int)i / TPR : 0, j = (int)i % TPR;
    const int t = row / rows, r = row - t * rows;
    const bool isq = ROPE && r < a.hq, isv = r >= a.hq + a.hkv;
    const int h = isq ? r : (isv ? r - a.hq - a.hkv : r - a.hq);
    bool live = in;
    int64_t pos = 0, slot = 0;
    // the row's values are on their way while its position and slot are looked up
    float x1[8], x2[8];
    uint4 u1 = make_uint4(0, 0, 0, 0), u2 = u1;
    if (in) {
      const uint4* src = (isq ? a.q : (isv ? a.v : a.k)) + (isq ? (int64_t)t * a.hq + h : (int64_t)t * a.hkv + h) * (D / 8) + j;
      u1 = ld_plain_v4(src);
      u2 = ld_plain_v4(src + TPR);
    }
    if (ROPE && in) {
      pos = __ldg(a.positions + t);
      if (pos < 0 || pos >= a.max_position) {  // broken caller invariant: record once per token, write nothing
        if (r == 0 && j == 0) PA_RECORD_ERROR(PA_ERRBIT_INDEX);
        live = false;
      }
    }
    if (live && !isq) {
      slot = __ldg(a.slots + t);
      if (slot >= a.num_slots && r == a.hq && j == 0) PA_RECORD_ERROR(PA_ERRBIT_INDEX);
      live = slot >= 0 && slot < a.num_slots;
    }
    const int64_t src_row = isq ? (int64_t)t * a.hq + h : (int64_t)t * a.hkv + h;
    const int64_t vec = src_row * (D / 8) + j;
    if (live) {
      unpack8<DT>(u1, x1);
      unpack8<DT>(u2, x2);
      if (ROPE && !isv) {
        const int64_t tb = pos * (D / 8) + 2 * j;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const float4 c = __ldg(a.cos_t + tb + half), s = __ldg(a.sin_t + tb + half);
          const float cv[4] = {c.x, c.y, c.z, c.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float p = x1[4 * half + e], w = x2[4 * half + e];
            x1[4 * half + e] = fmaf(p, cv[e], -__fmul_rn(w, sv[e]));
            x2[4 * half + e] = fmaf(w, cv[e], __fmul_rn(p, sv[e]));
          }
        }
        u1 = pack8<DT>(x1);
        u2 = pack8<DT>(x2);
        if (isq) {
          st_v4(a.q_out + vec, u1);
          st_v4(a.q_out + vec + TPR, u2);
        }
        unpack8<DT>(u1, x1);  // the key as the 16-bit cache would hold it
        unpack8<DT>(u2, x2);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x1[e] = x2[e] = 0.f;
    }
    if (ROPE && __all_sync(0xffffffffu, isq || !in)) return;
    float lo1 = min8(x1), hi1 = max8(x1), lo2 = min8(x2), hi2 = max8(x2);
    if constexpr (NG == 1) {
      lo1 = min_nan(lo1, lo2);
      hi1 = max_nan(hi1, hi2);
    }
#pragma unroll
    for (int o = TPR / 2; o > 0; o >>= 1) {
      lo1 = min_nan(lo1, __shfl_xor_sync(0xffffffffu, lo1, o));
      hi1 = max_nan(hi1, __shfl_xor_sync(0xffffffffu, hi1, o));
      if constexpr (NG == 2) {
        lo2 = min_nan(lo2, __shfl_xor_sync(0xffffffffu, lo2, o));
        hi2 = max_nan(hi2, __shfl_xor_sync(0xffffffffu, hi2, o));
      }
    }
    // Four quotients a group, each an IEEE division: taken by one lane each (two a lane, not eight) and handed round.
    // Lane j of the row: group (j / 2) mod n, the even lane hi / 15 and lo / s, the odd one lo / 15 and 1 / s.
    const bool odd = j & 1, second = NG == 2 && (j & 2);
    const float lo = second ? lo2 : lo1, hi = second ? hi2 : hi1;
    const float q15 = __fdiv_rn(odd ? lo : hi, 15.f), other = __shfl_xor_sync(0xffffffffu, q15, 1);
    float s = Elt<DT>::to_f2(Elt<DT>::from_f2(odd ? __fsub_rn(other, q15) : __fsub_rn(q15, other), 0.f)).x;
    const bool alike = s < 1.17549435e-38f;  // a NaN is not: s and z are NaN then, every code 0
    float quot = __fdiv_rn(odd ? 1.f : lo, alike ? 1.f : s);
    if (alike) {
      s = fabsf(lo);
      quot = odd ? 0.f : (lo > 0.f ? 1.f : (lo < 0.f ? -1.f : 0.f));  // 1 / s taken as 0: every code is 0
    }
    const uint32_t pword = Elt<DT>::from_f2(s, quot);  // (s, z) in the even lane
    if (!odd) quot = Elt<DT>::to_f2(pword).y;
    const float s1 = __shfl_sync(0xffffffffu, s, 0, TPR), z1 = __shfl_sync(0xffffffffu, quot, 0, TPR),
                inv1 = __shfl_sync(0xffffffffu, quot, 1, TPR);
    float s2 = s1, z2 = z1, inv2 = inv1;
    if constexpr (NG == 2) {
      s2 = __shfl_sync(0xffffffffu, s, 2, TPR);
      z2 = __shfl_sync(0xffffffffu, quot, 2, TPR);
      inv2 = __shfl_sync(0xffffffffu, quot, 3, TPR);
    }
    if (!live || isq) return;
    // where 1 / s is taken as 0 every code is to be 0: the shift 1 sees to it
    const float shift1 = inv1 == 0.f ? 1.f : z1, shift2 = inv2 == 0.f ? 1.f : z2;
    uint4* held = isv ? a.v_out : a.k_out;
    uint32_t w1, w2;
    if (held) {
      w1 = encode8<true>(x1, s1, z1, inv1, shift1);
      w2 = encode8<true>(x2, s2, z2, inv2, shift2);
      st_v4(held + vec, pack8<DT>(x1));
      st_v4(held + vec + TPR, pack8<DT>(x2));
    } else {
      w1 = encode8<false>(x1, s1, z1, inv1, shift1);
      w2 = encode8<false>(x2, s2, z2, inv2, shift2);
    }
    const int64_t blk = slot >> a.bs_shift;
    const int64_t crow = ((blk * a.hkv + h) << a.bs_shift) + (slot & ((1 << a.bs_shift) - 1));
    uint32_t* cw = reinterpret_cast<uint32_t*>(isv ? a.vc : a.kc) + crow * (D / 8);
    uint32_t* pw = (isv ? a.vp : a.kp) + crow * NG;
    if constexpr (NG == 2) {
      reinterpret_cast<uint2*>(cw)[j] = make_uint2(w1, w2);
    } else {
      cw[j] = w1;
      cw[j + 4] = w2;
    }
    if (!odd && j < 2 * NG) pw[j >> 1] = pword;
  }
}

// Block copy: CTA (pair, part); a part is up to kCopyLoads * 256 16-byte vectors of the pair's four runs, end to end.
// Every thread has its loads in flight before the first store: 4096 blocks of 16 x 8 x 128 (151 MB both ways) 25.0 us,
// 6.0 TB/s; with two loads in flight 26.1, with one 32.1.
constexpr int kCopyLoads = 5;
__global__ void __launch_bounds__(256) copy_blocks_int4_kernel(const int32_t* __restrict__ pairs, int code_vecs,
                                                               int param_vecs, int num_blocks, int per_part, uint4* kc,
                                                               uint4* vc, uint4* kp, uint4* vp) {
  // as the writes: let the next kernel's set-up begin, wait for the preceding one
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int32_t src = __ldg(pairs + 2 * (int64_t)blockIdx.x), dst = __ldg(pairs + 2 * (int64_t)blockIdx.x + 1);
  if (src < 0 || src >= num_blocks || dst < 0 || dst >= num_blocks) {
    if (threadIdx.x == 0 && blockIdx.y == 0) PA_RECORD_ERROR(PA_ERRBIT_INDEX);
    return;
  }
  const int total = 2 * (code_vecs + param_vecs);
  for (int64_t part = blockIdx.y * (int64_t)per_part; part < total; part += (int64_t)gridDim.y * per_part) {
    const int end = (int)min((int64_t)total, part + per_part);
    uint4 u[kCopyLoads];
    uint4* to[kCopyLoads];
#pragma unroll
    for (int e = 0; e < kCopyLoads; ++e) {
      const int i = (int)part + e * 256 + threadIdx.x;
      to[e] = nullptr;
      if (i < end) {
        const bool codes = i < 2 * code_vecs;
        const int per = codes ? code_vecs : param_vecs;
        int o = codes ? i : i - 2 * code_vecs;
        const bool isv = o >= per;
        if (isv) o -= per;
        uint4* base = codes ? (isv ? vc : kc) : (isv ? vp : kp);
        u[e] = ld_plain_v4(base + (int64_t)src * per + o);
        to[e] = base + (int64_t)dst * per + o;
      }
    }
#pragma unroll
    for (int e = 0; e < kCopyLoads; ++e)
      if (to[e]) st_v4(to[e], u[e]);
  }
}

// 8 codes of a word -> values s * (code + z), rounded to the type.  A code becomes a float by one permute, as the low
// byte of 2^23.
template <int DT>
__device__ __forceinline__ uint4 expand8(uint32_t w, uint32_t param) {
  const float2 p = Elt<DT>::to_f2(param);
  const uint32_t even = w & 0x0f0f0f0fu, odd = (w >> 4) & 0x0f0f0f0fu;
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t m = __byte_perm((i & 1) ? odd : even, 0x4B000000u, 0x7440u | (uint32_t)(i >> 1));
    x[i] = __fmul_rn(p.x, __fadd_rn(__fsub_rn(__uint_as_float(m), 8388608.f), p.y));
  }
  return pack8<DT>(x);
}

// Expansion: CTA (pair and K or V, part of the block's rows); rows in the order of the 16-bit block; a thread has the
// loads of kLoadItems items in flight before it expands the first: 4096 blocks of 16 x 8 x 128 (344 MB) 59.3 us, 5.8 TB/s,
// by the writes; with two items in flight 63, with one 76.
constexpr int kLoadItems = 4;
template <int DT, int D>
__global__ void __launch_bounds__(256) load_blocks_int4_kernel(const int32_t* __restrict__ pairs, int hkv,
                                                               int block_size, int num_blocks, int num_dst,
                                                               const uint32_t* __restrict__ kc,
                                                               const uint32_t* __restrict__ vc,
                                                               const uint32_t* __restrict__ kp,
                                                               const uint32_t* __restrict__ vp, uint4* __restrict__ k,
                                                               uint4* __restrict__ v) {
  // as the writes: let the next kernel's set-up begin, wait for the preceding one
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int TPR = D / 16, NG = D / 64;
  const int64_t pair = blockIdx.x >> 1;
  const bool isv = blockIdx.x & 1;
  const int32_t src = __ldg(pairs + 2 * pair), dst = __ldg(pairs + 2 * pair + 1);
  if (src < 0 || src >= num_blocks || dst < 0 || dst >= num_dst) {
    if (threadIdx.x == 0 && blockIdx.y == 0 && !isv) PA_RECORD_ERROR(PA_ERRBIT_INDEX);
    return;
  }
  const int64_t rows = (int64_t)hkv * block_size;
  const uint32_t* codes = (isv ? vc : kc) + src * rows * (D / 8);
  const uint32_t* params = (isv ? vp : kp) + src * rows * NG;
  uint4* out = (isv ? v : k) + dst * rows * (D / 8);
  const int total = (int)rows * TPR;
  for (int64_t part = blockIdx.y * (int64_t)(kLoadItems * 256); part < total; part += (int64_t)gridDim.y * (kLoadItems * 256)) {
    uint32_t w1[kLoadItems], w2[kLoadItems], p1[kLoadItems], p2[kLoadItems];
#pragma unroll
    for (int e = 0; e < kLoadItems; ++e) {
      const int i = (int)part + e * 256 + threadIdx.x;
      const int row = i / TPR, j = i % TPR;  // row = token * hkv + head of the 16-bit block
      const int tok = row / hkv, h = row - tok * hkv;
      const int64_t crow = (int64_t)h * block_size + tok;
      if (i >= total) continue;
      if constexpr (NG == 2) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(codes + crow * (D / 8)) + j);
        const uint2 p = __ldg(reinterpret_cast<const uint2*>(params + crow * NG));
        w1[e] = w.x; w2[e] = w.y; p1[e] = p.x; p2[e] = p.y;
      } else {
        w1[e] = __ldg(codes + crow * (D / 8) + j);
        w2[e] = __ldg(codes + crow * (D / 8) + j + 4);
        p1[e] = p2[e] = __ldg(params + crow);
      }
    }
#pragma unroll
    for (int e = 0; e < kLoadItems; ++e) {
      const int i = (int)part + e * 256 + threadIdx.x;
      if (i >= total) continue;
      uint4* o = out + (int64_t)(i / TPR) * (D / 8) + i % TPR;
      st_v4(o, expand8<DT>(w1[e], p1[e]));
      st_v4(o + TPR, expand8<DT>(w2[e], p2[e]));
    }
  }
}

int check_int4_cache(const void* kc, const void* vc, const void* kp, const void* vp, int num_blocks, int block_size,
                     int num_kv_heads, int head_dim) {
  if (!kc || !vc || !kp || !vp || num_blocks < 0 || num_kv_heads <= 0 || head_dim <= 0) return PA_ERR_INVALID;
  if (!valid_block_size(block_size) || !valid_head_dim(head_dim)) return PA_ERR_UNSUPPORTED;
  if ((int64_t)num_kv_heads * block_size * head_dim >= (1ll << 31)) return PA_ERR_UNSUPPORTED;  // 32-bit offsets in a block
  if (!aligned16(kc) || !aligned16(vc) || !aligned16(kp) || !aligned16(vp)) return PA_ERR_ALIGN;
  return PA_OK;
}

bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

template <bool ROPE>
int launch_write(const WriteArgs& a, int head_dim, int dtype, cudaStream_t st) {
  // one item a thread: the hardware keeps the SMs filled with fresh loads
  const int64_t blocks = ((int64_t)a.total + kWriteThreads - 1) / kWriteThreads;
  auto kern = dtype == PA_BF16
                  ? (head_dim == 128 ? write_kv_int4_kernel<PA_BF16, 128, ROPE> : write_kv_int4_kernel<PA_BF16, 64, ROPE>)
                  : (head_dim == 128 ? write_kv_int4_kernel<PA_F16, 128, ROPE> : write_kv_int4_kernel<PA_F16, 64, ROPE>);
  return launch_programmatic(kern, dim3((unsigned)blocks), dim3(kWriteThreads), 0, st, a);
}

}  // namespace

extern "C" int pa_write_kv_int4(const void* k, const void* v, const int64_t* slot_mapping, int num_tokens,
                                void* k_codes, void* v_codes, void* k_params, void* v_params, void* k_out,
                                void* v_out, int num_blocks, int block_size, int num_kv_heads, int head_dim, int dtype,
                                void* stream) {
  int s = check_int4_cache(k_codes, v_codes, k_params, v_params, num_blocks, block_size, num_kv_heads, head_dim);
  if (s != PA_OK) return s;
  if (!valid_dtype(dtype)) return PA_ERR_UNSUPPORTED;
  if (num_tokens < 0) return PA_ERR_INVALID;
  if (num_tokens == 0) return PA_OK;
  if (!k || !v || !slot_mapping) return PA_ERR_INVALID;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_out) || !aligned16(v_out) || !aligned8(slot_mapping))
    return PA_ERR_ALIGN;
  const int64_t total = (int64_t)num_tokens * 2 * num_kv_heads * (head_dim / 16);
  if (total >= (1ll << 31) - 32) return PA_ERR_UNSUPPORTED;
  WriteArgs a = {};
  a.k = (const uint4*)k;
  a.v = (const uint4*)v;
  a.slots = slot_mapping;
  a.kc = (uint8_t*)k_codes;
  a.vc = (uint8_t*)v_codes;
  a.kp = (uint32_t*)k_params;
  a.vp = (uint32_t*)v_params;
  a.k_out = (uint4*)k_out;
  a.v_out = (uint4*)v_out;
  a.num_slots = (int64_t)num_blocks * block_size;
  a.total = (int)total;
  a.hkv = num_kv_heads;
  a.bs_shift = __builtin_ctz((unsigned)block_size);
  return launch_write<false>(a, head_dim, dtype, (cudaStream_t)stream);
}

extern "C" int pa_rope_write_kv_int4(const void* q, void* q_out, const void* k, const void* v,
                                     const int64_t* positions, const float* cos_table, const float* sin_table,
                                     int max_position, const int64_t* slot_mapping, int num_tokens, int num_q_heads,
                                     void* k_codes, void* v_codes, void* k_params, void* v_params, void* k_out,
                                     void* v_out, int num_blocks, int block_size, int num_kv_heads, int head_dim,
                                     int dtype, void* stream) {
  if (num_tokens < 0 || num_q_heads <= 0 || max_position <= 0) return PA_ERR_INVALID;
  int s = check_int4_cache(k_codes, v_codes, k_params, v_params, num_blocks, block_size, num_kv_heads, head_dim);
  if (s != PA_OK) return s;
  if (!valid_dtype(dtype)) return PA_ERR_UNSUPPORTED;
  if (num_tokens == 0) return PA_OK;
  if (!q || !q_out || !k || !v || !positions || !cos_table || !sin_table || !slot_mapping) return PA_ERR_INVALID;
  if (!aligned16(q) || !aligned16(q_out) || !aligned16(k) || !aligned16(v) || !aligned16(k_out) ||
      !aligned16(v_out) || !aligned16(cos_table) || !aligned16(sin_table) || !aligned8(positions) ||
      !aligned8(slot_mapping))
    return PA_ERR_ALIGN;
  const int64_t total = (int64_t)num_tokens * ((int64_t)num_q_heads + 2ll * num_kv_heads) * (head_dim / 16);
  if (total >= (1ll << 31) - 32) return PA_ERR_UNSUPPORTED;
  WriteArgs a = {};
  a.q = (const uint4*)q;
  a.q_out = (uint4*)q_out;
  a.k = (const uint4*)k;
  a.v = (const uint4*)v;
  a.positions = positions;
  a.cos_t = (const float4*)cos_table;
  a.sin_t = (const float4*)sin_table;
  a.slots = slot_mapping;
  a.kc = (uint8_t*)k_codes;
  a.vc = (uint8_t*)v_codes;
  a.kp = (uint32_t*)k_params;
  a.vp = (uint32_t*)v_params;
  a.k_out = (uint4*)k_out;
  a.v_out = (uint4*)v_out;
  a.num_slots = (int64_t)num_blocks * block_size;
  a.max_position = max_position;
  a.total = (int)total;
  a.hq = num_q_heads;
  a.hkv = num_kv_heads;
  a.bs_shift = __builtin_ctz((unsigned)block_size);
  return launch_write<true>(a, head_dim, dtype, (cudaStream_t)stream);
}

extern "C" int pa_copy_blocks_int4(const int32_t* pairs, int num_pairs, void* k_codes, void* v_codes, void* k_params,
                                   void* v_params, int num_blocks, int block_size, int num_kv_heads, int head_dim,
                                   void* stream) {
  int s = check_int4_cache(k_codes, v_codes, k_params, v_params, num_blocks, block_size, num_kv_heads, head_dim);
  if (s != PA_OK) return s;
  if (num_pairs < 0) return PA_ERR_INVALID;
  if (num_pairs == 0) return PA_OK;
  if (!pairs) return PA_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(pairs) & 3u) return PA_ERR_ALIGN;
  const int rows = num_kv_heads * block_size;
  const int code_vecs = rows * (head_dim / 32), param_vecs = rows * (head_dim / 64) / 4;
  const int total = 2 * (code_vecs + param_vecs), parts = (total + kCopyLoads * 256 - 1) / (kCopyLoads * 256);
  const int per_part = (total + parts - 1) / parts;  // equal parts
  const dim3 grid((unsigned)num_pairs, (unsigned)(parts > 65535 ? 65535 : parts));
  return launch_programmatic(copy_blocks_int4_kernel, grid, dim3(256), 0, (cudaStream_t)stream, pairs, code_vecs,
                             param_vecs, num_blocks, per_part, (uint4*)k_codes, (uint4*)v_codes, (uint4*)k_params,
                             (uint4*)v_params);
}

extern "C" int pa_load_blocks_int4(const int32_t* pairs, int num_pairs, const void* k_codes, const void* v_codes,
                                   const void* k_params, const void* v_params, int num_blocks, void* k_cache,
                                   void* v_cache, int num_dst_blocks, int block_size, int num_kv_heads, int head_dim,
                                   int dtype, void* stream) {
  int s = check_int4_cache(k_codes, v_codes, k_params, v_params, num_blocks, block_size, num_kv_heads, head_dim);
  if (s != PA_OK) return s;
  if (!valid_dtype(dtype)) return PA_ERR_UNSUPPORTED;
  if (!k_cache || !v_cache || num_dst_blocks < 0 || num_pairs < 0) return PA_ERR_INVALID;
  if (!aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_ALIGN;
  if (num_pairs == 0) return PA_OK;
  if (!pairs || num_pairs >= (1 << 30)) return PA_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(pairs) & 3u) return PA_ERR_ALIGN;
  const int64_t total = (int64_t)num_kv_heads * block_size * (head_dim / 16);
  const int64_t parts = (total + kLoadItems * 256 - 1) / (kLoadItems * 256);
  auto kern = dtype == PA_BF16 ? (head_dim == 128 ? load_blocks_int4_kernel<PA_BF16, 128> : load_blocks_int4_kernel<PA_BF16, 64>)
                               : (head_dim == 128 ? load_blocks_int4_kernel<PA_F16, 128> : load_blocks_int4_kernel<PA_F16, 64>);
  const dim3 grid((unsigned)num_pairs * 2u, (unsigned)(parts > 65535 ? 65535 : parts));
  return launch_programmatic(kern, grid, dim3(256), 0, (cudaStream_t)stream, pairs, num_kv_heads, block_size, num_blocks,
                             num_dst_blocks, (const uint32_t*)k_codes, (const uint32_t*)v_codes,
                             (const uint32_t*)k_params, (const uint32_t*)v_params, (uint4*)k_cache, (uint4*)v_cache);
}
