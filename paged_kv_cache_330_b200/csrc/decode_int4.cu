// Paged decode attention over the INT4 KV cache (format: kv_int4.cu).
//
// For every sequence b and query head h,
//   out[b][h] = sum_t softmax_t(scale <q[b][h], Kd_b[t][h/G]>) Vd_b[t][h/G],
// with Kd, Vd the rows s * (code + z).  A row of D 128 is 72 bytes (64 of codes, 8 of parameters): 16-bit caches
// hold 256.  At that size the work per byte, not HBM, is what has to be kept small, so the kernel is built
// around warps that never wait for one another.
//
// Work split.  A segment is one (sequence, KV head), cut into tiles of 32 tokens; on a line of segments end to end it takes
// kStart places for what starting and ending it costs, then a place per tile.  Where segments are many and not long
// they are dealt to the CTAs whole, by falling length to and fro, and what a CTA gets is its line.  Otherwise there is one
// line of all segments, and CTA c takes places [T c / n, T (c+1) / n) of T.  A CTA's warps take equal parts of its line.
// Every warp walks its own part: it looks its blocks up, brings its tiles into a ring of its own with asynchronous
// 16-byte copies (cp.async, nine a lane per tile; no other warp involved) and keeps the softmax state and the output
// of the current segment in registers.  Bulk copies were measured first: one instruction per copy, but each of a
// tile's eight takes a turn of its own through the uniform path, 200 of the 700 instructions of a tile.
// What a warp holds of a segment is a piece: a whole segment is written out at once, a partial one goes to
// shared memory, and after the one barrier at the end of the tiles the pieces of a segment are joined, first
// within the CTA, then, for the at most two segments that a CTA shares with its neighbours, through the
// workspace by the CTA that counts last (a counter per cut segment, no waiting).  The joining order is the order of
// the line, so results do not depend on timing.
//
// Mathematics.  Products run on mma.m16n8k16 (fp16 in, fp32 out) with tokens (scores) or columns (PV) as the 16
// rows and up to 8 heads of the group as the 8 columns.  A group of 16 is two halves: CTAs 2i and 2i + 1 walk the same
// part of the line, each for 8 heads; what the second one reads comes from L2.
//   * Codes enter as fp16 subnormals: a nibble in the low four bits of a half is code * 2^-24, in the next four
//     code * 2^-20, exactly, with no offset to take out again.  Widening a word of 8 codes of V is one shift and four
//     ANDs; the factors 2^24 and 16 sit in the final scaling of the output rows.  The matrix unit lines products up by
//     the operands' exponent fields, and that of a subnormal is 2^-14 whatever its value: it cuts a product with a code
//     at 2^-24 where the products of normal numbers are cut at 2^-34.  With V that is 2^-14 of the largest weight in 16,
//     less than the weights' own rounding.  With K it would be 2^-14 of the largest q: errors of 2e-5 in scores of
//     ordinary size, against 2e-7 with all of K's codes 2^4 higher, in bits 4 to 7.  That costs two multiplications a
//     word, 2 % of the time (64 sequences of 4096 to 8192, 99 -> 101 us).
//   * Parameters are converted once per token (lane = token), not once per lane that needs them, and handed round
//     through shared memory: s_K times the score scale as fp32, s_V as fp32, both z as fp16.
//   * Scores: s_t = sum_group s_K (sum code q + z_K sum q).  The zero-point part is one more product per group, of z
//     (times 2^-6: below 2^-8 it loses bits worth 2^-19 of a code) with the group sum of q in two fp16 terms.
//   * PV: the weight of a token enters times its V scale, P' = 2^(x - R) s_V, in fp16.  The zero-point part is again one
//     product per group, of z_V with the same P', so code and zero-point parts carry the same rounding and the error
//     stays relative to the value, not to the code.  Rounded once (2^-11), P' adds an error as large as an fp16 output's
//     own rounding: against 64 bits 2.9e-4 where that rounding alone leaves 2.05e-4 (64 sequences of 1 to 64 tokens).
//     So where the output is fp16 P' enters in two terms (2^-22; 2.05e-4): up to 4 heads leave half of the products'
//     columns free for the second term (128 sequences of 100 to 1024, 16 heads, 22.4 -> 23.4 us), 8 heads take products of
//     their own (one sequence of 100001, 32 heads, 23.1 -> 24.9; 64 of 4096 to 8192, 64 heads, 90 -> 108 to 112: 60
//     products a tile for 40, of 8 cycles each).  A bf16 output's rounding leaves 1.65e-3, and one term makes it 1.66e-3:
//     one term.
//   * Online softmax with a reference R per head that moves only when it must: a piece starts with a guess, which
//     stays if it puts the first tile's largest P' into [2^3, 2^15) and is set so (to (2^3, 2^4]) otherwise; later R
//     is raised only when P' come near 2^15 or the sum l passes 2^100.  Any R gives the same quotient O / l;
//     the usual tile needs no maximum, no shuffles and no rescaling of O, one vote tells.  l and O are fp32.
//
// Measured (B200): 64 sequences of 4096 to 8192 tokens, 64 heads, 8 KV heads of 128 (455 MB): 91 to 95 us, 4.9 TB/s, in
// bursts, 102 to 106 at the power limit; the tiles go by at 6 TB/s.  128 sequences of 100 to 1024, 16 heads (84 MB): 22.4 us, of which
// 3 until the first loads, 2 until they land, 14 at 6 TB/s and 2 to 3 until the last CTA has joined its pieces.  One sequence
// of 100001, 32 heads, 2 KV heads, fp16: 24.9 us.  4 sequences of up to 64 tokens, fp16: 3.95 us.

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "host_common.h"
#include "join_int4.h"

PA_DEFINE_ERROR_WORD(pa__err_decode_int4)

namespace {

using namespace pa;

constexpr int kTile = 32;            // tokens per tile: two 16-token chunks, each within one block
// What a segment costs besides its tiles, in tiles: 256 sequences of 16 to 300 tokens 18.5 us with 1, 17.6 with 2, 17.7
// with 3; 128 of 100 to 1024 22.4, 22.2, 22.2; 40 of 100 to 4096 26.7, 26.8, 27.1.
constexpr int kStart = 2;
constexpr int kLens = 512;           // sequences whose lengths a CTA keeps in shared memory
constexpr float kLn2 = 0.6931471805599453f;
// Segments of up to kUncut tiles are dealt whole to the CTAs where the CTAs that get one less than the others wait for less
// than kJoin tiles, on the mean: joining a segment across CTAs costs about 5 us at the end, a tile 0.11 us (D 128).  Dealt
// against cut: 32 sequences of 1000 to 2048 tokens (256 segments) 19.1 and 22.1 us, 64 of 500 to 8000 (D 64, 256 segments)
// 24.2 and 28.3; 16 segments of 63 tiles on 48 CTAs, where 43 tiles would be waited for, 13.4 and 11.5.  Where
// there are too many to deal, those of up to kMove tiles are not cut either: the CTAs' cuts move to their ends.
constexpr int kUncut = 256, kMove = 32;
template <int D>
constexpr int kJoin = D == 128 ? 30 : 60;
constexpr float kGuess = -8.f;       // a piece's first reference: fits when its largest weight * V scale is 2^-5 .. 2^7
constexpr float kUnit = 16777216.f;  // 2^24: what a code's fp16 subnormal stands for, inverted
constexpr float kUnitK = 1048576.f;  // 2^20: the same for K's codes

struct Params {
  const void* q;
  void* out;
  float* lse;
  const uint8_t* k_codes;
  const uint8_t* k_params;
  long long v_codes;  // where V's codes and parameters lie, relative to K's (an address less in registers)
  long long v_params;
  const int32_t* block_tables;
  const int32_t* context_lens;
  int* ws_cnt;   // [3 kMaxGrid], zero between calls, see join_round
  float* ws_r;   // [slots][G] reference R of a share
  float* ws_l;   // [slots][G]
  float* ws_o;   // [slots][G][D]
  int max_blocks_per_seq, batch, num_q_heads, num_kv_heads, block_size, num_blocks;
  float scale_log2;
};

enum : int { F_VALID = 1, F_HEAD = 2, F_TAIL = 4 };

// A partial piece as the joining step sees it: its segment, whether it holds the segment's first (F_HEAD) and
// last (F_TAIL) tile, the segment's tiles and where they start on the line.
struct Piece {
  int b, g, flags, nt;
  long long seg_start;
};

// A piece on its way: filed by the walk that brings tiles in, taken up by the consumer.
struct Queued {
  int b, g, L, t0;      // sequence, KV head, length, first tile
  long long seg_start;  // where the segment starts on the line
  int end, pad;         // where the piece ends
};
// The walk of a warp between two windows of block lookups (kept in shared memory: it is looked at once in 16 tiles).
struct Walk {
  int b, g, L, t;       // segment, its length, next tile
  int end, item;        // where the piece ends; dealt segments: which of the CTA's it is (else -1)
  long long seg_start;  // where the segment starts on the line, and where the warp's part of the line ends
  long long line_end;
};

// Pieces of one segment within a CTA, for the joining step.
struct Run {
  unsigned mask;  // which pieces
  int b, g, whole;
};

template <int D, int G, int NW, int NS>
struct Layout {
  static constexpr int NG = D / 64, ROWB = D / 2, PARB = NG * 4;
  static constexpr int K_OFF = 0, V_OFF = kTile * ROWB, KP_OFF = 2 * kTile * ROWB, VP_OFF = KP_OFF + kTile * PARB;
  static constexpr int STAGE = VP_OFF + kTile * PARB;
  static constexpr int PART = (G * (D + 2) * 4 + 15) / 16 * 16;  // a partial piece: o [G][D], R [G], l [G]
  static constexpr int RING = NS * STAGE > PART ? NS * STAGE : (PART + 127) / 128 * 128;  // also the last piece
  static constexpr int RING_OFF = 0;
  static constexpr int SV_OFF = 0, Z_OFF = kTile * NG * 4, CONV = Z_OFF + kTile * NG * 2;  // a warp's converted V parameters
  static constexpr int PART_OFF = RING_OFF + NW * RING;          // the first piece of every warp
  static constexpr int PIECE_OFF = (PART_OFF + NW * PART + 15) / 16 * 16;  // Piece [NW][2]
  static constexpr int NQ = NS + 2;                              // pieces filed and not done: NS stages' and one more
  static constexpr int QUEUE_OFF = PIECE_OFF + NW * 2 * (int)sizeof(Piece);  // Queued [NW][NQ]
  static constexpr int WALK_OFF = QUEUE_OFF + NW * NQ * (int)sizeof(Queued);  // Walk [NW]
  static constexpr int WIN_OFF = (WALK_OFF + NW * (int)sizeof(Walk) + 15) / 16 * 16;  // uint64 [NW][32]: where the next 32 chunks' codes are
  static constexpr int SCAN_OFF = WIN_OFF + NW * 256;            // int64 [NW]: tiles of a warp's sequences
  static constexpr int LONG_OFF = QUEUE_OFF;                     // int [NW]: the longest of them, at the start
  static constexpr int INCL_OFF = WIN_OFF;                       // int64 [NW * 32]: the scan within the warps, at the start
  static constexpr int CONV_OFF = SCAN_OFF + NW * 8;             // CONV [NW]
  static constexpr int JOIN_OFF = WIN_OFF;                       // Run [2 NW], weights and sums: after the tiles
  static_assert(JOIN_OFF + 2 * NW * (16 + 12 * G) <= CONV_OFF + NW * CONV, "room for the joining step");
  static constexpr int LENS_OFF = CONV_OFF + NW * CONV;          // int [kLens]: lengths, for batches that fit
  // q rows of the pieces filed, for groups of heads small enough: their pieces may be short, and each would wait for q
  static constexpr bool QS = G <= 4;
  static constexpr int QB = QS ? G * D * 2 : 0;
  static constexpr int ITEMS_OFF = LENS_OFF + kLens * 4;         // int2 [32]: sequence and KV head of the segments dealt to the CTA
  static constexpr int QS_OFF = ITEMS_OFF + 256;                 // QB [NW][NQ]
  static constexpr int BYTES = QS_OFF + NW * NQ * QB;
  // Byte offset of word `word` (4 bytes) of row `row` among a tile's codes: 16-byte units of a row are exchanged so
  // that neighbouring rows' units lie in different banks.  Rows 8 apart are exchanged alike.
  static __device__ __forceinline__ int code_off(int row, int word) {
    const int unit = word >> 2;
    return row * ROWB + ((ROWB == 64 ? unit ^ (row >> 1 & 3) : unit ^ (row >> 2 & 1)) << 4) + (word & 3) * 4;
  }
  static_assert(STAGE % 128 == 0 && sizeof(Piece) % 8 == 0 && sizeof(Queued) == 32 && sizeof(Walk) == 40 && ITEMS_OFF % 8 == 0 && PIECE_OFF % 16 == 0 && QUEUE_OFF % 16 == 0 &&
                    WIN_OFF % 16 == 0 && CONV_OFF % 16 == 0 && CONV % 16 == 0,
                "alignment");
};

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}
__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same; `first` (a constant where it is called): from a zero accumulator.
__device__ __forceinline__ void mma_f16(bool first, float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  if (!first) return mma_f16(c, a0, a1, a2, a3, b0, b1);
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t trans8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ __half2 as_h2(uint32_t a) { return *reinterpret_cast<const __half2*>(&a); }
__device__ __forceinline__ uint32_t as_u32(__half2 a) { return *reinterpret_cast<const uint32_t*>(&a); }
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float rows_max(float v) {  // over the 8 lanes that share a column
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float rows_sum(float v) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// One more at a counter that starts at zero, with device scope: what the block wrote before (its barrier passed) is
// visible to whoever counts last, and the last finds everybody's.  The last one (of n) leaves the counter at zero.
__device__ __forceinline__ bool count_last(int* cnt, int n) {
  int old;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(old) : "l"(cnt) : "memory");
  if (old != n - 1) return false;
  *cnt = 0;
  return true;
}

constexpr uint32_t kOnes = 0x3c003c00u;  // fp16 1.0, twice
constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u;  // a nibble of each half, worth 2^-24 and 2^-20

// ------------------------------------------------------------------ a warp's state over one piece
template <int DT, int D, int G>
struct State {
  static constexpr int NG = D / 64, KS = D / 16, WPL = D / 32;  // WPL: K words a lane reads of a row
  // Where the output is fp16, a weight times its V scale enters in two fp16 terms.  Up to 4 heads leave columns free:
  // columns 4 to 7 are the same heads once more, with the second terms (SIDE); 8 heads take products of their own (TWICE).
  static constexpr bool SIDE = DT == PA_F16 && G <= 4, TWICE = DT == PA_F16 && G > 4;
  uint32_t qb[KS][2];  // q as B operand (fp16, prescaled)
  uint32_t qsum[NG];   // B operand of the zero-point product: lanes c = 0 the sum of q over a group, 2^-14 of it in two terms
  float o[KS][4];      // O^T times 2^-24 (rows g) and 2^-20 (rows g + 8), columns heads
  float z[NG][4];      // sum P' z_V (columns heads; all rows alike)
  float l[2];          // this lane's part of sum 2^(x - R)
  float R[2];
  float qs;            // scale * log2(e) * 2^20 / prescale
  bool fresh;          // some head has met no non-zero V scale yet: its R is not set

  // qrows: the group's [G][D] rows of q.  A lane loads just the values its operands hold.
  template <bool in_shared>
  __device__ __forceinline__ void begin(const uint8_t* qrows, float scale_log2, int lane) {
    const int g = lane >> 2, c = lane & 3;
    uint4 raw[WPL];
    using T2 = typename Elt<DT>::T2;
    uint32_t top = 0;  // largest magnitudes, two columns at once
#pragma unroll
    for (int i = 0; i < WPL; ++i) {
      // stored word WPL * c + i of a row: 8 values from `base` on
      const int base = D == 128 ? 64 * (i & 1) + 8 * (2 * c + (i >> 1)) : 8 * (2 * c + i);
      raw[i] = make_uint4(0, 0, 0, 0);
      const int h = SIDE ? g & 3 : g;
      if (h < G) {
        const uint4* at = reinterpret_cast<const uint4*>(qrows + (h * D + base) * 2);
        raw[i] = in_shared ? *at : __ldcg(at);
      }
    }
#pragma unroll
    for (int i = 0; i < WPL; ++i) {
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const T2 v = __hmax2(*reinterpret_cast<T2*>(&top), __habs2(*reinterpret_cast<const T2*>(&w[m])));
        top = *reinterpret_cast<const uint32_t*>(&v);
      }
    }
    const float2 top2 = Elt<DT>::to_f2(top);
    float amax = warp_max(fmaxf(top2.x, top2.y));
    if (amax == INFINITY) {  // a head of the group is lost; the scale of the others is that of the finite values
      float finite = 0.f;
#pragma unroll
      for (int i = 0; i < WPL; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const float2 v = Elt<DT>::to_f2(w[m]);
          if (fabsf(v.x) < INFINITY) finite = fmaxf(finite, fabsf(v.x));
          if (fabsf(v.y) < INFINITY) finite = fmaxf(finite, fabsf(v.y));
        }
      }
      amax = warp_max(finite);
    }
    int e = 0;
    if (amax > 0.f) {
      int k;
      frexpf(amax, &k);  // amax in [2^(k-1), 2^k)
      e = min(60, max(-60, 15 - k));
    }
    const float f = __int_as_float((127 + e) << 23), finv = __int_as_float((127 - e) << 23);
    qs = scale_log2 * finv * kUnitK;
#pragma unroll
    for (int i = 0; i < WPL; ++i) {
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
      float x[8];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const float2 v = Elt<DT>::to_f2(w[m]);
        x[2 * m] = v.x * f;
        x[2 * m + 1] = v.y * f;
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        qb[2 * i + s][0] = pack_h2(x[2 * s], x[2 * s + 4]);
        qb[2 * i + s][1] = pack_h2(x[2 * s + 1], x[2 * s + 5]);
      }
    }
#pragma unroll
    for (int grp = 0; grp < NG; ++grp) {
      float acc[4];
#pragma unroll
      for (int i = grp; i < WPL; i += NG)
#pragma unroll
        for (int s = 0; s < 2; ++s)
          mma_f16(i == grp && s == 0, acc, kOnes, kOnes, kOnes, kOnes, qb[2 * i + s][0], qb[2 * i + s][1]);
      // lane g takes head g, which column 2 (g / 2) + g % 2 of any row holds
      const float s0 = __shfl_sync(0xffffffffu, acc[0], g >> 1), s1 = __shfl_sync(0xffffffffu, acc[1], g >> 1);
      const float sum = ((g & 1) ? s1 : s0) * (64.f / kUnitK), hi = __half2float(__float2half_rn(sum));
      qsum[grp] = c == 0 ? pack_h2(hi, sum - hi) : 0u;
      z[grp][0] = z[grp][1] = z[grp][2] = z[grp][3] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < KS; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    l[0] = l[1] = 0.f;
    R[0] = R[1] = kGuess;
    fresh = true;
  }

  // Moves the references of the heads that need it, so that the tile's scores x (relative to R; -inf where
  // masked) give P' <= 2^4 and l <= 2^91.  svm: the larger finite V scale of each of this lane's rows.
  __device__ __forceinline__ void rebase(float (&x)[2][4], const float (&svm)[4]) {
    bool still = false;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float u = -INFINITY, v = l[e] > 0.f ? __log2f(l[e]) : -INFINITY;
      bool set = false;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float xr = x[r >> 1][2 * (r & 1) + e];
        v = fmaxf(v, xr);
        u = fmaxf(u, svm[r] > 0.f ? xr + __log2f(svm[r]) : -INFINITY);
      }
#pragma unroll
      for (int i = 0; i < KS; ++i) set |= o[i][e] != 0.f || o[i][2 + e] != 0.f;
#pragma unroll
      for (int grp = 0; grp < NG; ++grp) set |= z[grp][e] != 0.f;
      // every lane of a column has to agree on whether its O is still all zero
      float any = set ? 1.f : 0.f;
      u = rows_max(u);
      v = rows_max(v);
      any = rows_max(any);
      if constexpr (SIDE) any = fmaxf(any, __shfl_xor_sync(0xffffffffu, any, 2));  // and both columns of a head
      set = any > 0.f;
      float up = fmaxf(u - 4.f, v - 90.f);
      if (set) up = fmaxf(up, 0.f);
      else if (u == -INFINITY) up = v, still = true;
      up = ceilf(up);
      if (!(fabsf(up) < 1e30f)) up = 0.f;  // not-a-number inputs: leave the references alone
      const float f = exp2f(-up);
      if (l[e] > 0.f) l[e] *= f;
      if (set) {
#pragma unroll
        for (int i = 0; i < KS; ++i) o[i][e] *= f, o[i][2 + e] *= f;
#pragma unroll
        for (int grp = 0; grp < NG; ++grp) z[grp][e] *= f, z[grp][2 + e] *= f;
      }
      R[e] += up;
#pragma unroll
      for (int r = 0; r < 4; ++r) x[r >> 1][2 * (r & 1) + e] -= up;
    }
    fresh = __any_sync(0xffffffffu, still);
  }

  // One tile in shared memory at `st` (a stage), its first nv (32 and more: all) tokens valid; conv: the warp's room for
  // converted V parameters (those of K replace the stage's).
  template <typename LY>
  __device__ __forceinline__ void tile(uint8_t* st, uint8_t* conv, int nv, int lane) {
    const int g = lane >> 2, c = lane & 3;
    // ---- parameters of token `lane`
    uint32_t kw[NG], vw[NG];
    if constexpr (NG == 2) {
      const uint2 a = *reinterpret_cast<const uint2*>(st + LY::KP_OFF + lane * 8);
      const uint2 b = *reinterpret_cast<const uint2*>(st + LY::VP_OFF + lane * 8);
      kw[0] = a.x; kw[1] = a.y;
      vw[0] = b.x; vw[1] = b.y;
    } else {
      kw[0] = *reinterpret_cast<const uint32_t*>(st + LY::KP_OFF + lane * 4);
      vw[0] = *reinterpret_cast<const uint32_t*>(st + LY::VP_OFF + lane * 4);
    }
    // ---- K codes: rows tokens g, g + 8, g + 16, g + 24 (r = 2 mt + hh)
    uint32_t kc[4][WPL];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint8_t* a = st + LY::K_OFF + LY::code_off(g, WPL * c) + 8 * r * LY::ROWB;
      if constexpr (WPL == 4) {
        const uint4 u = *reinterpret_cast<const uint4*>(a);
        kc[r][0] = u.x; kc[r][1] = u.y; kc[r][2] = u.z; kc[r][3] = u.w;
      } else {
        const uint2 u = *reinterpret_cast<const uint2*>(a);
        kc[r][0] = u.x; kc[r][1] = u.y;
      }
    }
    __syncwarp();  // every lane holds its parameters: their place may be overwritten
    float vs[NG];
    {
      float ks[NG], kz[NG], vz[NG];
#pragma unroll
      for (int grp = 0; grp < NG; ++grp) {
        const float2 a = Elt<DT>::to_f2(kw[grp]), b = Elt<DT>::to_f2(vw[grp]);
        ks[grp] = a.x * qs;
        kz[grp] = a.y * 0.015625f;
        vs[grp] = lane < nv ? b.x : 0.f;  // rows past the end hold anything, NaN among it
        vz[grp] = lane < nv ? b.y : 0.f;
      }
      __half* z = reinterpret_cast<__half*>(conv + LY::Z_OFF) + (lane >> 1) * 2 * NG + (lane & 1);
      if constexpr (NG == 2) {
        *reinterpret_cast<uint4*>(st + LY::KP_OFF + lane * 16) = make_uint4(
            __float_as_uint(ks[0]), __float_as_uint(ks[1]), pack_h2(kz[0], kz[0]), pack_h2(kz[1], kz[1]));
        *reinterpret_cast<float2*>(conv + LY::SV_OFF + lane * 8) = make_float2(vs[0], vs[1]);
        const __half2 zz = __floats2half2_rn(vz[0], vz[1]);
        z[0] = __low2half(zz);
        z[2] = __high2half(zz);
      } else {
        *reinterpret_cast<uint2*>(st + LY::KP_OFF + lane * 8) = make_uint2(__float_as_uint(ks[0]), pack_h2(kz[0], kz[0]));
        *reinterpret_cast<float*>(conv + LY::SV_OFF + lane * 4) = vs[0];
        z[0] = __float2half_rn(vz[0]);
      }
    }
    // the tile's largest V scale (not negative: its bits order as its value does)
    const float sv_top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(NG == 2 ? fmaxf(vs[0], vs[NG - 1]) : vs[0])));
    __syncwarp();
    // ---- scores relative to R, columns heads 2c + {0,1}
    float x[2][4];
    uint32_t times16;  // a shift by 4 on the multiplier's pipe: the compiler, seeing the 16, would shift twice on the other
    asm("mov.u32 %0, 16;" : "=r"(times16));
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      float ks[2][NG];
      uint32_t kz[2][NG];
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const uint8_t* a = st + LY::KP_OFF + (16 * mt + 8 * hh + g) * 8 * NG;
        if constexpr (NG == 2) {
          const uint4 u = *reinterpret_cast<const uint4*>(a);
          ks[hh][0] = __uint_as_float(u.x); ks[hh][1] = __uint_as_float(u.y);
          kz[hh][0] = u.z; kz[hh][1] = u.w;
        } else {
          const uint2 u = *reinterpret_cast<const uint2*>(a);
          ks[hh][0] = __uint_as_float(u.x);
          kz[hh][0] = u.y;
        }
      }
      float acc[NG][4];
#pragma unroll
      for (int i = 0; i < WPL; ++i)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const uint32_t a = kc[2 * mt][i] >> (8 * s), b = kc[2 * mt + 1][i] >> (8 * s);
          mma_f16(i < NG && s == 0, acc[i % NG], a * times16 & kHigh, b * times16 & kHigh, a & kHigh, b & kHigh,
                  qb[2 * i + s][0], qb[2 * i + s][1]);
        }
#pragma unroll
      for (int grp = 0; grp < NG; ++grp) {
        mma_f16(acc[grp], kz[0][grp], kz[1][grp], kz[0][grp], kz[1][grp], qsum[grp], 0u);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[mt][e] = fmaf(acc[grp][e], ks[e >> 1][grp], grp == 0 ? -R[e & 1] : x[mt][e]);
      }
    }
    if (nv < kTile) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (8 * r + g >= nv) x[r >> 1][2 * (r & 1)] = x[r >> 1][2 * (r & 1) + 1] = -INFINITY;
    }
    // ---- weights; taken once more after a move of the references
    float sv[4][NG];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float* a = reinterpret_cast<const float*>(conv + LY::SV_OFF) + (8 * r + g) * NG;
      if constexpr (NG == 2) {
        const float2 u = *reinterpret_cast<const float2*>(a);
        sv[r][0] = u.x;
        sv[r][1] = u.y;
      } else {
        sv[r][0] = a[0];
      }
    }
    uint32_t pk[NG][4], pl[NG][4];  // the weights (TWICE: their first terms), their second terms
    const uint32_t second = SIDE && c >= 2 ? 0xffffffffu : 0u;
    float sum[2];
    for (bool moved = false;; moved = true) {
      bool move = false;
      sum[0] = sum[1] = 0.f;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float p0 = fast_exp2(x[r >> 1][2 * (r & 1)]), p1 = fast_exp2(x[r >> 1][2 * (r & 1) + 1]);
        sum[0] += p0;
        sum[1] += p1;
#pragma unroll
        for (int grp = 0; grp < NG; ++grp) {
          const float a = p0 * sv[r][grp], b = p1 * sv[r][grp];
          pk[grp][r] = pack_h2(a, b);
          if constexpr (SIDE || TWICE) {
            const float2 first = __half22float2(as_h2(SIDE ? pk[grp][r] & second : pk[grp][r]));
            (SIDE ? pk : pl)[grp][r] = pack_h2(a - first.x, b - first.y);
          }
        }
      }
      // each P' is at most the lane's sum times the largest scale: below 2^15, and l below 2^100
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        move |= !(sum[e] * sv_top < 32768.f);
        sum[e] += l[e];
        move |= !(sum[e] < 1.2676506e30f);
      }
      move = __any_sync(0xffffffffu, move);
      if (fresh && !move) {  // is the guess large enough for every head?
        bool low = false;
        __half2 top = as_h2(0u);
#pragma unroll
        for (int grp = 0; grp < NG; ++grp)
#pragma unroll
          for (int r = 0; r < 4; ++r) top = __hmax2(top, as_h2(pk[grp][r]));
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) top = __hmax2(top, as_h2(__shfl_xor_sync(0xffffffffu, as_u32(top), o)));
        low |= (!SIDE || c < 2) && (!(__low2float(top) >= 8.f) || !(__high2float(top) >= 8.f));
        move = __any_sync(0xffffffffu, low);
        fresh = move;
      }
      if (!move || moved) break;
      // An infinite scale fits with no reference: its group is lost, the other's weights go by its own.  Read once more
      // (volatile: or the compiler tests the registers that the usual tile holds, 96 us for 93 at 64 long sequences).
      float svm[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        svm[r] = 0.f;
#pragma unroll
        for (int grp = 0; grp < NG; ++grp) {
          const float s = *reinterpret_cast<volatile float*>(conv + LY::SV_OFF + ((8 * r + g) * NG + grp) * 4);
          if (s < INFINITY) svm[r] = fmaxf(svm[r], s);
        }
      }
      rebase(x, svm);
    }
    l[0] = sum[0];
    l[1] = sum[1];
#pragma unroll
    for (int grp = 0; grp < NG; ++grp)
#pragma unroll
      for (int r = 0; r < 4; ++r) {  // tokens along the rows of the B operand
        pk[grp][r] = trans8x8(pk[grp][r]);
        if constexpr (TWICE) pl[grp][r] = trans8x8(pl[grp][r]);
      }
    // ---- O^T += V^T P'^T: tokens 2c, 2c + 1, 2c + 8, 2c + 9 of each half; word `grp` of lane g's piece of a row holds
    // values 64 grp + 8 g ..
    // (codes lie swizzled, see bring; odd c take their two tokens in the other order, which with the swizzle spreads
    // a half-warp's 8-byte loads over all banks and costs only another permute selector)
    const int odd = c & 1;
    const uint8_t* vl = st + LY::V_OFF;
    const uint8_t* v0 = vl + LY::code_off(2 * c + odd, NG * g);
    const uint8_t* v1 = vl + LY::code_off(2 * c + (odd ^ 1), NG * g);
    const uint32_t sel_lo = odd ? 0x1054u : 0x5410u, sel_hi = odd ? 0x3276u : 0x7632u;
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      uint32_t w[4][NG];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint8_t* a = ((t & 1) ? v1 : v0) + (16 * mt + 8 * (t >> 1)) * LY::ROWB;
        if constexpr (NG == 2) {
          const uint2 u = *reinterpret_cast<const uint2*>(a);
          w[t][0] = u.x;
          w[t][1] = u.y;
        } else {
          w[t][0] = *reinterpret_cast<const uint32_t*>(a);
        }
      }
      uint32_t zp[2][NG];  // z of tokens 2c, 2c + 1 and of 2c + 8, 2c + 9
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const uint32_t* a = reinterpret_cast<const uint32_t*>(conv + LY::Z_OFF) + ((2 * mt + hh) * 4 + c) * NG;
#pragma unroll
        for (int grp = 0; grp < NG; ++grp) zp[hh][grp] = a[grp];
      }
#pragma unroll
      for (int grp = 0; grp < NG; ++grp) {
        mma_f16(z[grp], zp[0][grp], zp[0][grp], zp[1][grp], zp[1][grp], pk[grp][2 * mt], pk[grp][2 * mt + 1]);
        if constexpr (TWICE)
          mma_f16(z[grp], zp[0][grp], zp[0][grp], zp[1][grp], zp[1][grp], pl[grp][2 * mt], pl[grp][2 * mt + 1]);
      }
#pragma unroll
      for (int grp = 0; grp < NG; ++grp)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t sel = half ? sel_hi : sel_lo;
          const uint32_t a = prmt(w[0][grp], w[1][grp], sel), b = prmt(w[2][grp], w[3][grp], sel);
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const uint32_t as = a >> (8 * s), bs = b >> (8 * s);
            mma_f16(o[4 * grp + 2 * half + s], as & kLow, as & kHigh, bs & kLow, bs & kHigh,
                    pk[grp][2 * mt], pk[grp][2 * mt + 1]);
            if constexpr (TWICE)
              mma_f16(o[4 * grp + 2 * half + s], as & kLow, as & kHigh, bs & kLow, bs & kHigh,
                      pl[grp][2 * mt], pl[grp][2 * mt + 1]);
          }
        }
    }
  }

  // Completes the lanes' parts of l, and adds up the terms that lie side by side.
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int e = 0; e < 2; ++e) l[e] = rows_sum(l[e]);
    if constexpr (SIDE) {
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] += __shfl_xor_sync(0xffffffffu, o[i][e], 2);
#pragma unroll
      for (int grp = 0; grp < NG; ++grp)
#pragma unroll
        for (int e = 0; e < 2; ++e) z[grp][e] += __shfl_xor_sync(0xffffffffu, z[grp][e], 2);
    }
  }
  // The 8 output values 64 grp + 8 g .. of head 2c + e, relative to R.
  __device__ __forceinline__ void values(int grp, int e, float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = fmaf(o[4 * grp + i][e], kUnit, z[grp][e]);
      v[2 * i + 1] = fmaf(o[4 * grp + i][2 + e], kUnit / 16.f, z[grp][e]);
    }
  }
};

// ------------------------------------------------------------------ kernel
template <int DT, int D, int G, int HV, int NW, int NS>
__global__ void __launch_bounds__(NW * 32, 1) decode_int4_kernel(const Params p) {
  using LY = Layout<D, G, NW, NS>;
  using S = State<DT, D, G>;
  using T = typename Elt<DT>::T;
  static_assert(NW <= 16, "a warp's lanes hold all pieces of the CTA");
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // HV CTAs walk the same part of the line, each for G heads of a group of HV * G
  const int half = HV == 2 ? blockIdx.x & 1 : 0, cta = blockIdx.x / HV, line_ctas = gridDim.x / HV;
  long long* warp_tiles = reinterpret_cast<long long*>(smem + LY::SCAN_OFF);
  int* warp_longest = reinterpret_cast<int*>(smem + LY::LONG_OFF);
  long long* incl_s = reinterpret_cast<long long*>(smem + LY::INCL_OFF);
  long long* cut_s = reinterpret_cast<long long*>(smem + LY::ITEMS_OFF);  // [2], where nothing is dealt
  int* order = reinterpret_cast<int*>(smem + LY::PART_OFF);  // [NW * 32], at the start: the sequences by falling length
  int* hist = order + NW * 32;                               // [NW][32]: a warp's sequences by bin, the longest first
  static_assert(NW * 256 <= NW * LY::PART, "room for order and hist");
  int2* items = reinterpret_cast<int2*>(smem + LY::ITEMS_OFF);
  Piece* pieces = reinterpret_cast<Piece*>(smem + LY::PIECE_OFF);
  int* lens_s = reinterpret_cast<int*>(smem + LY::LENS_OFF);
  const int B = p.batch, Hkv = p.num_kv_heads, bs = p.block_size;
  const int cap = p.max_blocks_per_seq * bs;
  if (lane == 0) pieces[2 * warp].flags = pieces[2 * warp + 1].flags = 0;
  // The block tables come from HBM on their first use: ask for them (a line a thread, at most) while the lengths are
  // added up.
  {
    const size_t line = (size_t)blockIdx.x * (NW * 32) + threadIdx.x, bytes = (size_t)B * p.max_blocks_per_seq * 4;
    if (line * 128 < bytes)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const uint8_t*>(p.block_tables) + line * 128));
  }

  // ---- the line: thread i counts the tiles of sequences [i * per, (i + 1) * per), a scan within every warp; each warp
  // then looks its first tile up in the scans
  const int per = (B + NW * 32 - 1) / (NW * 32);
  auto len_of = [&](int i) { return i < kLens ? lens_s[i] : min(max(__ldg(p.context_lens + i), 0), cap); };
  auto tiles_of = [](int L) { return (L + kTile - 1) / kTile; };
  auto places_of = [](int L) { return L > 0 ? (L + kTile - 1) / kTile + kStart : 0; };
  {
    long long incl = 0;
    int longest = 0;
    bool clamped = false;
    for (int i = threadIdx.x * per, e = min(B, i + per); i < e; ++i) {
      const int L = __ldg(p.context_lens + i), Lc = min(max(L, 0), cap);
      clamped |= L != Lc;
      if (i < kLens) lens_s[i] = Lc;
      incl += places_of(Lc);
      longest = max(longest, tiles_of(Lc));
    }
    if (clamped && blockIdx.x == 0) PA_RECORD_ERROR(PA_ERRBIT_INDEX);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    incl_s[threadIdx.x] = incl;
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 31) {
      warp_tiles[warp] = incl;
      warp_longest[warp] = longest;
    }
  }
  __syncthreads();
  long long wincl = lane < NW ? warp_tiles[lane] * Hkv : 0;  // places up to and with warp `lane`'s sequences
#pragma unroll
  for (int o = 1; o < NW; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, wincl, o);
    if (lane >= o) wincl += t;
  }
  const long long total = __shfl_sync(0xffffffffu, wincl, NW - 1);
  const long long ctas = min((long long)line_ctas, total);
  const bool narrow = (total + 1) * (ctas + 1) < (1ll << 32);
  // The segment at place x of the line, and the tile (the segment's first one, if x is one of its kStart places).
  auto find = [&](long long x) {
    Walk w = {};
    w.item = -1;
    const int wsel = __popc(__ballot_sync(0xffffffffu, lane < NW && wincl <= x));
    const long long before = wsel ? __shfl_sync(0xffffffffu, wincl, wsel - 1) : 0;
    const long long li = incl_s[wsel * 32 + lane] * Hkv + before;
    const int tsel = __popc(__ballot_sync(0xffffffffu, li <= x));
    long long in_seq = x - (tsel ? __shfl_sync(0xffffffffu, li, tsel - 1) : before);
    w.b = (wsel * 32 + tsel) * per;
    for (;; ++w.b) {
      w.L = len_of(w.b);
      const long long all = (long long)places_of(w.L) * Hkv;
      if (in_seq < all) break;
      in_seq -= all;
    }
    // a quotient below Hkv, from one in floating point that is off by less than 1
    w.g = min((int)__fdividef((float)in_seq, (float)places_of(w.L)), Hkv - 1);
    const long long rest = in_seq - (long long)w.g * places_of(w.L);
    w.g += rest < 0 ? -1 : (rest >= places_of(w.L) ? 1 : 0);
    const int place = (int)(in_seq - (long long)w.g * places_of(w.L));
    w.seg_start = x - place;
    w.t = max(0, place - kStart);
    return w;
  };
  // The next segment in line (sequences without tokens have none).
  auto step_on = [&](Walk& w) {
    w.seg_start += places_of(w.L);
    w.t = 0;
    if (w.item >= 0) {
      const int2 it = items[++w.item];
      w.b = it.x;
      w.g = it.y;
      w.L = len_of(w.b);
    } else if (++w.g == p.num_kv_heads) {
      w.g = 0;
      do w.L = len_of(++w.b);
      while (w.L == 0 && w.b < p.batch - 1);
    }
  };
  Walk w0 = {};  // this warp's part of the line: from w0 to w0.line_end
  bool any = false;
  const int longest = __reduce_max_sync(0xffffffffu, lane < NW ? warp_longest[lane] : 0);
  bool dealt = longest <= kUncut && B <= NW * 32 && (long long)B * Hkv <= 32ll * line_ctas;
  const bool one = (long long)B * Hkv <= line_ctas;  // a segment a CTA at most: in any order
  int segs = B * Hkv, first = 0, last = longest;     // the last round: its first segment, and that one's tiles
  if (dealt && !one) {  // order the sequences by falling length, in 32 bins (31 - length / width; 32: empty), by place within one
    const int width = (longest + 31) / 32, mine = threadIdx.x < B ? tiles_of(lens_s[threadIdx.x]) : 0;
    const int my_bin = mine ? 31 - (mine - 1) / width : 32;
    const unsigned alike = __match_any_sync(0xffffffffu, my_bin);
    hist[warp * 32 + lane] = 0;
    __syncwarp();
    if (my_bin < 32 && lane == __ffs(alike) - 1) hist[warp * 32 + my_bin] = __popc(alike);
    __syncthreads();
    int before = 0, all = 0;  // sequences in bin `lane`: in the warps before this one, and in all
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const int n = hist[w * 32 + lane];
      before += w < warp ? n : 0;
      all += n;
    }
    int longer = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, longer, o);
      if (lane >= o) longer += t;
    }
    const int seqs = __shfl_sync(0xffffffffu, longer, 31);  // that are not empty
    const int rank0 = __shfl_sync(0xffffffffu, longer - all + before, min(my_bin, 31));
    if (my_bin < 32) order[rank0 + __popc(alike & ((1u << lane) - 1u))] = threadIdx.x;
    segs = seqs * Hkv;
    __syncthreads();
    first = max(segs - 1, 0) / line_ctas * line_ctas;
    last = segs ? tiles_of(lens_s[order[first / Hkv]]) : 0;
  }
  dealt = dealt && last * (line_ctas - (segs - first)) <= kJoin<D> * line_ctas;
  if (dealt) {  // to the CTAs in turn and back again; a CTA's segments are its line
    const int k = lane * line_ctas + (lane & 1 ? line_ctas - 1 - cta : cta);  // the CTA's segment `lane`
    const bool have = k < segs;
    const int rank = have ? k / Hkv : 0, kvh = k - rank * Hkv, b = one ? rank : (have ? order[rank] : 0), L = have ? lens_s[b] : 0;
    int incl = places_of(L);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    if (warp == 0 && have) items[lane] = make_int2(b, kvh);
    const int own = __shfl_sync(0xffffffffu, incl, 31), xs = own * warp / NW, xe = own * (warp + 1) / NW;
    if (xs < xe) {
      const int at = __popc(__ballot_sync(0xffffffffu, incl <= xs));
      w0.b = __shfl_sync(0xffffffffu, b, at);
      w0.g = __shfl_sync(0xffffffffu, kvh, at);
      w0.L = __shfl_sync(0xffffffffu, L, at);
      w0.seg_start = __shfl_sync(0xffffffffu, incl, at) - places_of(w0.L);
      w0.t = max(0, xs - (int)w0.seg_start - kStart);
      w0.line_end = xe;
      w0.item = at;
      any = w0.t < xe - (int)w0.seg_start - kStart;
    }
  } else if (cta < ctas) {
    long long x0 = udiv(total * cta, ctas, narrow), x1 = udiv(total * (cta + 1), ctas, narrow);
    // first (where segments are short) even warps move the CTA's first cut to the nearest end of a segment, odd ones its
    // last; then each warp looks its own part up.  One copy of the search: its instructions come from far.
#pragma unroll 1
    for (bool cuts = longest <= kMove;; cuts = false) {
      const long long xs = x0 + (x1 - x0) * warp / NW, xe = x0 + (x1 - x0) * (warp + 1) / NW;
      const long long x = cuts ? (warp & 1 ? x1 : x0) : xs;
      if (cuts || xs < xe) w0 = find(min(x, total - 1));
      if (!cuts) {
        w0.line_end = xe;
        // a part that ends in a segment's kStart places, or starts behind its last tile, may hold no tile of it
        any = xs < xe && w0.t < xe - w0.seg_start - kStart;
        break;
      }
      const long long next = w0.seg_start + places_of(w0.L);
      if (lane == 0 && warp < 2) cut_s[warp] = 2 * (x - w0.seg_start) < places_of(w0.L) ? w0.seg_start : next;
      __syncthreads();
      x0 = cut_s[0];
      x1 = cut_s[1];
    }
  }
  __syncthreads();  // the scans are done with: the windows take their place

  // ---- what this lane copies of a tile: of each chunk's codes the 16-byte units lane, lane + 32, .. (K and V
  // alike); of the parameters one unit of the tile's four runs (K chunk 0, K chunk 1, V chunk 0, V chunk 1)
  constexpr int PER = LY::ROWB / 32, UPR = LY::ROWB / 16, PUNITS = LY::PARB;
  static_assert(LY::ROWB == 8 * LY::PARB, "offsets of parameters follow from those of codes");
  const uint32_t ring = smem_u32(smem + LY::RING_OFF) + warp * LY::RING;
  const int par_run = lane / PUNITS;
  const uint8_t* kbase = p.k_codes + lane * 16;
  const uint8_t* par_base = p.k_params + ((par_run & 2) ? p.v_params : 0) + (lane % PUNITS) * 16;
  const uint32_t par_dst = ((par_run & 2) ? LY::VP_OFF : LY::KP_OFF) + (par_run & 1) * 16 * LY::PARB + (lane % PUNITS) * 16;
  uint32_t code_dst[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) code_dst[e] = LY::code_off((lane + 32 * e) / UPR, ((lane + 32 * e) % UPR) * 4);
  Queued* queue = reinterpret_cast<Queued*>(smem + LY::QUEUE_OFF) + warp * LY::NQ;
  uint64_t* win = reinterpret_cast<uint64_t*>(smem + LY::WIN_OFF) + warp * 32;
  Walk* walk = reinterpret_cast<Walk*>(smem + LY::WALK_OFF) + warp;
  const ulonglong2* win_at = nullptr;  // the next tile's two chunks
  int win_left = 0;                    // tiles the window still holds
  int filed = 0;                       // pieces filed

  auto file_piece = [&](Walk& w) {
    w.end = (int)min((long long)tiles_of(w.L), w.line_end - w.seg_start - kStart);
    if (lane == 0) {
      Queued& q = queue[filed % LY::NQ];
      *reinterpret_cast<int4*>(&q) = make_int4(w.b, w.g, w.L, w.t);
      q.seg_start = w.seg_start;
      q.end = w.end;
    }
    ++filed;
  };
  auto head0 = [&](size_t seg) { return (seg * HV + half) * G; };  // of a segment: the first row of q, out and lse
  auto q_rows = [&](int b, int kvh) {
    return reinterpret_cast<const uint8_t*>(p.q) + head0((size_t)b * p.num_kv_heads + kvh) * D * 2;
  };
  auto bring_q = [&](const Walk& w) {  // of the piece filed last, with its first tile
    if constexpr (LY::QS) {
      const uint8_t* src = q_rows(w.b, w.g);
      const uint32_t dst = smem_u32(smem + LY::QS_OFF + (warp * LY::NQ + (filed - 1) % LY::NQ) * LY::QB);
      for (int i = lane; i < LY::QB / 16; i += 32) cp_async16(dst + i * 16, src + i * 16);
    }
  };
  auto look_up = [&](Walk& w) {  // where the codes of the next 32 chunks of the piece are
    const int tok = (2 * w.t + lane) * 16;
    uint64_t off = ~0ull;        // no such chunk
    if (tok < w.L) {
      const int bs = p.block_size;
      int phys = __ldg(p.block_tables + (size_t)w.b * p.max_blocks_per_seq + (tok >> (__ffs(bs) - 1)));
      if (phys < 0 || phys >= p.num_blocks) {  // broken caller invariant: record, read block 0 instead
        PA_RECORD_ERROR(PA_ERRBIT_INDEX);
        phys = 0;
      }
      const uint32_t code_block = p.num_kv_heads * bs * LY::ROWB;  // bytes; below 2^31 (checked on the host)
      off = (uint64_t)(uint32_t)phys * code_block + (uint32_t)(w.g * bs + (tok & (bs - 1))) * LY::ROWB;
    }
    win_left = min(16, w.end - w.t);
    w.t += win_left;
    __syncwarp();
    win[lane] = off;
    if (lane == 0) *walk = w;
    win_at = reinterpret_cast<const ulonglong2*>(win);
    __syncwarp();
  };
  auto next_window = [&]() {
    Walk w = *walk;
    if (w.t == w.end) {
      if (w.seg_start + places_of(w.L) + kStart >= w.line_end) return;  // no tile of the next segment is this warp's
      step_on(w);
      file_piece(w);
      bring_q(w);
    }
    look_up(w);
  };
  auto bring = [&](uint32_t stage) {  // the walk's next tile into the stage at this shared address
    const ulonglong2 off = *win_at++;
    const uint8_t* k0 = kbase + off.x;
    const uint8_t* v0 = k0 + p.v_codes;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      cp_async16(stage + LY::K_OFF + code_dst[e], k0 + 512 * e);
      cp_async16(stage + LY::V_OFF + code_dst[e], v0 + 512 * e);
    }
    const bool two = (uint32_t)(off.y >> 32) != 0xffffffffu;
    if (two) {
      const uint8_t* k1 = kbase + off.y;
      const uint8_t* v1 = k1 + p.v_codes;
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        cp_async16(stage + LY::K_OFF + 16 * LY::ROWB + code_dst[e], k1 + 512 * e);
        cp_async16(stage + LY::V_OFF + 16 * LY::ROWB + code_dst[e], v1 + 512 * e);
      }
    }
    if (par_run < 4 && (two || !(par_run & 1)))
      cp_async16(stage + par_dst, par_base + (((par_run & 1) ? off.y : off.x) >> 3));
    if (--win_left == 0) next_window();
  };
  if (any) {
    file_piece(w0);
    look_up(w0);
  }

  // The cache, q and the output may be in use by the preceding kernel (programmatic dependent launch; lengths and
  // block tables are not its outputs): wait for it before the first load of them and before any write.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (any) bring_q(w0);
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    if (win_left) bring(ring + s * LY::STAGE);
    cp_async_commit();
  }
  // sequences without a token: zeros, and a log-sum-exp of -inf
  for (int i = blockIdx.x * NW + warp; i < B; i += gridDim.x * NW) {
    if (len_of(i) != 0) continue;
    uint4* o4 = reinterpret_cast<uint4*>(reinterpret_cast<T*>(p.out) + (size_t)i * p.num_q_heads * D);
    for (int e = lane; e < p.num_q_heads * D / 8; e += 32) o4[e] = make_uint4(0, 0, 0, 0);
    if (p.lse)
      for (int h = lane; h < p.num_q_heads; h += 32) p.lse[(size_t)i * p.num_q_heads + h] = -INFINITY;
  }

  // ---- pieces and their tiles
  S st;
  int stage_at = 0;  // byte offset of the current stage
  for (int piece = 0; piece < filed; ++piece) {  // a piece's successor is filed before its last tile is done
    const Queued& d = queue[piece % LY::NQ];     // written before a warp barrier that this warp has passed
    int rem;  // tokens of the segment from the current tile on
    {
      const int4 e = *reinterpret_cast<const int4*>(&d);
      int m = d.end - e.w;  // the piece's tiles
      rem = e.z - e.w * kTile;
      if constexpr (LY::QS) {
        cp_async_wait<NS - 1>();
        __syncwarp();
        st.template begin<true>(smem + LY::QS_OFF + (warp * LY::NQ + piece % LY::NQ) * LY::QB, p.scale_log2, lane);
      } else {  // q is on its way while the tile lands
        st.template begin<false>(q_rows(e.x, e.y), p.scale_log2, lane);
      }
      do {
        cp_async_wait<NS - 1>();
        __syncwarp();
        st.template tile<LY>(smem + LY::RING_OFF + warp * LY::RING + stage_at, smem + LY::CONV_OFF + warp * LY::CONV, rem,
                             lane);
        __syncwarp();
        if (win_left) bring(ring + stage_at);
        cp_async_commit();
        stage_at = stage_at == (NS - 1) * LY::STAGE ? 0 : stage_at + LY::STAGE;
        rem -= kTile;
      } while (--m);
    }
    st.finish();
    const int4 de = *reinterpret_cast<const int4*>(&d);
    const int b = de.x, kvh = de.y;
    const bool head = de.w == 0, tail = rem <= 0;
    const int g = lane >> 2, c = lane & 3;
    if (head && tail) {
      const size_t row0 = head0((size_t)b * p.num_kv_heads + kvh);
      T* out = reinterpret_cast<T*>(p.out) + row0 * D;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int h = 2 * c + e;
        if (h >= G) continue;
        const float inv = 1.f / st.l[e];
#pragma unroll
        for (int grp = 0; grp < S::NG; ++grp) {
          float v[8];
          st.values(grp, e, v);
          uint4 u;
          u.x = Elt<DT>::from_f2(v[0] * inv, v[1] * inv);
          u.y = Elt<DT>::from_f2(v[2] * inv, v[3] * inv);
          u.z = Elt<DT>::from_f2(v[4] * inv, v[5] * inv);
          u.w = Elt<DT>::from_f2(v[6] * inv, v[7] * inv);
          st_v4(out + h * D + 64 * grp + 8 * g, u);
        }
        if (p.lse && g == 0) p.lse[row0 + h] = (st.R[e] + __log2f(st.l[e])) * kLn2;
      }
    } else {
      const int which = piece + 1 == filed;  // the warp's last piece lies in its ring, which is done with
      float* part = reinterpret_cast<float*>(which ? smem + LY::RING_OFF + warp * LY::RING
                                                   : smem + LY::PART_OFF + warp * LY::PART);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int h = 2 * c + e;
        if (h >= G) continue;
#pragma unroll
        for (int grp = 0; grp < S::NG; ++grp) {
          float v[8];
          st.values(grp, e, v);
          float4* o4 = reinterpret_cast<float4*>(part + h * D + 64 * grp + 8 * g);
          o4[0] = make_float4(v[0], v[1], v[2], v[3]);
          o4[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
        if (g == 0) {
          part[G * D + h] = st.R[e];
          part[G * D + G + h] = st.l[e];
        }
      }
      if (lane == 0) {
        Piece pc;
        pc.b = b;
        pc.g = kvh;
        pc.flags = F_VALID | (head ? F_HEAD : 0) | (tail ? F_TAIL : 0);
        pc.nt = tiles_of(de.z);
        pc.seg_start = d.seg_start;
        pieces[2 * warp + which] = pc;
      }
    }
  }
  // let the next programmatically launched kernel begin its set-up; it waits for this grid before it touches memory
  asm volatile("griddepcontrol.launch_dependents;");
  __syncthreads();

  // ---- join the pieces of each segment.  Lane i holds piece i of the CTA; a run is the pieces of one segment.  (This
  // code runs once a launch, so its instructions come from far: few of them, and threads side by side, count.)
  Piece pc;
  pc.flags = 0;
  pc.b = pc.g = pc.nt = 0;
  pc.seg_start = 0;
  if (lane < 2 * NW) pc = pieces[lane];
  const bool valid = pc.flags & F_VALID;
  const unsigned vmask = __ballot_sync(0xffffffffu, valid);
  if (vmask == 0) return;
  Run* run_s = reinterpret_cast<Run*>(smem + LY::JOIN_OFF);
  float* w_s = reinterpret_cast<float*>(run_s + 2 * NW);    // [2 NW][G]: weight of a piece within its run
  float2* md_s = reinterpret_cast<float2*>(w_s + 2 * NW * G);  // [2 NW][G]: reference M and sum of a run
  const unsigned below = vmask & ((1u << lane) - 1u);
  const long long prev = __shfl_sync(0xffffffffu, pc.seg_start, below ? 31 - __clz(below) : lane);
  const bool starts = valid && (!below || prev != pc.seg_start);
  const unsigned smask = __ballot_sync(0xffffffffu, starts);
  const int runs = __popc(smask);
  const unsigned after = lane < 31 ? smask & ~((2u << lane) - 1u) : 0u;
  const unsigned rmask = vmask & ~((1u << lane) - 1u) & (after ? (1u << (__ffs(after) - 1)) - 1u : 0xffffffffu);
  const int end_flags = __shfl_sync(0xffffffffu, pc.flags, starts ? 31 - __clz(rmask) : lane);
  const bool whole = (pc.flags & F_HEAD) && (end_flags & F_TAIL);
  // Segments cut between CTAs: the first run or the last at most.
  const bool cut0 = __shfl_sync(0xffffffffu, starts && !whole, __ffs(smask) - 1);
  const bool cut1 = runs > 1 && __shfl_sync(0xffffffffu, starts && !whole, 31 - __clz(smask));
  const int cuts = cut0 + cut1;
  if (starts) {  // every warp writes the same table, and reads its own writes
    Run r;
    r.mask = rmask;
    r.b = pc.b;
    r.g = pc.g;
    r.whole = whole;
    run_s[__popc(smask & ((1u << lane) - 1u))] = r;
  }
  __syncwarp();
  auto part_of = [&](int i) {
    return reinterpret_cast<const float*>((i & 1) ? smem + LY::RING_OFF + (i >> 1) * LY::RING
                                                  : smem + LY::PART_OFF + (i >> 1) * LY::PART);
  };
  // weights: eight lanes to a (run, head)
  for (int item = warp * 4 + (lane >> 3); item - (lane >> 3) < runs * G; item += NW * 4) {
    const int r = min(item / G, runs - 1), h = item % G;
    const unsigned mask = run_s[r].mask;
    float R[(2 * NW + 7) / 8], l[(2 * NW + 7) / 8], M = -INFINITY;
#pragma unroll
    for (int k = 0; k < (2 * NW + 7) / 8; ++k) {
      const int i = k * 8 + (lane & 7);
      const bool on = mask >> i & 1;
      R[k] = on ? part_of(i)[G * D + h] : 0.f;
      l[k] = on ? part_of(i)[G * D + G + h] : 0.f;
      M = fmaxf(M, l[k] > 0.f ? R[k] + __log2f(l[k]) : -INFINITY);  // of the pieces' log-sum-exps: nothing overflows
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float den = 0.f;
#pragma unroll
    for (int k = 0; k < (2 * NW + 7) / 8; ++k) {
      const int i = k * 8 + (lane & 7);
      const float w = l[k] > 0.f ? exp2f(R[k] - M) : 0.f;
      den = fmaf(w, l[k], den);
      if ((mask >> i & 1) && item < runs * G) w_s[i * G + h] = w;
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    if ((lane & 7) == 0 && item < runs * G) md_s[r * G + h] = make_float2(M, den);
  }
  __syncthreads();
  // columns: a thread takes 4 of a head.  Cut segments first: this CTA's shares of them go to the workspace.
  constexpr int QUADS = G * D / 4;
  const size_t ws_row0 = (size_t)half * (B * (size_t)Hkv + line_ctas) * G;  // each half has slots and counters of its own
  float *ws_r = p.ws_r + ws_row0, *ws_l = p.ws_l + ws_row0, *ws_o = p.ws_o + ws_row0 * D;
  int* ws_cnt = p.ws_cnt + half * (kMaxGrid / 2);
  auto columns = [&](int from, int to) {
    for (int q = from * QUADS + threadIdx.x; q < to * QUADS; q += NW * 32) {
      const int k = q / QUADS, e = q - k * QUADS, h = e / (D / 4), col = e % (D / 4) * 4;
      const int r = k >= cuts ? k - cuts + cut0 : (k == 0 && cut0 ? 0 : runs - 1);
      const Run run = run_s[r];
      const float2 md = md_s[r * G + h];
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (unsigned m = run.mask; m; m &= m - 1) {
        const int i = __ffs(m) - 1;
        const float w = w_s[i * G + h];
        const float4 o = *reinterpret_cast<const float4*>(part_of(i) + h * D + col);
        acc.x = fmaf(w, o.x, acc.x); acc.y = fmaf(w, o.y, acc.y);
        acc.z = fmaf(w, o.z, acc.z); acc.w = fmaf(w, o.w, acc.w);
      }
      const size_t seg = (size_t)run.b * Hkv + run.g;
      if (run.whole) {
        const float inv = 1.f / md.y;
        uint2 u;
        u.x = Elt<DT>::from_f2(acc.x * inv, acc.y * inv);
        u.y = Elt<DT>::from_f2(acc.z * inv, acc.w * inv);
        *reinterpret_cast<uint2*>(reinterpret_cast<T*>(p.out) + (head0(seg) + h) * D + col) = u;
        if (p.lse && col == 0) p.lse[head0(seg) + h] = (md.x + __log2f(md.y)) * kLn2;
      } else {
        const size_t row = (seg + cta) * G + h;
        *reinterpret_cast<float4*>(ws_o + row * D + col) = acc;
        if (col == 0) {
          ws_r[row] = md.x;
          ws_l[row] = md.y;
        }
      }
    }
  };
  columns(0, cuts);
  // The cut segments (0: of the first run, 1: of the last), in lanes 0 and 1 of every warp.
  Cut cut = {0, 0, 0};
  if (lane < 2 && (lane == 0 ? cut0 : cut1)) {
    const Piece& mine = pieces[__ffs(run_s[lane == 0 ? 0 : runs - 1].mask) - 1];
    cut = cut_of((long long)mine.b * Hkv + mine.g, mine.seg_start + kStart, mine.nt, ctas, total, narrow);
  }
  int* done_s = reinterpret_cast<int*>(smem + LY::LENS_OFF);
  if (cuts) {
    __syncthreads();  // the CTA's shares are written
    if (warp == 0 && lane < 2) {
      const Round r = join_round(0, cut, cta);
      done_s[lane] = cut.n > 0 && count_last(ws_cnt + r.counter, r.n);
    }
  }
  columns(cuts, runs);  // meanwhile the segments that lie within the CTA
  if (!cuts) return;
  // Cut segments whose shares this CTA counted last: a thread takes 4 columns of a head, 8 shares at a time.  Each round
  // follows from the segment alone: nothing is carried from one segment, or one round, to the next.
  constexpr int PASSES = (QUADS + NW * 32 - 1) / (NW * 32), U = 8;
  for (int which = 0; which < 2; ++which) {
    Cut k;
    k.seg = __shfl_sync(0xffffffffu, cut.seg, which);
    k.c0 = __shfl_sync(0xffffffffu, cut.c0, which);
    k.n = __shfl_sync(0xffffffffu, cut.n, which);
    for (int round = 0;; ++round) {
      __syncthreads();
      if (!done_s[which]) break;
      const Round jr = join_round(round, k, cta);
      float4 acc[PASSES];
      float M[PASSES], den[PASSES];
#pragma unroll
      for (int ps = 0; ps < PASSES; ++ps) {
        acc[ps] = make_float4(0.f, 0.f, 0.f, 0.f);
        M[ps] = -INFINITY;
        den[ps] = 0.f;
        const int quad = ps * NW * 32 + threadIdx.x, h = quad / (D / 4), col = quad % (D / 4) * 4;
        if (quad >= QUADS) break;
        for (int i0 = 0; i0 < jr.n; i0 += U) {
          float r[U], l[U];
          float4 v[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int i = min(i0 + u, jr.n - 1);
            const size_t row = (size_t)(i == 0 ? jr.slot0 : jr.slots + (long long)i * jr.step) * G + h;
            r[u] = __ldcg(ws_r + row);
            l[u] = i0 + u < jr.n ? __ldcg(ws_l + row) : 0.f;
            v[u] = __ldcg(reinterpret_cast<const float4*>(ws_o + row * D + col));
          }
          float top = M[ps];
#pragma unroll
          for (int u = 0; u < U; ++u) top = fmaxf(top, l[u] > 0.f ? r[u] + __log2f(l[u]) : -INFINITY);
          const float f = M[ps] > -INFINITY ? exp2f(M[ps] - top) : 0.f;
          M[ps] = top;
          den[ps] *= f;
          acc[ps].x *= f; acc[ps].y *= f; acc[ps].z *= f; acc[ps].w *= f;
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const float w = l[u] > 0.f ? exp2f(r[u] - top) : 0.f;
            den[ps] = fmaf(w, l[u], den[ps]);
            acc[ps].x = fmaf(w, v[u].x, acc[ps].x); acc[ps].y = fmaf(w, v[u].y, acc[ps].y);
            acc[ps].z = fmaf(w, v[u].z, acc[ps].z); acc[ps].w = fmaf(w, v[u].w, acc[ps].w);
          }
        }
      }
      if (jr.again) __syncthreads();  // the group's shares are read: their joint share takes the first one's slot
#pragma unroll
      for (int ps = 0; ps < PASSES; ++ps) {
        const int quad = ps * NW * 32 + threadIdx.x, h = quad / (D / 4), col = quad % (D / 4) * 4;
        if (quad >= QUADS) break;
        if (jr.again) {
          const size_t row = (size_t)jr.slot0 * G + h;
          *reinterpret_cast<float4*>(ws_o + row * D + col) = acc[ps];
          if (col == 0) {
            ws_r[row] = M[ps];
            ws_l[row] = den[ps];
          }
        } else {
          const size_t at = head0((size_t)k.seg) + h;
          const float inv = 1.f / den[ps];
          uint2 u;
          u.x = Elt<DT>::from_f2(acc[ps].x * inv, acc[ps].y * inv);
          u.y = Elt<DT>::from_f2(acc[ps].z * inv, acc[ps].w * inv);
          *reinterpret_cast<uint2*>(reinterpret_cast<T*>(p.out) + at * D + col) = u;
          if (p.lse && col == 0) p.lse[at] = (M[ps] + __log2f(den[ps])) * kLn2;
        }
      }
      if (!jr.again) break;
      __syncthreads();  // the joint share is written
      if (threadIdx.x == 0) {
        const Round up = join_round(round + 1, k, cta);
        done_s[which] = count_last(ws_cnt + up.counter, up.n);
      }
    }
  }
}

// ------------------------------------------------------------------ host side
// Warps of a CTA (one CTA fills an SM) and stages of each warp's ring.  D 128, G <= 8: 12 warps of 168 registers; 16 warps
// of 128 need 590 instructions a tile instead of 522 (values kept and fetched again): 64 sequences of 4096 to 8192
// tokens, 64 heads, take 92.9 us with 16, 89.5 with 12, 101 with 10, 107 with 8.  D 64 fits 16 (27.4 against 28.6 us,
// 64 sequences of 500 to 8000).  A third stage changes nothing.  (Measured with K's codes low in their halves and segments cut.)
// G 16 as one piece (two column tiles, 8 warps of 250 registers) against two halves on two CTAs: one sequence of 2000
// tokens 14.7 and 11.3 us, of 100001 26.8 and 23.7, 16 of 8000 26.6 and 25.6, 64 of 100 to 8000 38.7 and 40.1 (D 128, 2
// KV heads; D 64 10.3 and 9.8 to 27.7 and 29.4).  Halves for all sizes: they win where segments are few, by up to 23 %, and
// lose up to 6 % where they are many; one form keeps one set of kernels.  (Measured with one term of the weights.)
constexpr int kWarps = 12;

template <int D, int G>
struct Shape {
  static constexpr int NW = D == 64 ? 16 : kWarps;
  static constexpr int NS = 2;
};

struct Plan {
  int grid;
  size_t off_r, off_l, off_o, bytes;
};

bool make_plan(int batch, int Hq, int Hkv, int D, int max_context_len, int num_partitions, Plan* pl) {
  if (batch < 0 || Hq <= 0 || Hkv <= 0 || num_partitions < 0 || max_context_len < 0 || Hq % Hkv) return false;
  if (!valid_head_dim(D) || !valid_group(Hq / Hkv)) return false;
  if ((int64_t)batch * Hq >= (1ll << 31)) return false;
  const int G = Hq / Hkv, HV = G == 16 ? 2 : 1;
  // One CTA fills an SM.  A small batch takes no more CTAs than give every warp about two tiles (were all contexts as
  // long as they may be), and a multiple of its segments, so that equal lengths are cut where CTAs meet or not at
  // all: joining across CTAs costs about 4 us.  (One sequence of 300 tokens, 8 KV heads: 8 CTAs 7 us, 20 CTAs 8.8 us.)
  const int64_t segs = std::max<int64_t>(1, (int64_t)batch * Hkv);
  const int64_t tiles = segs * ((max_context_len + (int64_t)kTile - 1) / kTile);
  const int64_t sms = sm_count() / HV, want = (tiles + 2 * kWarps - 1) / (2 * kWarps);
  int64_t grid = std::min(sms, std::max<int64_t>(1, want));
  if (segs <= sms) {
    const int64_t up = std::min(sms / segs, (grid + segs - 1) / segs) * segs;
    if (up >= grid || up * 20 >= grid * 19) grid = up;
  }
  if (num_partitions) grid = (num_partitions + (int64_t)HV - 1) / HV;
  pl->grid = (int)std::min<int64_t>(grid, kMaxGrid / HV) * HV;
  auto align256 = [](size_t x) { return (x + 255) & ~size_t(255); };
  const size_t slots = (size_t)batch * Hkv + pl->grid;
  pl->off_r = 3 * kMaxGrid * 4;
  pl->off_l = pl->off_r + align256(slots * G * 4);
  pl->off_o = pl->off_l + align256(slots * G * 4);
  pl->bytes = pl->off_o + align256(slots * G * D * 4);
  return true;
}

template <int DT, int D, int G, int HV = 1>
int launch(const Params& p, int grid, cudaStream_t st) {
  constexpr int NW = Shape<D, G>::NW, NS = Shape<D, G>::NS;
  using LY = Layout<D, G, NW, NS>;
  static_assert(LY::BYTES <= 227 * 1024, "shared memory of one CTA");
  auto kern = decode_int4_kernel<DT, D, G, HV, NW, NS>;
  // per instantiation and device; host threads may race to set it, which only repeats an idempotent call
  static std::atomic<bool> attr_set[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PA_ERR_CUDA;
  if (dev < 0 || dev >= 64 || !attr_set[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, LY::BYTES) != cudaSuccess)
      return PA_ERR_CUDA;
    if (dev >= 0 && dev < 64) attr_set[dev].store(true, std::memory_order_release);
  }
  return launch_programmatic(kern, dim3((unsigned)grid), dim3(NW * 32), LY::BYTES, st, p);
}

template <int DT, int D>
int dispatch_g(int G, const Params& p, int grid, cudaStream_t st) {
  switch (G) {
    case 1: return launch<DT, D, 1>(p, grid, st);
    case 2: return launch<DT, D, 2>(p, grid, st);
    case 4: return launch<DT, D, 4>(p, grid, st);
    case 8: return launch<DT, D, 8>(p, grid, st);
    case 16: return launch<DT, D, 8, 2>(p, grid, st);
  }
  return PA_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" int pa_decode_int4_plan(int batch, int num_q_heads, int num_kv_heads, int head_dim, int max_context_len,
                                   int num_partitions_or_0, int* grid_out, int* max_pieces_out,
                                   size_t* workspace_bytes_out) {
  Plan pl;
  if (!make_plan(batch, num_q_heads, num_kv_heads, head_dim, max_context_len, num_partitions_or_0, &pl))
    return PA_ERR_INVALID;
  if (grid_out) *grid_out = pl.grid;
  if (max_pieces_out) *max_pieces_out = batch * num_kv_heads + pl.grid;
  if (workspace_bytes_out) *workspace_bytes_out = pl.bytes;
  return PA_OK;
}

extern "C" size_t pa_decode_int4_workspace_size(int batch, int num_q_heads, int num_kv_heads, int head_dim,
                                                int max_context_len, int num_partitions_or_0) {
  Plan pl;
  return make_plan(batch, num_q_heads, num_kv_heads, head_dim, max_context_len, num_partitions_or_0, &pl) ? pl.bytes
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
  // the kernel counts tokens in 32 bits, up to a window of look-ups (32 chunks of 16) past a sequence's end
  if ((int64_t)max_blocks_per_seq * block_size > (1ll << 31) - 1024) return PA_ERR_UNSUPPORTED;
  if ((int64_t)num_kv_heads * block_size * head_dim >= (1ll << 31)) return PA_ERR_UNSUPPORTED;
  Plan pl;
  if (!make_plan(batch, num_q_heads, num_kv_heads, head_dim, max_context_len, num_partitions_or_0, &pl))
    return PA_ERR_INVALID;
  if (!workspace || workspace_bytes < pl.bytes) return PA_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return PA_ERR_ALIGN;
  uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
  Params p;
  p.q = q;
  p.out = out;
  p.lse = lse_out;
  p.k_codes = (const uint8_t*)k_codes;
  p.k_params = (const uint8_t*)k_params;
  p.v_codes = (long long)((intptr_t)v_codes - (intptr_t)k_codes);
  p.v_params = (long long)((intptr_t)v_params - (intptr_t)k_params);
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.ws_cnt = reinterpret_cast<int*>(ws);
  p.ws_r = reinterpret_cast<float*>(ws + pl.off_r);
  p.ws_l = reinterpret_cast<float*>(ws + pl.off_l);
  p.ws_o = reinterpret_cast<float*>(ws + pl.off_o);
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.batch = batch;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.block_size = block_size;
  p.num_blocks = num_blocks;
  p.scale_log2 = scale * 1.4426950408889634f;
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == PA_BF16)
    return head_dim == 128 ? dispatch_g<PA_BF16, 128>(G, p, pl.grid, st) : dispatch_g<PA_BF16, 64>(G, p, pl.grid, st);
  return head_dim == 128 ? dispatch_g<PA_F16, 128>(G, p, pl.grid, st) : dispatch_g<PA_F16, 64>(G, p, pl.grid, st);
}
