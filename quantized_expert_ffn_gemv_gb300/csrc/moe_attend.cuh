// What the attention kernels share: their arguments, a sequence as they see
// it, partial results.
//
// Both kernels cut a line of work into equal parts, one a CTA.  A (sequence,
// kv head, row tile) segment that lies in one part is finished by its CTA; of
// one that is cut, every CTA leaves a partial result (output relative to a
// reference maximum, the maximum, the sum): in its slot 1 where it begins at
// the segment's first tile, in slot 0 otherwise, and the CTA that has the
// last tile notes the segment in `ends`.  attend_join_kernel merges those.
//
// With a shared prefix, attend_tiles_kernel runs over its keys with the rows
// of all sequences as one, attend_rows_kernel over what is behind it, and
// attend_join_shared_kernel merges both for every row: then no kernel finishes
// a segment, whole ones leave their result in `whole`, and every segment's
// parts are noted in `spans`.
#pragma once

#include <cfloat>
#include <cmath>

#include "moe_kv.cuh"
#include "moe_ptx.cuh"

namespace moe {

constexpr float kPShift = 8.f;  // probabilities are held times 2^8
constexpr uint32_t kNaN = 0x7FFFFFFFu;

// A cut segment, noted by the CTA with its last tile: where the segment is,
// and the CTA that has its first tile (-1: the CTA ends none).
struct SegmentEnd {
  int first, b, head, rt;
};

// The parts of a segment: first .. last, or kWhole for one that a single CTA finished.
constexpr int kWhole = -2;
struct Span {
  int first, last;
};

struct AttArgs {
  const uint16_t* q;
  int64_t q_ts, q_hs;
  uint16_t* out;
  int64_t o_ts, o_hs;
  float* lse;
  float scale_log2;  // scale * log2(e)
  int nq, group;
  int tile_rows;     // rows of a row tile
  int parts;         // CTAs
  float* partial;    // [parts][2][tile_rows][D]
  float2* stats;     // [parts][2][tile_rows] (maximum, sum)
  SegmentEnd* ends;  // [parts]
  int shared;          // keys of the shared prefix, 0 = none; what follows is for it
  int max_row_tiles;   // row tiles of a sequence at most (attend_rows_kernel's segments)
  float* whole;        // [segments][tile_rows][D]
  float2* whole_stats; // [segments][tile_rows]
  Span* spans;         // [segments]
};

// A sequence's arrays, made harmless: new tokens that cannot be are none
// (flag_batch reports them), a length is not negative.
struct Seq {
  int row0, n, len;  // first row, new tokens, length
  bool over;         // longer than the block table is wide
};

__device__ __forceinline__ Seq seq_at(const KvArgs& a, int b) {
  Seq s;
  s.row0 = __ldg(a.cu + b);
  s.n = __ldg(a.cu + b + 1) - s.row0;
  s.len = max(__ldg(a.lens + b), 0);
  if (s.row0 < 0 || s.n < 0 || s.n > a.max_tokens || s.row0 > a.n_tokens - s.n) s.n = 0;
  s.over = s.len > a.max_pages * a.page_size;
  return s;
}

__device__ __forceinline__ void flag_batch(const KvArgs& a, int b) {
  int bad = kv_seq_ok(a, b) ? 0 : MOE_KV_BAD_BATCH;
  if (__ldg(a.lens + b) > a.max_pages * a.page_size) bad |= MOE_KV_BAD_PAGE;
  if (bad) kv_flag(a, bad);
}

// Natural logarithm of the sum of exp(score) from a maximum in units of log2 and a sum held times 2^8.
__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l) - kPShift) * 0.6931471805599453f;
}

// Probabilities and values enter the products rounded to fp16 once each.  With
// fp16 outputs, whose own rounding is no larger, the two together made up to
// 1.6 times its error: there a second product takes up the rest, of the values
// in attend_rows_kernel, of keys and probabilities in attend_tiles_kernel,
// whose shared memory has no room for a second V.
// What rounding to fp16 left of a and b:
__device__ __forceinline__ uint32_t rest_of(uint32_t held, float a, float b) {
  float x, y;
  unpack2<false>(held, x, y);
  return pack2<false>(a - x, b - y);
}

// (v & mask) | bits in one instruction; `bits` has to be a register the
// compiler cannot see through (two constants would take two instructions).
template <uint32_t MASK>
__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(v), "n"(MASK), "r"(bits));
  return r;
}

// The power of two that brings a row's largest magnitude below 2 (2^8 at the
// end of bf16's range), as an exponent; infinities and NaN leave it at 0.
__device__ __forceinline__ int row_exponent(float big) {
  const int e = ((__float_as_uint(big) >> 23) & 255) - 127;
  return big > 0.f && e < 128 ? min(max(e, -120), 120) : 0;
}
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
// What a query is multiplied by: 2^-e with the scale's sign, 0 for a scale of 0, so that the scores' factor is positive.
__device__ __forceinline__ float query_factor(float scale_log2, int e) {
  return scale_log2 == 0.f ? 0.f : scale_log2 < 0.f ? -pow2i(-e) : pow2i(-e);
}
// What a product of scaled query and key is multiplied by, > 0.
__device__ __forceinline__ float score_factor(float scale_log2, int e) {
  return scale_log2 == 0.f ? 1.f : fmaxf(fabsf(scale_log2) * pow2i(e), FLT_MIN);
}

// Launches, one translation unit each (moe_attend_rows8.cu and so on).  The
// number of CTAs an SM holds is part of the plan.
int rows_blocks(int dim, int bits, int tile_rows);
moe_status_t launch_rows8(const KvArgs& kv, const AttArgs& t, int dim, bool bf16, cudaStream_t st);
moe_status_t launch_rows4(const KvArgs& kv, const AttArgs& t, int dim, bool bf16, cudaStream_t st);
moe_status_t launch_tiles8(const KvArgs& kv, const AttArgs& t, int dim, bool bf16, cudaStream_t st);
moe_status_t launch_tiles4(const KvArgs& kv, const AttArgs& t, int dim, bool bf16, cudaStream_t st);

}  // namespace moe
