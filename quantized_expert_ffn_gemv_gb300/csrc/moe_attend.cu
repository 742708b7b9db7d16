// Attention of a batch's new tokens over the quantised paged cache.
//
// attend_rows_kernel: few rows a sequence (decode, speculation).  Rows are
// (new token, query head of the kv head's group), 16 to a row tile, the M of
// mma.sync m16n8k16.  A call is a line of work units, one for each 32-token
// tile of keys that a (sequence, kv head, row tile) segment has to see; the
// line is cut into equal parts, one a CTA, whatever the lengths are.  A CTA's
// four warps take every fourth tile of a segment, each with a ring of its own
// that one lane fills by bulk copies (half a tile, its K or its V with the
// scales, is contiguous in the pool), and keep a running maximum, sum and
// output in registers (one pass over the keys).  The warps' results are
// merged in shared memory; a segment that ends in another CTA leaves a
// partial result in the workspace and attend_join_kernel merges those.
//
// Dequantisation happens on the way into the tensor core.  K: a lane's 8
// elements of a 32-element block are the operands of two k16 steps (the order
// of the reduction is free, so the natural byte order serves as the
// fragment's), as exact fp16 integers (1024 + u through the exponent, minus
// 1024 + bias); the block's scale multiplies the fp32 product.  V: a byte
// permutation pairs the same element of two keys; integer times scale is
// rounded to fp16 once.  Queries are scaled by a power of two per row so that
// fp16 holds them whatever their range; probabilities carry 2^8 so that small
// ones keep their precision in fp16.
#include <cfloat>
#include <cmath>

#include "moe_kv.cuh"
#include "moe_ptx.cuh"

namespace moe {
namespace {

using namespace ptx;

constexpr int kAttWarps = 4;
constexpr int kAttThreads = 32 * kAttWarps;
constexpr int kRows = 16;          // rows of a row tile
constexpr int kMinTiles = 4;       // tiles a CTA takes at least: one a warp
constexpr float kPShift = 8.f;     // probabilities are held times 2^8
constexpr int kRingBytes = 26112;  // a warp's ring, at most (two CTAs an SM)

struct AttArgs {
  const uint16_t* q;
  int64_t q_ts, q_hs;
  uint16_t* out;
  int64_t o_ts, o_hs;
  float* lse;
  float scale_log2;  // scale * log2(e)
  int nq, group, max_row_tiles;
  int parts;        // CTAs of attend_rows_kernel
  float* partial;   // [parts][2][16][D]
  float2* stats;    // [parts][2][16] (maximum, sum)
  int64_t* starts;  // [segments]: where the segment begins on the line of work; [-1]: units a CTA takes
};

// A sequence as the kernels see it.
struct Seq {
  int row0, n, len, tiles, row_tiles;  // first row, new tokens, length, 32-token tiles of keys, row tiles
  bool over;                           // longer than the block table is wide
};

__device__ __forceinline__ Seq seq_at(const KvArgs& a, int group, int b) {
  Seq s;
  s.row0 = __ldg(a.cu + b);
  s.n = __ldg(a.cu + b + 1) - s.row0;
  s.len = max(__ldg(a.lens + b), 0);
  if (s.row0 < 0 || s.n < 0 || s.n > a.max_tokens || s.row0 > a.n_tokens - s.n) s.n = 0;  // flagged by flag_batch
  const int cap = a.max_pages * a.page_size;
  s.over = s.len > cap;
  s.tiles = max(1, (min(s.len, cap) + kKvTile - 1) / kKvTile);
  s.row_tiles = (s.n * group + kRows - 1) / kRows;
  return s;
}

__device__ void flag_batch(const KvArgs& a, int b) {
  const int c0 = __ldg(a.cu + b), c1 = __ldg(a.cu + b + 1), len = __ldg(a.lens + b);
  int bad = 0;
  if (c0 < 0 || c1 < c0 || c1 - c0 > a.max_tokens || c1 > a.n_tokens || c1 - c0 > len) bad |= MOE_KV_BAD_BATCH;
  if (len > a.max_pages * a.page_size) bad |= MOE_KV_BAD_PAGE;
  if (bad) kv_flag(a, bad);
}

// Element of column c (0..7) of the value product's n-tile j: the lanes of
// column c hold a contiguous run of a key's bytes.
template <int D, int BITS>
__device__ __forceinline__ int out_dim(int j, int c) {
  if (BITS == 8 && D == 256) return (j >> 4) * 128 + 16 * c + (j & 15);
  return (D / 8) * c + j;
}

template <int D, int BITS>
struct RowsPlan {
  static constexpr int kHalf = kv_half_bytes(D, BITS);
  static constexpr int kEntries = (kRingBytes / kHalf) < 12 ? (kRingBytes / kHalf) : 12;
  static constexpr int kRing = kEntries * kHalf;      // bytes a warp
  static constexpr int kQBytes = kRows * D * 2;       // query fragments
  static constexpr int kMerge = kRows * (D + 4) * 4;  // a warp's output for the merge, inside its ring
  static constexpr int kSmem = kAttWarps * kRing + kQBytes + 64 + kAttWarps * kEntries * 8;
  static_assert(kMerge <= kRing, "the merge buffer lies in the ring");
  static_assert(kEntries >= 3, "a ring of three halves at least");
};

// One warp's products of a 32-key tile: scores s[4 n-tiles][4] as the exact
// product of integers and queries times the block scale.
template <int D, int BITS>
__device__ __forceinline__ void score_tile(float (&s)[4][4], uint32_t kb, uint32_t qf, int lane) {
  constexpr int R = kv_row_bytes(D, BITS), NC = R / 16;
  const int g = lane >> 2, t = lane & 3, turn = kv_turn(g) & (NC - 1);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll
  for (int b = 0; b < D / 32; ++b) {
    const uint4 qa = lds128(qf + (2 * b) * 512 + lane * 16), qb = lds128(qf + (2 * b + 1) * 512 + lane * 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t k0, k1, k2, k3;
      if (BITS == 8) {
        const uint2 w = lds64(kb + (8 * i + g) * R + (((2 * b + (t >> 1)) ^ turn) << 4) + (t & 1) * 8);
        k0 = hsub2(prmt(w.x, 0x64646464u, 0x4140), 0x64806480u);
        k1 = hsub2(prmt(w.x, 0x64646464u, 0x4342), 0x64806480u);
        k2 = hsub2(prmt(w.y, 0x64646464u, 0x4140), 0x64806480u);
        k3 = hsub2(prmt(w.y, 0x64646464u, 0x4342), 0x64806480u);
      } else {
        const uint32_t w = lds32(kb + (8 * i + g) * R + ((b ^ turn) << 4) + t * 4), w8 = w >> 8;
        k0 = hsub2((w & 0x000F000Fu) | 0x64006400u, 0x64086408u);
        k1 = hfma2((w & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD480D480u);
        k2 = hsub2((w8 & 0x000F000Fu) | 0x64006400u, 0x64086408u);
        k3 = hfma2((w8 & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD480D480u);
      }
      float p[4] = {0.f, 0.f, 0.f, 0.f};
      mma_f16(p, qa.x, qa.y, qa.z, qa.w, k0, k1);
      mma_f16(p, qb.x, qb.y, qb.z, qb.w, k2, k3);
      const uint32_t sc = lds32(kb + kKvTile * R + (b * kKvTile + 8 * i + 2 * t) * 2);
      const float2 d = __half22float2(*reinterpret_cast<const __half2*>(&sc));
      s[i][0] = fmaf(p[0], d.x, s[i][0]);
      s[i][1] = fmaf(p[1], d.y, s[i][1]);
      s[i][2] = fmaf(p[2], d.x, s[i][2]);
      s[i][3] = fmaf(p[3], d.y, s[i][3]);
    }
  }
}

// o += p v for 16 keys (step u of a tile).  edge: keys from lim on (within
// the tile) are seen by no row and count as 0 whatever their bytes say, and so
// do non-finite scales (the caller deals with the rows that see them).
template <int D, int BITS>
__device__ __forceinline__ void value_step(float (&o)[D / 8][4], const uint32_t (&p)[4], uint32_t vb, int u, int lane,
                                           bool edge, int lim) {
  constexpr int R = kv_row_bytes(D, BITS), NC = R / 16, RUN = D / 8;
  constexpr int kRuns = (BITS == 8 && D == 256) ? 2 : 1;  // runs of RUN / kRuns elements a lane column has
  constexpr int kWords = RUN / kRuns * BITS / 32;         // 32-bit words of a run: 1, 2 or 4
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int r = 0; r < kRuns; ++r) {
    const int first = r * 128 + g * (RUN / kRuns);  // first element of the run
    const int blk = first / 32;
    uint32_t v[4][4], sc[2];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int key = 16 * u + 2 * t + (x & 1) + (x >> 1) * 8;
      const int turn = kv_turn(key) & (NC - 1);
      const int byte = first * BITS / 8;
      const uint32_t a = vb + key * R + (((byte >> 4) ^ turn) << 4) + (byte & 15);
      if (kWords == 4) {
        const uint4 w = lds128(a);
        v[x][0] = w.x, v[x][1] = w.y, v[x][2] = w.z, v[x][3] = w.w;
      } else if (kWords == 2) {
        const uint2 w = lds64(a);
        v[x][0] = w.x, v[x][1] = w.y;
      } else {
        v[x][0] = lds32(a);
      }
    }
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int key = 16 * u + 2 * t + 8 * y;
      sc[y] = lds32(vb + kKvTile * R + (blk * kKvTile + key) * 2);
      if (edge) {
        if (key >= lim || (sc[y] & 0x7C00u) == 0x7C00u) sc[y] &= 0xFFFF0000u;
        if (key + 1 >= lim || (sc[y] & 0x7C000000u) == 0x7C000000u) sc[y] &= 0x0000FFFFu;
      }
    }
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      if (BITS == 8) {
        const uint32_t x0 = prmt(v[0][w], v[1][w], 0x5140), x1 = prmt(v[0][w], v[1][w], 0x7362);
        const uint32_t y0 = prmt(v[2][w], v[3][w], 0x5140), y1 = prmt(v[2][w], v[3][w], 0x7362);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t sel = (e & 1) ? 0x4342u : 0x4140u;
          const uint32_t b0 = hmul2(hsub2(prmt(e < 2 ? x0 : x1, 0x64646464u, sel), 0x64806480u), sc[0]);
          const uint32_t b1 = hmul2(hsub2(prmt(e < 2 ? y0 : y1, 0x64646464u, sel), 0x64806480u), sc[1]);
          mma_f16(o[r * 16 + 4 * w + e], p[0], p[1], p[2], p[3], b0, b1);
        }
      } else {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t x = prmt(v[0][w], v[1][w], q ? 0x7632 : 0x5410), y = prmt(v[2][w], v[3][w], q ? 0x7632 : 0x5410);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t b0 = hmul2(hsub2((x & 0x000F000Fu) | 0x64006400u, 0x64086408u), sc[0]);
            uint32_t b1 = hmul2(hsub2((y & 0x000F000Fu) | 0x64006400u, 0x64086408u), sc[1]);
            mma_f16(o[8 * w + 4 * q + 2 * e], p[0], p[1], p[2], p[3], b0, b1);
            b0 = hmul2(hfma2((x & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD480D480u), sc[0]);
            b1 = hmul2(hfma2((y & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD480D480u), sc[1]);
            mma_f16(o[8 * w + 4 * q + 2 * e + 1], p[0], p[1], p[2], p[3], b0, b1);
            x >>= 8, y >>= 8;
          }
        }
      }
    }
  }
}

__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l) - kPShift) * 0.6931471805599453f;
}

constexpr uint32_t kNaN = 0x7FFFFFFFu;

template <int D, int BITS, bool BF16>
__global__ void __launch_bounds__(kAttThreads, 2) attend_rows_kernel(const KvArgs a, const AttArgs t) {
  using P = RowsPlan<D, BITS>;
  constexpr int R = kv_row_bytes(D, BITS);
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring = smem_u32(smem) + warp * P::kRing;
  float* merge = reinterpret_cast<float*>(smem);  // warp w's part starts at its ring
  uint8_t* misc = smem + kAttWarps * P::kRing;
  const uint32_t qf = smem_u32(misc);
  uint32_t* qs = reinterpret_cast<uint32_t*>(misc);
  float* row_exp = reinterpret_cast<float*>(misc + P::kQBytes);  // [16] 2^e of the query scaling
  const uint32_t bars = smem_u32(misc + P::kQBytes + 64) + warp * P::kEntries * 8;
  __shared__ long long s_sum[kAttWarps];
  __shared__ long long s_base;
  __shared__ int s_b;
  __shared__ float2 s_stat[kAttWarps][kRows];

  if (lane < P::kEntries) mbar_init(bars + lane * 8, 1);
  fence_mbar_init();

  // the line of work: each thread sums its share of the sequences
  const int chunk = (a.n_seqs + kAttThreads - 1) / kAttThreads;
  const int b_lo = min(tid * chunk, a.n_seqs), b_hi = min(b_lo + chunk, a.n_seqs);
  long long mine = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const Seq s = seq_at(a, t.group, b);
    mine += (long long)s.row_tiles * a.heads * s.tiles;
    if (blockIdx.x == 0) flag_batch(a, b);
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_sum[warp] = incl;
  __syncthreads();
  long long total = 0, before = incl - mine;
#pragma unroll
  for (int w = 0; w < kAttWarps; ++w) {
    if (w < warp) before += s_sum[w];
    total += s_sum[w];
  }
  const long long part = max((total + gridDim.x - 1) / gridDim.x, (long long)kMinTiles);
  const long long w0 = (long long)blockIdx.x * part, w1 = min(w0 + part, total);
  if (blockIdx.x == 0 && tid == 0) t.starts[-1] = part;
  if (w0 < total && before <= w0 && w0 < before + mine) {
    s_base = before;
    s_b = b_lo;
  }
  __syncthreads();
  grid_launch_dependents();
  if (w0 >= total) return;

  int b = s_b;
  long long base = s_base, cur = w0;
  unsigned issued = 0, used = 0;  // halves over the life of the warp's ring
  bool timed_out = false;
  const int g = lane >> 2, tq = lane & 3;
  while (cur < w1) {
    const Seq sq = seq_at(a, t.group, b);
    const long long size = (long long)sq.row_tiles * a.heads * sq.tiles;
    const long long local = cur - base;
    if (local >= size) {
      base += size;
      ++b;
      continue;
    }
    const int seg = (int)(local / sq.tiles), t0 = (int)(local - (long long)seg * sq.tiles);
    const int head = seg / sq.row_tiles, rt = seg - head * sq.row_tiles;
    const int t1 = (int)min((long long)sq.tiles, t0 + (w1 - cur));
    const int rows = min(kRows, sq.n * t.group - rt * kRows);
    cur += t1 - t0;

    __syncthreads();  // the previous piece's merge has been read
    if (lane == 0) fence_async_shared();
    __syncwarp();
    // this warp's tiles t0 + warp, + 4, ...; lane j holds the page of the (first + j)-th
    const int nt = (t1 - t0 - warp + kAttWarps - 1) / kAttWarps;
    int first = 0, pages = -1;
    bool bad_page = false;
    auto load_pages = [&](int from) {
      first = from;
      const int i = from + lane;
      pages = 0;
      if (i < nt) {
        const int pi = kv_page_of(a, (t0 + warp + kAttWarps * i) * kKvTile);
        pages = pi < a.max_pages ? __ldg(a.table + (size_t)b * a.table_stride + pi) : -1;
        if ((unsigned)pages >= (unsigned)a.n_pages) {
          if (sq.len > 0) bad_page = true;  // an empty sequence's one tile holds nothing that is seen
          pages = 0;                        // in bounds; the rows become NaN
        }
      }
    };
    const uint8_t* head_data = a.data + (size_t)head * a.head_bytes;
    int sent = 0;  // halves of this piece issued
    auto issue = [&]() {
      const int i = sent >> 1;
      if (i >= nt) return;
      if (i >= first + 32) load_pages(i);
      const int page = __shfl_sync(0xffffffffu, pages, i - first);
      if (lane == 0) {
        const int pos = (t0 + warp + kAttWarps * i) * kKvTile;
        const int in_page = pos - kv_page_of(a, pos) * a.page_size;
        const uint8_t* src = head_data + (size_t)page * a.page_bytes + (size_t)(in_page / kKvTile) * (2 * P::kHalf) +
                             (sent & 1) * P::kHalf;
        const unsigned slot = issued % P::kEntries;
        mbar_expect_tx(bars + slot * 8, P::kHalf);
        bulk_g2s(ring + slot * P::kHalf, src, P::kHalf, bars + slot * 8);
      }
      ++issued;
      ++sent;
    };
    load_pages(0);
    for (int e = 0; e < P::kEntries; ++e) issue();

    // queries: 8 threads a row; the row's largest magnitude sets the power of two it is divided by
    {
      constexpr int NE = D / 8;
      const int row = tid >> 3, part8 = tid & 7;
      const int fr = rt * kRows + row, tok = fr / t.group, gh = fr - tok * t.group;
      const bool live = row < rows;
      const uint16_t* src = t.q + (int64_t)(sq.row0 + tok) * t.q_ts + (int64_t)(head * t.group + gh) * t.q_hs + part8 * NE;
      float f[NE];
      float big = 0.f;
#pragma unroll
      for (int i = 0; i < NE; i += 8) {
        const uint4 w = live ? *reinterpret_cast<const uint4*>(src + i) : make_uint4(0, 0, 0, 0);
        unpack2<BF16>(w.x, f[i], f[i + 1]);
        unpack2<BF16>(w.y, f[i + 2], f[i + 3]);
        unpack2<BF16>(w.z, f[i + 4], f[i + 5]);
        unpack2<BF16>(w.w, f[i + 6], f[i + 7]);
      }
#pragma unroll
      for (int i = 0; i < NE; ++i) big = fmaxf(big, fabsf(f[i]));
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
      // exponent of the largest: |f| * 2^-e stays below 2 (2^8 at the end of bf16's range); infinities and NaN stay what they are
      int e = ((__float_as_uint(big) >> 23) & 255) - 127;
      e = big > 0.f && e < 128 ? min(max(e, -120), 120) : 0;
      const float down = __uint_as_float((uint32_t)(127 - e) << 23);
      if (part8 == 0) row_exp[row] = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
      for (int i = 0; i < NE; i += 8) {
        const int d = part8 * NE + i, blk = d >> 5, tt = (d & 31) >> 3;
        uint32_t h[4];  // operand pairs of the block's two k16 steps
#pragma unroll
        for (int j = 0; j < 4; ++j)
          h[j] = BITS == 8 ? pack2<false>(f[i + 2 * j] * down, f[i + 2 * j + 1] * down)
                           : pack2<false>(f[i + j] * down, f[i + j + 4] * down);
        const int ln = (row & 7) * 4 + tt, hi = row >> 3;
#pragma unroll
        for (int j = 0; j < 4; ++j) qs[((2 * blk + (j >> 1)) * 32 + ln) * 4 + (j & 1) * 2 + hi] = h[j];
      }
    }
    __syncthreads();

    float o[D / 8][4], m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[j][i] = 0.f;
    // last position each of the lane's two rows sees; rows that are none see nothing
    const int f0 = rt * kRows + g, f1 = f0 + 8;
    const int see0 = g < rows ? sq.len - sq.n + f0 / t.group : -1;
    const int see1 = g + 8 < rows ? sq.len - sq.n + f1 / t.group : -1;
    const int see_min = sq.len - sq.n + (rt * kRows) / t.group;
    const int see_max = sq.len - sq.n + (rt * kRows + rows - 1) / t.group;
    const float c0 = t.scale_log2 * row_exp[g], c1 = t.scale_log2 * row_exp[g + 8];

    for (int i = 0; i < nt; ++i) {
      const int key0 = (t0 + warp + kAttWarps * i) * kKvTile;
      const bool edge = key0 + kKvTile - 1 > see_min;
      float s[4][4];
      {
        const unsigned slot = used % P::kEntries;
        if (!mbar_wait(bars + slot * 8, (used / P::kEntries) & 1)) timed_out = true;
        score_tile<D, BITS>(s, ring + slot * P::kHalf, qf, lane);
        ++used;
        __syncwarp();
        issue();
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        s[x][0] *= c0, s[x][1] *= c0, s[x][2] *= c1, s[x][3] *= c1;
      }
      if (edge) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int key = key0 + 8 * x + 2 * tq;
          if (key > see0) s[x][0] = -INFINITY;
          if (key + 1 > see0) s[x][1] = -INFINITY;
          if (key > see1) s[x][2] = -INFINITY;
          if (key + 1 > see1) s[x][3] = -INFINITY;
        }
      }
      float n0 = m0, n1 = m1;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        n0 = fmaxf(n0, fmaxf(s[x][0], s[x][1]));
        n1 = fmaxf(n1, fmaxf(s[x][2], s[x][3]));
      }
#pragma unroll
      for (int of = 1; of < 4; of <<= 1) {
        n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, of));
        n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, of));
      }
      if (__any_sync(0xffffffffu, n0 > m0 || n1 > m1)) {
        const float r0 = n0 > m0 ? ex2(m0 - n0) : 1.f, r1 = n1 > m1 ? ex2(m1 - n1) : 1.f;
        l0 *= r0, l1 *= r1;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          o[j][0] *= r0, o[j][1] *= r0, o[j][2] *= r1, o[j][3] *= r1;
        }
        m0 = n0, m1 = n1;
      }
      const float z0 = (m0 == -INFINITY ? 0.f : m0) - kPShift, z1 = (m1 == -INFINITY ? 0.f : m1) - kPShift;
      uint32_t p[2][4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float e0 = ex2(s[x][0] - z0), e1 = ex2(s[x][1] - z0), e2 = ex2(s[x][2] - z1), e3 = ex2(s[x][3] - z1);
        l0 += e0 + e1;
        l1 += e2 + e3;
        p[x >> 1][(x & 1) * 2] = pack2<false>(e0, e1);
        p[x >> 1][(x & 1) * 2 + 1] = pack2<false>(e2, e3);
      }
      {
        const unsigned slot = used % P::kEntries;
        if (!mbar_wait(bars + slot * 8, (used / P::kEntries) & 1)) timed_out = true;
        const uint32_t vb = ring + slot * P::kHalf;
        const int lim = see_max + 1 - key0;
        value_step<D, BITS>(o, p[0], vb, 0, lane, edge, lim);
        value_step<D, BITS>(o, p[1], vb, 1, lane, edge, lim);
        if (edge) {
          // value_step took non-finite scales for 0, so that rows that do not see such a key stay clean; the rows that do become NaN
          bool odd = false;
          for (int blk = 0; blk < D / 32; ++blk) {
            const uint32_t w = lds32(vb + kKvTile * R + (blk * kKvTile + (lane & ~1)) * 2);
            odd |= (((lane & 1) ? w >> 16 : w) & 0x7C00u) == 0x7C00u;
          }
          unsigned keys = __ballot_sync(0xffffffffu, odd && lane < lim);
          while (keys) {
            const int key = __ffs(keys) - 1;
            keys &= keys - 1;
            if (key0 + key <= see0) l0 = __uint_as_float(kNaN);
            if (key0 + key <= see1) l1 = __uint_as_float(kNaN);
          }
        }
        ++used;
        __syncwarp();
        issue();
      }
    }
#pragma unroll
    for (int of = 1; of < 4; of <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, of);
      l1 += __shfl_xor_sync(0xffffffffu, l1, of);
    }
    if (__any_sync(0xffffffffu, bad_page) || sq.over) {
      if (lane == 0) kv_flag(a, MOE_KV_BAD_PAGE);
      l0 = l1 = __uint_as_float(kNaN);
    }
    if (timed_out) {
      if (lane == 0) kv_flag(a, MOE_KV_TIMEOUT);
      l0 = l1 = __uint_as_float(kNaN);
    }

    // merge: the ring is drained (every half issued was used)
    float* mine_o = merge + warp * (P::kRing / 4);
    __syncwarp();
    if (nt > 0) {
#pragma unroll
      for (int j = 0; j < D / 8; j += 4) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int d = out_dim<D, BITS>(j, 2 * tq + (c & 1));
          *reinterpret_cast<float4*>(mine_o + (g + (c >> 1) * 8) * (D + 4) + d) =
              make_float4(o[j][c], o[j + 1][c], o[j + 2][c], o[j + 3][c]);
        }
      }
    }
    if (tq == 0) {
      s_stat[warp][g] = make_float2(m0, l0);
      s_stat[warp][g + 8] = make_float2(m1, l1);
    }
    __syncthreads();
    {
      constexpr int NE = D / 8;
      const int row = tid >> 3, part8 = tid & 7;
      float m = -INFINITY, l = 0.f, wgt[kAttWarps];
#pragma unroll
      for (int w = 0; w < kAttWarps; ++w) m = fmaxf(m, s_stat[w][row].x);
#pragma unroll
      for (int w = 0; w < kAttWarps; ++w) {
        const float2 st = s_stat[w][row];
        wgt[w] = st.x == -INFINITY ? 0.f : ex2(st.x - m);
        l += st.y != st.y ? st.y : st.y * wgt[w];
      }
      float acc[NE];
#pragma unroll
      for (int i = 0; i < NE; ++i) acc[i] = 0.f;
#pragma unroll
      for (int w = 0; w < kAttWarps; ++w) {
        if (w >= t1 - t0) break;  // that warp had no tile
        const float* src = merge + w * (P::kRing / 4) + row * (D + 4) + part8 * 4;
#pragma unroll
        for (int i = 0; i < NE; i += 4) {
          const float4 v = *reinterpret_cast<const float4*>(src + i * 8);
          acc[i] = fmaf(wgt[w], v.x, acc[i]);
          acc[i + 1] = fmaf(wgt[w], v.y, acc[i + 1]);
          acc[i + 2] = fmaf(wgt[w], v.z, acc[i + 2]);
          acc[i + 3] = fmaf(wgt[w], v.w, acc[i + 3]);
        }
      }
      if (row < rows) {
        if (t0 == 0 && t1 == sq.tiles) {
          const int fr = rt * kRows + row, tok = fr / t.group, gh = fr - tok * t.group;
          const float inv = l == 0.f ? 0.f : 1.f / l;
          uint16_t* dst = t.out + (int64_t)(sq.row0 + tok) * t.o_ts + (int64_t)(head * t.group + gh) * t.o_hs + part8 * 4;
#pragma unroll
          for (int i = 0; i < NE; i += 4)
            *reinterpret_cast<uint2*>(dst + i * 8) =
                make_uint2(pack2<BF16>(acc[i] * inv, acc[i + 1] * inv), pack2<BF16>(acc[i + 2] * inv, acc[i + 3] * inv));
          if (t.lse && part8 == 0) t.lse[(int64_t)(sq.row0 + tok) * t.nq + head * t.group + gh] = lse_of(m, l);
        } else {
          const size_t at = ((size_t)blockIdx.x * 2 + (t0 > 0 ? 0 : 1)) * kRows + row;
#pragma unroll
          for (int i = 0; i < NE; i += 4)
            *reinterpret_cast<float4*>(t.partial + at * D + part8 * 4 + i * 8) =
                make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
          if (part8 == 0) t.stats[at] = make_float2(m, l);
        }
      }
      if (t0 == 0 && tid == 0) t.starts[((int64_t)b * a.heads + head) * t.max_row_tiles + rt] = cur - (t1 - t0);
    }
  }
}

// Merges the partial results of the segments that several CTAs worked on:
// one CTA a row, its warps every fourth part.
template <int D, bool BF16>
__global__ void __launch_bounds__(kAttThreads) attend_join_kernel(const KvArgs a, const AttArgs t) {
  constexpr int NE = D / 32;  // elements a lane holds
  __shared__ float s_o[kAttWarps][D];
  __shared__ float2 s_stat[kAttWarps];
  grid_wait();
  const int seg = blockIdx.x, row = blockIdx.y;
  const int rt = seg % t.max_row_tiles, bh = seg / t.max_row_tiles, head = bh % a.heads, b = bh / a.heads;
  const Seq sq = seq_at(a, t.group, b);
  if (rt >= sq.row_tiles || rt * kRows + row >= sq.n * t.group) return;
  const long long part = t.starts[-1], start = t.starts[seg];
  const int c0 = (int)(start / part), c1 = (int)((start + sq.tiles - 1) / part);
  if (c0 == c1) return;  // one CTA had it all
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // a part that begins at the segment's first tile lies in its CTA's slot 1, the others in slot 0
  float m = -INFINITY, l = 0.f, o[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) o[i] = 0.f;
  for (int c = c0 + warp; c <= c1; c += kAttWarps) {
    const size_t at = ((size_t)c * 2 + (c == c0 ? 1 : 0)) * kRows + row;
    const float2 st = t.stats[at];
    const float n = fmaxf(m, st.x);
    const float wo = m == -INFINITY ? 0.f : ex2(m - n), wn = st.x == -INFINITY ? 0.f : ex2(st.x - n);
    l = (l != l ? l : l * wo) + (st.y != st.y ? st.y : st.y * wn);
    const float* src = t.partial + at * D + lane * NE;
#pragma unroll
    for (int i = 0; i < NE; ++i) o[i] = o[i] * wo + src[i] * wn;
    m = n;
  }
#pragma unroll
  for (int i = 0; i < NE; ++i) s_o[warp][lane * NE + i] = o[i];
  if (lane == 0) s_stat[warp] = make_float2(m, l);
  __syncthreads();
  float mm = -INFINITY, ll = 0.f;
#pragma unroll
  for (int w = 0; w < kAttWarps; ++w) mm = fmaxf(mm, s_stat[w].x);
  float wgt[kAttWarps];
#pragma unroll
  for (int w = 0; w < kAttWarps; ++w) {
    wgt[w] = s_stat[w].x == -INFINITY ? 0.f : ex2(s_stat[w].x - mm);
    ll += s_stat[w].y != s_stat[w].y ? s_stat[w].y : s_stat[w].y * wgt[w];
  }
  const float inv = ll == 0.f ? 0.f : 1.f / ll;
  const int fr = rt * kRows + row, tok = fr / t.group, gh = fr - tok * t.group;
  uint16_t* dst = t.out + (int64_t)(sq.row0 + tok) * t.o_ts + (int64_t)(head * t.group + gh) * t.o_hs;
  for (int d = 2 * tid; d < D; d += 2 * kAttThreads) {
    float v0 = 0.f, v1 = 0.f;
#pragma unroll
    for (int w = 0; w < kAttWarps; ++w) {
      v0 = fmaf(wgt[w], s_o[w][d], v0);
      v1 = fmaf(wgt[w], s_o[w][d + 1], v1);
    }
    *reinterpret_cast<uint32_t*>(dst + d) = pack2<BF16>(v0 * inv, v1 * inv);
  }
  if (t.lse && tid == 0) t.lse[(int64_t)(sq.row0 + tok) * t.nq + head * t.group + gh] = lse_of(mm, ll);
}

struct Workspace {
  size_t partial, stats, starts, bytes;
};

size_t up16(size_t v) { return (v + 15) & ~(size_t)15; }

Workspace plan_workspace(int parts, int dim, int64_t segments) {
  Workspace w{};
  w.partial = 0;
  w.stats = up16(w.partial + (size_t)parts * 2 * kRows * dim * 4);
  w.starts = up16(w.stats + (size_t)parts * 2 * kRows * 8);
  w.bytes = up16(w.starts + 16 + (size_t)segments * 8);
  return w;
}

template <typename K>
bool raise_smem(K kernel, int bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
}

template <int D, int BITS, bool BF16>
moe_status_t launch_rows_kernel(const KvArgs& kv, const AttArgs& t, int64_t segments, cudaStream_t st) {
  constexpr int smem = RowsPlan<D, BITS>::kSmem;
  if (!raise_smem(attend_rows_kernel<D, BITS, BF16>, smem)) return MOE_ERR_CUDA;
  attend_rows_kernel<D, BITS, BF16><<<t.parts, kAttThreads, smem, st>>>(kv, t);
  if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  const int64_t rows = (int64_t)kv.max_tokens * t.group;
  cfg.gridDim = dim3((unsigned)segments, (unsigned)(rows < kRows ? rows : kRows));
  cfg.blockDim = dim3(kAttThreads);
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attend_join_kernel<D, BF16>, kv, t) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <int D, int BITS>
moe_status_t launch_rows_type(const KvArgs& kv, const AttArgs& t, int64_t segments, bool bf16, cudaStream_t st) {
  return bf16 ? launch_rows_kernel<D, BITS, true>(kv, t, segments, st) : launch_rows_kernel<D, BITS, false>(kv, t, segments, st);
}

// What both entries derive from their arguments.
moe_status_t attend_plan(const moe_kv_cache_t* cache, const moe_kv_batch_t* batch, int32_t n_q, int32_t shared_tokens,
                         KvArgs* kv, int* parts, int* row_tiles, int64_t* segments, Workspace* ws) {
  moe_status_t st = kv_args(cache, batch, kv);
  if (st != MOE_OK) return st;
  if (n_q < 1 || n_q % cache->n_kv_heads || shared_tokens < 0 || shared_tokens % cache->page_size) return MOE_ERR_INVALID_ARG;
  if (shared_tokens / cache->page_size > batch->max_pages) return MOE_ERR_INVALID_ARG;
  const int64_t rows = (int64_t)batch->max_tokens * (n_q / cache->n_kv_heads);
  if (rows > 1 << 24) return MOE_ERR_UNSUPPORTED;
  *row_tiles = (int)((rows + kRows - 1) / kRows);
  *segments = (int64_t)batch->n_seqs * cache->n_kv_heads * *row_tiles;
  if (*segments > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  int sms = 0;
  st = device_sms(&sms);
  if (st != MOE_OK) return st;
  *parts = 2 * sms;
  *ws = plan_workspace(*parts, cache->head_dim, *segments);
  return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" MOE_API moe_status_t moe_kv_attend_workspace(const moe_kv_cache_t* cache, const moe_kv_batch_t* batch, int32_t n_q,
                                                        int32_t shared_tokens, size_t* bytes) {
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = 0;
  moe::KvArgs kv;
  moe::Workspace ws;
  int parts, row_tiles;
  int64_t segments;
  const moe_status_t st = moe::attend_plan(cache, batch, n_q, shared_tokens, &kv, &parts, &row_tiles, &segments, &ws);
  if (st == MOE_OK) *bytes = ws.bytes;
  return st;
}

extern "C" MOE_API moe_status_t moe_kv_attend(const moe_kv_cache_t* cache, const moe_kv_batch_t* batch, int32_t dtype,
                                              int32_t n_q, const moe_heads_t* q, const moe_heads_t* out, float* lse,
                                              float scale, int32_t shared_tokens, void* workspace, size_t workspace_bytes,
                                              void* cuda_stream) {
  if (dtype != MOE_BF16 && dtype != MOE_FP16) return dtype == MOE_FP32 ? MOE_ERR_UNSUPPORTED : MOE_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || ((uintptr_t)lse & 3)) return MOE_ERR_INVALID_ARG;
  moe::KvArgs kv;
  moe::Workspace ws;
  int parts, row_tiles;
  int64_t segments;
  const moe_status_t st = moe::attend_plan(cache, batch, n_q, shared_tokens, &kv, &parts, &row_tiles, &segments, &ws);
  if (st != MOE_OK) return st;
  if (kv.n_tokens == 0) return MOE_OK;
  const int dim = cache->head_dim;
  if (!moe::heads_ok(q, dim) || !moe::out_heads_ok(out, n_q, kv.n_tokens, dim)) return MOE_ERR_INVALID_ARG;
  if (!workspace || ((uintptr_t)workspace & 15)) return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < ws.bytes) return MOE_ERR_OUT_OF_MEMORY;
  uint8_t* w = (uint8_t*)workspace;
  moe::AttArgs t{};
  t.q = (const uint16_t*)q->data;
  t.q_ts = q->token_stride;
  t.q_hs = q->head_stride;
  t.out = (uint16_t*)out->data;
  t.o_ts = out->token_stride;
  t.o_hs = out->head_stride;
  t.lse = lse;
  t.scale_log2 = scale * 1.4426950408889634f;
  t.nq = n_q;
  t.group = n_q / cache->n_kv_heads;
  t.max_row_tiles = row_tiles;
  t.parts = parts;
  t.partial = (float*)(w + ws.partial);
  t.stats = (float2*)(w + ws.stats);
  t.starts = (int64_t*)(w + ws.starts + 16);
  const bool bf = dtype == MOE_BF16;
  const cudaStream_t s = (cudaStream_t)cuda_stream;
  if (cache->bits == 8) {
    if (dim == 64) return moe::launch_rows_type<64, 8>(kv, t, segments, bf, s);
    if (dim == 128) return moe::launch_rows_type<128, 8>(kv, t, segments, bf, s);
    return moe::launch_rows_type<256, 8>(kv, t, segments, bf, s);
  }
  if (dim == 64) return moe::launch_rows_type<64, 4>(kv, t, segments, bf, s);
  if (dim == 128) return moe::launch_rows_type<128, 4>(kv, t, segments, bf, s);
  return moe::launch_rows_type<256, 4>(kv, t, segments, bf, s);
}
