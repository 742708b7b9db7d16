// Attention with few rows a sequence (decode, speculation).  Rows are
// (new token, query head of the kv head's group), 8 * NT to a row tile.  A
// call is a line of work units, one for each 32-token tile of keys that a
// (sequence, kv head, row tile) segment has to see and kSegment for the
// segment itself; the line is cut into equal parts, one a CTA, whatever the
// lengths are.  A CTA's four warps take every fourth tile of a segment, each
// with a ring of its own that one lane fills by bulk copies (half a tile, its
// K or its V with the scales, is contiguous in the pool), and keep a running
// maximum, sum and output in registers (one pass over the keys).  The warps'
// results are merged in shared memory; a segment that ends in another CTA
// leaves a partial result.
//
// The products run on mma.sync m16n8k16 with keys (or output elements) as M
// and rows as N, so that a group of 8 query heads fills the tile: with rows
// as M half of it was padding.  Warp instructions bound the 4-bit case: 64
// sequences of 8,192 tokens take 80 us (45 of memory time), in 8 bits 103 (84).  S^T = K Q^T has its
// probabilities transposed in registers (movmatrix) into the operand of
// O^T = V^T P^T.
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
#pragma once

#include "moe_attend.cuh"

namespace moe {
namespace {

using namespace ptx;

constexpr int kAttWarps = 4;
constexpr int kAttThreads = 32 * kAttWarps;
// Units of work that a segment costs beside its tiles: its queries, its first
// copy's latency, its merge.  Measured on 64 sequences of 1 to 24,001 tokens:
// 73 us with 2, 54 with 4, 42 with 8 and 16; equal lengths do not notice.
constexpr int kSegment = 12;
constexpr int kMinUnits = 8;  // units a CTA takes at least

// Element j of lane group c's (0..7) share of the output: a contiguous run of
// a key's bytes, or two for 8-bit heads of 256.
template <int D, int BITS>
__device__ __forceinline__ int out_dim(int j, int c) {
  if (BITS == 8 && D == 256) return (j >> 4) * 128 + 16 * c + (j & 15);
  return (D / 8) * c + j;
}

// Shared memory of attend_rows_kernel.  Three CTAs an SM where registers
// (the output is D / 4 * NT of them) and the rings allow it, else two.
template <int D, int BITS, int NT>
struct RowsPlan {
  static constexpr int kHalf = kv_half_bytes(D, BITS);
  static constexpr int kBlocks = NT == 4 || D * NT >= 512 || (D == 256 && BITS == 8) ? 2 : 3;
  static constexpr int kRingBytes = kBlocks == 2 ? 26112 : D == 256 ? 13824 : 17408;
  static constexpr int kEntries = (kRingBytes / kHalf) < 12 ? (kRingBytes / kHalf) : 12;
  static constexpr int kRing = kEntries * kHalf;          // bytes a warp
  static constexpr int kRows = 8 * NT;
  static constexpr int kQBytes = kRows * D * 2;           // query fragments
  static constexpr int kMerge = kRows * (D + 4) * 4;      // a warp's output for the merge, inside its ring
  static constexpr int kSmem = kAttWarps * kRing + kQBytes + kRows * 4 + kAttWarps * kEntries * 8;
  static_assert(kMerge <= kRing, "the merge buffer lies in the ring");
  static_assert(kEntries >= 3, "a ring of three halves at least");
};

// Eight stored integers of a key as the fp16 operand pairs of two k16 steps.
// magic: 0x6400 in both halves, the fp16 exponent at which a mantissa step is 1.
template <int BITS>
__device__ __forceinline__ void key_operands(uint32_t (&k)[4], uint32_t at, uint32_t magic) {
  if (BITS == 8) {
    const uint2 w = lds64(at);
    k[0] = hsub2(prmt(w.x, magic, 0x5150), 0x64806480u);
    k[1] = hsub2(prmt(w.x, magic, 0x5352), 0x64806480u);
    k[2] = hsub2(prmt(w.y, magic, 0x5150), 0x64806480u);
    k[3] = hsub2(prmt(w.y, magic, 0x5352), 0x64806480u);
  } else {
    const uint32_t w = lds32(at), w8 = w >> 8;
    k[0] = hsub2(and_or<0x000F000Fu>(w, magic), 0x64086408u);
    k[1] = hfma2(and_or<0x00F000F0u>(w, magic), 0x2C002C00u, 0xD480D480u);
    k[2] = hsub2(and_or<0x000F000Fu>(w8, magic), 0x64086408u);
    k[3] = hfma2(and_or<0x00F000F0u>(w8, magic), 0x2C002C00u, 0xD480D480u);
  }
}

// One warp's products of a 32-key tile: s[i][n] holds keys 16 i + g and
// 16 i + 8 + g (g = lane / 4) against rows 8 n + 2 t and + 1 (t = lane % 4).
template <int D, int BITS, int NT>
__device__ __forceinline__ void score_tile(float (&s)[2][NT][4], uint32_t kb, uint32_t qf, int lane, uint32_t magic) {
  constexpr int R = kv_row_bytes(D, BITS), NC = R / 16;
  const int g = lane >> 2, t = lane & 3, turn = kv_turn(g) & (NC - 1);
#pragma unroll
  for (int b = 0; b < D / 32; ++b) {
    uint4 q[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) q[n] = lds128(qf + ((b * NT + n) * 32 + lane) * 16);
    const int at = BITS == 8 ? (((2 * b + (t >> 1)) ^ turn) << 4) + (t & 1) * 8 : ((b ^ turn) << 4) + t * 4;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t k0[4], k1[4];
      key_operands<BITS>(k0, kb + (16 * i + g) * R + at, magic);
      key_operands<BITS>(k1, kb + (16 * i + 8 + g) * R + at, magic);
      const uint32_t sc = kb + kKvTile * R + (b * kKvTile + 16 * i + g) * 2;
      const float d0 = __half2float(__ushort_as_half((uint16_t)lds16(sc)));
      const float d1 = __half2float(__ushort_as_half((uint16_t)lds16(sc + 16)));
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float p[4];
        mma_f16_zero(p, k0[0], k1[0], k0[1], k1[1], q[n].x, q[n].y);
        mma_f16(p, k0[2], k1[2], k0[3], k1[3], q[n].z, q[n].w);
        s[i][n][0] = b ? fmaf(p[0], d0, s[i][n][0]) : p[0] * d0;
        s[i][n][1] = b ? fmaf(p[1], d0, s[i][n][1]) : p[1] * d0;
        s[i][n][2] = b ? fmaf(p[2], d1, s[i][n][2]) : p[2] * d1;
        s[i][n][3] = b ? fmaf(p[3], d1, s[i][n][3]) : p[3] * d1;
      }
    }
  }
}

// An m-tile of integers times scales, and with REST what rounding that to fp16
// left (exact in fp16 too), against the probabilities.
template <int NT, bool REST>
__device__ __forceinline__ void value_product(float (&o)[NT][4], const uint32_t (&w)[4], const uint32_t (&sc)[2], const uint32_t (&p)[NT][2]) {
  uint32_t a[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) a[j] = hmul2(w[j], sc[j >> 1]);
#pragma unroll
  for (int n = 0; n < NT; ++n) mma_f16(o[n], a[0], a[1], a[2], a[3], p[n][0], p[n][1]);
  if (REST) {
#pragma unroll
    for (int j = 0; j < 4; ++j) a[j] = hfma2(w[j], sc[j >> 1], a[j] ^ 0x80008000u);
#pragma unroll
    for (int n = 0; n < NT; ++n) mma_f16(o[n], a[0], a[1], a[2], a[3], p[n][0], p[n][1]);
  }
}

// o += p v for 16 keys (step u of a tile).  edge: keys from lim on (within
// the tile) are seen by no row and count as 0 whatever their bytes say, and so
// do non-finite scales (the caller deals with the rows that see them).  REST: what
// their rounding to fp16 left of integer times scale is a second operand.
template <int D, int BITS, int NT, bool REST>
__device__ __forceinline__ void value_step(float (&o)[D / 16][NT][4], const uint32_t (&p)[NT][2], uint32_t vb, int u, int lane,
                                           bool edge, int lim, uint32_t magic) {
  constexpr int R = kv_row_bytes(D, BITS), NC = R / 16, RUN = D / 8;
  constexpr int kRuns = (BITS == 8 && D == 256) ? 2 : 1;  // runs of RUN / kRuns elements a lane group has
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
      // m-tiles of two elements each: a[0], a[1] keys 2t, 2t + 1 of the first and second; a[2], a[3] keys 2t + 8, 2t + 9
      if (BITS == 8) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t x = prmt(v[0][w], v[1][w], h ? 0x7362 : 0x5140), y = prmt(v[2][w], v[3][w], h ? 0x7362 : 0x5140);
          const uint32_t w4[4] = {hsub2(prmt(x, magic, 0x5150), 0x64806480u), hsub2(prmt(x, magic, 0x5352), 0x64806480u),
                                  hsub2(prmt(y, magic, 0x5150), 0x64806480u), hsub2(prmt(y, magic, 0x5352), 0x64806480u)};
          value_product<NT, REST>(o[r * 8 + 2 * w + h], w4, sc, p);
        }
      } else {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t x = prmt(v[0][w], v[1][w], q ? 0x7632 : 0x5410), y = prmt(v[2][w], v[3][w], q ? 0x7632 : 0x5410);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t w4[4] = {
                hsub2(and_or<0x000F000Fu>(x, magic), 0x64086408u), hfma2(and_or<0x00F000F0u>(x, magic), 0x2C002C00u, 0xD480D480u),
                hsub2(and_or<0x000F000Fu>(y, magic), 0x64086408u), hfma2(and_or<0x00F000F0u>(y, magic), 0x2C002C00u, 0xD480D480u)};
            value_product<NT, REST>(o[4 * w + 2 * q + h], w4, sc, p);
            x >>= 8, y >>= 8;
          }
        }
      }
    }
  }
}

// 32-token tiles of keys that a sequence's segments have (behind a shared prefix there may be none), and its row tiles.
__device__ __forceinline__ int key_tiles(const KvArgs& a, const AttArgs& t, const Seq& s) {
  const int keys = min(s.len, a.max_pages * a.page_size) - t.shared;
  return max(t.shared ? 0 : 1, (keys + kKvTile - 1) / kKvTile);
}
template <int ROWS>
__device__ __forceinline__ int row_tiles(const AttArgs& t, const Seq& s) {
  return (s.n * t.group + ROWS - 1) / ROWS;
}

template <int D, int BITS, bool BF16, int NT>
__global__ void __launch_bounds__(kAttThreads, (RowsPlan<D, BITS, NT>::kBlocks)) attend_rows_kernel(const KvArgs a, const AttArgs t) {
  using P = RowsPlan<D, BITS, NT>;
  constexpr int R = kv_row_bytes(D, BITS), kRows = P::kRows;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring = smem_u32(smem) + warp * P::kRing;
  float* merge = reinterpret_cast<float*>(smem);  // warp w's part starts at its ring
  uint8_t* misc = smem + kAttWarps * P::kRing;
  const uint32_t qf = smem_u32(misc);
  uint4* qs = reinterpret_cast<uint4*>(misc);
  float* row_factor = reinterpret_cast<float*>(misc + P::kQBytes);  // [kRows] score_factor
  const uint32_t bars = smem_u32(misc + P::kQBytes + kRows * 4) + warp * P::kEntries * 8;
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
    const Seq s = seq_at(a, b);
    mine += (long long)row_tiles<kRows>(t, s) * a.heads * (key_tiles(a, t, s) + kSegment);
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
  const long long part = max((total + gridDim.x - 1) / gridDim.x, (long long)kMinUnits);
  const long long w0 = (long long)blockIdx.x * part, w1 = min(w0 + part, total);
  if (tid == 0) t.ends[blockIdx.x].first = -1;
  if (w0 < total && before <= w0 && w0 < before + mine) {
    s_base = before;
    s_b = b_lo;
  }
  __syncthreads();
  grid_launch_dependents();
  if (w0 >= total) {
    if (t.shared) grid_wait();
    return;
  }

  int b = s_b;
  long long base = s_base, cur = w0;
  int in_slot = 0, out_slot = 0;  // the ring's next entry to fill and to use
  uint32_t phase = 0;             // of the entry to use
  bool in_time = true;
  // the exponent of the dequantisation in a register the compiler cannot see through: with two constants an
  // and-or would take two instructions
  uint32_t magic = 0x64006400u;
  asm volatile("" : "+r"(magic));
  const int g = lane >> 2, tq = lane & 3;
  while (cur < w1) {
    const Seq sq = seq_at(a, b);
    const int tiles = key_tiles(a, t, sq), n_rt = row_tiles<kRows>(t, sq), units = tiles + kSegment;
    const long long size = (long long)n_rt * a.heads * units;
    const long long local = cur - base;
    if (local >= size) {
      base += size;
      ++b;
      continue;
    }
    const int seg = (int)(local / units), u0 = (int)(local - (long long)seg * units);
    const int u1 = (int)min((long long)units, u0 + (w1 - cur));
    const int t0 = max(u0 - kSegment, 0), t1 = max(u1 - kSegment, 0);
    cur += u1 - u0;
    if (t1 <= t0) continue;  // the part ends before the segment's first tile
    const int head = seg / n_rt, rt = seg - head * n_rt;
    const int rows = min(kRows, sq.n * t.group - rt * kRows);

    __syncthreads();  // the previous piece's merge has been read
    fence_async_shared();
    // this warp's tiles t0 + warp, + 4, ...; lane j holds the address of the (first + j)-th, and issues its copies
    const int nt = (t1 - t0 - warp + kAttWarps - 1) / kAttWarps;
    int first = 0;
    const uint8_t* mine_src = nullptr;
    int bad = INT32_MAX;  // the first position on a bad page that the lane looked up
    auto load_pages = [&](int from) {
      first = from;
      const int i = from + lane;
      if (i < nt) {
        const int pos = t.shared + (t0 + warp + kAttWarps * i) * kKvTile, pi = kv_page_of(a, pos);
        int page = pi < a.max_pages ? __ldg(a.table + (size_t)b * a.table_stride + pi) : -1;
        if ((unsigned)page >= (unsigned)a.n_pages) {
          if (sq.len > 0) bad = min(bad, pos);  // an empty sequence's one tile holds nothing that is seen
          page = 0;                             // in bounds; the rows that see it become NaN
        }
        mine_src = a.data + (size_t)page * a.page_bytes + (size_t)head * a.head_bytes +
                   (size_t)((pos - pi * a.page_size) / kKvTile) * (2 * P::kHalf);
      }
    };
    int sent = 0;  // halves of this piece issued
    auto issue = [&]() {
      if (sent >= 2 * nt) return;
      const int i = sent >> 1;
      if (i >= first + 32) load_pages(i);
      if (lane == i - first && in_time) {  // (an entry whose copy did not come is not filled again)
        mbar_expect_tx(bars + in_slot * 8, P::kHalf);
        bulk_g2s(ring + in_slot * P::kHalf, mine_src + (sent & 1) * P::kHalf, P::kHalf, bars + in_slot * 8);
      }
      in_slot = in_slot + 1 == P::kEntries ? 0 : in_slot + 1;
      ++sent;
    };
    // Gives the slot just read back to the producer and moves on.
    auto release = [&]() {
      if (++out_slot == P::kEntries) out_slot = 0, phase ^= 1;
      __syncwarp();
      issue();
    };
    load_pages(0);
    for (int e = 0; e < P::kEntries; ++e) issue();

    // Queries: D / 8 threads a row, 8 elements each, in the order of the
    // operand pairs.
    {
      constexpr int TPR = D / 8;
#pragma unroll
      for (int r0 = 0; r0 < kRows; r0 += kAttThreads / TPR) {
        const int row = r0 + tid / TPR, d8 = tid % TPR;
        const int fr = rt * kRows + row, tok = fr / t.group, gh = fr - tok * t.group;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (row < rows)
          w = *reinterpret_cast<const uint4*>(t.q + (int64_t)(sq.row0 + tok) * t.q_ts + (int64_t)(head * t.group + gh) * t.q_hs + d8 * 8);
        float f[8];
        unpack2<BF16>(w.x, f[0], f[1]);
        unpack2<BF16>(w.y, f[2], f[3]);
        unpack2<BF16>(w.z, f[4], f[5]);
        unpack2<BF16>(w.w, f[6], f[7]);
        float big = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) big = fmaxf(big, fabsf(f[i]));
#pragma unroll
        for (int o = 1; o < TPR; o <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
        const int e = row_exponent(big);
        const float down = query_factor(t.scale_log2, e);
        if (row < kRows) {
          if (d8 == 0) row_factor[row] = score_factor(t.scale_log2, e);
          uint32_t h[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            h[j] = BITS == 8 ? pack2<false>(f[2 * j] * down, f[2 * j + 1] * down) : pack2<false>(f[j] * down, f[j + 4] * down);
          qs[((d8 >> 2) * NT + (row >> 3)) * 32 + (row & 7) * 4 + (d8 & 3)] = make_uint4(h[0], h[1], h[2], h[3]);
        }
      }
    }
    __syncthreads();

    float o[D / 16][NT][4], m[NT][2], l[NT][2], c[NT][2];
    int see[NT][2];  // last position that the lane's rows see; rows that are none see nothing
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = 8 * n + 2 * tq + h;
        m[n][h] = -INFINITY;
        l[n][h] = 0.f;
        c[n][h] = row_factor[row];
        see[n][h] = row < rows ? sq.len - sq.n + (rt * kRows + row) / t.group : -1;
      }
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][n][i] = 0.f;
    const int see_min = sq.len - sq.n + (rt * kRows) / t.group;
    const int see_max = sq.len - sq.n + (rt * kRows + rows - 1) / t.group;

    for (int i = 0; i < nt; ++i) {
      const int key0 = t.shared + (t0 + warp + kAttWarps * i) * kKvTile;
      const bool edge = key0 + kKvTile - 1 > see_min;
      float s[2][NT][4];
      {
        mbar_wait(bars + out_slot * 8, phase, in_time);
        score_tile<D, BITS, NT>(s, ring + out_slot * P::kHalf, qf, lane, magic);
        release();
      }
      if (edge) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const int key = key0 + 16 * x + g;
            if (key > see[n][0]) s[x][n][0] = -INFINITY;
            if (key > see[n][1]) s[x][n][1] = -INFINITY;
            if (key + 8 > see[n][0]) s[x][n][2] = -INFINITY;
            if (key + 8 > see[n][1]) s[x][n][3] = -INFINITY;
          }
      }
      // maxima in units of log2 (c > 0, so the largest product has the largest score)
      float top[NT][2];
      bool grew = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float v = fmaxf(fmaxf(s[0][n][h], s[0][n][h + 2]), fmaxf(s[1][n][h], s[1][n][h + 2]));
#pragma unroll
          for (int of = 4; of < 32; of <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, of));
          top[n][h] = v * c[n][h];
          grew |= top[n][h] > m[n][h];
        }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float r[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const bool up = top[n][h] > m[n][h];
            r[h] = up ? ex2(m[n][h] - top[n][h]) : 1.f;
            if (up) m[n][h] = top[n][h];
            l[n][h] *= r[h];
          }
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            o[j][n][0] *= r[0], o[j][n][1] *= r[1], o[j][n][2] *= r[0], o[j][n][3] *= r[1];
          }
        }
      }
      uint32_t p[2][NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float z0 = kPShift - (m[n][0] == -INFINITY ? 0.f : m[n][0]), z1 = kPShift - (m[n][1] == -INFINITY ? 0.f : m[n][1]);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float e[4];
#pragma unroll
          for (int h = 0; h < 4; ++h) e[h] = ex2(fmaf(s[x][n][h], c[n][h & 1], h & 1 ? z1 : z0));
          l[n][0] += e[0] + e[2];
          l[n][1] += e[1] + e[3];
          p[x][n][0] = transpose8(pack2<false>(e[0], e[1]));
          p[x][n][1] = transpose8(pack2<false>(e[2], e[3]));
        }
      }
      {
        mbar_wait(bars + out_slot * 8, phase, in_time);
        const uint32_t vb = ring + out_slot * P::kHalf;
        const int lim = see_max + 1 - key0;
        value_step<D, BITS, NT, !BF16>(o, p[0], vb, 0, lane, edge, lim, magic);
        value_step<D, BITS, NT, !BF16>(o, p[1], vb, 1, lane, edge, lim, magic);
        if (edge) {
          // value_step took non-finite scales for 0, so that rows that do not see such a key stay clean; the rows that do become NaN
          bool odd = false;
          for (int blk = 0; blk < D / 32; ++blk) odd |= (lds16(vb + kKvTile * R + (blk * kKvTile + lane) * 2) & 0x7C00u) == 0x7C00u;
          unsigned keys = __ballot_sync(0xffffffffu, odd && lane < lim);
          while (keys) {
            const int key = key0 + __ffs(keys) - 1;
            keys &= keys - 1;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                if (key <= see[n][h]) l[n][h] = __uint_as_float(kNaN);
          }
        }
        release();
      }
    }
    bad = __reduce_min_sync(0xffffffffu, bad);
    if (bad != INT32_MAX && lane == 0) kv_flag(a, MOE_KV_BAD_PAGE);
    if (sq.over) bad = min(bad, a.max_pages * a.page_size);  // (flagged with the batch)
    in_time = __all_sync(0xffffffffu, in_time);
    if (!in_time) {
      if (lane == 0) kv_flag(a, MOE_KV_TIMEOUT);
      bad = INT32_MIN;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int of = 4; of < 32; of <<= 1) l[n][h] += __shfl_xor_sync(0xffffffffu, l[n][h], of);
        if (see[n][h] >= bad) l[n][h] = __uint_as_float(kNaN);
        if (g == 0) s_stat[warp][8 * n + 2 * tq + h] = make_float2(m[n][h], l[n][h]);
      }

    // merge: the ring is drained (every half issued was used, unless a wait ran out)
    float* mine_o = merge + warp * (P::kRing / 4);
    __syncwarp();
    if (nt > 0) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < D / 16; j += 2)
            *reinterpret_cast<float4*>(mine_o + (8 * n + 2 * tq + h) * (D + 4) + out_dim<D, BITS>(2 * j, g)) =
                make_float4(o[j][n][h], o[j][n][h + 2], o[j + 1][n][h], o[j + 1][n][h + 2]);
    }
    __syncthreads();
    {
      constexpr int TPR = kAttThreads / kRows, NE = D / TPR;  // threads a row, elements a thread
      const int row = tid / TPR, sub = tid % TPR;
      float mm = -INFINITY, ll = 0.f, wgt[kAttWarps];
#pragma unroll
      for (int w = 0; w < kAttWarps; ++w) mm = fmaxf(mm, s_stat[w][row].x);
#pragma unroll
      for (int w = 0; w < kAttWarps; ++w) {
        const float2 st = s_stat[w][row];
        wgt[w] = st.x == -INFINITY ? 0.f : ex2(st.x - mm);
        ll += st.y != st.y ? st.y : st.y * wgt[w];
      }
      const bool whole = t0 == 0 && t1 == tiles;
      const int64_t segment = ((int64_t)b * a.heads + head) * t.max_row_tiles + rt;  // (with a shared prefix)
      const int fr = rt * kRows + row, tok = fr / t.group, gh = fr - tok * t.group;
      const float inv = ll == 0.f ? 0.f : 1.f / ll;
      const bool finish = whole && !t.shared;
      const size_t at = whole ? (size_t)segment * kRows + row : ((size_t)blockIdx.x * 2 + (t0 > 0 ? 0 : 1)) * kRows + row;
      float* partial = whole ? t.whole : t.partial;
      if (row < rows) {
#pragma unroll
        for (int i = 0; i < NE; i += 4) {
          const int d = sub * 4 + i * TPR;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < kAttWarps; ++w) {
            if (w >= t1 - t0) break;  // that warp had no tile
            const float4 v = *reinterpret_cast<const float4*>(merge + w * (P::kRing / 4) + row * (D + 4) + d);
            acc.x = fmaf(wgt[w], v.x, acc.x);
            acc.y = fmaf(wgt[w], v.y, acc.y);
            acc.z = fmaf(wgt[w], v.z, acc.z);
            acc.w = fmaf(wgt[w], v.w, acc.w);
          }
          if (finish)
            *reinterpret_cast<uint2*>(t.out + (int64_t)(sq.row0 + tok) * t.o_ts + (int64_t)(head * t.group + gh) * t.o_hs + d) =
                make_uint2(pack2<BF16>(acc.x * inv, acc.y * inv), pack2<BF16>(acc.z * inv, acc.w * inv));
          else
            *reinterpret_cast<float4*>(partial + at * D + d) = acc;
        }
        if (sub == 0) {
          if (!finish)
            (whole ? t.whole_stats : t.stats)[at] = make_float2(mm, ll);
          else if (t.lse)
            t.lse[(int64_t)(sq.row0 + tok) * t.nq + head * t.group + gh] = lse_of(mm, ll);
        }
      }
      if (t1 == tiles && tid == 0) {
        const int first_part = (int)((cur - u1 + kSegment) / part);  // (cur - u1: the segment's place on the line)
        if (t.shared)
          t.spans[segment] = Span{whole ? kWhole : first_part, (int)blockIdx.x};
        else if (!whole)
          t.ends[blockIdx.x] = SegmentEnd{first_part, b, head, rt};
      }
    }
  }
  if (!in_time) settle();
  if (t.shared) grid_wait();  // the merge waits for this kernel, and through it for the prefix's pass
}

template <int D, int BITS, bool BF16, int NT>
moe_status_t launch_rows_kernel(const KvArgs& kv, const AttArgs& t, cudaStream_t st) {
  constexpr int smem = RowsPlan<D, BITS, NT>::kSmem;
  const moe_status_t ok = raise_smem<attend_rows_kernel<D, BITS, BF16, NT>>(smem);
  if (ok != MOE_OK) return ok;
  if (!t.shared) {
    attend_rows_kernel<D, BITS, BF16, NT><<<t.parts, kAttThreads, smem, st>>>(kv, t);
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  }
  // beside the prefix's pass, which it does not read, as SMs become free
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)t.parts);
  cfg.blockDim = dim3(kAttThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attend_rows_kernel<D, BITS, BF16, NT>, kv, t) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <int D, int BITS, bool BF16>
moe_status_t launch_rows_tile(const KvArgs& kv, const AttArgs& t, cudaStream_t st) {
  if (t.tile_rows == 8) return launch_rows_kernel<D, BITS, BF16, 1>(kv, t, st);
  if constexpr (D < 256)
    if (t.tile_rows == 32) return launch_rows_kernel<D, BITS, BF16, 4>(kv, t, st);
  return launch_rows_kernel<D, BITS, BF16, 2>(kv, t, st);
}

template <int BITS>
moe_status_t launch_rows(const KvArgs& kv, const AttArgs& t, int dim, bool bf16, cudaStream_t st) {
  if (dim == 64) return bf16 ? launch_rows_tile<64, BITS, true>(kv, t, st) : launch_rows_tile<64, BITS, false>(kv, t, st);
  if (dim == 128) return bf16 ? launch_rows_tile<128, BITS, true>(kv, t, st) : launch_rows_tile<128, BITS, false>(kv, t, st);
  return bf16 ? launch_rows_tile<256, BITS, true>(kv, t, st) : launch_rows_tile<256, BITS, false>(kv, t, st);
}

}  // namespace
}  // namespace moe
