// Per-head norm + rotation, and the quantised paged cache written and read.
//
// One kernel (head_rows_kernel) serves the norm + rotation, the append and
// both in one pass; they differ in which rows of heads it is given and in
// where a finished row goes.  All of it is bound by memory traffic (or, for a
// few tokens, by latency): D/8 lanes hold a head's row, 8 elements (one
// 16-byte load) each, so the mean square is a butterfly over those lanes, a
// rotation partner is one shuffle away and a scale block of 32 is 4 lanes.
#include <cmath>
#include <utility>

#include "moe_kv.cuh"

namespace moe {

constexpr int kMaxTokens = INT32_MAX - 256;  // a block's tokens more still fit an int

moe_status_t kv_args(const moe_kv_cache_t* c, const moe_kv_batch_t* b, KvArgs* out) {
  if (!c || !b || !c->data || !c->status || !b->block_table || !b->seq_lens || !b->cu_tokens) return MOE_ERR_INVALID_ARG;
  if (((uintptr_t)c->data & 15) || ((uintptr_t)c->status & 3) || ((uintptr_t)b->block_table & 3) ||
      ((uintptr_t)b->seq_lens & 3) || ((uintptr_t)b->cu_tokens & 3))
    return MOE_ERR_INVALID_ARG;
  const size_t page = moe_kv_page_bytes(c->page_size, c->n_kv_heads, c->head_dim, c->bits);
  if (!page || c->n_pages < 1 || c->data_bytes / page < (size_t)c->n_pages) return MOE_ERR_INVALID_ARG;
  if (b->n_seqs < 1 || b->n_seqs > 65536 || b->max_pages < 1 || b->table_stride < b->max_pages || b->n_tokens < 0 ||
      b->n_tokens > kMaxTokens)
    return MOE_ERR_INVALID_ARG;
  if ((int64_t)b->max_pages * c->page_size > INT32_MAX) return MOE_ERR_INVALID_ARG;
  if (b->n_tokens > 0 && (b->max_tokens < 1 || b->max_tokens > b->n_tokens)) return MOE_ERR_INVALID_ARG;
  int shift = -1;
  for (int s = 5; s <= 12; ++s)
    if (c->page_size == 1 << s) shift = s;
  *out = KvArgs{(uint8_t*)c->data, c->status,     b->block_table, b->seq_lens,     b->cu_tokens, c->n_pages,
                c->page_size,      shift,         c->n_kv_heads,  b->table_stride, b->max_pages, b->n_seqs,
                b->n_tokens,       b->max_tokens, page,           page / c->n_kv_heads};
  return MOE_OK;
}

bool heads_ok(const moe_heads_t* h, int dim) {
  return h && h->data && !((uintptr_t)h->data & 15) && h->token_stride >= 0 && h->head_stride >= 0 &&
         h->token_stride % 8 == 0 && h->head_stride % 8 == 0 && (h->token_stride == 0 || h->token_stride >= dim) &&
         (h->head_stride == 0 || h->head_stride >= dim);
}

// No two of n_tokens x n_heads rows of dim elements share one.
static bool rows_apart(int64_t n_tokens, int64_t n_heads, int64_t ts, int64_t hs, int64_t dim) {
  if (n_tokens < 2 && n_heads < 2) return true;
  if (n_heads < 2) return ts >= dim;
  if (n_tokens < 2) return hs >= dim;
  if (ts < hs) std::swap(ts, hs), std::swap(n_tokens, n_heads);
  using wide = __int128;
  if (hs < dim) return false;
  if ((wide)(n_heads - 1) * hs + dim <= ts) return true;  // the usual ones
  // the smaller steps end up among later rows of the larger: the distance of each to the two nearest of those
  for (int64_t j = 1; j < n_heads; ++j) {
    const wide at = (wide)j * hs;
    const int64_t i = (int64_t)(at / ts);
    if ((i > 0 && i < n_tokens && at - (wide)i * ts < dim) || (i + 1 < n_tokens && (wide)(i + 1) * ts - at < dim)) return false;
    if (i >= n_tokens) break;  // behind all of them
  }
  return true;
}

bool out_heads_ok(const moe_heads_t* h, int n_heads, int n_tokens, int dim) {
  return heads_ok(h, dim) && rows_apart(n_tokens, n_heads, h->token_stride, h->head_stride, dim);
}

moe_status_t device_sms(int* sms) {
  static int known[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return MOE_ERR_CUDA;
  int n = __atomic_load_n(&known[dev], __ATOMIC_RELAXED);
  if (!n) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return MOE_ERR_CUDA;
    __atomic_store_n(&known[dev], n, __ATOMIC_RELAXED);
  }
  *sms = n;
  return MOE_OK;
}

namespace {

constexpr int kRowThreads = 256;
constexpr int kRowsPerUnit = 4;  // heads of one token that a group of lanes takes when there are many rows

struct HeadSrc {
  const uint16_t* p;
  int64_t ts, hs;
};
struct HeadDst {
  uint16_t* p;
  int64_t ts, hs;
};

struct RowArgs {
  HeadSrc q, k, v;
  HeadDst qo, ko;
  const uint16_t *wq, *wk;
  const float* table;
  const int32_t* positions;
  int n_positions, rot, inter;
  float eps, woff, inv_dim;
  int n_tokens, nq, nk, dim;
  int per, q_slots, k_slots;  // heads a unit takes; units of a token for q, and for k (and for v)
};

// Two fp32 operations an instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{.reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mul.rn.f32x2 z, x, y; mov.b64 {%0, %1}, z;}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{.reg .b64 x, y, z, w; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mov.b64 z, {%6, %7}; fma.rn.f32x2 w, x, y, z; mov.b64 {%0, %1}, w;}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
template <bool BF16>
__device__ __forceinline__ float2 pair_of(uint32_t w) {
  float2 r;
  unpack2<BF16>(w, r.x, r.y);
  return r;
}

// One element's integer from its quotient by d, and its half-even tie from the exact rest.
__device__ __forceinline__ uint32_t quantise_slowly(float x, float d, float inv, float low, float top) {
  float q = rintf(x * inv);
  const float rest = fmaf(-q, d, x);
  if (fabsf(rest) * 2.f == d && q != 2.f * rintf(0.5f * q)) q += copysignf(1.f, rest);
  q = d > 0.f ? fminf(fmaxf(q, low), top) : 0.f;
  return (uint32_t)(int)q;
}

// w, 8 values packed, of a scale block's 4 lanes -> the block's fp16 scale, and
// this lane's 8 integers packed (8 bytes, or 4 bytes in x of the result).
template <bool BF16, int BITS>
__device__ __forceinline__ uint2 quantise8(const uint32_t (&w)[4], uint16_t& scale) {
  // the largest magnitude, as the type's bits: a NaN is above infinity, infinity above every number
  uint32_t big = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu), __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
  big = __vmaxu2(big, __shfl_xor_sync(0xffffffffu, big, 1));
  big = __vmaxu2(big, __shfl_xor_sync(0xffffffffu, big, 2));
  const float m = pair_of<BF16>(max(big >> 16, big & 0xFFFFu)).x;
  constexpr float top = BITS == 8 ? 127.f : 7.f, low = BITS == 8 ? -127.f : -8.f;
  scale = __half_as_ushort(__float2half_rn(m / top));
  if (!(m <= 65024.f)) scale = 0x7FFFu;  // the block reads back as NaN
  const float d = __half2float(__ushort_as_half(scale));
  // round_half_even(x / d) without eight divisions.  x and d have at most 11
  // significant bits and the quotient's half-integers h / 2 at most 8, so
  // 2 x = h d or the two are 2^-19 apart, relative: x * (1 / d), off by less
  // than 2^-22, rounds as the quotient does unless that is a half-integer
  // exactly.  Then |x - q d| = d / 2 (an exact fma), and an odd q goes to its
  // even neighbour.  A normal d is within 2^-11 of m / top, which keeps |q|
  // within top; the sum with 1.5 * 2^23 rounds and holds q in its low bits.
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(d));
  constexpr float kMagic = 12582912.f;
  uint32_t u[8];
  float far = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = pair_of<BF16>(w[j]);
    const float2 y = fma2(x, make_float2(inv, inv), make_float2(kMagic, kMagic));
    const float qx = kMagic - y.x, qy = kMagic - y.y;  // -q
    far = fmaxf(far, fmaxf(fabsf(fmaf(qx, d, x.x)), fabsf(fmaf(qy, d, x.y))));
    u[2 * j] = __float_as_uint(y.x);
    u[2 * j + 1] = __float_as_uint(y.y);
  }
  if (!(d >= 6.103515625e-05f) || far * 2.f == d) {
    const float slow = d > 0.f ? 1.f / d : 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 x = pair_of<BF16>(w[j]);
      u[2 * j] = quantise_slowly(x.x, d, slow, low, top);
      u[2 * j + 1] = quantise_slowly(x.y, d, slow, low, top);
    }
  }
  // the low bytes of four words, in order
  const auto bytes = [](uint32_t a, uint32_t b, uint32_t c, uint32_t e) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, e, 0x0040), 0x5410);
  };
  if (BITS == 8) return make_uint2(bytes(u[0], u[1], u[2], u[3]) ^ 0x80808080u, bytes(u[4], u[5], u[6], u[7]) ^ 0x80808080u);
  const uint32_t even = bytes(u[0], u[2], u[4], u[6]), odd = bytes(u[1], u[3], u[5], u[7]);
  return make_uint2(((even & 0x0F0F0F0Fu) | (odd << 4 & 0xF0F0F0F0u)) ^ 0x88888888u, 0u);
}

// The first blocks look through the batch's sequences, a thread one or (with few threads) several.  A thread's first is
// loaded beside what finds its own token, so that looking costs no trip to memory of its own.
struct SeqCheck {
  bool on;  // the block has sequences to look at
  int64_t b;
  int c0, c1, len;
  __device__ __forceinline__ SeqCheck(const KvArgs& kv)
      : on(blockIdx.y == 0 && blockIdx.x < (unsigned)(kv.n_seqs + kRowThreads - 1) / kRowThreads), c0(0), c1(0), len(0) {
    if (!on) return;
    b = (int64_t)blockIdx.x * kRowThreads + threadIdx.x;
    if (b < kv.n_seqs) c0 = __ldg(kv.cu + b), c1 = __ldg(kv.cu + b + 1), len = __ldg(kv.lens + b);
  }
  __device__ __forceinline__ void flag(const KvArgs& kv) const {
    if (!on) return;
    bool ok = kv_seq_ok(kv, c0, c1, len);
    const int64_t threads = (int64_t)gridDim.x * kRowThreads;
    for (int64_t i = b + threads; i < kv.n_seqs; i += threads) ok &= kv_seq_ok(kv, (int)i);
    if (!ok) kv_flag(kv, MOE_KV_BAD_BATCH);
  }
};

// LPR lanes a row.  NORM: q and k rows are normalised and rotated.  BITS > 0:
// k and v rows go to the cache (else k goes to ko and there is no v).
// blockIdx.y is a unit's place within its token, so that all of a block's
// rows are q, k or v rows and what they share (weights, angles) is prepared
// once a unit: with 4 rows a unit the kernel is bound by the instructions it
// issues.  4,096 tokens with 76 MB of q and k in heads of 256 take 18 us (24 with
// rows of all three kinds side by side, each preparing its own).
template <int LPR, bool BF16, bool NORM, int BITS>
__global__ void __launch_bounds__(kRowThreads, 4) head_rows_kernel(const RowArgs r, const KvArgs kv) {
  constexpr bool STORE = BITS > 0;
  const int lane = threadIdx.x % LPR;
  const int t = blockIdx.x * (kRowThreads / LPR) + threadIdx.x / LPR;
  int slot = blockIdx.y;
  const int kind = slot < r.q_slots ? 0 : slot < r.q_slots + r.k_slots ? 1 : 2;
  const bool flags = STORE && slot == 0 && lane == 0;
  slot -= kind == 0 ? 0 : kind == 1 ? r.q_slots : r.q_slots + r.k_slots;
  const int h0 = slot * r.per, n = min(r.per, (kind == 0 ? r.nq : r.nk) - h0);  // the unit's heads
  const HeadSrc src = kind == 0 ? r.q : kind == 1 ? r.k : r.v;
  bool live = t < r.n_tokens;
  const bool in = lane * 8 < r.dim;

  uint4 x[kRowsPerUnit];
  const uint16_t* from = src.p + (int64_t)t * src.ts + h0 * src.hs + lane * 8;
#pragma unroll
  for (int i = 0; i < kRowsPerUnit; ++i) {
    x[i] = make_uint4(0, 0, 0, 0);
    if (live && in && i < n) x[i] = *reinterpret_cast<const uint4*>(from + i * src.hs);
  }

  int pos = 0;
  uint8_t* tile = nullptr;
  if constexpr (STORE) {
    const SeqCheck seqs(kv);
    if (live) {
      const int b = kv_seq_of(kv, t);
      live = b >= 0;
      if (live) {
        const int c0 = __ldg(kv.cu + b), fresh = __ldg(kv.cu + b + 1) - c0, len = __ldg(kv.lens + b);
        pos = len - fresh + (t - c0);
        if (pos >= 0) tile = kv_tile_of(kv, b, pos, kv_tile_bytes(LPR * 8, BITS));
        if (flags && pos >= 0 && !tile) kv_flag(kv, MOE_KV_BAD_PAGE);
      }
    }
    seqs.flag(kv);
  }
  const int row = pos & (kKvTile - 1);
  const bool turns = NORM && kind < 2;
  const int half8 = r.rot / 16;  // lanes of the rotated part's first half
  const bool rotated = turns && lane < 2 * half8;
  const int partner = rotated && !r.inter ? (lane < half8 ? lane + half8 : lane - half8) : lane;
  // out = inv * (x * cw + g * sw): g is the rotation's partner of x, cw and sw hold the weights, cos and +-sin
  float2 cw[4], sw[4];
  float nan_pos = 0.f;
  if (NORM) {
    int angle = pos;
    if (live && r.positions) angle = __ldg(r.positions + t);
    if (angle < 0) live = false;  // padding
    const uint16_t* wt = kind == 0 ? r.wq : r.wk;
#pragma unroll
    for (int j = 0; j < 4; ++j) cw[j] = sw[j] = make_float2(1.f, 1.f);
    if (turns && wt != nullptr && in) {
      const uint4 a = __ldg(reinterpret_cast<const uint4*>(wt + lane * 8)), b = __ldg(reinterpret_cast<const uint4*>(wt + partner * 8));
      const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        cw[j] = pair_of<BF16>(wa[j]);
        cw[j].x += r.woff, cw[j].y += r.woff;
        sw[j] = pair_of<BF16>(r.inter ? __byte_perm(wb[j], wb[j], 0x1032) : wb[j]);
        sw[j].x += r.woff, sw[j].y += r.woff;
      }
    }
    const bool beyond = turns && r.rot > 0 && live && angle >= r.n_positions;
    if (beyond) nan_pos = __uint_as_float(0x7FFFFFFFu);
    if (rotated && live && !beyond) {
      // a pair of the table is (cos, sin) of one angle
      const float* tab = r.table + (int64_t)angle * r.rot;
      if (r.inter) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 a = __ldg(reinterpret_cast<const float2*>(tab + lane * 8) + j);
          cw[j].x *= a.x, cw[j].y *= a.x;
          sw[j].x *= -a.y, sw[j].y *= a.y;
        }
      } else {
        const bool first = lane < half8;
        const float4* p = reinterpret_cast<const float4*>(tab + (first ? lane : lane - half8) * 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 a = __ldg(p + j);
          cw[j].x *= a.x, cw[j].y *= a.z;
          sw[j].x *= first ? -a.y : a.y, sw[j].y *= first ? -a.w : a.w;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) sw[j] = make_float2(0.f, 0.f);
    }
  }
  const bool to_cache = STORE && kind > 0;
  const HeadDst dst = kind == 0 ? r.qo : r.ko;
  uint16_t* to = dst.p + (int64_t)t * dst.ts + h0 * dst.hs + lane * 8;
#pragma unroll
  for (int i = 0; i < kRowsPerUnit; ++i) {
    if (i >= n) break;  // (the whole block)
    uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    if (turns) {
      float2 f[4], sum = make_float2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = pair_of<BF16>(w[j]), sum = fma2(f[j], f[j], sum);
      float ss = sum.x + sum.y;
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float inv = rsqrtf(fmaf(ss, r.inv_dim, r.eps)) + nan_pos;
      const float2 inv2 = make_float2(inv, inv);
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = mul2(mul2(f[j], inv2), cw[j]);
      if (r.rot > 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t o = r.inter ? __byte_perm(w[j], w[j], 0x1032) : __shfl_sync(0xffffffffu, w[j], partner, LPR);
          f[j] = fma2(mul2(pair_of<BF16>(o), inv2), sw[j], f[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = pack2<BF16>(f[j].x, f[j].y);
    }
    if (!to_cache) {
      if (live && in) *reinterpret_cast<uint4*>(to + i * dst.hs) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      constexpr int B = STORE ? BITS : 8, R = kv_row_bytes(LPR * 8, B);
      uint16_t scale;
      const uint2 u = quantise8<BF16, B>(w, scale);  // the whole warp: shuffles
      if (live && tile) {
        uint8_t* base = tile + (size_t)(h0 + i) * kv.head_bytes + (kind == 2 ? kv_half_bytes(LPR * 8, B) : 0);
        const int turn = kv_turn(row) & (R / 16 - 1);
        if (B == 8)
          *reinterpret_cast<uint2*>(base + row * R + (((lane >> 1) ^ turn) << 4) + (lane & 1) * 8) = u;
        else
          *reinterpret_cast<uint32_t*>(base + row * R + (((lane >> 2) ^ turn) << 4) + (lane & 3) * 4) = u.x;
        if ((lane & 3) == 0) reinterpret_cast<uint16_t*>(base + kKvTile * R)[(lane >> 2) * kKvTile + row] = scale;
      }
    }
  }
}

// Neighbouring groups of lanes take neighbouring tokens of the same heads, so
// that a tile's 2-byte scales (32 tokens side by side) come from the same
// sectors; a unit reads kReadHeads heads' K and V with all loads in flight.
// 74 MB of 4-bit heads of 128 and the 262 they become take 58 us (5.8 TB/s).
constexpr int kReadHeads = 2;

template <int LPR, bool BF16, int BITS>
__global__ void __launch_bounds__(kRowThreads) kv_read_kernel(const KvArgs kv, const HeadDst ko, const HeadDst vo, int slots) {
  constexpr int D = LPR * 8, R = kv_row_bytes(D, BITS), HB = kv_half_bytes(D, BITS);
  const int lane = threadIdx.x % LPR;
  const int s = blockIdx.y, t = (int)(blockIdx.x * (kRowThreads / LPR) + threadIdx.x / LPR);
  const SeqCheck seqs(kv);
  const int b = t < kv.n_tokens ? kv_seq_of(kv, t) : -1;
  seqs.flag(kv);
  if (b < 0) return;
  const int c0 = __ldg(kv.cu + b), n = __ldg(kv.cu + b + 1) - c0, len = __ldg(kv.lens + b);
  const int pos = len - n + (t - c0);
  const uint8_t* tile = pos >= 0 ? kv_tile_of(kv, b, pos, kv_tile_bytes(D, BITS)) : nullptr;
  if (lane == 0 && s == 0 && pos >= 0 && !tile) kv_flag(kv, MOE_KV_BAD_PAGE);
  const int row = pos & (kKvTile - 1), turn = kv_turn(row) & (R / 16 - 1);
  const int at = BITS == 8 ? row * R + (((lane >> 1) ^ turn) << 4) + (lane & 1) * 8
                           : row * R + (((lane >> 2) ^ turn) << 4) + (lane & 3) * 4;
  uint2 u[2 * kReadHeads];
  uint16_t sc[2 * kReadHeads];
#pragma unroll
  for (int i = 0; i < 2 * kReadHeads; ++i) {
    const int h = s + (i >> 1) * slots;
    u[i] = make_uint2(0, 0);
    sc[i] = 0x7FFFu;
    if (tile && h < kv.heads) {
      const uint8_t* base = tile + (size_t)h * kv.head_bytes + (i & 1) * HB;
      if (BITS == 8)
        u[i] = *reinterpret_cast<const uint2*>(base + at);
      else
        u[i].x = *reinterpret_cast<const uint32_t*>(base + at);
      sc[i] = reinterpret_cast<const uint16_t*>(base + kKvTile * R)[(lane >> 2) * kKvTile + row];
    }
  }
#pragma unroll
  for (int i = 0; i < 2 * kReadHeads; ++i) {
    const int h = s + (i >> 1) * slots;
    if (h >= kv.heads) continue;
    const float d = __half2float(__ushort_as_half(sc[i]));
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int q = BITS == 8 ? (int)(((j < 4 ? u[i].x : u[i].y) >> (8 * (j & 3))) & 255u) - 128
                              : (int)((u[i].x >> (4 * j)) & 15u) - 8;
      f[j] = d * (float)q;
    }
    const HeadDst& o = (i & 1) ? vo : ko;
    *reinterpret_cast<uint4*>(o.p + (int64_t)t * o.ts + h * o.hs + lane * 8) =
        make_uint4(pack2<BF16>(f[0], f[1]), pack2<BF16>(f[2], f[3]), pack2<BF16>(f[4], f[5]), pack2<BF16>(f[6], f[7]));
  }
}

HeadSrc src_of(const moe_heads_t* h) {
  return h ? HeadSrc{(const uint16_t*)h->data, h->token_stride, h->head_stride} : HeadSrc{nullptr, 0, 0};
}
HeadDst dst_of(const moe_heads_t* h) {
  return h ? HeadDst{(uint16_t*)h->data, h->token_stride, h->head_stride} : HeadDst{nullptr, 0, 0};
}

template <int LPR, bool NORM, int BITS>
moe_status_t launch_rows(RowArgs r, const KvArgs& kv, bool bf16, cudaStream_t st) {
  const int64_t H = (int64_t)r.nq + r.nk + (BITS ? r.nk : 0);
  // One row a group while its threads fill the 152 SMs (1,024 of them each, by
  // the launch bounds) at most twice over, so that a small call's rows run
  // side by side; several rows of a token a group above that, which reuses the
  // token's angles and page.
  if (H > 65535) return MOE_ERR_UNSUPPORTED;
  const int64_t rows = (int64_t)r.n_tokens * H;
  r.per = rows * LPR <= 152 * 2048 ? 1 : kRowsPerUnit;
  r.q_slots = (r.nq + r.per - 1) / r.per;
  r.k_slots = (r.nk + r.per - 1) / r.per;
  r.inv_dim = 1.f / (float)r.dim;
  const unsigned slots = (unsigned)(r.q_slots + (BITS ? 2 : 1) * r.k_slots);
  const dim3 blocks((unsigned)(((int64_t)r.n_tokens * LPR + kRowThreads - 1) / kRowThreads), slots);
  if (bf16)
    head_rows_kernel<LPR, true, NORM, BITS><<<blocks, kRowThreads, 0, st>>>(r, kv);
  else
    head_rows_kernel<LPR, false, NORM, BITS><<<blocks, kRowThreads, 0, st>>>(r, kv);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <bool NORM>
moe_status_t launch_store(const RowArgs& r, const KvArgs& kv, int bits, bool bf16, cudaStream_t st) {
  if (bits == 8) {
    if (r.dim == 64) return launch_rows<8, NORM, 8>(r, kv, bf16, st);
    if (r.dim == 128) return launch_rows<16, NORM, 8>(r, kv, bf16, st);
    return launch_rows<32, NORM, 8>(r, kv, bf16, st);
  }
  if (r.dim == 64) return launch_rows<8, NORM, 4>(r, kv, bf16, st);
  if (r.dim == 128) return launch_rows<16, NORM, 4>(r, kv, bf16, st);
  return launch_rows<32, NORM, 4>(r, kv, bf16, st);
}

template <int LPR, int BITS>
moe_status_t launch_read(const KvArgs& kv, const HeadDst& ko, const HeadDst& vo, bool bf16, cudaStream_t st) {
  const int slots = (kv.heads + kReadHeads - 1) / kReadHeads;
  const dim3 grid((unsigned)(((int64_t)kv.n_tokens * LPR + kRowThreads - 1) / kRowThreads), slots);
  if (bf16)
    kv_read_kernel<LPR, true, BITS><<<grid, kRowThreads, 0, st>>>(kv, ko, vo, slots);
  else
    kv_read_kernel<LPR, false, BITS><<<grid, kRowThreads, 0, st>>>(kv, ko, vo, slots);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// Fills the norm + rotation part of `r`; the activations are checked by the caller.
moe_status_t norm_args(const moe_norm_rope_t* d, int dim, const int32_t* positions, bool need_positions, RowArgs* r) {
  if (!d || !(d->eps >= 0.f) || !std::isfinite(d->eps) || !std::isfinite(d->weight_offset)) return MOE_ERR_INVALID_ARG;
  if (((uintptr_t)d->q_weight & 15) || ((uintptr_t)d->k_weight & 15)) return MOE_ERR_INVALID_ARG;
  if (d->rot_dim < 0 || d->rot_dim % 16 || d->rot_dim > dim) return MOE_ERR_INVALID_ARG;
  if (d->rot_dim > 0 && (!d->table || ((uintptr_t)d->table & 15) || d->n_positions < 1)) return MOE_ERR_INVALID_ARG;
  if (d->rot_dim > 0 && need_positions && !positions) return MOE_ERR_INVALID_ARG;
  if ((uintptr_t)positions & 3) return MOE_ERR_INVALID_ARG;
  r->wq = (const uint16_t*)d->q_weight;
  r->wk = (const uint16_t*)d->k_weight;
  r->table = d->table;
  r->positions = positions;
  r->n_positions = d->n_positions;
  r->rot = d->rot_dim;
  r->inter = d->interleaved != 0;
  r->eps = d->eps;
  r->woff = d->weight_offset;
  return MOE_OK;
}

moe_status_t half_type(int32_t dtype) {
  if (dtype == MOE_BF16 || dtype == MOE_FP16) return MOE_OK;
  return dtype == MOE_FP32 ? MOE_ERR_UNSUPPORTED : MOE_ERR_INVALID_ARG;
}

}  // namespace
}  // namespace moe

extern "C" MOE_API size_t moe_kv_page_bytes(int32_t page_size, int32_t n_kv_heads, int32_t head_dim, int32_t bits) {
  if (page_size < 32 || page_size > 4096 || page_size % 32 || n_kv_heads < 1 || n_kv_heads > 1024) return 0;
  if ((head_dim != 64 && head_dim != 128 && head_dim != 256) || (bits != 8 && bits != 4)) return 0;
  return (size_t)n_kv_heads * (page_size / 32) * moe::kv_tile_bytes(head_dim, bits);
}

extern "C" MOE_API moe_status_t moe_rope_table(int32_t n_positions, int32_t rot_dim, double base, float* table_host) {
  if (!table_host || n_positions < 1 || rot_dim < 16 || rot_dim % 16 || !(base > 0.0) || !std::isfinite(base))
    return MOE_ERR_INVALID_ARG;
  const int half = rot_dim / 2;
  for (int i = 0; i < half; ++i) {
    const double f = std::pow(base, -2.0 * i / rot_dim);
    for (int64_t p = 0; p < n_positions; ++p) {
      table_host[(p * half + i) * 2] = (float)std::cos((double)p * f);
      table_host[(p * half + i) * 2 + 1] = (float)std::sin((double)p * f);
    }
  }
  return MOE_OK;
}

extern "C" MOE_API moe_status_t moe_qk_norm_rope(const moe_norm_rope_t* desc, int32_t dtype, int32_t n_tokens,
                                                 int32_t head_dim, int32_t n_q, const moe_heads_t* q,
                                                 const moe_heads_t* q_out, int32_t n_kv, const moe_heads_t* k,
                                                 const moe_heads_t* k_out, const int32_t* positions, void* cuda_stream) {
  moe_status_t st = moe::half_type(dtype);
  if (st != MOE_OK) return st;
  if (n_tokens < 0 || n_tokens > moe::kMaxTokens || head_dim < 8 || head_dim > 256 || head_dim % 8 || n_q < 0 || n_kv < 0 || n_q > 65536 || n_kv > 65536)
    return MOE_ERR_INVALID_ARG;
  moe::RowArgs r{};
  st = moe::norm_args(desc, head_dim, positions, n_tokens > 0, &r);
  if (st != MOE_OK) return st;
  if (n_tokens == 0 || n_q + n_kv == 0) return MOE_OK;
  if (n_q + n_kv > 65535) return MOE_ERR_UNSUPPORTED;
  if (n_q && (!moe::heads_ok(q, head_dim) || !moe::out_heads_ok(q_out, n_q, n_tokens, head_dim))) return MOE_ERR_INVALID_ARG;
  if (n_kv && (!moe::heads_ok(k, head_dim) || !moe::out_heads_ok(k_out, n_kv, n_tokens, head_dim))) return MOE_ERR_INVALID_ARG;
  r.q = moe::src_of(n_q ? q : nullptr);
  r.qo = moe::dst_of(n_q ? q_out : nullptr);
  r.k = moe::src_of(n_kv ? k : nullptr);
  r.ko = moe::dst_of(n_kv ? k_out : nullptr);
  r.n_tokens = n_tokens;
  r.nq = n_q;
  r.nk = n_kv;
  r.dim = head_dim;
  const cudaStream_t s = (cudaStream_t)cuda_stream;
  const moe::KvArgs none{};
  if (head_dim <= 64) return moe::launch_rows<8, true, 0>(r, none, dtype == MOE_BF16, s);
  if (head_dim <= 128) return moe::launch_rows<16, true, 0>(r, none, dtype == MOE_BF16, s);
  return moe::launch_rows<32, true, 0>(r, none, dtype == MOE_BF16, s);
}

extern "C" MOE_API moe_status_t moe_kv_append(const moe_kv_cache_t* cache, const moe_kv_batch_t* batch, int32_t dtype,
                                              const moe_heads_t* k, const moe_heads_t* v, void* cuda_stream) {
  moe_status_t st = moe::half_type(dtype);
  if (st != MOE_OK) return st;
  moe::KvArgs kv;
  st = moe::kv_args(cache, batch, &kv);
  if (st != MOE_OK) return st;
  if (kv.n_tokens == 0) return MOE_OK;
  if (!moe::heads_ok(k, cache->head_dim) || !moe::heads_ok(v, cache->head_dim)) return MOE_ERR_INVALID_ARG;
  moe::RowArgs r{};
  r.k = moe::src_of(k);
  r.v = moe::src_of(v);
  r.n_tokens = kv.n_tokens;
  r.nk = kv.heads;
  r.dim = cache->head_dim;
  return moe::launch_store<false>(r, kv, cache->bits, dtype == MOE_BF16, (cudaStream_t)cuda_stream);
}

extern "C" MOE_API moe_status_t moe_kv_append_norm_rope(const moe_kv_cache_t* cache, const moe_kv_batch_t* batch,
                                                        const moe_norm_rope_t* desc, int32_t dtype, int32_t n_q,
                                                        const moe_heads_t* q, const moe_heads_t* q_out,
                                                        const moe_heads_t* k, const moe_heads_t* v,
                                                        const int32_t* positions, void* cuda_stream) {
  moe_status_t st = moe::half_type(dtype);
  if (st != MOE_OK) return st;
  moe::KvArgs kv;
  st = moe::kv_args(cache, batch, &kv);
  if (st != MOE_OK) return st;
  const int dim = cache->head_dim;
  moe::RowArgs r{};
  st = moe::norm_args(desc, dim, positions, false, &r);
  if (st != MOE_OK) return st;
  if (n_q < 0 || n_q > 65536) return MOE_ERR_INVALID_ARG;
  if (kv.n_tokens == 0) return MOE_OK;
  if (n_q && (!moe::heads_ok(q, dim) || !moe::out_heads_ok(q_out, n_q, kv.n_tokens, dim))) return MOE_ERR_INVALID_ARG;
  if (!moe::heads_ok(k, dim) || !moe::heads_ok(v, dim)) return MOE_ERR_INVALID_ARG;
  r.q = moe::src_of(n_q ? q : nullptr);
  r.qo = moe::dst_of(n_q ? q_out : nullptr);
  r.k = moe::src_of(k);
  r.v = moe::src_of(v);
  r.n_tokens = kv.n_tokens;
  r.nq = n_q;
  r.nk = kv.heads;
  r.dim = dim;
  return moe::launch_store<true>(r, kv, cache->bits, dtype == MOE_BF16, (cudaStream_t)cuda_stream);
}

extern "C" MOE_API moe_status_t moe_kv_read(const moe_kv_cache_t* cache, const moe_kv_batch_t* batch, int32_t dtype,
                                            const moe_heads_t* k_out, const moe_heads_t* v_out, void* cuda_stream) {
  moe_status_t st = moe::half_type(dtype);
  if (st != MOE_OK) return st;
  moe::KvArgs kv;
  st = moe::kv_args(cache, batch, &kv);
  if (st != MOE_OK) return st;
  if (kv.n_tokens == 0) return MOE_OK;
  const int dim = cache->head_dim;
  if (!moe::out_heads_ok(k_out, kv.heads, kv.n_tokens, dim) || !moe::out_heads_ok(v_out, kv.heads, kv.n_tokens, dim))
    return MOE_ERR_INVALID_ARG;
  const moe::HeadDst ko = moe::dst_of(k_out), vo = moe::dst_of(v_out);
  const cudaStream_t s = (cudaStream_t)cuda_stream;
  const bool bf = dtype == MOE_BF16;
  if (cache->bits == 8) {
    if (dim == 64) return moe::launch_read<8, 8>(kv, ko, vo, bf, s);
    if (dim == 128) return moe::launch_read<16, 8>(kv, ko, vo, bf, s);
    return moe::launch_read<32, 8>(kv, ko, vo, bf, s);
  }
  if (dim == 64) return moe::launch_read<8, 4>(kv, ko, vo, bf, s);
  if (dim == 128) return moe::launch_read<16, 4>(kv, ko, vo, bf, s);
  return moe::launch_read<32, 4>(kv, ko, vo, bf, s);
}
