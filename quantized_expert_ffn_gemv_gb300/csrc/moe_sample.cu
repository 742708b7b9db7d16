// Sampling: one thread-block cluster a row.  The row is read from memory once,
// as fp32 into the cluster's shared memory, and everything else happens
// there: the maximum, the cut that top-k and top-p make, the kept mass, and
// the token.  With the row at hand the bound is the one read of the logits;
// for a single row it is the chain of cluster barriers.  256 rows of 151,552
// fp32 logits take 55 us greedy (23 to read them), 129 with top-k 50, 355 with
// top-p 0.9 alone; one row of bf16 logits, top-k 50, 13.
//
// Weights w = 2^-y, y = (max - z) log2(e) / T, are evaluated to about 2^-31
// relative (float pairs for y, a 512-entry table and a cubic for the rest)
// and summed as integers in units of 2^-45: integer sums have no order, so
// any split of the work gives the same bits, and the sums that top-p, min-p
// and the draw compare are exact.  Conversions go through the float's
// mantissa (adding 1.5 * 2^23): the conversion unit is a quarter as wide, and the 64-bit
// one that a first version used took half of its time.
//
// The cut.  Kept elements are a prefix of the order (logit descending, index
// ascending).  A histogram of y (1/16 octave a bin; counts, or masses as two
// 16-bit halves in units of which every weight of the bin is a whole number)
// finds the bin the cut falls into.  Each CTA lists its elements of that bin and those in front of it.
// If both fit one list, the first CTA ranks them all and draws the token by
// itself; if only the bin's do, it ranks those for the cut's last element
// and the cluster draws; otherwise the bin is histogrammed again, a thousand
// times finer in y and then by the logits' bits, until few are left or all
// have the same logit, whose cut is then an index.  The histogram's bound is
// its shared-memory atomics (10 us for the counts of 256 rows' elements, an SM
// having two), so for a small k a histogram of each thread's largest logit is
// tried first: the k-th largest of those is at most the k-th of all, and
// seldom many lie between.
#include <cooperative_groups.h>
#include <algorithm>
#include <cmath>

#include "moe_kv.cuh"

namespace cg = cooperative_groups;

namespace moe {
namespace {

constexpr int kSThreads = 512, kSWarps = kSThreads / 32;
constexpr int kBins = 1024, kPerOctave = 16;  // 64 octaves: beyond them a weight is 0 in units of 2^-45
constexpr int kUnit = 45;                     // 2^18 weights of 2^45 fit 64 bits
constexpr int kList = kSThreads;              // elements sorted at most: one a thread
constexpr int kDirect = 256;                  // up to here each element is compared with all others, beyond they are sorted
constexpr int kHalfList = 384;                // what a CTA lists of either sort
constexpr int kMaxVocab = 262144;
constexpr int kMaxCluster = 8;
constexpr int kTable = 512;

struct Pow2Table {
  float2 v[kTable];
};
// 2^(-(i + 1) / 512) as float pairs: the exponential's power series in binary64.
constexpr Pow2Table make_pow2() {
  Pow2Table t{};
  for (int i = 0; i < kTable; ++i) {
    const double x = -0.69314718055994530942 * (i + 1) / kTable;
    double term = 1.0, sum = 1.0;
    for (int n = 1; n < 24; ++n) {
      term *= x / n;
      sum += term;
    }
    t.v[i].x = (float)sum;
    t.v[i].y = (float)(sum - (double)t.v[i].x);
  }
  return t;
}
__device__ const Pow2Table g_pow2 = make_pow2();

struct SampleArgs {
  const void* logits;
  int64_t row_stride;
  int rows, vocab, slice;
  int ahead;  // rows that run at a time
  const float *u, *temperature, *top_p, *min_p;
  const int32_t* top_k;
  int32_t* tokens;
  float* probs;
};

// log2(e) / T as a float pair.
struct Rate {
  float h, l;
};
__device__ __forceinline__ Rate rate_of(float T) {
  const float lh = 1.44269502162933349609f, ll = 1.925963033500e-08f;  // log2(e)
  Rate r;
  r.h = lh / T;
  r.l = (fmaf(-r.h, T, lh) + ll) / T;
  return r;
}

constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: the low mantissa bits of a sum with it are the other term, rounded
constexpr int kMagicBits = 0x4B400000;

// y of a logit z <= m rounded to fp32, which orders logits weakly, at most
// 100 (infinity for -infinity before the minimum); and its bin.
__device__ __forceinline__ float y_of(float z, float m, const Rate& c) { return fminf((m - z) * c.h, 100.f); }
__device__ __forceinline__ int bin_of(float y) { return min(__float_as_int(fmaf(y, (float)kPerOctave, kMagic)) - kMagicBits, kBins - 1); }

// w = W 2^-(31 + s - 1), W in 2^30 .. 2^31.  From 64 octaves on W is
// anything and s at least 64, which to_units makes 0.
__device__ __forceinline__ uint32_t weight31(float z, float m, const Rate& c, const float2* tab, int& s) {
  const float x = m - z;
  const float kf = fmaf(fminf(x * c.h, 100.f), (float)kTable, kMagic);  // (y_of's product)
  const int k = __float_as_int(kf) - kMagicBits - 1;                    // round(512 y) - 1
  // r = y - round(512 y) / 512, small, from y = (x + xl) (c.h + c.l)
  float r = fmaf(x, c.h, (kf - kMagic) * (-1.f / kTable));
  r = fmaf(x, c.l, r);
  const float bb = x - m;
  r = fmaf((m - (x - bb)) + (-z - bb), c.h, r);  // m - z = x + that
  // 2^-r - 1 by its series: |r| < 2^-10
  const float p = r * fmaf(r, fmaf(r, -0.0555041087f, 0.2402265070f), -0.6931471806f);
  const float2 t = tab[k & (kTable - 1)];  // t.x in 1/2 .. 1
  const float low = fmaf(fmaf(t.x, p, t.y), 2147483648.f, kMagic);
  s = (k >> 9) + 1;
  return (((__float_as_uint(t.x) & 0x7FFFFFu) | 0x800000u) << 7) + (uint32_t)(__float_as_int(low) - kMagicBits);
}
// W 2^(15 - s) rounded to units of 2^-45 is v 2^up, with 32-bit shifts.
constexpr int kUp = kUnit - 30;
__device__ __forceinline__ uint32_t rounded(uint32_t W, int s) {
  const uint32_t down = (uint32_t)(s - min(s, kUp));
  uint32_t half, v;
  asm("shl.b32 %0, 1, %1;" : "=r"(half) : "r"(down));  // 0 from 32 on
  asm("shr.u32 %0, %1, %2;" : "=r"(v) : "r"(W + (half >> 1)), "r"(down));
  return v;
}
__device__ __forceinline__ uint64_t to_units(uint32_t W, int s) { return (uint64_t)rounded(W, s) * (1u << (kUp - min(s, kUp))); }
// The units that the masses of an octave's bins are held in: their weights have s = octave or octave + 1, so that each is a
// whole number of 2^bin_unit, at most 2^31 1.022 of them.
__device__ __forceinline__ int bin_unit(int octave) { return kUp - min(octave + 1, kUp); }
__device__ __forceinline__ uint32_t in_bin_units(uint32_t W, int s, int octave) {
  return rounded(W, s) << (min(octave + 1, kUp) - min(s, kUp));
}
__device__ __forceinline__ uint64_t weight(float z, float m, const Rate& c, const float2* tab) {
  int s;
  const uint32_t W = weight31(z, m, c, tab, s);
  return to_units(W, s);
}

// Order-preserving image of a logit (no NaN): larger logit, larger key; -0 equals 0.
__device__ __forceinline__ uint32_t key_of(float z) {
  const uint32_t b = __float_as_uint(z + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key & 0x7FFFFFFFu : ~key);
}

// floor(x * f), or ceil(x * f) with up, for 0 <= f < 1, exactly.
__device__ __forceinline__ uint64_t mul_frac(uint64_t x, float f, bool up) {
  if (!(f > 0.f)) return 0;
  const uint32_t b = __float_as_uint(f);
  const int e = (int)(b >> 23);
  const uint64_t mant = e ? (b & 0x7FFFFFu) | 0x800000u : (b & 0x7FFFFFu);
  const int sh = 150 - (e ? e : 1);  // f = mant * 2^-sh, sh = 24 .. 149
  const uint64_t lo = x * mant, hi = __umul64hi(x, mant);
  uint64_t q, rest;
  if (sh < 64) {
    q = (hi << (64 - sh)) | (lo >> sh);
    rest = lo << (64 - sh);
  } else if (sh < 128) {
    q = hi >> (sh - 64);
    rest = lo | (sh == 64 ? 0 : hi << (128 - sh));
  } else {
    q = 0;
    rest = lo | hi;
  }
  return q + (up && rest ? 1 : 0);
}

// The elements kept: those of a key above, or of the key itself up to an index.
struct Cut {
  uint32_t key, idx;
};
__device__ __forceinline__ bool kept(uint32_t key, uint32_t idx, const Cut& c) { return key > c.key || (key == c.key && idx <= c.idx); }

// An element of a list by its place in the order: larger first.
__device__ __forceinline__ uint64_t entry(uint32_t key, uint32_t idx) { return (uint64_t)key << 32 | ~idx; }
__device__ __forceinline__ uint32_t key_in(uint64_t e) { return (uint32_t)(e >> 32); }
__device__ __forceinline__ uint32_t idx_in(uint64_t e) { return ~(uint32_t)e; }

struct alignas(16) Shared {
  // this CTA's histogram, and later its lists: elements of the cut's bin, and in front of it
  union {
    struct {
      uint32_t count[kBins], hi[kBins], lo[kBins];
    } h;
    uint64_t part[2][kHalfList];
  };
  // first CTA: the cluster's histogram, and later the cluster's list and what sorting it takes
  union {
    struct {
      uint64_t mass[kBins];
      uint32_t count[kBins];
    } all;
    struct {
      uint64_t list[kList], w[kList], swap[2][kList];
    };
  };
  float2 pow2[kTable];
  uint64_t wsum[kSWarps], bsum[kSWarps];
  uint32_t wcnt[kSWarps];
  float wmax[kSWarps];
  // written by the CTA, read by the cluster
  float cmax;
  uint32_t cfirst, ccount;  // greedy: the maximum's lowest index; find_cut: lowest and highest key, or a count
  uint32_t part_n[2];
  uint64_t ctotal;
  // written by the first CTA, read by the cluster
  int cut_bin;
  uint32_t cut_count, cut_need, cut_front;
  uint64_t cut_before, cut_target;
  Cut cut;
};

// Exclusive prefixes of a count and a mass over the block's threads.
__device__ __forceinline__ void block_scan(Shared& s, uint32_t& c, uint64_t& m) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t ci = c;
  uint64_t mi = m;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t cv = __shfl_up_sync(0xffffffffu, ci, o);
    const uint64_t mv = __shfl_up_sync(0xffffffffu, mi, o);
    if (lane >= o) ci += cv, mi += mv;
  }
  __syncthreads();
  if (lane == 31) s.wcnt[warp] = ci, s.wsum[warp] = mi;
  __syncthreads();
  uint32_t cb = 0;
  uint64_t mb = 0;
  for (int w = 0; w < warp; ++w) cb += s.wcnt[w], mb += s.wsum[w];
  c = cb + ci - c;
  m = mb + mi - m;
}

// The sum over the block's threads, for all of them.
__device__ __forceinline__ uint64_t block_sum(Shared& s, uint64_t v) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if (lane == 0) s.wsum[warp] = v;
  __syncthreads();
  v = 0;
  for (int w = 0; w < kSWarps; ++w) v += s.wsum[w];
  return v;
}

static_assert(kSWarps == 2 * kMaxCluster, "a warp for each of the cluster's lists");

// The slice of a row that a CTA holds, n4 float4 (the end filled with
// -infinity), and what is asked of the row.
struct Slice {
  const float4* z;
  int n4;
  uint32_t base;
  float m;
  Rate c;
  uint32_t k;     // top-k, 0 = all
  float p;        // top-p, 1 = all
  uint64_t least; // min-p in units
  float u;
  float top;  // the largest of this thread's own
  int32_t* token;
  float* prob;
};

// Sorts one value a thread, descending, over the block's first P threads (P a
// power of two from 32; the others have 0): a bitonic network, by shuffles
// within a warp and through shared memory across.
__device__ __forceinline__ uint64_t sort_values(Shared& s, uint64_t v, int P) {
  const int tid = threadIdx.x;
  int buf = 0;
  for (int size = 2; size <= P; size *= 2) {
    const bool down = (tid & size) == 0;
    for (int stride = size / 2; stride >= 32; stride /= 2) {
      s.swap[buf][tid] = v;
      __syncthreads();
      const uint64_t o = s.swap[buf][tid ^ stride];
      v = (((tid & stride) == 0) == down) == (o > v) ? o : v;
      buf ^= 1;  // (the next barrier is behind every read of this one)
    }
    if (tid < P) {
#pragma unroll
      for (int stride = 16; stride > 0; stride /= 2) {
        if (stride >= size) continue;
        const uint64_t o = __shfl_xor_sync(0xffffffffu, v, stride);
        v = (((tid & stride) == 0) == down) == (o > v) ? o : v;
      }
    }
  }
  return v;
}

// A thread's element of a list in the first CTA: its weight, how many are
// ahead of it in the order, and their mass.  Threads without one have w = 0
// and a place behind all.
struct Ranked {
  uint64_t e, w, front;
  uint32_t place;
};
// How many neighbouring threads share an element of a list compared directly.
__device__ __forceinline__ int sharers(int n) {
  int share = 1;
  while (share < 32 && n * share * 2 <= kSThreads) share *= 2;
  return share;
}
// The sum of w over the list's elements before(i, mine), this thread's part by part.
template <typename F>
__device__ __forceinline__ uint64_t sum_before(const Shared& s, int n, int share, F before, uint32_t& ahead) {
  uint64_t sum = 0;
  ahead = 0;
#pragma unroll 4
  for (int i = threadIdx.x % share; i < n; i += share)
    if (before(s.list[i])) ++ahead, sum += s.w[i];
  for (int o = 1; o < share; o <<= 1) {
    ahead += __shfl_xor_sync(0xffffffffu, ahead, o);
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  return sum;
}
// Ranks the list's n <= kList elements.  500 of them take 18 us by comparing
// all with all and 3 by sorting; 50 take 2 and 4.
__device__ __forceinline__ Ranked rank_list(Shared& s, const Slice& v, int n) {
  const int tid = threadIdx.x;
  Ranked r{tid < n ? s.list[tid] : 0, 0, 0, (uint32_t)tid};
  if (n > kDirect) r.e = sort_values(s, r.e, 1 << (32 - __clz(n - 1)));
  if (tid < n) r.w = weight(logit_of(key_in(r.e)), v.m, v.c, s.pow2);
  if (n > kDirect) {
    uint32_t none = 0;
    r.front = r.w;
    block_scan(s, none, r.front);
    return r;
  }
  if (tid < n) s.w[tid] = r.w;
  __syncthreads();
  const int share = sharers(n), mine = tid / share;
  r.e = mine < n ? s.list[mine] : 0;
  r.front = sum_before(s, n, share, [&](uint64_t o) { return o > r.e; }, r.place);
  r.w = mine < n && tid % share == 0 ? s.w[mine] : 0;
  if (mine >= n || tid % share) r.place = kList;
  return r;
}

// The first CTA alone: every element that top-k and top-p can keep is in the
// list, n of them; cut them, and draw the token.  target: the mass that top-p
// asks for, or 0: its share of what top-k keeps of the list.
__device__ void draw_from_list(Shared& s, const Slice& v, int n, uint64_t target) {
  const int tid = threadIdx.x;
  const Ranked r = rank_list(s, v, n);
  uint64_t w = v.k > 0 && r.place >= v.k ? 0 : r.w;
  if (v.p < 1.f) {
    // front < sum * p  <=>  front < ceil(sum * p)
    if (!target) target = max(mul_frac(block_sum(s, w), v.p, true), (uint64_t)1);
    if (r.front >= target) w = 0;
  }
  if (w < v.least && r.place != 0) w = 0;
  const uint64_t total = block_sum(s, w);  // (its barriers: all have read the list)
  uint64_t below, e = r.e;
  if (n > kDirect) {  // the kept ones in index order, each with its place in the list
    s.w[tid] = w;
    const uint64_t i = sort_values(s, w ? (uint64_t)(uint32_t)e << 32 | tid : 0, 1 << (32 - __clz(n - 1)));
    __syncthreads();
    w = i ? s.w[(uint32_t)i] : 0;
    e = i >> 32;
    below = w;
    uint32_t none = 0;
    block_scan(s, none, below);
  } else {
    const int share = sharers(n), mine = tid / share;
    if (tid % share == 0 && mine < n) s.w[mine] = w;
    __syncthreads();
    uint32_t ahead;
    below = sum_before(s, n, share, [&](uint64_t o) { return (uint32_t)o > (uint32_t)e; }, ahead);  // (~index)
  }
  // running sum > u * total  <=>  running sum > floor(u * total)
  const uint64_t at = mul_frac(total, v.u, false);
  if (w != 0 && below <= at && at < below + w) {
    *v.token = (int32_t)idx_in(e);
    if (v.prob) *v.prob = (float)w / (float)total;
  }
}

// Calls f(logit, index in the row) for the slice's elements, several loads of four in flight.
template <typename F>
__device__ __forceinline__ void each(const Slice& v, F f) {
  constexpr int kAhead = 2;
  for (int i0 = threadIdx.x; i0 < v.n4; i0 += kAhead * kSThreads) {
    float4 q[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      q[j] = i0 + j * kSThreads < v.n4 ? v.z[i0 + j * kSThreads] : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int i = i0 + j * kSThreads;
      if (j > 0 && i >= v.n4) break;
      f(q[j].x, v.base + 4 * i);
      f(q[j].y, v.base + 4 * i + 1);
      f(q[j].z, v.base + 4 * i + 2);
      f(q[j].w, v.base + 4 * i + 3);
    }
  }
}

// The same for the logits that pred accepts, when they are few: a thread goes
// through the ones among its eight, instead of all threads through all eight.
// STEP threads go through the float4 from first, this thread's, to end.
template <int STEP, typename P, typename F>
__device__ __forceinline__ void each_of(const Slice& v, int first, int end, P pred, F f) {
  for (int i0 = first; i0 < end; i0 += 2 * STEP) {
    float4 q[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      q[j] = i0 + j * STEP < end ? v.z[i0 + j * STEP] : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    uint32_t hit = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      hit |= (pred(q[j].x) ? 1u : 0u) << 4 * j;
      hit |= (pred(q[j].y) ? 2u : 0u) << 4 * j;
      hit |= (pred(q[j].z) ? 4u : 0u) << 4 * j;
      hit |= (pred(q[j].w) ? 8u : 0u) << 4 * j;
    }
    if (i0 + STEP >= end) hit &= 15u;
    for (; hit; hit &= hit - 1) {
      const int b = __ffs(hit) - 1, at = 4 * (i0 + (b >> 2) * STEP) + (b & 3);
      f(reinterpret_cast<const float*>(v.z)[at], v.base + at);
    }
  }
}

// The cut among the elements that `limit` keeps (all, when not limited): at
// the top-k'th of the order, or, by mass, at the first where the running mass
// reaches top-p of it all.  The whole cluster calls it.  True: the token is
// drawn.  Otherwise the cut is in the first CTA's Shared::cut until the
// caller's next cluster barrier.
__device__ bool find_cut(cg::cluster_group& cluster, Shared& s, Shared* s0, const Slice& v, const Cut limit, bool limited,
                         bool by_mass) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cluster.block_rank(), C = (int)cluster.num_blocks();
  int level = 0, shift = 0, octave = 0, bin0 = 0, bin1 = 0;  // level 0 looks at all, 1 at bin0 of it, 2 and up at bin1 of that
  float y0 = 0.f, finer = 0.f;                               // level 1: where its bins begin, bins an octave
  uint32_t top_key = 0, low_key = 0;                         // level 2 and up: the range of keys looked at
  bool quick = !by_mass && !limited && v.k * 4 <= (uint32_t)(kSThreads * C);  // only the threads' largest
  uint32_t need = v.k;
  uint64_t before = 0, target = 0;  // mass in front of the range; the mass to reach (set at level 0)
  // is an element among those looked at, and in which bin
  auto place = [&](uint32_t idx, float z) -> int {
    const float y = y_of(z, v.m, v.c);
    const int b0 = bin_of(y);
    if (level > 0 && b0 != bin0) return -1;
    if (level == 0 && !limited) return b0;
    const uint32_t key = key_of(z);
    if (limited && !kept(key, idx, limit)) return -1;
    if (level == 0) return b0;
    const int b1 = min((int)((y - y0) * finer), kBins - 2);
    if (level == 1) return b1;
    return b1 == bin1 && key <= top_key && key >= low_key ? (int)((top_key - key) >> shift) : -1;
  };
  for (;;) {
    for (int i = tid; i < kBins; i += kSThreads) s.h.count[i] = s.h.hi[i] = s.h.lo[i] = 0;
    __syncthreads();
    // counts, or masses.  The last bin collects most elements when the temperature is low: counted apart; its mass is taken for 0
    uint32_t far = 0;
    if (quick) {
      const int bin = bin_of(y_of(v.top, v.m, v.c));
      if (bin < kBins - 1) atomicAdd(&s.h.count[bin], 1u);
    } else each(v, [&](float z, uint32_t idx) {
      const int bin = place(idx, z);
      if (bin < 0) return;
      if (by_mass) {
        if (bin == kBins - 1) return;
        int sh;
        uint32_t W = weight31(z, v.m, v.c, s.pow2, sh);
        W = in_bin_units(W, sh, level == 0 ? (int)((uint32_t)bin / kPerOctave) : octave);
        atomicAdd(&s.h.hi[bin], W >> 16);
        atomicAdd(&s.h.lo[bin], W & 0xFFFFu);
      } else if (bin == kBins - 1) {
        ++far;
      } else {
        atomicAdd(&s.h.count[bin], 1u);
      }
    });
    far = __reduce_add_sync(0xffffffffu, far);
    if (lane == 0 && far) atomicAdd(&s.h.count[kBins - 1], far);
    cluster.sync();
    // every CTA adds up its share of the bins over the cluster, for the first one
    for (int i = rank * (kBins / C) + tid; i < (rank + 1) * (kBins / C); i += kSThreads) {
      uint32_t cnt = 0;
      uint64_t mass = 0;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        if (r >= C) continue;
        const Shared* o = cluster.map_shared_rank(&s, r);
        cnt += o->h.count[i];
        if (by_mass) mass += ((uint64_t)o->h.hi[i] << 16) + o->h.lo[i];
      }
      // (by mass a lower bound of the count: a weight is at most 2^most 1.022 of the bin's units)
      const int of = level == 0 ? i / kPerOctave : octave, most = max(kUnit - max(of, kUp - 1), 0);
      s0->all.count[i] = by_mass ? (uint32_t)((mass >> most) - (mass >> (most + 5))) : cnt;
      s0->all.mass[i] = mass << bin_unit(of);
    }
    if (tid < 2) s.part_n[tid] = 0;
    cluster.sync();
    if (rank == 0) {
      constexpr int kPer = kBins / kSThreads;
      uint32_t cnt[kPer], cb = 0;
      uint64_t mass[kPer], mb = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        cb += cnt[j] = s.all.count[tid * kPer + j];
        mb += mass[j] = s.all.mass[tid * kPer + j];
      }
      if (tid == 0) s.cut_bin = -1;
      const uint64_t own = mb;
      block_scan(s, cb, mb);
      if (by_mass && level == 0) {
        if (tid == kSThreads - 1) s.cut_target = max(mul_frac(mb + own, v.p, true), (uint64_t)1);
        __syncthreads();
        target = s.cut_target;
      }
      mb += before;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const bool here = by_mass ? mb < target && target <= mb + mass[j] : cb < need && need <= cb + cnt[j];
        if (here) {
          s.cut_bin = tid * kPer + j;
          s.cut_count = cnt[j];
          s.cut_need = need - cb;
          s.cut_front = cb;
          s.cut_before = mb;
        }
        cb += cnt[j];
        mb += mass[j];
      }
    }
    cluster.sync();
    const int bin = s0->cut_bin;
    const uint32_t count = quick ? 0 : s0->cut_count;
    if (quick && bin < 0) {  // (too few of them have a weight)
      quick = false;
      cluster.sync();  // the cut's bin has been read
      continue;
    }
    const bool front_too = quick || level == 0 && s0->cut_front + count <= kList;  // (by mass, maybe not)
    before = s0->cut_before;
    if (by_mass) target = s0->cut_target;
    if (!by_mass && !quick) need = s0->cut_need;
    const bool one_key = level > 1 && shift == 0;
    if (level == 0) {
      bin0 = bin;
      octave = bin / kPerOctave;
      y0 = ((float)bin0 - 0.5f) / kPerOctave;
      finer = bin0 == kBins - 1 ? 27.f : 16000.f;  // 1,000 for the bin; the last one ends at 100
    } else if (level == 1) {
      bin1 = bin;
    } else {
      top_key -= (uint32_t)bin << shift;
      const uint32_t span = shift ? (1u << shift) - 1u : 0u;
      low_key = top_key - low_key > span ? top_key - span : low_key;
    }
    if (count <= kList) {
      // list the bin's elements, and at level 0 those in front of it where they may fit
      const float y_end = bin0 == kBins - 1 ? 100.f : (float)(bin0 + 1) / kPerOctave;
      const float y_begin = front_too ? 0.f : ((float)bin0 - 0.5f) / kPerOctave;
      const auto near = [&](float z) {
        const float y = y_of(z, v.m, v.c);
        return y >= y_begin && y <= y_end;
      };
      each_of<kSThreads>(v, tid, v.n4, near, [&](float z, uint32_t idx) {
        const int b = place(idx, z);
        if (b < 0 || (level == 0 && b > bin0) || (level == 1 && b != bin1)) return;
        const int sort = level == 0 && b < bin0;
        if (*(volatile uint32_t*)&s.part_n[sort] > kHalfList) return;  // (a race that at most counts a few more)
        const uint32_t at = atomicAdd(&s.part_n[sort], 1u);
        if (at < kHalfList) s.part[sort][at] = entry(key_of(z), idx);
      });
      cluster.sync();
      uint32_t n0 = 0, n1 = 0;
      if (lane < C) {
        const Shared* o = cluster.map_shared_rank(&s, lane);
        n0 = o->part_n[0];
        n1 = o->part_n[1];
      }
      const bool whole0 = __all_sync(0xffffffffu, n0 <= kHalfList), whole1 = __all_sync(0xffffffffu, n1 <= kHalfList);
      const bool fits = front_too && whole0 && whole1 && __reduce_add_sync(0xffffffffu, n0 + n1) <= kList;
      if (quick ? fits : whole0 && __reduce_add_sync(0xffffffffu, n0) <= kList) {
        if (rank == 0) {
          // gather the CTAs' lists: one warp a list
          uint32_t mine = fits ? n0 + n1 : n0, start = mine;
#pragma unroll
          for (int o = 1; o < kMaxCluster; o <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, start, o);
            if (lane >= o) start += x;
          }
          const int to = (int)__shfl_sync(0xffffffffu, start, kMaxCluster - 1);
          start -= mine;
          const int r = warp >> 1, sort = warp & 1;  // kSWarps = 2 kMaxCluster
          const uint32_t at = __shfl_sync(0xffffffffu, start, r) + (sort ? __shfl_sync(0xffffffffu, n0, r) : 0);
          const uint32_t len0 = __shfl_sync(0xffffffffu, n0, r), len1 = __shfl_sync(0xffffffffu, n1, r);
          const uint32_t len = sort ? (fits ? len1 : 0) : len0;
          if (r < C) {
            const Shared* o = cluster.map_shared_rank(&s, r);
            for (uint32_t e = lane; e < len; e += 32) s.list[at + e] = o->part[sort][e];
          }
          __syncthreads();
          if (fits) {
            draw_from_list(s, v, to, by_mass ? target : 0);
          } else {
            const Ranked r = rank_list(s, v, to);
            // the need-th, or the one whose weight takes the mass to the target
            const uint64_t front = before + r.front;
            if (by_mass ? front < target && target <= front + r.w : r.place == need - 1)
              s.cut = Cut{key_in(r.e), idx_in(r.e)};
          }
        }
        cluster.sync();
        return fits;
      }
    }
    if (quick) {
      quick = false;
      before = 0;
      cluster.sync();  // the lists' lengths have been read
      continue;
    }
    if (one_key) {
      // all elements of the bin have the key top_key and one weight: the cut is the want-th of them in index order
      const uint32_t k = top_key;
      uint32_t want = need;
      if (by_mass) {
        const uint64_t w = weight(logit_of(k), v.m, v.c, s.pow2), more = target > before ? target - before : 1;
        want = w ? (uint32_t)min((more + w - 1) / w, (uint64_t)UINT32_MAX) : UINT32_MAX;
      }
      const float* z = reinterpret_cast<const float*>(v.z);
      const int n = 4 * v.n4, seg = (n + kSWarps - 1) / kSWarps, lo = min(warp * seg, n), hi = min(lo + seg, n);
      auto equal = [&](int i) { return i < hi && key_of(z[i]) == k && (!limited || kept(k, v.base + i, limit)); };
      uint32_t mine = 0;
      for (int i0 = lo; i0 < hi; i0 += 32) mine += __popc(__ballot_sync(0xffffffffu, equal(i0 + lane)));
      __syncthreads();
      if (lane == 0) s.wcnt[warp] = mine;
      __syncthreads();
      if (tid == 0) {
        uint32_t all = 0;
        for (int x = 0; x < kSWarps; ++x) all += s.wcnt[x];
        s.ccount = all;
      }
      cluster.sync();
      uint32_t front = 0, equals = 0;
      for (int r = 0; r < C; ++r) {
        const uint32_t x = cluster.map_shared_rank(&s, r)->ccount;
        front += r < rank ? x : 0;
        equals += x;
      }
      want = min(want, equals);
      for (int x = 0; x < warp; ++x) front += s.wcnt[x];
      if (front < want && want <= front + mine) {
        for (int i0 = lo; i0 < hi; i0 += 32) {
          const bool eq = equal(i0 + lane);
          const unsigned b = __ballot_sync(0xffffffffu, eq);
          if (eq && front + __popc(b & ((1u << lane) - 1u)) + 1 == want) s0->cut = Cut{k, v.base + i0 + lane};
          front += __popc(b);
        }
      }
      cluster.sync();
      return false;
    }
    // the bin again, finer: from level 2 on within the keys it spans
    if (level == 1) {
      uint32_t hi = 0, lo = 0xFFFFFFFFu;
      each(v, [&](float z, uint32_t idx) {
        if (place(idx, z) == bin1) hi = max(hi, key_of(z)), lo = min(lo, key_of(z));
      });
      hi = __reduce_max_sync(0xffffffffu, hi);
      lo = __reduce_min_sync(0xffffffffu, lo);
      if (tid == 0) s.cfirst = 0xFFFFFFFFu, s.ccount = 0;
      __syncthreads();
      if (lane == 0) {
        atomicMax(&s.ccount, hi);
        atomicMin(&s.cfirst, lo);
      }
      cluster.sync();
      for (int r = 0; r < C; ++r) {
        const Shared* o = cluster.map_shared_rank(&s, r);
        hi = max(hi, o->ccount);
        lo = min(lo, o->cfirst);
      }
      top_key = hi;
      low_key = lo;
    }
    shift = 0;
    while (level > 0 && ((top_key - low_key) >> shift) >= (uint32_t)(kBins - 1)) ++shift;  // the far bin stays free
    ++level;
    cluster.sync();  // ccount, cfirst, the lists' lengths and the cut have been read
  }
}

__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ float as_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float as_f32(__half v) { return __half2float(v); }

template <typename T>
__global__ void __launch_bounds__(kSThreads, 2) sample_kernel(const SampleArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  cg::cluster_group cluster = cg::this_cluster();
  Shared& s = *reinterpret_cast<Shared*>(smem);
  float* z = reinterpret_cast<float*>(smem + sizeof(Shared));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cluster.block_rank(), C = (int)cluster.num_blocks();
  const int row = blockIdx.x / C;
  Shared* s0 = cluster.map_shared_rank(&s, 0);
  const uint32_t base = (uint32_t)rank * a.slice;
  const int n = max(0, min(a.slice, a.vocab - (int)base));
  const T* src = reinterpret_cast<const T*>(a.logits) + (int64_t)row * a.row_stride + base;

  // the one read: scalar up to a 16-byte boundary, 16 bytes a thread from there
  constexpr int kVec = 16 / sizeof(T);
  float top = -INFINITY;
  auto clean = [&](float v) {
    v = v != v ? -INFINITY : v;  // a NaN ranks below every number and weighs nothing, like -infinity
    top = fmaxf(top, v);
    return v;
  };
  auto put = [&](int i, float v) { z[i] = clean(v); };
  const int head = min(n, (int)(((16 - ((uintptr_t)src & 15)) & 15) / sizeof(T)));
  const int vecs = (n - head) / kVec;
  if (tid < head) put(tid, as_f32(src[tid]));
  const uint4* vsrc = reinterpret_cast<const uint4*>(src + head);
  constexpr int kAhead = 4;
  for (int v0 = 0; v0 < vecs; v0 += kSThreads * kAhead) {
    uint4 w[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int v = v0 + j * kSThreads + tid;
      if (v < vecs) w[j] = __ldcs(vsrc + v);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int v = v0 + j * kSThreads + tid;
      if (v < vecs) {
        const T* e = reinterpret_cast<const T*>(&w[j]);
        if (head == 0) {
#pragma unroll
          for (int i = 0; i < kVec; i += 4)
            reinterpret_cast<float4*>(z + v * kVec)[i / 4] =
                make_float4(clean(as_f32(e[i])), clean(as_f32(e[i + 1])), clean(as_f32(e[i + 2])), clean(as_f32(e[i + 3])));
        } else {
#pragma unroll
          for (int i = 0; i < kVec; ++i) put(head + v * kVec + i, as_f32(e[i]));
        }
      }
    }
  }
  for (int i = head + vecs * kVec + tid; i < n; i += kSThreads) put(i, as_f32(src[i]));
  // the slice that is read when this one's place is free, into L2 while the row is worked on
  if (tid == 0 && row < a.rows - a.ahead) {
    const uintptr_t from = (uintptr_t)(src + (int64_t)a.ahead * a.row_stride), at = (from + 15) & ~(uintptr_t)15;
    const uintptr_t bytes = (from + (uintptr_t)n * sizeof(T) - at) & ~(uintptr_t)15;
    if (n * (int)sizeof(T) >= 32) asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(at), "r"((uint32_t)bytes) : "memory");
  }
  const int n4 = (n + 3) / 4;
  if (tid < 4 * n4 - n) z[n + tid] = -INFINITY;
  for (int i = tid; i < kTable; i += kSThreads) s.pow2[i] = g_pow2.v[i];

  const float T0 = a.temperature ? a.temperature[row] : 1.f;
  const int k0 = a.top_k ? a.top_k[row] : 0;
  const float p0 = a.top_p ? a.top_p[row] : 1.f, q0 = a.min_p ? a.min_p[row] : 0.f;
  const float u0 = a.u[row];

  float wtop = top;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) wtop = fmaxf(wtop, __shfl_xor_sync(0xffffffffu, wtop, o));
  if (lane == 0) s.wmax[warp] = wtop;
  __syncthreads();
  if (tid == 0) {
    float v = s.wmax[0];
    for (int w = 1; w < kSWarps; ++w) v = fmaxf(v, s.wmax[w]);
    s.cmax = v;
    s.cfirst = 0xFFFFFFFFu;
  }
  cluster.sync();
  float m = lane < C ? cluster.map_shared_rank(&s, lane)->cmax : -INFINITY;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));

  if (m == -INFINITY) {
    if (rank == 0 && tid == 0) {
      a.tokens[row] = -1;
      if (a.probs) a.probs[row] = 0.f;
    }
    cluster.sync();  // no CTA leaves while another may read its sums
    return;
  }
  if (!(T0 > 0.f) || k0 == 1 || p0 <= 0.f || q0 > 1.f) {  // greedy, or only the first of the order is kept
    uint32_t first = 0xFFFFFFFFu;
    for (int i = tid; i < n; i += kSThreads)
      if (z[i] == m) first = min(first, base + i);
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0 && first != 0xFFFFFFFFu) atomicMin(&s.cfirst, first);
    cluster.sync();
    if (rank == 0 && tid == 0) {
      for (int r = 0; r < C; ++r) first = min(first, cluster.map_shared_rank(&s, r)->cfirst);
      a.tokens[row] = (int32_t)first;
      if (a.probs) a.probs[row] = 1.f;
    }
    cluster.sync();
    return;
  }
  if (m == INFINITY) {  // infinite logits share the weight
    top = top == INFINITY ? 0.f : -INFINITY;
    for (int i = tid; i < n; i += kSThreads) z[i] = z[i] == INFINITY ? 0.f : -INFINITY;
    m = 0.f;
    __syncthreads();
  }
  const bool top_k = k0 > 1 && k0 < a.vocab, top_p = p0 < 1.f;
  const uint64_t least = q0 > 0.f ? (q0 >= 1.f ? 1ull << kUnit : mul_frac(1ull << kUnit, q0, true)) : 0;
  const Slice v{reinterpret_cast<const float4*>(z), n4, base, m, rate_of(fminf(fmaxf(T0, 1e-30f), 1e30f)), top_k ? (uint32_t)k0 : 0,
                top_p ? p0 : 1.f, least, u0 > 0.f ? fminf(u0, 0.99999994f) : 0.f, top, a.tokens + row, a.probs ? a.probs + row : nullptr};

  Cut cut{0, 0xFFFFFFFFu};
  bool limited = false;
  for (int step = 0; step < 2; ++step) {
    if (step == 0 ? !top_k : !top_p) continue;
    if (find_cut(cluster, s, s0, v, cut, limited, step == 1)) return;  // drawn
    cut = s0->cut;
    limited = true;
    cluster.sync();
  }
  // each warp's contiguous share of the slice, four neighbours a lane: its kept mass goes to wsum, the CTA's to ctotal
  const int seg = (n4 + kSWarps - 1) / kSWarps, lo = min(warp * seg, n4), hi = min(lo + seg, n4);
  const float z_cut = limited ? logit_of(cut.key) : -INFINITY;
  auto is_kept = [&](float zi, uint32_t idx) { return zi >= z_cut && (!limited || kept(key_of(zi), idx, cut)); };
  auto weigh = [&](float zi) -> uint64_t {
    const uint64_t w = weight(zi, m, v.c, s.pow2);
    return w >= least ? w : 0;
  };
  auto load4 = [&](int i) { return i < hi ? v.z[i] : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY); };
  {
    uint64_t sum = 0;
    if (!limited) {
      for (int i0 = lo + lane; i0 < hi; i0 += 64) {
        const float4 q[2] = {load4(i0), load4(i0 + 32)};
#pragma unroll
        for (int j = 0; j < 2; ++j) sum += (weigh(q[j].x) + weigh(q[j].y)) + (weigh(q[j].z) + weigh(q[j].w));
      }
    } else {
      each_of<32>(v, lo + lane, hi, [&](float zi) { return zi >= z_cut; },
                  [&](float zi, uint32_t idx) { sum += is_kept(zi, idx) ? weigh(zi) : 0; });
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncthreads();
    if (lane == 0) s.wsum[warp] = sum;
    __syncthreads();
    if (tid == 0) {
      uint64_t all = 0;
      for (int w = 0; w < kSWarps; ++w) all += s.wsum[w];
      s.ctotal = all;
    }
    cluster.sync();
  }
  uint64_t part = lane < C ? cluster.map_shared_rank(&s, lane)->ctotal : 0, total = part, front = lane < rank ? part : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, o);
    front += __shfl_xor_sync(0xffffffffu, front, o);
  }
  // sum > u * total  <=>  sum > floor(u * total)
  const uint64_t at = mul_frac(total, v.u, false);
  int of = 0;  // the warp whose share holds the token, if this CTA's does
  while (of < kSWarps && !(front <= at && at < front + s.wsum[of])) front += s.wsum[of++];
  if (of < kSWarps) {
    // all warps take that share, 32 float4 each at a time
    const int first = min(of * seg, n4), end = min(first + seg, n4);
    for (int i0 = first; i0 < end; i0 += 32 * kSWarps) {
      const int i = i0 + 32 * warp + lane;
      const float4 q = i < end ? v.z[i] : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      const float zs[4] = {q.x, q.y, q.z, q.w};
      const uint32_t idx = base + 4 * i;
      uint64_t w[4], incl = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) incl += w[e] = i < end && is_kept(zs[e], idx + e) ? weigh(zs[e]) : 0;
      const uint64_t four = incl;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      __syncthreads();
      if (lane == 31) s.bsum[warp] = incl;
      __syncthreads();
      uint64_t below = front + incl - four;
      for (int w2 = 0; w2 < kSWarps; ++w2) {
        below += w2 < warp ? s.bsum[w2] : 0;
        front += s.bsum[w2];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (below <= at && at < below + w[e]) {
          *v.token = (int32_t)(idx + e);
          if (v.prob) *v.prob = (float)w[e] / (float)total;
        }
        below += w[e];
      }
      if (front > at) break;
    }
  }
  cluster.sync();
}

template <typename T>
moe_status_t launch_sample(SampleArgs a, cudaStream_t st) {
  int sms = 0;
  moe_status_t ok = device_sms(&sms);
  if (ok != MOE_OK) return ok;
  // Slices of at most 80 KB leave room for two CTAs an SM (larger rows than 163,840 words go without); few rows take larger
  // clusters, down to slices of 4,096, so that one row's read and passes are
  // spread over more SMs.
  int C = 1;
  while (C < kMaxCluster && (a.vocab + C - 1) / C > 20480) C *= 2;
  while (C < kMaxCluster && (int64_t)a.rows * C * 2 <= sms && a.vocab / C > 4096) C *= 2;
  a.slice = (((a.vocab + C - 1) / C) + 7) & ~7;  // a multiple of the float4 and of 16 bytes of any type
  const int smem = (int)sizeof(Shared) + a.slice * 4;
  ok = raise_smem<sample_kernel<T>>((int)sizeof(Shared) + kMaxVocab / kMaxCluster * 4);
  if (ok != MOE_OK) return ok;
  // what runs at a time: an SM's 228 KB hold two CTAs (with 1 KB each of the system's) up to slices of 20,480
  a.ahead = std::max(1, sms * (2 * (smem + 1024) <= 228 * 1024 ? 2 : 1) / C);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.rows * C));
  cfg.blockDim = dim3(kSThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = C;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T>, a) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace
}  // namespace moe

extern "C" MOE_API moe_status_t moe_sample(const void* logits, int32_t dtype, int32_t rows, int32_t vocab, int64_t row_stride,
                                           const float* u, const float* temperature, const int32_t* top_k,
                                           const float* top_p, const float* min_p, int32_t* tokens, float* probs,
                                           void* cuda_stream) {
  if (dtype != MOE_BF16 && dtype != MOE_FP16 && dtype != MOE_FP32) return MOE_ERR_INVALID_ARG;
  const int size = dtype == MOE_FP32 ? 4 : 2;
  if (rows < 0 || vocab < 1 || row_stride < 0 || (rows > 1 && row_stride < vocab)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!logits || !u || !tokens || ((uintptr_t)logits % size) || ((uintptr_t)u & 3) || ((uintptr_t)temperature & 3) ||
      ((uintptr_t)top_k & 3) || ((uintptr_t)top_p & 3) || ((uintptr_t)min_p & 3) || ((uintptr_t)tokens & 3) ||
      ((uintptr_t)probs & 3))
    return MOE_ERR_INVALID_ARG;
  if (vocab > moe::kMaxVocab || rows > 1 << 28) return MOE_ERR_UNSUPPORTED;
  const moe::SampleArgs a{logits, row_stride, rows, vocab, 0, 0, u, temperature, top_p, min_p, top_k, tokens, probs};
  const cudaStream_t s = (cudaStream_t)cuda_stream;
  if (dtype == MOE_FP32) return moe::launch_sample<float>(a, s);
  if (dtype == MOE_BF16) return moe::launch_sample<__nv_bfloat16>(a, s);
  return moe::launch_sample<__half>(a, s);
}
