// Attention of a batch's new tokens over the quantised paged cache: the plan,
// the merge of partial results and the C entries.  The kernels:
//   attend_rows_kernel  (moe_attend_rows.cuh)   few rows a sequence, mma.sync
//   attend_tiles_kernel (moe_attend_tiles.cuh)  many rows a sequence, tcgen05
#include <algorithm>

#include "moe_attend.cuh"

namespace moe {
namespace {

using namespace ptx;

// Merges the partial results of the cut segments, the one that ends in part
// blockIdx.x.  A lone long sequence has up to a hundred parts a segment: then
// (WARPS 8) a CTA takes one row, its warps every eighth part; many segments
// have a part or two each: then (WARPS 1) every warp takes a row.
constexpr int kJoinThreads = 256;

template <int D, bool BF16, int WARPS>
__global__ void __launch_bounds__(kJoinThreads) attend_join_kernel(const KvArgs a, const AttArgs t) {
  constexpr int NE = D / 32;  // elements a lane holds
  __shared__ float s_o[WARPS > 1 ? WARPS : 1][D];
  __shared__ float2 s_stat[WARPS > 1 ? WARPS : 1];
  grid_wait();
  const SegmentEnd end = t.ends[blockIdx.x];
  if (end.first < 0) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = WARPS > 1 ? tid >> 5 : 0;
  const int row = WARPS > 1 ? blockIdx.y : blockIdx.y * (kJoinThreads / 32) + (tid >> 5);
  const int c0 = end.first, c1 = blockIdx.x, head = end.head;
  const Seq sq = seq_at(a, end.b);
  const int fr = end.rt * t.tile_rows + row;
  if (row >= t.tile_rows || fr >= sq.n * t.group) return;
  // the part that begins at the segment's first tile lies in its CTA's slot 1, the others in slot 0; four parts' loads in flight
  float m = -INFINITY, l = 0.f, o[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) o[i] = 0.f;
  constexpr int kAhead = 4;
  for (int c = c0 + warp; c <= c1; c += WARPS * kAhead) {
    float2 st[kAhead];
    float v[kAhead][NE];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int ck = c + k * WARPS;
      st[k] = make_float2(-INFINITY, 0.f);
      if (ck > c1) continue;
      const size_t at = ((size_t)ck * 2 + (ck == c0 ? 1 : 0)) * t.tile_rows + row;
      st[k] = t.stats[at];
      const float* src = t.partial + at * D + lane * NE;
#pragma unroll
      for (int i = 0; i < NE; ++i) v[k][i] = src[i];
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (c + k * WARPS > c1) break;
      const float n = fmaxf(m, st[k].x);
      const float wo = m == -INFINITY ? 0.f : ex2(m - n), wn = st[k].x == -INFINITY ? 0.f : ex2(st[k].x - n);
      l = (l != l ? l : l * wo) + (st[k].y != st[k].y ? st[k].y : st[k].y * wn);
#pragma unroll
      for (int i = 0; i < NE; ++i) o[i] = o[i] * wo + v[k][i] * wn;
      m = n;
    }
  }
  const int tok = fr / t.group, gh = fr - tok * t.group;
  uint16_t* dst = t.out + (int64_t)(sq.row0 + tok) * t.o_ts + (int64_t)(head * t.group + gh) * t.o_hs;
  float* lse = t.lse ? t.lse + (int64_t)(sq.row0 + tok) * t.nq + head * t.group + gh : nullptr;
  if constexpr (WARPS == 1) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int i = 0; i < NE; i += 2) *reinterpret_cast<uint32_t*>(dst + lane * NE + i) = pack2<BF16>(o[i] * inv, o[i + 1] * inv);
    if (lse && lane == 0) *lse = lse_of(m, l);
  } else {
#pragma unroll
    for (int i = 0; i < NE; ++i) s_o[warp][lane * NE + i] = o[i];
    if (lane == 0) s_stat[warp] = make_float2(m, l);
    __syncthreads();
    float mm = -INFINITY, ll = 0.f, wgt[WARPS];
#pragma unroll
    for (int w = 0; w < WARPS; ++w) mm = fmaxf(mm, s_stat[w].x);
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      wgt[w] = s_stat[w].x == -INFINITY ? 0.f : ex2(s_stat[w].x - mm);
      ll += s_stat[w].y != s_stat[w].y ? s_stat[w].y : s_stat[w].y * wgt[w];
    }
    const float inv = ll == 0.f ? 0.f : 1.f / ll;
    for (int d = 2 * tid; d < D; d += 2 * kJoinThreads) {
      float v0 = 0.f, v1 = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        v0 = fmaf(wgt[w], s_o[w][d], v0);
        v1 = fmaf(wgt[w], s_o[w][d + 1], v1);
      }
      *reinterpret_cast<uint32_t*>(dst + d) = pack2<BF16>(v0 * inv, v1 * inv);
    }
    if (lse && tid == 0) *lse = lse_of(mm, ll);
  }
}

// Merges a segment's parts, or its whole, into a row's running result; the warp's lanes hold D / 32 elements each.
template <int D>
__device__ __forceinline__ void merge_span(const AttArgs& t, int64_t segment, int row, int lane, float& m, float& l, float (&o)[D / 32]) {
  constexpr int NE = D / 32, kAhead = D == 256 ? 4 : 8;
  const Span s = t.spans[segment];
  const bool whole = s.first == kWhole;
  const int c0 = whole ? 0 : s.first, c1 = whole ? 0 : s.last;
  for (int c = c0; c <= c1; c += kAhead) {
    float2 st[kAhead];
    float v[kAhead][NE];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int ck = c + k;
      st[k] = make_float2(-INFINITY, 0.f);
      if (ck > c1) continue;
      const size_t at = (whole ? (size_t)segment : (size_t)ck * 2 + (ck == c0 ? 1 : 0)) * t.tile_rows + row;
      st[k] = (whole ? t.whole_stats : t.stats)[at];
      const float* src = (whole ? t.whole : t.partial) + at * D + lane * NE;
#pragma unroll
      for (int i = 0; i < NE; ++i) v[k][i] = src[i];
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (c + k > c1) break;
      const float n = fmaxf(m, st[k].x);
      const float wo = m == -INFINITY ? 0.f : ex2(m - n), wn = st[k].x == -INFINITY ? 0.f : ex2(st[k].x - n);
      l = (l != l ? l : l * wo) + (st[k].y != st[k].y ? st[k].y : st[k].y * wn);
#pragma unroll
      for (int i = 0; i < NE; ++i) o[i] = o[i] * wo + v[k][i] * wn;
      m = n;
    }
  }
}

// A warp a row (token, query head): what it saw of the shared prefix (`pre`) and behind it (`t`).
template <int D, bool BF16>
__global__ void __launch_bounds__(kJoinThreads) attend_join_shared_kernel(const KvArgs a, const AttArgs t, const AttArgs pre) {
  constexpr int NE = D / 32;
  grid_wait();
  const int lane = threadIdx.x & 31;
  const int64_t r = (int64_t)blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5);
  const int tok = (int)(r / t.nq), qh = (int)(r - (int64_t)tok * t.nq);
  if (tok >= a.n_tokens) return;
  const int b = kv_seq_of(a, tok);
  if (b < 0) return;
  const Seq sq = seq_at(a, b);
  if (tok - sq.row0 >= sq.n) return;
  const int head = qh / t.group, g = qh - head * t.group;
  float m = -INFINITY, l = 0.f, o[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) o[i] = 0.f;
  const int see = sq.len - sq.n + tok - sq.row0;
  const int n = min(max(__ldg(a.cu + a.n_seqs), 0), a.n_tokens);
  if (see >= 0 && tok < n) {  // (a batch whose token counts decrease, which is flagged, has rows that the prefix's pass did not see)
    const int tiles = (n * t.group + pre.tile_rows - 1) / pre.tile_rows;
    const int fr = tok * t.group + g, rt = fr / pre.tile_rows;
    merge_span<D>(pre, (int64_t)head * tiles + rt, fr - rt * pre.tile_rows, lane, m, l, o);
  }
  if (min(sq.len, a.max_pages * a.page_size) > t.shared) {
    const int fr = (tok - sq.row0) * t.group + g, rt = fr / t.tile_rows;
    merge_span<D>(t, ((int64_t)b * a.heads + head) * t.max_row_tiles + rt, fr - rt * t.tile_rows, lane, m, l, o);
  }
  if (see >= a.max_pages * a.page_size) l = __uint_as_float(kNaN);  // (neither pass has a tile there where the prefix fills the table)
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint16_t* dst = t.out + (int64_t)tok * t.o_ts + (int64_t)qh * t.o_hs;
#pragma unroll
  for (int i = 0; i < NE; i += 2) *reinterpret_cast<uint32_t*>(dst + lane * NE + i) = pack2<BF16>(o[i] * inv, o[i + 1] * inv);
  if (t.lse && lane == 0) t.lse[(int64_t)tok * t.nq + qh] = lse_of(m, l);
}

// Where a kernel's results lie in the workspace, from `at` on.
struct Workspace {
  size_t partial, stats, ends, whole, whole_stats, spans, end;
};

size_t up16(size_t v) { return (v + 15) & ~(size_t)15; }

// segments: those that leave results of their own (with a shared prefix).
Workspace plan_workspace(size_t at, int parts, int tile_rows, int dim, int64_t segments) {
  Workspace w{};
  w.partial = at;
  w.stats = up16(w.partial + (size_t)parts * 2 * tile_rows * dim * 4);
  w.ends = up16(w.stats + (size_t)parts * 2 * tile_rows * 8);
  w.whole = up16(w.ends + (size_t)parts * sizeof(SegmentEnd));
  w.whole_stats = up16(w.whole + (size_t)segments * tile_rows * dim * 4);
  w.spans = up16(w.whole_stats + (size_t)segments * tile_rows * 8);
  w.end = up16(w.spans + (size_t)segments * sizeof(Span));
  return w;
}
void place(AttArgs* t, uint8_t* base, const Workspace& w) {
  t->partial = (float*)(base + w.partial);
  t->stats = (float2*)(base + w.stats);
  t->ends = (SegmentEnd*)(base + w.ends);
  t->whole = (float*)(base + w.whole);
  t->whole_stats = (float2*)(base + w.whole_stats);
  t->spans = (Span*)(base + w.spans);
}

template <int D, bool BF16>
moe_status_t launch_join_type(const KvArgs& kv, const AttArgs& t, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  const int64_t most = (int64_t)kv.max_tokens * t.group;
  const int rows = (int)(most < t.tile_rows ? most : t.tile_rows);
  const int64_t segments = (int64_t)kv.n_seqs * kv.heads * ((most + t.tile_rows - 1) / t.tile_rows);
  const bool wide = t.parts >= 8 * segments || t.tile_rows <= 32;
  cfg.gridDim = dim3((unsigned)t.parts, (unsigned)(wide ? rows : (rows + kJoinThreads / 32 - 1) / (kJoinThreads / 32)));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  const cudaError_t e = wide ? cudaLaunchKernelEx(&cfg, attend_join_kernel<D, BF16, 8>, kv, t)
                             : cudaLaunchKernelEx(&cfg, attend_join_kernel<D, BF16, 1>, kv, t);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
template <int D>
moe_status_t launch_join(const KvArgs& kv, const AttArgs& t, bool bf16, cudaStream_t st) {
  return bf16 ? launch_join_type<D, true>(kv, t, st) : launch_join_type<D, false>(kv, t, st);
}

template <int D>
moe_status_t launch_join_shared(const KvArgs& kv, const AttArgs& t, const AttArgs& pre, bool bf16, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  const int64_t rows = (int64_t)kv.n_tokens * t.nq, warps = kJoinThreads / 32;
  cfg.gridDim = dim3((unsigned)((rows + warps - 1) / warps));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  const cudaError_t e = bf16 ? cudaLaunchKernelEx(&cfg, attend_join_shared_kernel<D, true>, kv, t, pre)
                             : cudaLaunchKernelEx(&cfg, attend_join_shared_kernel<D, false>, kv, t, pre);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// What both entries derive from their arguments.
struct AttPlan {
  KvArgs kv;
  bool tiles;   // attend_tiles_kernel
  int shared;   // keys that are read once for the batch
  int parts, tile_rows, max_row_tiles;
  int pre_parts, pre_rows;
  Workspace ws, pre_ws;
  size_t bytes;
};

moe_status_t attend_plan(const moe_kv_cache_t* cache, const moe_kv_batch_t* batch, int32_t n_q, int32_t shared_tokens, AttPlan* p) {
  moe_status_t st = kv_args(cache, batch, &p->kv);
  if (st != MOE_OK) return st;
  if (n_q < 1 || n_q % cache->n_kv_heads || shared_tokens < 0 || shared_tokens % cache->page_size) return MOE_ERR_INVALID_ARG;
  if (shared_tokens / cache->page_size > batch->max_pages) return MOE_ERR_INVALID_ARG;
  const int64_t rows = batch->n_tokens ? (int64_t)batch->max_tokens * (n_q / cache->n_kv_heads) : 0;
  if (rows > 1 << 24) return MOE_ERR_UNSUPPORTED;
  int sms = 0;
  st = device_sms(&sms);
  if (st != MOE_OK) return st;
  // A sequence's rows in tiles of 8 while they suffice, then 16 and 32, which
  // share the dequantised keys and values.  Above one such tile (two of them
  // for heads of 64) the tensor cores' tiles of 256, 128 for heads of 256.  In
  // us there and here, 32 sequences of 8,192 tokens, 4 kv heads of 128, 8 bits:
  // 32 rows 118 and 109, 48 rows 122 and 188, 64 rows 125 and 193 (4 bits 118
  // and 107, 121 and 185, 124 and 190); heads of 64, 64 rows: 109 and 117 (4 bits
  // 101 and 112; with fp16 activations the tiles take a third longer, rows do
  // not).  Heads of 256, which have registers for 16 rows here: 12
  // sequences of 60,000 to 131,072 tokens in 4 bits, 32 rows, 219 and 328.
  const int dim = cache->head_dim, heads = cache->n_kv_heads, group = n_q / heads;
  const int big = dim == 256 ? 128 : 256;
  p->tiles = rows > (dim == 256 ? 16 : dim == 128 ? 32 : 64);
  p->tile_rows = p->tiles ? big : rows <= 8 ? 8 : rows <= 16 || dim == 256 ? 16 : 32;
  p->parts = p->tiles ? sms : sms * rows_blocks(dim, cache->bits, p->tile_rows);
  p->max_row_tiles = (int)((rows + p->tile_rows - 1) / p->tile_rows);
  // A prefix gets a pass of its own where that spares the rows' kernel a
  // million keys (counted a kv head), whose reading takes about as long as the
  // pass and the merge.  In us, with the pass and without (where all but the
  // first read come from L2), 8 bits, heads of 128, 4 kv heads: 16 sequences x
  // 16,384 tokens (1.0 million) 37 and 42, 64 x 4,096 (1.0) 41 and 48, 128 x
  // 4,096 (2.1) 53 and 84, 48 x 16,384 (3.1) 52 and 106; 64 x 2,048 (0.5) 33
  // without, and with one that the rows' kernel had to wait for 42.  4 bits, 64
  // x 4,096: 40 and 48; heads of 256, 2 kv heads, 16 x 32,768 (1.0) 63 and 68;
  // of 64, 8 kv heads, 64 x 4,096 (2.1) 36 and 58.
  const int64_t all_rows = (int64_t)batch->n_tokens * group;
  const int64_t passes = std::max<int64_t>(all_rows / p->tile_rows, std::min(batch->n_seqs, batch->n_tokens));
  p->shared = !p->tiles && (double)(passes - 1) * shared_tokens * heads >= 0.98e6 ? shared_tokens : 0;
  p->pre_parts = sms;
  p->pre_rows = big;
  const int64_t segments = (int64_t)batch->n_seqs * heads * p->max_row_tiles, pre_segments = heads * ((all_rows + big - 1) / big);
  if (segments > INT32_MAX || pre_segments > INT32_MAX || all_rows * heads > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  p->ws = plan_workspace(0, p->parts, p->tile_rows, dim, p->shared ? segments : 0);
  p->bytes = p->ws.end;
  if (p->shared) {
    p->pre_ws = plan_workspace(p->bytes, p->pre_parts, p->pre_rows, dim, pre_segments);
    p->bytes = p->pre_ws.end;
  }
  return MOE_OK;
}

}  // namespace

// As RowsPlan::kBlocks.
int rows_blocks(int dim, int bits, int tile_rows) {
  return tile_rows == 32 || dim * tile_rows >= 4096 || (dim == 256 && bits == 8) ? 2 : 3;
}

}  // namespace moe

extern "C" MOE_API moe_status_t moe_kv_attend_workspace(const moe_kv_cache_t* cache, const moe_kv_batch_t* batch, int32_t n_q,
                                                        int32_t shared_tokens, size_t* bytes) {
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = 0;
  moe::AttPlan p;
  const moe_status_t st = moe::attend_plan(cache, batch, n_q, shared_tokens, &p);
  if (st == MOE_OK) *bytes = p.bytes;
  return st;
}

extern "C" MOE_API moe_status_t moe_kv_attend(const moe_kv_cache_t* cache, const moe_kv_batch_t* batch, int32_t dtype,
                                              int32_t n_q, const moe_heads_t* q, const moe_heads_t* out, float* lse,
                                              float scale, int32_t shared_tokens, void* workspace, size_t workspace_bytes,
                                              void* cuda_stream) {
  if (dtype != MOE_BF16 && dtype != MOE_FP16) return dtype == MOE_FP32 ? MOE_ERR_UNSUPPORTED : MOE_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || ((uintptr_t)lse & 3)) return MOE_ERR_INVALID_ARG;
  moe::AttPlan p;
  const moe_status_t st = moe::attend_plan(cache, batch, n_q, shared_tokens, &p);
  if (st != MOE_OK) return st;
  if (p.kv.n_tokens == 0) return MOE_OK;
  const int dim = cache->head_dim;
  if (!moe::heads_ok(q, dim) || !moe::out_heads_ok(out, n_q, p.kv.n_tokens, dim)) return MOE_ERR_INVALID_ARG;
  if (!workspace || ((uintptr_t)workspace & 15)) return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < p.bytes) return MOE_ERR_OUT_OF_MEMORY;
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
  t.tile_rows = p.tile_rows;
  t.parts = p.parts;
  t.shared = p.shared;
  t.max_row_tiles = p.max_row_tiles;
  moe::place(&t, w, p.ws);
  const bool bf = dtype == MOE_BF16;
  const cudaStream_t s = (cudaStream_t)cuda_stream;
  const bool wide = cache->bits == 8;
  moe_status_t done;
  if (!p.shared) {
    const auto launch = p.tiles ? (wide ? moe::launch_tiles8 : moe::launch_tiles4) : (wide ? moe::launch_rows8 : moe::launch_rows4);
    done = launch(p.kv, t, dim, bf, s);
    if (done != MOE_OK) return done;
    if (dim == 64) return moe::launch_join<64>(p.kv, t, bf, s);
    if (dim == 128) return moe::launch_join<128>(p.kv, t, bf, s);
    return moe::launch_join<256>(p.kv, t, bf, s);
  }
  moe::AttArgs pre = t;
  pre.parts = p.pre_parts;
  pre.tile_rows = p.pre_rows;
  moe::place(&pre, w, p.pre_ws);
  done = (wide ? moe::launch_tiles8 : moe::launch_tiles4)(p.kv, pre, dim, bf, s);
  if (done == MOE_OK) done = (wide ? moe::launch_rows8 : moe::launch_rows4)(p.kv, t, dim, bf, s);
  if (done != MOE_OK) return done;
  if (dim == 64) return moe::launch_join_shared<64>(p.kv, t, pre, bf, s);
  if (dim == 128) return moe::launch_join_shared<128>(p.kv, t, pre, bf, s);
  return moe::launch_join_shared<256>(p.kv, t, pre, bf, s);
}
